"""ep_route and ep_route_grad against the definition in 64 bits.

Choices have to be equal.  Weights: exp of a rounded difference of logits (R the logits' range) is
within (R + 4) steps of 2^-24 of itself, and so are the sum's terms; the sum of n terms adds n steps,
quotient and scale two: (2 R + n + 12) steps in all, and as many for a gradient's sums of at most n
terms, relative to the sum of their magnitudes."""
import math

import pytest
import torch

import block_ref as ref
from combine_moe_layout_amd import binding as B
from products_ref import half_step

pytestmark = pytest.mark.gpu
TYPES = {"fp32": (B.EP_F32, torch.float32), "bf16": (B.EP_BF16, torch.bfloat16), "fp16": (B.EP_F16, torch.float16)}
SCORES = {"softmax": B.EP_SCORE_SOFTMAX, "sigmoid": B.EP_SCORE_SIGMOID}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def steps(logits, n):
    l = logits.double()
    l = l[torch.isfinite(l)]
    r = (l.max() - l.min()).item() if l.numel() else 0.0
    return (2 * min(r, 200.0) + n + 12) * ref.STEP


def route(logits, name, router, bias=None):
    T, k = logits.shape[0], router.num_topk
    idx = torch.full((T, k), -7, dtype=torch.int64, device="cuda")
    w = torch.full((T, k), 7.0, device="cuda")
    B.ep_route(logits, router, idx, w, TYPES[name][0], bias=bias)
    torch.cuda.synchronize()
    return idx, w


def check_weights(logits, idx, w, score, renorm, scale):
    want = ref.weights(ref.usable(logits)[0], idx, score, renorm, scale)
    tol = steps(logits, logits.shape[1]) * want + 2.0 ** -126
    assert torch.isfinite(w).all()
    assert ((w.double() - want).abs() <= tol).all(), ((w.double() - want).abs() / tol).max().item()
    assert (w[idx < 0] == 0).all()


SHAPES = [  # T, E, k, groups, topk_groups, group_top
    (1, 1, 1, 1, 1, 1), (3, 2, 1, 1, 1, 1), (5, 5, 5, 1, 1, 1), (33, 24, 3, 1, 1, 1), (64, 64, 6, 1, 1, 1),
    (257, 64, 33, 1, 1, 1), (100, 256, 8, 8, 4, 2), (100, 256, 8, 8, 3, 1), (31, 160, 6, 8, 3, 2), (17, 96, 7, 3, 2, 1),
    (9, 100, 64, 1, 1, 1), (40, 255, 9, 5, 2, 2), (40, 40, 4, 40, 7, 1), (13, 300, 10, 1, 1, 1), (13, 512, 16, 16, 4, 2),
    (7, 1024, 8, 8, 2, 2), (7, 1000, 64, 10, 5, 2), (5, 1024, 3, 1024, 100, 1), (2, 1024, 3, 512, 100, 2),
    (2000, 128, 8, 4, 1, 2)]


@pytest.mark.parametrize("T,E,k,groups,topk_groups,group_top", SHAPES)
def test_choice_and_weights(T, E, k, groups, topk_groups, group_top):
    print("[gpu-route]", T, E, k, groups, topk_groups, group_top, flush=True)
    for n, (name, score, biased, renorm) in enumerate([
            ("fp32", "softmax", False, True), ("fp32", "sigmoid", True, True), ("bf16", "sigmoid", False, False),
            ("fp16", "softmax", True, False), ("bf16", "softmax", False, True), ("fp32", "softmax", True, True)]):
        g = gen(T * 1000 + n)
        logits = torch.randn((T, E), device="cuda", generator=g).to(TYPES[name][1])
        bias = torch.randn(E, device="cuda", generator=g) * 0.1 if biased else None
        router = B.EpRouter(E, k, SCORES[score], groups, topk_groups, group_top, renorm, 1.5)
        idx, w = route(logits, name, router, bias)
        assert torch.equal(idx, ref.choice(logits, bias, k, score, groups, topk_groups, group_top)), (name, score, biased)
        check_weights(logits, idx, w, score, renorm, 1.5)


@pytest.mark.parametrize("E,k,groups,topk_groups,group_top", [(64, 6, 1, 1, 1), (256, 8, 8, 4, 2), (33, 5, 3, 2, 2),
                                                              (512, 9, 4, 2, 1)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_go_to_the_lower_index(E, k, groups, topk_groups, group_top, score):
    """Logits of five values, with and without a bias of two values: whole runs of equal keys."""
    g = gen(E + k)
    logits = torch.randint(-2, 3, (300, E), device="cuda", generator=g).float()
    logits[0] = 0.0
    logits[1] = -0.0
    logits[2, ::2] = -0.0
    bias = torch.randint(0, 2, (E,), device="cuda", generator=g).float() * 0.25
    router = B.EpRouter(E, k, SCORES[score], groups, topk_groups, group_top)
    for b in (None, bias, torch.zeros_like(bias)):
        idx, _ = route(logits, "fp32", router, b)
        assert torch.equal(idx, ref.choice(logits, b, k, score, groups, topk_groups, group_top))


@pytest.mark.parametrize("E,groups,topk_groups,group_top", [(64, 1, 1, 1), (256, 8, 3, 2), (250, 5, 2, 2), (1024, 1, 1, 1)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_keys_closer_than_fp32_can_tell(E, groups, topk_groups, group_top, score):
    """A bias that makes all keys of a token the same to within fp32's rounding: their order is that
    of the sums in 64 bits.  (Those differ by about 2^-26, far above 64 bits' own rounding.)"""
    for seed in range(4):
        logits = torch.randn((1, E), device="cuda", generator=gen(seed))
        bias = (0.75 - ref.scores(logits, score)[0]).float()
        key = (ref.scores(logits, score) + bias.double())[0]
        assert (key.max() - key.min()).item() < 2.0 ** -23     # the test means what it says
        many = logits.repeat(5, 1)
        many[2] = torch.randn(E, device="cuda", generator=gen(seed + 50))   # an ordinary token among them
        router = B.EpRouter(E, 8, SCORES[score], groups, topk_groups, group_top)
        idx, w = route(many, "fp32", router, bias)
        assert torch.equal(idx, ref.choice(many, bias, 8, score, groups, topk_groups, group_top)), seed
        check_weights(many, idx, w, score, True, 1.0)


@pytest.mark.parametrize("E,groups,topk_groups", [(32, 8, 3), (64, 4, 2), (24, 8, 3), (600, 5, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups_of_keys_that_cancel(E, groups, topk_groups, score):
    """A group's two largest keys are large and of opposite signs: what fp32 rounds off of each is more
    than the groups' sums, which are those of the scores alone, differ by."""
    n, T = E // groups, 500
    logits = torch.randn((T, E), device="cuda", generator=gen(E))
    bias = torch.full((groups, n), -90000.0, device="cuda")
    bias[:, 0], bias[:, 1] = 30000.0, -30000.0
    router = B.EpRouter(E, 2, SCORES[score], groups, topk_groups, 2)
    idx, w = route(logits, "fp32", router, bias.view(-1))
    assert torch.equal(idx, ref.choice(logits, bias.view(-1), 2, score, groups, topk_groups, 2))
    check_weights(logits, idx, w, score, True, 1.0)


@pytest.mark.parametrize("E,groups,topk_groups,group_top", [(64, 1, 1, 1), (256, 8, 3, 2), (250, 5, 2, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_infinite_biases(E, groups, topk_groups, group_top, score):
    """Experts with a bias of +inf come first, in their order; those with -inf never."""
    logits = torch.randn((40, E), device="cuda", generator=gen(E))
    bias = 0.1 * torch.randn(E, device="cuda", generator=gen(E + 1))
    bias[torch.tensor([5, E - 3, E // 2])] = math.inf
    bias[::4] = -math.inf
    bias[7] = 3e38
    router = B.EpRouter(E, 8, SCORES[score], groups, topk_groups, group_top)
    idx, w = route(logits, "fp32", router, bias)
    assert torch.equal(idx, ref.choice(logits, bias, 8, score, groups, topk_groups, group_top))
    check_weights(logits, idx, w, score, True, 1.0)


@pytest.mark.parametrize("E,k,groups,topk_groups", [(8, 3, 1, 1), (64, 6, 1, 1), (256, 8, 8, 4), (100, 8, 5, 2), (600, 16, 1, 1)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_masked_experts(E, k, groups, topk_groups, score, renorm):
    """-inf and NaN are never chosen, a token with too few experts is filled with -1, a token with
    none is all -1; +inf is the largest value.  The gradient there is 0."""
    g = gen(E + k)
    T = 70
    logits = torch.randn((T, E), device="cuda", generator=g)
    logits.masked_fill_(torch.rand((T, E), device="cuda", generator=g) < 0.3, -math.inf)
    logits.masked_fill_(torch.rand((T, E), device="cuda", generator=g) < 0.1, math.nan)
    logits[0], logits[1], logits[2] = -math.inf, math.nan, -math.inf
    logits[2, E - 1] = 1.0
    logits[3, 3], logits[4, :2] = math.inf, math.inf
    logits[5], logits[6] = torch.finfo(torch.float32).min, math.inf
    bias = torch.randn(E, device="cuda", generator=g) * 0.1
    bias[1], bias[2] = -math.inf, math.nan
    router = B.EpRouter(E, k, SCORES[score], groups, topk_groups, 1, renorm)
    for b in (None, bias):
        idx, w = route(logits, "fp32", router, b)
        assert torch.equal(idx, ref.choice(logits, b, k, score, groups, topk_groups))
        assert (idx[0] == -1).all() and (idx[1] == -1).all() and (w[:2] == 0).all()
        rest = torch.cat([torch.arange(3), torch.arange(7, T)]).cuda()
        check_weights(logits[rest], idx[rest], w[rest], score, renorm, 1.0)
        assert torch.isfinite(w).all()
        d = torch.full_like(logits, 7.0)
        dw = torch.randn((T, k), device="cuda", generator=g)
        dw[idx < 0] = math.nan                     # not used
        B.ep_route_grad(dw, logits, idx, router, d, B.EP_F32)
        assert torch.isfinite(d).all()
        assert (d[~ref.usable(logits)[1]] == 0).all()


def exact_gradient(dw, logits, idx, score, renorm, scale):
    """By autograd through the weights in 64 bits, and the sum of the magnitudes of its terms.  Where
    those cancel exactly (the unchosen experts of a renormalised softmax), autograd's own rounding
    is left: E terms of at most scale * sum |dw|, each within 2^-52 of itself.  `size` has it in
    units of a step of fp32."""
    l, live = ref.usable(logits)
    l = l.detach().requires_grad_(True)
    dw = torch.where(idx >= 0, dw.double(), 0.0)
    (ref.weights(l, idx, score, renorm, scale) * dw).sum().backward()
    with torch.no_grad():
        w = ref.weights(l, idx, score, renorm, scale)
        size = torch.zeros_like(l)
        if renorm:
            term = w * (w[:, None, :] / scale * (dw[:, :, None] - dw[:, None, :]).abs()).sum(2)
        else:
            term = w * dw.abs()
        size.scatter_add_(1, idx.clamp(min=0), torch.where(idx >= 0, term, 0.0))
        if score == "softmax" and not renorm:
            size += ref.scores(logits, score) * term.sum(1, keepdim=True)
        size += logits.shape[1] * 2.0 ** -52 / ref.STEP * scale * dw.abs().sum(1, keepdim=True)
    return torch.where(live, l.grad, 0.0), size


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 2, 2), (65, 24, 3), (64, 64, 6), (130, 256, 8), (9, 100, 64),
                                   (13, 300, 10), (7, 1000, 16), (6, 1024, 64), (1025, 16, 4)])
@pytest.mark.parametrize("name", ["fp32", "bf16", "fp16"])
def test_gradient(T, E, k, name):
    print("[gpu-route] gradient", T, E, k, name, flush=True)
    code, dt = TYPES[name]
    for score in SCORES:
        for renorm in (True, False):
            g = gen(T + E)
            logits = torch.randn((T, E), device="cuda", generator=g).to(dt)
            dw = torch.randn((T, k), device="cuda", generator=g)
            router = B.EpRouter(E, k, SCORES[score], renormalize=renorm, scale=2.5)
            idx, _ = route(logits, name, router)
            d = torch.full_like(logits, 7.0)
            B.ep_route_grad(dw, logits, idx, router, d, code)
            want, size = exact_gradient(dw, logits, idx, score, renorm, 2.5)
            tol = (2 * steps(logits, E) + k * ref.STEP) * size
            tol = tol + half_step(want.abs() + tol, dt)
            assert torch.isfinite(d).all()
            assert ((d.double() - want).abs() <= tol).all(), ((d.double() - want).abs() / tol).max().item()


def test_gradient_of_given_choices():
    """Choices that a caller made: the same id twice adds up in order, ids out of range and -1 add nothing."""
    T, E, k = 50, 40, 6
    g = gen(3)
    logits = torch.randn((T, E), device="cuda", generator=g)
    dw = torch.randn((T, k), device="cuda", generator=g)
    idx = torch.randint(0, E, (T, k), device="cuda", generator=g)
    idx[:, 1] = idx[:, 0]
    bad = idx.clone()
    bad[::3, 4] = -1
    bad[::4, 5] = E
    bad[1, 2], bad[2, 3] = -2 ** 40, 2 ** 40
    none = torch.where((bad < 0) | (bad >= E), -1, bad)
    for score in SCORES:
        for renorm in (True, False):
            router = B.EpRouter(E, k, SCORES[score], renormalize=renorm)
            d = torch.empty_like(logits)
            B.ep_route_grad(dw, logits, bad, router, d, B.EP_F32)
            want, size = exact_gradient(dw, logits, none, score, renorm, 1.0)
            tol = (2 * steps(logits, E) + (k + 1) * ref.STEP) * size + 2.0 ** -126
            assert ((d.double() - want).abs() <= tol).all(), ((d.double() - want).abs() / tol).max().item()
            again = torch.empty_like(d)
            B.ep_route_grad(dw, logits, bad, router, again, B.EP_F32)
            assert torch.equal(d, again)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(score, renorm):
    """Along random directions, the choice being all experts: (f(l + h v) - f(l - h v)) / 2h of the
    kernel's own weights, h = 2^-6.  Weights are within 40 steps of 2^-24, which h makes 2^-12.7 of
    them each; the third derivative of a weight along v is below 13 |v|^3 w (five terms of softmax's
    or sigmoid's, each of a product of slopes below 2 |v|), times h^2 / 6: 2^-10.8 |v|^3 w."""
    T, E = 64, 8
    g = gen(5)
    logits, v = (torch.randn((T, E), device="cuda", generator=g) for _ in range(2))
    v = v / v.abs().amax(1, keepdim=True)
    dw = torch.randn((T, E), device="cuda", generator=g)      # by expert
    router = B.EpRouter(E, E, SCORES[score], renormalize=renorm)

    def by_expert(l):
        idx, w = route(l, "fp32", router)
        return torch.zeros((T, E), device="cuda").scatter_(1, idx, w).double()

    h = 2.0 ** -6
    diff = ((by_expert(logits + h * v) - by_expert(logits - h * v)) / (2 * h) * dw.double()).sum(1)
    idx, w = route(logits, "fp32", router)
    d = torch.empty_like(logits)
    B.ep_route_grad(dw.gather(1, idx), logits, idx, router, d, B.EP_F32)
    tol = (2.0 ** -12.7 + 2.0 ** -10.8) * (by_expert(logits) * dw.double().abs()).sum(1) * 2
    assert ((diff - (d.double() * v.double()).sum(1)).abs() <= tol).all()


def test_extreme_logits():
    """Scores that underflow: the shares over the chosen still add up, relative to the largest."""
    logits = torch.tensor([[-200.0, -201.0, -300.0, -202.0], [-3e38, -3e38, -1e38, -3e38], [200.0, 100.0, 150.0, -200.0],
                           [-88.0, -89.0, -104.0, -120.0]], device="cuda")
    for score in SCORES:
        router = B.EpRouter(4, 2, SCORES[score])
        idx, w = route(logits, "fp32", router)
        assert torch.equal(idx, ref.choice(logits, None, 2, score))
        want = ref.weights(logits.double(), idx, score, True, 1.0)
        assert (w.double() - want).abs().max() <= 64 * ref.STEP, score
        d = torch.empty_like(logits)
        B.ep_route_grad(torch.ones((4, 2), device="cuda"), logits, idx, router, d, B.EP_F32)
        assert (d == 0).all()


def test_many_tokens():
    """More tokens than one wave of workgroups holds, and the whole range written."""
    T, E, k = 70001, 48, 4
    logits = torch.randn((T, E), device="cuda", generator=gen(9)).bfloat16()
    router = B.EpRouter(E, k, B.EP_SCORE_SIGMOID)
    idx, w = route(logits, "bf16", router)
    key, order = torch.sort(logits.double(), dim=1, descending=True, stable=True)
    assert torch.equal(idx, order[:, :k])
    check_weights(logits, idx, w, "sigmoid", True, 1.0)


def test_offsets_past_32_bits():
    """More logits than 2^31: the last tokens come out as by themselves, forward and gradient."""
    T, E, k = 2_100_000, 1024, 2
    logits = torch.zeros((T, E), device="cuda", dtype=torch.bfloat16)
    logits[-9:] = torch.randn((9, E), device="cuda", generator=gen(3)).bfloat16()
    router = B.EpRouter(E, k, B.EP_SCORE_SOFTMAX, 8, 4, 1, False)
    idx, w = route(logits, "bf16", router)
    few, few_w = route(logits[-9:].clone(), "bf16", router)
    assert torch.equal(idx[-9:], few) and torch.equal(w[-9:], few_w) and (idx[:-9] == torch.arange(k, device="cuda")).all()
    d, few_d = torch.empty_like(logits), torch.empty_like(logits[-9:])
    B.ep_route_grad(w, logits, idx, router, d, B.EP_BF16)
    B.ep_route_grad(few_w, logits[-9:].clone(), few, router, few_d, B.EP_BF16)
    assert torch.equal(d[-9:], few_d)


def test_no_tokens():
    router = B.EpRouter(8, 2)
    e = lambda *s, dt=torch.float32: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
    B.ep_route(e(0, 8), router, e(0, 2, dt=torch.int64), e(0, 2), B.EP_F32)
    B.ep_route_grad(e(0, 2), e(0, 8), e(0, 2, dt=torch.int64), router, e(0, 8), B.EP_F32)
    torch.cuda.synchronize()
