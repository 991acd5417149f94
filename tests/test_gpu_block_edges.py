"""The router, the block norms and the 8-bit products at the ends of their ranges, against the
definitions in 64 bits."""
import math

import pytest
import torch

import block_ref as ref
import test_gpu_block_norm as norms
import test_gpu_int8 as int8
import test_gpu_route as routes
from combine_moe_layout_amd import binding as B
from products_ref import half_step

pytestmark = pytest.mark.gpu
BF = torch.bfloat16

# groups of 2, 3 and 60 experts meet in LDS, groups of 8, 32 and 256 by lanes of 4, 8 and 16 experts
GROUPS = [(4, 2, 1), (24, 8, 3), (64, 8, 3), (300, 5, 2), (512, 16, 4), (1024, 4, 2)]


@pytest.mark.parametrize("E,groups,topk_groups", GROUPS)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_group_sums_past_fp32(E, groups, topk_groups, score):
    """Biases whose sums by two leave fp32's range, above and below: groups go by the sums in fp64, and a
    group without any usable expert comes after all of them."""
    print("[gpu-edges] group sums", E, groups, topk_groups, score, flush=True)
    T, n = 60, E // groups
    for sign in (1.0, -1.0):
        for seed in range(4):
            g = routes.gen(E + seed)
            logits = torch.randn((T, E), device="cuda", generator=g)
            logits.view(T, groups, n)[1::3, 0] = -math.inf              # the group of the lowest index is dead
            bias = sign * (1.8e38 + 1.6e38 * torch.rand(E, device="cuda", generator=g))
            if E == 4 and seed == 0:
                bias = sign * torch.tensor([3e38, 2e38, 3e38, 3e38], device="cuda")
            router = B.EpRouter(E, 2, routes.SCORES[score], groups, topk_groups, 2)
            idx, _ = routes.route(logits, "fp32", router, bias)
            assert torch.equal(idx, ref.choice(logits, bias, 2, score, groups, topk_groups, 2)), (sign, seed)


@pytest.mark.parametrize("E,k,groups,topk_groups,group_top", [(64, 6, 1, 1, 1), (256, 8, 8, 3, 2), (250, 5, 5, 2, 1)])
def test_keys_that_fp64_cannot_tell(E, k, groups, topk_groups, group_top):
    """Sigmoids of logits past 37 are 1 in fp64, and scores beside a bias of 1e17 add nothing: with a bias
    those are ties and go to the lower index, without one the logits decide."""
    logits = 38 + 22 * torch.rand((30, E), device="cuda", generator=routes.gen(E))
    router = B.EpRouter(E, k, B.EP_SCORE_SIGMOID, groups, topk_groups, group_top)
    first = torch.arange(k, device="cuda").expand(30, k)
    for l, b in ((logits, 0.0), (logits, 0.5), (logits - 49, 1e17)):
        idx, _ = routes.route(l, "fp32", router, torch.full((E,), b, device="cuda"))
        assert torch.equal(idx, first), b
    if group_top == 1:
        idx, _ = routes.route(logits, "fp32", router)
        assert torch.equal(idx, ref.choice(logits, None, k, "sigmoid", groups, topk_groups, group_top))
        if groups == 1:
            assert torch.equal(idx, torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k])


@pytest.mark.parametrize("rows,H", [(5, 64), (9, 1032), (3, 8200), (3, 16392)])
def test_norm_gradients_of_large_rows(rows, H):
    """Rows whose root mean square is 1e12 to 1e16: sums of squares are in range, and the part of the
    gradient along the row is as right as any other."""
    print("[gpu-edges] large rows", rows, H, flush=True)
    for kind, scale in ((k, s) for k in ("all", "post", "add", "first") for s in (1e12, 1e14, 1e15, 1e16)):
        v = norms.inputs(rows, H, kind, BF)
        for n in ("y", "residual"):
            v[n] = None if v[n] is None else (v[n].float() * scale).to(BF)
        if v["d_normed"] is not None:
            v["d_out"] = None
        want, size = norms.exact_gradients(v, 0.75), norms.sizes(v, 0.75)
        got = norms.gradients(v, B.EP_BF16, BF, 0.75, B.EP_GRAD_F32)
        for k in got:
            norms.near(got[k], want[k], size[k], (kind, scale, k))


@pytest.mark.parametrize("rows,H", [(5, 64), (9, 1032), (3, 8200), (3, 16392)])
@pytest.mark.parametrize("eps", [1e-24, 1e-30, 1e-36])
def test_norm_gradients_of_empty_rows_with_a_small_eps(rows, H, eps, monkeypatch):
    """A row of zeros has an inverse root mean square of 1e12 to 1e18 and the gradients that go with it;
    the weights' gradients do not see it."""
    monkeypatch.setattr(norms, "EPS", eps)
    for kind in ("all", "post", "add", "first"):
        v = norms.inputs(rows, H, kind, BF)
        for n in ("y", "residual"):
            if v[n] is not None:
                v[n][1] = 0
        want, size = norms.exact_gradients(v, 0.75), norms.sizes(v, 0.75)
        got = norms.gradients(v, B.EP_BF16, BF, 0.75, B.EP_GRAD_F32)
        for k in got:
            norms.near(got[k], want[k], size[k], (kind, k))


@pytest.mark.parametrize("H", [64, 1032, 8200, 16392])
def test_gradient_by_an_infinite_y_without_its_norm(H):
    """Without norms d_y = gate d_out and d_residual = alpha d_out, whatever y holds."""
    v = norms.inputs(6, H, "gate", BF)
    v["pre"] = v["d_normed"] = None
    v["y"][1, 3], v["y"][2, H - 1], v["y"][4] = math.inf, math.nan, -math.inf
    got = norms.gradients(v, B.EP_BF16, BF, 0.75, only=("y", "residual"))
    assert torch.equal(got["y"], (v["d_out"].float() * v["gate"][:, None]).to(BF))
    assert torch.equal(got["residual"], (v["d_out"].float() * 0.75).to(BF))


@pytest.mark.parametrize("E,k", [(2, 1), (64, 1), (64, 2), (256, 8), (300, 3), (1000, 1)])
@pytest.mark.parametrize("name", ["fp32", "bf16"])
def test_gradient_of_confident_softmax(E, k, name):
    """Shares of all experts where the chosen have nearly everything:
       d_j = scale p_j (sum_i p_i (dw_j - dw_i) + q dw_j),  q = the share of those not chosen,
    and no digits are lost on the way.  A share is a term over a sum, (R + 4) and (R + n + 4) steps of
    2^-24 off, R the range of the logits (as for the weights in test_gpu_route); a term of the gradient
    has two of them, and k + 6 sums and products."""
    print("[gpu-edges] confident softmax", E, k, name, flush=True)
    code, dt = routes.TYPES[name]
    T, scale = 48, 2.5
    g = routes.gen(E + k)
    logits = torch.randn((T, E), device="cuda", generator=g)
    first = torch.randint(0, E, (T,), device="cuda", generator=g)
    gap = torch.linspace(8.0, 60.0, T, device="cuda")
    for j in range(k):
        logits[torch.arange(T, device="cuda"), (first + j * 7) % E] = gap + 0.5 * j
    logits = logits.to(dt)
    dw = torch.randn((T, k), device="cuda", generator=g)
    if k > 1:
        dw[::2, 1] = dw[::2, 0]                        # equal gradients: the difference is 0
        dw[1::4, 1] = dw[1::4, 0] * (1 + 2.0 ** -20)   # and nearly equal ones
    router = B.EpRouter(E, k, B.EP_SCORE_SOFTMAX, renormalize=False, scale=scale)
    idx, _ = routes.route(logits, name, router)
    given = [idx] if k < 3 else [idx, torch.cat([idx[:, :1], idx[:, :1], idx[:, 2:]], 1)]   # one of them twice
    for at in given:
        d = torch.full_like(logits, 7.0)
        B.ep_route_grad(dw, logits, at, router, d, code)
        p = ref.scores(logits, "softmax")
        by = torch.zeros_like(p).scatter_add_(1, at, dw.double())
        chosen = torch.zeros_like(p, dtype=torch.bool).scatter_(1, at, True)
        q = torch.where(chosen, 0.0, p).sum(1, keepdim=True)
        pc = torch.where(chosen, p, 0.0)
        want, size = torch.empty_like(p), torch.empty_like(p)
        for t in range(T):
            c = chosen[t].nonzero()[:, 0]
            diff = by[t, :, None] - by[t, None, c]
            want[t] = scale * p[t] * ((pc[t, c] * diff).sum(1) + q[t] * by[t])
            size[t] = scale * p[t] * ((pc[t, c] * diff.abs()).sum(1) + q[t] * by[t].abs())
        size = torch.where(chosen, size, scale * p * (pc * by.abs()).sum(1, keepdim=True))
        # (a sum of two dw is rounded: half a step of the largest, in both factors of a difference)
        dup = 0.0 if at is idx else 2 * ref.STEP * scale * pc * by.abs().amax(1, keepdim=True)
        tol = (2 * routes.steps(logits, E) + (k + 6) * ref.STEP) * size + dup + 2.0 ** -126
        tol = tol + half_step(want.abs() + tol, dt)
        assert ((d.double() - want).abs() <= tol).all(), ((d.double() - want).abs() / tol).max().item()


@pytest.mark.parametrize("T,K,N", [(3, 208, 48), (16, 400, 4096), (200, 144, 4096), (700, 1040, 4096), (2300, 272, 4096)])
@pytest.mark.parametrize("name", ["none", "swiglu"])
def test_large_and_small_scales(T, K, N, name):
    """Rows' scales of up to 2^117 with columns' as small, and the other way round: a sum times one scale
    leaves fp32's range, the result does not.  (Below fp32's normal range a product is off by half of 2^-149.)"""
    print("[gpu-edges] scales", T, K, N, name, flush=True)
    N = N // 2 if name == "swiglu" else N
    q, s, w, ws, bias = int8.operands(1, int8.width(N, name), K, T, T + N)
    q[T // 2] = 0
    out = torch.empty((T, N), dtype=BF, device="cuda")
    pre = torch.empty((T, int8.width(N, name)), dtype=BF, device="cuda")
    for half in (2.0 ** 64, 2.0 ** -52):
        ws2 = ws[0] / half / half
        for rows in (slice(None), slice(1, None, 2)):      # all of them, every other
            s2 = s.clone()
            s2[rows] = s2[rows] * half * half
            z, off = int8.exact_product(q, s2, w[0], ws2, bias[0])
            off = off + 2.0 ** -149
            B.ep_linear_int8(q, s2, w[0], ws2, out, act=int8.ACTS[name], bias=bias[0], preact=pre)
            # (the rows left as they were times 2^104: what they give is not of interest)
            at = slice(None) if half > 1 else rows
            int8.check(pre[at], z[at], off[at], "preact")
            int8.check(out[at], int8.act(z, name)[at], int8.act_error(z, off, name)[at], "out")
