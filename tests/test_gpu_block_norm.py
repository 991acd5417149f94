"""ep_block_norm and ep_block_norm_grad against the formulas in 64 bits.

Before its one rounding to 16 bits a value is the result of fp32 sums and products.  A sum over a row
passes at most 8 * 8 additions in a lane, 6 between lanes and 16 between waves, so it is within
90 steps of 2^-24 of the sum of its terms' magnitudes, and the inverse root of a sum of squares
within 48 steps of itself.  A gradient's term is a product of at most two such roots' powers (three
factors each), a sum and ten other factors or additions: within 512 steps of the sum of magnitudes
that `sizes` below takes through the same formulas.  A weight's gradient adds its sum over rows:
a workgroup's own (rows / 512 or fewer than 40 here), then at most 2048 / 16 + 16."""
import pytest
import torch

import block_ref as ref
from combine_moe_layout_amd import binding as B
from products_ref import half_step

pytestmark = pytest.mark.gpu
TYPES = {"bf16": (B.EP_BF16, torch.bfloat16), "fp16": (B.EP_F16, torch.float16)}
OFF = 512 * ref.STEP
EPS = 1e-6
KINDS = {  # post norm, gate, residual, pre norm, y
    "all": (True, True, True, True, True), "add": (False, False, True, True, True),
    "post": (True, False, True, False, True), "gate": (False, True, True, True, True),
    "alone": (True, True, False, True, True), "first": (False, False, True, True, False)}


def inputs(rows, H, kind, dt, seed=0):
    post, gate, residual, pre, y = KINDS[kind]
    g = torch.Generator(device="cuda")
    g.manual_seed(rows * 7 + H + seed)
    rn = lambda *s: torch.randn(s, device="cuda", generator=g)  # noqa: E731
    return dict(y=rn(rows, H).to(dt) if y else None, post=(1 + rn(H) * 0.1).to(dt) if post else None,
                gate=torch.rand(rows, device="cuda", generator=g) if gate else None,
                residual=rn(rows, H).mul_(2).to(dt) if residual else None,
                pre=(1 + rn(H) * 0.1).to(dt) if pre else None, d_out=rn(rows, H).to(dt),
                d_normed=rn(rows, H).to(dt) if pre else None)


def double(t):
    return None if t is None else t.double()


def near(got, want, size, what):
    tol = OFF * size
    tol = tol + half_step(want.abs() + tol, got.dtype)
    assert torch.isfinite(got).all(), what
    worst = ((got.double() - want).abs() / tol).max().item() if got.numel() else 0.0
    assert worst <= 1, (what, worst)


SHAPES = [(1, 8), (3, 24), (5, 512), (9, 520), (2, 1000), (37, 1024), (4, 1032), (600, 72), (17, 4096), (3, 7168),
          (2, 8200), (2, 16384), (2, 16392), (2, 32768), (1, 65536), (1300, 264)]


@pytest.mark.parametrize("rows,H", SHAPES)
@pytest.mark.parametrize("name", ["bf16", "fp16"])
def test_forward(rows, H, name):
    print("[gpu-norm]", rows, H, name, flush=True)
    code, dt = TYPES[name]
    for kind in KINDS:
        v = inputs(rows, H, kind, dt)
        alpha = 0.75
        out = torch.full((rows, H), 7.0, dtype=dt, device="cuda")
        normed = torch.full_like(out, 7.0) if v["pre"] is not None else None
        B.ep_block_norm(v["y"], v["residual"], out, code, EPS, v["post"], v["gate"], alpha, v["pre"], normed)
        d = {k: double(t) for k, t in v.items()}
        x, n = ref.block_norm(d["y"], d["residual"], EPS, d["post"], d["gate"], alpha, d["pre"])
        size, _ = ref.block_norm(None if d["y"] is None else d["y"].abs(), None if d["residual"] is None else d["residual"].abs(),
                                 EPS, d["post"], d["gate"], alpha)
        near(out, x, size, (kind, "out"))
        if normed is not None:
            inv = 1 / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)
            # x off by OFF * size moves its root mean square by no more than theirs
            spread = x.abs() * inv * torch.sqrt((size * size).mean(1, keepdim=True)) * inv
            near(normed, n, (size * inv + spread) * d["pre"].abs(), (kind, "normed"))
            again = torch.full_like(normed, 7.0)
            B.ep_block_norm(v["y"], v["residual"], None, code, EPS, v["post"], v["gate"], alpha, v["pre"], again)
            assert torch.equal(normed, again)


def exact_gradients(v, alpha):
    d = {k: double(t) for k, t in v.items()}
    leaves = {k: d[k].requires_grad_(True) for k in ("y", "post", "gate", "residual", "pre") if d[k] is not None}
    x, n = ref.block_norm(d["y"], d["residual"], EPS, d["post"], d["gate"], alpha, d["pre"])
    total = 0.0
    if d["d_out"] is not None:
        total = total + (x * d["d_out"]).sum()
    if n is not None and d["d_normed"] is not None:
        total = total + (n * d["d_normed"]).sum()
    total.backward()
    return {k: t.grad for k, t in leaves.items()}


def sizes(v, alpha):
    """The gradients' formulas with every term's magnitude."""
    d = {k: double(t) for k, t in v.items()}
    x, _ = ref.block_norm(d["y"], d["residual"], EPS, d["post"], d["gate"], alpha)
    big, _ = ref.block_norm(None if d["y"] is None else d["y"].abs(), None if d["residual"] is None else d["residual"].abs(),
                            EPS, d["post"], d["gate"], alpha)
    mean = lambda t: t.mean(1, keepdim=True)  # noqa: E731
    dx = torch.zeros_like(x) if d["d_out"] is None else d["d_out"].abs()
    out = {}
    if d["pre"] is not None:
        r = 1 / torch.sqrt(mean(x * x) + EPS)
        # how much x's own error counts: its terms may be larger than x
        big = torch.maximum(big, torch.sqrt(mean(big * big)))
        a = d["pre"].abs() * d["d_normed"].abs()
        worse = (big * r).amax(1, keepdim=True).clamp(min=1.0)
        dx = dx + (r * a + big * r ** 3 * mean(a * big)) * worse
        out["pre"] = (d["d_normed"].abs() * big * r * worse).sum(0)
    out["residual"] = abs(alpha) * dx
    if d["y"] is not None:
        y = d["y"].abs()
        gate = torch.ones_like(dx[:, :1]) if d["gate"] is None else d["gate"][:, None]
        if d["post"] is None:
            out["gate"], out["y"] = (dx * y).sum(1), gate * dx
        else:
            s, post = 1 / torch.sqrt(mean(y * y) + EPS), d["post"].abs()
            out["gate"] = (dx * y * s * post).sum(1)
            out["post"] = (gate * dx * y * s).sum(0)
            out["y"] = gate * (s * post * dx + y * s ** 3 * mean(post * dx * y))
    return out


def gradients(v, code, dt, alpha, flags=0, fill=7.0, only=None):
    rows, H = v["d_out"].shape if v["d_out"] is not None else v["d_normed"].shape
    gt = torch.float32 if flags & B.EP_GRAD_F32 else dt
    want = [k for k in ("y", "residual", "gate", "post", "pre") if v[k] is not None and (only is None or k in only)]
    got = {k: torch.full(v[k].shape, fill, dtype=gt if k in ("post", "pre") else v[k].dtype, device="cuda") for k in want}
    ws = torch.empty(B.ep_block_norm_grad_workspace_bytes(rows, H), dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)                       # scratch needs no initial value
    B.ep_block_norm_grad(v["d_out"], v["d_normed"], v["y"], v["residual"], code | flags, ws, EPS, v["post"], v["gate"],
                         alpha, v["pre"], d_y=got.get("y"), d_residual=got.get("residual"), d_gate=got.get("gate"),
                         d_post_weight=got.get("post"), d_pre_weight=got.get("pre"))
    torch.cuda.synchronize()
    return got


@pytest.mark.parametrize("rows,H", SHAPES)
@pytest.mark.parametrize("name", ["bf16", "fp16"])
def test_gradient(rows, H, name):
    print("[gpu-norm] gradient", rows, H, name, flush=True)
    code, dt = TYPES[name]
    for kind in KINDS:
        v = inputs(rows, H, kind, dt)
        want, size = exact_gradients(v, 0.75), sizes(v, 0.75)
        for flags in (0, B.EP_GRAD_F32):
            got = gradients(v, code, dt, 0.75, flags)
            for k in got:
                near(got[k], want[k], size[k], (kind, k, flags))
        again = gradients(v, code, dt, 0.75, B.EP_GRAD_F32)
        assert all(torch.equal(again[k], got[k]) for k in got)
        for only in (("y",), ("pre",), ("gate", "post"), ("residual",)):     # any of them alone
            some = gradients(v, code, dt, 0.75, B.EP_GRAD_F32, only=only) if any(v[k] is not None for k in only) else {}
            assert all(torch.equal(some[k], got[k]) for k in some), only


@pytest.mark.parametrize("name", ["bf16", "fp16"])
def test_one_incoming_gradient(name):
    code, dt = TYPES[name]
    for kind, gone in (("all", "d_out"), ("all", "d_normed"), ("add", "d_out"), ("alone", "d_out")):
        v = inputs(21, 1032, kind, dt)
        v[gone] = None
        if gone == "d_normed":
            v["pre"] = None
        want, size = exact_gradients(v, 1.0), sizes(v, 1.0)
        got = gradients(v, code, dt, 1.0)
        for k in got:
            near(got[k], want[k], size[k], (kind, gone, k))


@pytest.mark.parametrize("name", ["bf16", "fp16"])
@pytest.mark.parametrize("flags", [B.EP_GRAD_ACCUMULATE, B.EP_GRAD_ACCUMULATE | B.EP_GRAD_F32])
def test_accumulate(name, flags):
    code, dt = TYPES[name]
    v = inputs(45, 264, "all", dt)
    want, size = exact_gradients(v, 1.0), sizes(v, 1.0)
    got = gradients(v, code, dt, 1.0, flags, fill=3.0)
    for k in ("post", "pre"):
        near(got[k], want[k] + 3.0, size[k] + 3.0, k)
    none = dict(v, **{k: v[k][:0] for k in ("y", "residual", "gate", "d_out", "d_normed")})
    got = gradients(none, code, dt, 1.0, flags, fill=3.0)
    assert (got["post"] == 3).all() and (got["pre"] == 3).all()
    got = gradients(none, code, dt, 1.0, flags & ~B.EP_GRAD_ACCUMULATE, fill=3.0)
    assert (got["post"] == 0).all() and (got["pre"] == 0).all()


def test_gradient_against_differences():
    """(f(v + h d) - f(v - h d)) / 2h of f = sum(d_out x) + sum(d_normed n), fp16 results of the forward
    kernel summed in 64 bits.  Inputs move by whole multiples of 2^-4 (exact in fp16), h d = 2^-4 on
    one row in one direction: f is off by the rounding of 2 * 64 results of at most 4, 2^-10 each at
    most, times weights of at most 1: 2^-10 * 2 * 64 * 2 / 2h = 4; the truncation, h^2 / 6 of the third
    derivative along a direction of length 0.5 (64 entries of 1 times h), is below that.  The gradient
    along d is made large for it: the test asks for 4 of about 30."""
    H = 64
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    v = {"y": None, "post": None, "gate": None, "pre": torch.ones(H, device="cuda").half(),
         "residual": (torch.randint(-32, 33, (1, H), device="cuda", generator=g) / 16).half()}
    d_n = torch.sign(torch.randn((1, H), device="cuda", generator=g)).half()
    v["d_normed"], v["d_out"] = d_n, d_n.clone()
    step = d_n * 2.0 ** -4                       # along the gradient's main direction

    def f(residual):
        out, n = torch.empty_like(residual), torch.empty_like(residual)
        B.ep_block_norm(None, residual, out, B.EP_F16, EPS, pre_weight=v["pre"], normed=n)
        return ((out.double() + n.double()) * d_n.double()).sum().item()

    got = gradients(v, B.EP_F16, torch.float16, 1.0)["residual"]
    along = (got.double() * d_n.double()).sum().item()
    diff = (f(v["residual"] + step) - f(v["residual"] - step)) / (2 * 2.0 ** -4)
    assert abs(diff) > 30 and abs(diff - along) <= 4, (diff, along)


@pytest.mark.parametrize("rows,H", [(600, 16_392), (515, 32_768)])
def test_many_wide_rows(rows, H):
    """Rows that no workgroup holds in registers, several to a workgroup: whole, in place, and with one
    incoming gradient."""
    print("[gpu-norm] wide", rows, H, flush=True)
    for kind in KINDS:
        v = inputs(rows, H, kind, torch.bfloat16)
        want, size = exact_gradients(v, 0.75), sizes(v, 0.75)
        got = gradients(v, 0, torch.bfloat16, 0.75, B.EP_GRAD_F32)
        for k in got:
            near(got[k], want[k], size[k], (kind, k))
        again = gradients(v, 0, torch.bfloat16, 0.75, B.EP_GRAD_F32)
        assert all(torch.equal(again[k], got[k]) for k in got)
        for only in (("y",), ("pre",), ("gate", "post"), ("residual",)):
            some = gradients(v, 0, torch.bfloat16, 0.75, B.EP_GRAD_F32, only=only) if any(v[k] is not None for k in only) else {}
            assert all(torch.equal(some[k], got[k]) for k in some), only
        if kind == "all":
            a, b = v["d_out"].clone(), v["d_normed"].clone()
            B.ep_block_norm_grad(a, b, v["y"], v["residual"], 0, None, EPS, v["post"], v["gate"], 0.75, v["pre"], d_y=a,
                                 d_residual=b)
            assert torch.equal(a, got["y"]) and torch.equal(b, got["residual"])
            for gone in ("d_out", "d_normed"):
                w = dict(v)
                w[gone] = None
                if gone == "d_normed":
                    w["pre"] = None
                want, size = exact_gradients(w, 1.0), sizes(w, 1.0)
                got = gradients(w, 0, torch.bfloat16, 1.0)
                for k in got:
                    near(got[k], want[k], size[k], (gone, k))


def test_outputs_in_place():
    for kind in ("all", "add"):
        v = inputs(33, 1000, kind, torch.bfloat16)
        out, normed = torch.empty_like(v["y"]), torch.empty_like(v["y"])
        B.ep_block_norm(v["y"], v["residual"], out, 0, EPS, v["post"], v["gate"], 1.0, v["pre"], normed)
        y, res = v["y"].clone(), v["residual"].clone()
        B.ep_block_norm(y, res, res, 0, EPS, v["post"], v["gate"], 1.0, v["pre"], y)
        assert torch.equal(res, out) and torch.equal(y, normed)
        got = gradients(v, 0, torch.bfloat16, 1.0)
        a, b = v["d_out"].clone(), v["d_normed"].clone()
        B.ep_block_norm_grad(a, b, v["y"], v["residual"], 0, None, EPS, v["post"], v["gate"], 1.0, v["pre"], d_y=b,
                             d_residual=a)
        assert torch.equal(a, got["residual"]) and torch.equal(b, got["y"])


def test_nonfinite_rows_stay_apart():
    """A row with a NaN or an infinity is its own affair; rows of zeros are finite."""
    v = inputs(12, 520, "all", torch.bfloat16)
    clean = torch.empty_like(v["y"]), torch.empty_like(v["y"])
    B.ep_block_norm(v["y"], v["residual"], clean[0], 0, EPS, v["post"], v["gate"], 1.0, v["pre"], clean[1])
    v["y"][3, 17], v["residual"][5, 1] = float("nan"), float("inf")
    v["y"][7], v["residual"][7] = 0, 0
    out, normed = torch.empty_like(v["y"]), torch.empty_like(v["y"])
    B.ep_block_norm(v["y"], v["residual"], out, 0, EPS, v["post"], v["gate"], 1.0, v["pre"], normed)
    others = [r for r in range(12) if r not in (3, 5, 7)]
    assert torch.equal(out[others], clean[0][others]) and torch.equal(normed[others], clean[1][others])
    assert torch.isnan(out[3]).all() and torch.isinf(out[5, 1]) and (out[7] == 0).all() and (normed[7] == 0).all()


def test_offsets_past_32_bits():
    """Tensors of more than 2^32 elements: the last rows come out as by themselves."""
    rows, H = 70_000, 65_536
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    last = torch.randn((3, H), device="cuda", generator=g).bfloat16()
    w = torch.randn(H, device="cuda", generator=g).bfloat16()
    y = torch.ones((rows, H), dtype=torch.bfloat16, device="cuda")
    y[-3:] = last
    out, few = torch.empty_like(y), torch.empty_like(last)
    B.ep_block_norm(y, None, out, 0, EPS, post_weight=w)
    B.ep_block_norm(last, None, few, 0, EPS, post_weight=w)
    assert torch.equal(out[-3:], few)
    B.ep_block_norm_grad(y, None, y, None, 0, None, EPS, post_weight=w, d_y=out)
    B.ep_block_norm_grad(last, None, last, None, 0, None, EPS, post_weight=w, d_y=few)
    assert torch.equal(out[-3:], few)


def test_no_rows():
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    B.ep_block_norm(e, None, torch.empty_like(e), 0)
    B.ep_block_norm_grad(e, None, e, None, 0, d_y=torch.empty_like(e))
    torch.cuda.synchronize()
