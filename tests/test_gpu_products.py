"""The experts' products, the dense product and their gradients against 64 bits (products_ref.py
derives the tolerances): types, activations, both receive layouts, sizes from one row to several
tiles, reductions that end inside a stage, experts without rows, rows that nobody uses."""
import pytest
import torch

from combine_moe_layout_amd import binding as B
from products_ref import (ACTS, SUM, TYPES, act, act_error, act_grad, act_grad_error, check, fp8_group_error,
                          segments, used_rows, width)

pytestmark = pytest.mark.gpu


def note(*a):
    print("[gpu-products]", *a, flush=True)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(shape, dt, g, scale=1.0):
    return (torch.randn(shape, device="cuda", generator=g) * scale).to(dt)


def layout(T, k, E, cap, g, masked=0.0, skew=False):
    if T:
        score = torch.rand((T, E), device="cuda", generator=g)
        if skew:
            score[:, 0] += 1
            score[:, E // 2:] -= 1
        idx = score.topk(k, 1).indices
        idx[torch.rand((T, k), device="cuda", generator=g) < masked] = -1
    else:
        idx = torch.zeros((0, k), dtype=torch.int64, device="cuda")
    lay = B.EpLayout(T, k, E, 1, cap)
    B.ep_get_layout(idx, lay)
    return lay


# (T, k, E, capacity, masked, skew): ragged, padded with drops, one expert, more experts than rows,
# experts without rows, nothing routed, no tokens
LAYOUTS = [(37, 3, 5, 0, 0.2, False), (50, 4, 8, 9, 0.0, True), (300, 1, 1, 0, 0.0, False),
           (5, 2, 70, 0, 0.0, False), (140, 2, 12, 0, 0.0, True), (9, 2, 4, 3, 1.0, False),
           (0, 2, 4, 0, 0.0, False)]


@pytest.mark.parametrize("name", ["bf16", "fp16"])
@pytest.mark.parametrize("a", list(ACTS))
@pytest.mark.parametrize("lay_i", range(len(LAYOUTS)))
def test_expert_gemm(name, a, lay_i):
    note("expert_gemm", name, a, LAYOUTS[lay_i])
    dtype, dt = TYPES[name]
    g = gen(lay_i)
    T, k, E, cap, masked, skew = LAYOUTS[lay_i]
    lay = layout(T, k, E, cap, g, masked, skew)
    R = lay.num_recv_rows
    K, N = [(64, 72), (200, 136), (8, 8), (264, 40), (1024, 264), (72, 16), (64, 64)][lay_i]
    W = width(N, a)
    used = used_rows(lay)
    x = randn((R, K), dt, g)
    x[~used] = float("nan")               # rows that nobody uses are not read
    w = randn((E, W, K), dt, g, K ** -0.5)
    bias = randn((E, W), dt, g) if lay_i % 2 == 0 else None
    out = torch.full((R, N), 7.0, dtype=dt, device="cuda")
    pre = torch.full((R, W), 7.0, dtype=dt, device="cuda")
    B.ep_expert_gemm(x, w, lay, out, dtype, act=ACTS[a], bias=bias, preact=pre)
    torch.cuda.synchronize()
    assert (out[~used] == 7).all() and (pre[~used] == 7).all()
    for e, (b, n) in enumerate(segments(lay)):
        if not n:
            continue
        xe, we = x[b:b + n].double(), w[e].double()
        z, s = xe @ we.T, xe.abs() @ we.abs().T
        if bias is not None:
            z, s = z + bias[e].double(), s + bias[e].double().abs()
        dz = (K + 1) * SUM * s
        check(pre[b:b + n], z, dz, "preact of expert %d" % e)
        check(out[b:b + n], act(z, a), act_error(z, dz, a), "out of expert %d" % e)
    if bias is None:                       # the same without the pre-activation
        again = torch.full((R, N), 7.0, dtype=dt, device="cuda")
        B.ep_expert_gemm(x, w, lay, again, dtype, act=ACTS[a])
        assert torch.equal(again, out)


@pytest.mark.parametrize("name", ["bf16", "fp16"])
@pytest.mark.parametrize("T,K,N", [(700, 320, 520), (257, 2048, 256), (2100, 136, 1032)])
def test_expert_gemm_large_groups(name, T, K, N):
    """Groups of several 128- and 256-row tiles; swiglu."""
    note("large groups", name, T, K, N)
    dtype, dt = TYPES[name]
    g = gen(T)
    lay = layout(T, 2, 3, 0, g, 0.0, True)
    R, E = lay.num_recv_rows, 3
    x, w = randn((R, K), dt, g), randn((E, 2 * N, K), dt, g, K ** -0.5)
    out = torch.zeros((R, N), dtype=dt, device="cuda")
    B.ep_expert_gemm(x, w, lay, out, dtype, act=B.EP_ACT_SWIGLU)
    for e, (b, n) in enumerate(segments(lay)):
        xe, we = x[b:b + n].double(), w[e].double()
        z, s = xe @ we.T, xe.abs() @ we.abs().T
        check(out[b:b + n], act(z, "swiglu"), act_error(z, K * SUM * s, "swiglu"), "expert %d" % e)


@pytest.mark.parametrize("name", ["bf16", "fp16"])
@pytest.mark.parametrize("T,k,E,cap,D,F", [(1500, 2, 6, 0, 136, 5440), (900, 2, 4, 500, 312, 72),
                                           (2000, 1, 5, 0, 264, 136), (900, 2, 4, 500, 264, 8200)])
def test_expert_products_in_tiles_of_every_size(name, T, k, E, cap, D, F):
    """256 tiles of 256 x 256 and more, or a few of 64 x 64, of every kind: up with a bias, its gradients by rows and by
    weights (adding to what was there, and in the operands' type)."""
    note("large tiles", name, T, k, E, cap, D, F)
    dtype, dt = TYPES[name]
    g = gen(T)
    lay = layout(T, k, E, cap, g, 0.05, cap > 0)
    R, used = lay.num_recv_rows, used_rows(lay)
    x, w, bias = randn((R, D), dt, g), randn((E, 2 * F, D), dt, g, D ** -0.5), randn((E, 2 * F), dt, g)
    dy, back, pre_in = randn((R, D), dt, g), randn((E, D, F), dt, g, D ** -0.5), randn((R, 2 * F), dt, g)
    x[~used] = float("nan")
    dy[~used] = float("inf")
    out, pre = (torch.full((R, n), 7.0, dtype=dt, device="cuda") for n in (F, 2 * F))
    B.ep_expert_gemm(x, w, lay, out, dtype, act=B.EP_ACT_SWIGLU, bias=bias, preact=pre)
    dx = torch.full((R, 2 * F), 7.0, dtype=dt, device="cuda")
    B.ep_expert_gemm_grad_x(dy, back, lay, dx, dtype, act=B.EP_ACT_SWIGLU, preact=pre_in)
    wide = randn((R, 2 * F), dt, g)
    wide[~used] = float("nan")
    dw, db = torch.full((E, 2 * F, D), 7.0, dtype=dt, device="cuda"), torch.full((E, 2 * F), 7.0, dtype=dt, device="cuda")
    B.ep_expert_gemm_grad_w(wide, x, lay, dw, dtype, dbias=db)
    old = randn((E, D, 2 * F), torch.float32, g)
    acc = old.clone()
    B.ep_expert_gemm_grad_w(x, wide, lay, acc, dtype | B.EP_GRAD_F32 | B.EP_GRAD_ACCUMULATE)
    torch.cuda.synchronize()
    for t in (out, pre, dx):
        assert (t[~used] == 7).all()
    for e, (b, n) in enumerate(segments(lay)):
        xe, ye, we, v = x[b:b + n].double(), wide[b:b + n].double(), w[e].double(), back[e].double()
        z, m = xe @ we.T + bias[e].double(), xe.abs() @ we.abs().T + bias[e].double().abs()
        dz = (D + 1) * SUM * m
        check(pre[b:b + n], z, dz, "preact of expert %d" % e)
        check(out[b:b + n], act(z, "swiglu"), act_error(z, dz, "swiglu"), "out of expert %d" % e)
        de, p = dy[b:b + n].double(), pre_in[b:b + n].double()
        d, dd = de @ v, D * SUM * (de.abs() @ v.abs())
        check(dx[b:b + n], act_grad(d, p, "swiglu"), act_grad_error(d, dd, p, "swiglu"), "dx of expert %d" % e)
        ref, m = ye.T @ xe, ye.abs().T @ xe.abs()
        check(dw[e], ref, n * SUM * m, "dweights of expert %d" % e)
        check(db[e], ye.sum(0), n * SUM * ye.abs().sum(0), "dbias of expert %d" % e)
        o = old[e].double()
        check(acc[e], o + ref.T, (n + 1) * SUM * (m.T + o.abs()), "accumulated dweights of expert %d" % e)


# ------------------------------------------------------------------------------------- FP8
def quant_rows(x, block):
    """E4M3 codes and per-block scales of rows: fp32 per 128, or E8M0 per 32 (with widely spread scales)."""
    b = x.reshape(x.shape[0], -1, block)
    a = b.abs().amax(-1).clamp(min=1e-4)
    if block == 32:
        e = torch.floor(torch.log2(a)) - 8
        return ((b / torch.exp2(e)[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                .reshape(x.shape)), (e + 127).to(torch.uint8)
    s = a / 448
    return (b / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).reshape(x.shape), s


def codes(q):
    return q.view(torch.float8_e4m3fn).double()


@pytest.mark.parametrize("kind", ["fp8", "pow2", "mn", "mxfp8"])
@pytest.mark.parametrize("a,bias", [("none", True), ("swiglu", False), ("gelu", True)])
@pytest.mark.parametrize("T,k,E,cap,K,N", [(37, 3, 5, 0, 128, 128), (50, 4, 8, 9, 640, 256),
                                             (3, 2, 70, 0, 256, 128), (900, 1, 2, 0, 384, 384),
                                             # few rows on average, many for some; large tiles
                                             (400, 2, 70, 0, 256, 640), (900, 1, 2, 0, 384, 2304),
                                             (700, 2, 3, 300, 640, 4608), (1500, 1, 1, 0, 128, 2944),
                                             # scales four stages at a time
                                             (37, 3, 5, 0, 512, 128), (50, 4, 8, 9, 2560, 256),
                                             (900, 1, 2, 0, 512, 2304), (1500, 1, 1, 0, 2560, 2944)])
def test_expert_gemm_fp8(kind, a, bias, T, k, E, cap, K, N):
    note("fp8", kind, a, T, k, E, cap, K, N)
    g = gen(T + K)
    mx = kind == "mxfp8"
    dtype = {"fp8": B.EP_FP8_E4M3, "pow2": B.EP_FP8_E4M3_POW2, "mxfp8": B.EP_MXFP8_E4M3,
             "mn": B.EP_FP8_E4M3 | B.EP_SCALES_MN_MAJOR}[kind]
    lay = layout(T, k, E, cap, g, 0.1 if cap else 0.0, T > 100)
    R, W = lay.num_recv_rows, width(N, a)
    # magnitudes that differ from block to block, so that a scale out of place shows
    spread = torch.exp2(torch.randint(-3, 4, (R, K // 32), device="cuda", generator=g).float())
    xf = torch.randn((R, K), device="cuda", generator=g) * spread.repeat_interleave(32, 1)
    used = used_rows(lay)
    q, s = quant_rows(xf, 32 if mx else 128)
    if kind == "pow2":
        s = torch.exp2(torch.ceil(torch.log2(s)))
    q[~used] = 0x7F                        # NaN codes in rows that nobody uses
    wf = torch.randn((E, W, K), device="cuda", generator=g) * K ** -0.5
    wf = wf * torch.exp2(torch.randint(-2, 3, (E, W // 128, K // 128), device="cuda", generator=g).float()
                         ).repeat_interleave(128, 1).repeat_interleave(128, 2)
    if mx:
        wq, ws = quant_rows(wf.reshape(E * W, K), 32)
        wq, ws = wq.reshape(E, W, K), ws.reshape(E, W, K // 32)
        wd = codes(wq) * torch.exp2(ws.double() - 127).repeat_interleave(32, 2)
        xd = codes(q) * torch.exp2(s.double() - 127).repeat_interleave(32, 1)
    else:
        blk = wf.reshape(E, W // 128, 128, K // 128, 128)
        ws = blk.abs().amax((2, 4)) / 448
        wq = (blk / ws[:, :, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).reshape(E, W, K)
        wd = codes(wq) * ws.double().repeat_interleave(128, 1).repeat_interleave(128, 2)
        xd = codes(q) * s.double().repeat_interleave(128, 1)
    bv = randn((E, W), torch.bfloat16, g) if bias else None
    out = torch.full((R, N), 7.0, dtype=torch.bfloat16, device="cuda")
    pre = torch.full((R, W), 7.0, dtype=torch.bfloat16, device="cuda")
    sc = s.t().contiguous() if kind == "mn" else s
    B.ep_expert_gemm(q, wq, lay, out, dtype, act=ACTS[a], x_scales=sc, weight_scales=ws, bias=bv, preact=pre)
    torch.cuda.synchronize()
    assert (out[~used] == 7).all() and (pre[~used] == 7).all()
    for e, (b, n) in enumerate(segments(lay)):
        if not n:
            continue
        xe, we = xd[b:b + n], wd[e]
        z, m = xe @ we.T, xe.abs() @ we.abs().T
        if bv is not None:
            z, m = z + bv[e].double(), m + bv[e].double().abs()
        # + 4: the scales' product and its use
        dz = (K + 4) * SUM * m + fp8_group_error(xe, we)
        check(pre[b:b + n], z, dz, "preact of expert %d" % e)
        check(out[b:b + n], act(z, a), act_error(z, dz, a), "out of expert %d" % e)


def test_expert_gemm_reads_what_dispatch_writes():
    """Rows and scales as ep_dispatch left them, every FP8 kind and both scale layouts."""
    g = gen(5)
    T, k, E, K, N = 61, 2, 6, 384, 128
    x = randn((T, K), torch.bfloat16, g)
    lay = layout(T, k, E, 0, g)
    R = lay.num_recv_rows
    for kind in (B.EP_FP8_E4M3, B.EP_FP8_E4M3_POW2, B.EP_MXFP8_E4M3, B.EP_FP8_E4M3 | B.EP_SCALES_MN_MAJOR):
        note("after dispatch", kind)
        mx, mn = kind == B.EP_MXFP8_E4M3, bool(kind & B.EP_SCALES_MN_MAJOR)
        q = torch.zeros((R, K), dtype=torch.uint8, device="cuda")
        shape = (R, K // 32) if mx else (K // 128, R) if mn else (R, K // 128)
        s = torch.zeros(shape, dtype=torch.uint8 if mx else torch.float32, device="cuda")
        B.ep_dispatch(x, lay, kind, q, s)
        w = torch.randint(0, 0x70, (E, N, K), device="cuda", generator=g, dtype=torch.uint8)
        ws = (torch.full((E, N, K // 32), 120, dtype=torch.uint8, device="cuda") if mx else
              torch.full((E, N // 128, K // 128), 2.0 ** -7, device="cuda"))
        out = torch.zeros((R, N), dtype=torch.bfloat16, device="cuda")
        B.ep_expert_gemm(q, w, lay, out, kind, x_scales=s, weight_scales=ws)
        rows = s.t() if mn else s
        xd = codes(q) * (torch.exp2(rows.double() - 127).repeat_interleave(32, 1) if mx
                         else rows.double().repeat_interleave(128, 1))
        wd = codes(w) * 2.0 ** -7
        for e, (b, n) in enumerate(segments(lay)):
            z, m = xd[b:b + n] @ wd[e].T, xd[b:b + n].abs() @ wd[e].abs().T
            check(out[b:b + n], z, (K + 4) * SUM * m + fp8_group_error(xd[b:b + n], wd[e]),
                  "kind %d expert %d" % (kind, e))


# -------------------------------------------------------------------------------- gradients
@pytest.mark.parametrize("name", ["bf16", "fp16"])
@pytest.mark.parametrize("a", list(ACTS))
@pytest.mark.parametrize("lay_i", range(len(LAYOUTS)))
def test_expert_gemm_grad_x(name, a, lay_i):
    note("grad_x", name, a, LAYOUTS[lay_i])
    dtype, dt = TYPES[name]
    g = gen(100 + lay_i)
    T, k, E, cap, masked, skew = LAYOUTS[lay_i]
    lay = layout(T, k, E, cap, g, masked, skew)
    R = lay.num_recv_rows
    K, N = [(72, 64), (136, 200), (8, 8), (40, 264), (264, 1024), (16, 72), (64, 64)][lay_i]
    used = used_rows(lay)
    dy, w = randn((R, N), dt, g), randn((E, N, K), dt, g, N ** -0.5)
    dy[~used] = float("nan")
    pre = None if a == "none" else randn((R, width(K, a)), dt, g)
    dx = torch.full((R, width(K, a)), 7.0, dtype=dt, device="cuda")
    B.ep_expert_gemm_grad_x(dy, w, lay, dx, dtype, act=ACTS[a], preact=pre)
    torch.cuda.synchronize()
    assert (dx[~used] == 7).all()
    for e, (b, n) in enumerate(segments(lay)):
        if not n:
            continue
        d, m = dy[b:b + n].double() @ w[e].double(), dy[b:b + n].double().abs() @ w[e].double().abs()
        z = None if pre is None else pre[b:b + n].double()
        dd = N * SUM * m
        check(dx[b:b + n], d if z is None else act_grad(d, z, a),
              dd if z is None else act_grad_error(d, dd, z, a), "dx of expert %d" % e)


@pytest.mark.parametrize("name", ["bf16", "fp16"])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("lay_i", range(len(LAYOUTS)))
def test_expert_gemm_grad_w(name, f32, lay_i):
    note("grad_w", name, f32, LAYOUTS[lay_i])
    dtype, dt = TYPES[name]
    g = gen(200 + lay_i)
    T, k, E, cap, masked, skew = LAYOUTS[lay_i]
    lay = layout(T, k, E, cap, g, masked, skew)
    R = lay.num_recv_rows
    K, N = [(64, 72), (200, 136), (8, 8), (264, 40), (520, 264), (72, 16), (64, 64)][lay_i]
    used = used_rows(lay)
    dy, x = randn((R, N), dt, g), randn((R, K), dt, g)
    dy[~used] = float("nan")
    x[~used] = float("inf")
    gt = torch.float32 if f32 else dt
    flag = dtype | (B.EP_GRAD_F32 if f32 else 0)
    dw = torch.full((E, N, K), 7.0, dtype=gt, device="cuda")
    db = torch.full((E, N), 7.0, dtype=gt, device="cuda")
    B.ep_expert_gemm_grad_w(dy, x, lay, dw, flag, dbias=db)
    old_w, old_b = randn((E, N, K), gt, g), randn((E, N), gt, g)
    acc_w, acc_b = old_w.clone(), old_b.clone()
    B.ep_expert_gemm_grad_w(dy, x, lay, acc_w, flag | B.EP_GRAD_ACCUMULATE, dbias=acc_b)
    torch.cuda.synchronize()
    for e, (b, n) in enumerate(segments(lay)):
        d, v = dy[b:b + n].double(), x[b:b + n].double()
        ref, m = d.T @ v, d.abs().T @ v.abs()
        check(dw[e], ref, n * SUM * m, "dweights of expert %d" % e)
        check(db[e], d.sum(0), n * SUM * d.abs().sum(0), "dbias of expert %d" % e)
        ow, ob = old_w[e].double(), old_b[e].double()
        check(acc_w[e], ow + ref, (n + 1) * SUM * (m + ow.abs()), "accumulated dweights of expert %d" % e)
        check(acc_b[e], ob + d.sum(0), (n + 1) * SUM * (d.abs().sum(0) + ob.abs()), "accumulated dbias")


def test_neighbours_infinities_stay_with_their_expert():
    """A NaN or infinity in one expert's rows or matrix does not reach another expert's results,
    though they share tiles' stages."""
    g = gen(9)
    dt, dtype = torch.bfloat16, B.EP_BF16
    lay = layout(45, 1, 3, 0, g)
    seg = segments(lay)
    R, K, N = lay.num_recv_rows, 72, 40
    x, w, dy = randn((R, K), dt, g), randn((3, N, K), dt, g), randn((R, N), dt, g)
    outs = []
    for bad in (False, True):
        if bad:
            b, n = seg[1]
            x[b:b + n, ::3] = float("inf")
            dy[b:b + n] = float("nan")
            w[1] = float("nan")
        out, dx = torch.zeros((R, N), dtype=dt, device="cuda"), torch.zeros((R, K), dtype=dt, device="cuda")
        dw, db = torch.zeros((3, N, K), dtype=dt, device="cuda"), torch.zeros((3, N), dtype=dt, device="cuda")
        B.ep_expert_gemm(x, w, lay, out, dtype)
        B.ep_expert_gemm_grad_x(dy, w, lay, dx, dtype)
        B.ep_expert_gemm_grad_w(dy, x, lay, dw, dtype, dbias=db)
        outs.append((out, dx, dw, db))
    for e in (0, 2):
        b, n = seg[e]
        for i in (0, 1):
            assert torch.equal(outs[0][i][b:b + n], outs[1][i][b:b + n])
        for i in (2, 3):
            assert torch.equal(outs[0][i][e], outs[1][i][e])
    b, n = seg[1]
    assert torch.isnan(outs[1][0][b:b + n]).all() and torch.isnan(outs[1][2][1]).all()


# ------------------------------------------------------------------------------------- dense
@pytest.mark.parametrize("name", ["bf16", "fp16"])
@pytest.mark.parametrize("a", list(ACTS))
@pytest.mark.parametrize("T,K,N", [(1, 64, 64), (3, 1032, 24), (16, 8, 8), (17, 520, 264), (64, 2048, 40),
                                     (129, 72, 136), (300, 256, 520),
                                     # chunks that go round every ring, rows at the block edges
                                     (15, 4616, 40), (32, 4616, 24), (33, 4616, 136), (63, 584, 72),
                                     (65, 1544, 72), (200, 2056, 200),
                                     # 128 x 128 and 256 x 256 tiles
                                     (130, 200, 5640), (2100, 136, 7240), (2304, 72, 7424)])
def test_linear(name, a, T, K, N):
    note("linear", name, a, T, K, N)
    dtype, dt = TYPES[name]
    g = gen(T + K)
    W = width(N, a)
    x, w = randn((T, K), dt, g), randn((W, K), dt, g, K ** -0.5)
    bias, res = randn((W,), dt, g), randn((T, N), dt, g)
    z, m = x.double() @ w.double().T, x.double().abs() @ w.double().abs().T
    for use_bias, use_res in ((True, True), (False, False), (True, False), (False, True)):
        out = torch.zeros((T, N), dtype=dt, device="cuda")
        pre = torch.zeros((T, W), dtype=dt, device="cuda") if use_bias else None
        B.ep_linear(x, w, out, dtype, act=ACTS[a], bias=bias if use_bias else None,
                    residual=res if use_res else None, preact=pre)
        zb = z + bias.double() if use_bias else z
        dz = (K + 1) * SUM * (m + (bias.double().abs() if use_bias else 0))
        ref, err = act(zb, a), act_error(zb, dz, a)
        if use_res:
            ref, err = ref + res.double(), err + SUM * (ref.abs() + err + res.double().abs())
        check(out, ref, err, "out")
        if pre is not None:
            check(pre, zb, dz, "preact")
    into = res.clone()                     # out may be the residual itself
    B.ep_linear(x, w, into, dtype, act=ACTS[a], residual=into)
    want = torch.zeros_like(into)
    B.ep_linear(x, w, want, dtype, act=ACTS[a], residual=res)
    assert torch.equal(into, want)


@pytest.mark.parametrize("name", ["bf16", "fp16"])
@pytest.mark.parametrize("a", list(ACTS))
@pytest.mark.parametrize("T,K,N", [(1, 64, 64), (5, 24, 1032), (17, 264, 520), (300, 520, 256), (0, 64, 72),
                                     (2100, 7240, 200), (200, 7240, 2104),
                                     # waves that share the reduction; none left over in the last chunk
                                     (70, 392, 1160), (1100, 72, 136), (65, 1000, 256), (256, 64, 72)])
def test_linear_gradients(name, a, T, K, N):
    note("linear grads", name, a, T, K, N)
    dtype, dt = TYPES[name]
    g = gen(T + K + 7)
    dy, w, x = randn((T, N), dt, g), randn((N, K), dt, g, N ** -0.5), randn((T, K), dt, g)
    Kw = width(K, a)
    pre = None if a == "none" else randn((T, Kw), dt, g)
    dx = torch.zeros((T, Kw), dtype=dt, device="cuda")
    dw = torch.full((N, K), 7.0, device="cuda")
    db = torch.full((N,), 7.0, device="cuda")
    B.ep_linear_grad_x(dy, w, dx, dtype, act=ACTS[a], preact=pre)
    B.ep_linear_grad_w(dy, x, dw, dtype | B.EP_GRAD_F32, dbias=db)
    d, m = dy.double() @ w.double(), dy.double().abs() @ w.double().abs()
    z = None if pre is None else pre.double()
    check(dx, d if z is None else act_grad(d, z, a),
          N * SUM * m if z is None else act_grad_error(d, N * SUM * m, z, a), "dx")
    check(dw, dy.double().T @ x.double(), T * SUM * (dy.double().abs().T @ x.double().abs()), "dweights")
    check(db, dy.double().sum(0), T * SUM * dy.double().abs().sum(0), "dbias")
    # the activation's own gradient, apart from any product
    h = randn((T, K), dt, g)
    if pre is not None:
        dz = torch.zeros((T, Kw), dtype=dt, device="cuda")
        B.ep_act_grad(h, pre, dz, dtype, ACTS[a])
        hd = h.double()
        check(dz, act_grad(hd, z, a), act_grad_error(hd, 0 * hd, z, a), "dz")


@pytest.mark.parametrize("a", ["gelu", "silu", "swiglu"])
def test_gradients_against_differences(a):
    """Directional derivatives of the 64-bit forward pass against the kernels' gradients: a central
    difference with step h is off by h^2/6 times a third derivative (below 1e-6 here) and the
    kernels' gradients by half a step of bf16 each and the sums' errors (inside 2^-8)."""
    g = gen(31)
    dt, dtype = torch.bfloat16, B.EP_BF16
    T, K, N, M = 33, 40, 24, 48
    x, w1 = randn((T, K), dt, g), randn((width(N, a), K), dt, g, K ** -0.5)
    b1, w2, dout = randn((width(N, a),), dt, g), randn((M, N), dt, g, N ** -0.5), randn((T, M), dt, g)
    h, pre = torch.zeros((T, N), dtype=dt, device="cuda"), torch.zeros((T, width(N, a)), dtype=dt, device="cuda")
    B.ep_linear(x, w1, h, dtype, act=ACTS[a], bias=b1, preact=pre)
    dz = torch.zeros_like(pre)
    B.ep_linear_grad_x(dout, w2, dz, dtype, act=ACTS[a], preact=pre)
    dx = torch.zeros_like(x)
    B.ep_linear_grad_x(dz, w1, dx, dtype)
    dw1, db1 = torch.zeros((width(N, a), K), device="cuda"), torch.zeros((width(N, a),), device="cuda")
    B.ep_linear_grad_w(dz, x, dw1, dtype | B.EP_GRAD_F32, dbias=db1)
    dw2 = torch.zeros((M, N), device="cuda")
    B.ep_linear_grad_w(dout, h, dw2, dtype | B.EP_GRAD_F32)

    def loss(x_, w1_, b1_, w2_):
        return (act(x_ @ w1_.T + b1_, a) @ w2_.T * dout.double()).sum()

    leaves = [x.double(), w1.double(), b1.double(), w2.double()]
    grads = [dx.double(), dw1.double(), db1.double(), dw2.double()]
    for i in range(4):
        d = torch.randn(leaves[i].shape, device="cuda", generator=g, dtype=torch.float64)
        step = 1e-4
        up, down = list(leaves), list(leaves)
        up[i], down[i] = leaves[i] + step * d, leaves[i] - step * d
        diff = ((loss(*up) - loss(*down)) / (2 * step)).item()
        got = (grads[i] * d).sum().item()
        # at most four roundings to bf16 lie on the way to a gradient (preact, h or dz, dx), each
        # half a step of the terms that it rounds: 4 * 2^-8 of the sum of magnitudes
        bound = 4 * 2.0 ** -8 * magnitude(i, leaves, dout.double(), a, d)
        assert abs(diff - got) <= bound + 1e-5 * abs(diff), (i, diff, got, bound)


def magnitude(i, leaves, dout, a, d):
    """Sum of the magnitudes that the i-th gradient's directional derivative adds up."""
    x, w1, b1, w2 = [t.abs() for t in leaves]
    z = leaves[0] @ leaves[1].T + leaves[2]
    dh = dout.abs() @ w2
    if a == "swiglu":
        n = z.shape[1] // 2
        dz = torch.cat([dh * 1.1 * (z[:, n:].abs() + 1), dh * (z[:, :n].abs() + 1)], 1)
    else:
        dz = dh * 1.13 * (1 + z.abs())
    if i == 0:
        return (dz @ w1 * d.abs()).sum().item()
    if i == 1:
        return (dz.T @ x * d.abs()).sum().item()
    if i == 2:
        return (dz.sum(0) * d.abs()).sum().item()
    return (dout.abs().T @ (act(z, a).abs() + 1) * d.abs()).sum().item()


# --------------------------------------------------------------------------- combine's gradient
@pytest.mark.parametrize("name", ["bf16", "fp16"])
@pytest.mark.parametrize("T,k,E,cap,H,masked", [(1, 1, 2, 0, 8, 0.0), (37, 3, 5, 0, 200, 0.3), (50, 8, 16, 11, 1024, 0.0),
                                                 (300, 2, 4, 0, 8200, 0.0), (130, 9, 12, 0, 64, 0.1),
                                                 (1100, 4, 8, 0, 512, 0.0), (6, 2, 4, 2, 72, 1.0), (0, 2, 4, 0, 64, 0.0),
                                                 (1000, 5, 8, 0, 72, 0.1),
                                                 # more than 128 MiB of rows
                                                 (6000, 3, 6, 0, 4104, 0.1), (2500, 8, 16, 1100, 4096, 0.0)])
def test_combine_grad(name, T, k, E, cap, H, masked):
    note("combine_grad", name, T, k, E, cap, H)
    dtype, dt = TYPES[name]
    g = gen(T + H)
    lay = layout(T, k, E, cap, g, masked)
    R = lay.num_recv_rows
    dout, y, w = randn((T, H), dt, g), randn((R, H), dt, g), torch.rand((T, k), device="cuda", generator=g)
    used = used_rows(lay)
    y[~used] = float("nan")
    dy = torch.full((R, H), 7.0, dtype=dt, device="cuda")
    dw = torch.full((T, k), 7.0, device="cuda")
    B.ep_combine_grad(dout, y, w, lay, dy, dw, dtype)
    torch.cuda.synchronize()
    assert (dy[~used] == 7).all()
    slot = lay.slot_idx.long()
    for j in range(k):
        t = torch.nonzero(slot[:, j] >= 0)[:, 0]
        r = slot[t, j]
        d, v = dout[t].double(), y[r].double()
        ref = w[t, j].double()[:, None] * d
        check(dy[r], ref, SUM * ref.abs(), "dy of choice %d" % j)
        check(dw[t, j], (d * v).sum(1), H * SUM * (d * v).abs().sum(1), "dw of choice %d" % j)
        gone = torch.nonzero(slot[:, j] < 0)[:, 0]
        assert (dw[gone, j] == 0).all()
    only = torch.full((R, H), 7.0, dtype=dt, device="cuda")
    B.ep_combine_grad(dout, None, w, lay, only, None, dtype)
    assert torch.equal(only, dy)


# ------------------------------------------------------------------- matrices beyond 2^32 bytes
@pytest.mark.parametrize("T", [3, 200])
def test_linear_offsets_past_32_bits(T):
    """A swiglu product whose ups begin 4 GiB into the matrix and whose last rows lie past 8 GiB:
    columns from both ends against 64 bits (few rows and many take different kernels)."""
    note("past 32 bits", T)
    dtype, dt, K, N = B.EP_BF16, torch.bfloat16, 32768, 65536
    g = gen(T)
    x = randn((T, K), dt, g)
    w = torch.empty((2 * N, K), dtype=dt, device="cuda").normal_(0, K ** -0.5, generator=g)
    out, pre = torch.zeros((T, N), dtype=dt, device="cuda"), torch.zeros((T, 2 * N), dtype=dt, device="cuda")
    B.ep_linear(x, w, out, dtype, act=B.EP_ACT_SWIGLU, preact=pre)
    cols = torch.tensor([0, 1, 17, N // 2 - 1, N // 2, N - 129, N - 1], device="cuda")
    both = torch.cat([cols, cols + N])
    z, m = x.double() @ w[both].double().T, x.double().abs() @ w[both].double().abs().T
    dz = K * SUM * m
    check(pre[:, both], z, dz, "preact")
    check(out[:, cols], act(z, "swiglu"), act_error(z, dz, "swiglu"), "out")


@pytest.mark.parametrize("T", [5, 300])
def test_expert_gemm_fp8_offsets_past_32_bits(T):
    note("fp8 past 32 bits", T)
    K, N = 65536, 65536
    g = gen(T)
    lay = B.EpLayout(T, 1, 1, 1)
    B.ep_get_layout(torch.zeros((T, 1), dtype=torch.int64, device="cuda"), lay)
    q, s = quant_rows(torch.randn((T, K), device="cuda", generator=g), 128)
    w = torch.randint(0, 0x60, (1, 2 * N, K), dtype=torch.uint8, device="cuda", generator=g)
    ws = torch.full((1, 2 * N // 128, K // 128), 2.0 ** -8, device="cuda")
    out, pre = (torch.zeros((T, n), dtype=torch.bfloat16, device="cuda") for n in (N, 2 * N))
    B.ep_expert_gemm(q, w, lay, out, B.EP_FP8_E4M3, act=B.EP_ACT_SWIGLU, x_scales=s, weight_scales=ws, preact=pre)
    cols = torch.tensor([0, 130, N // 2, N - 1], device="cuda")
    both = torch.cat([cols, cols + N])
    xd, wd = codes(q) * s.double().repeat_interleave(128, 1), codes(w[0, both]) * 2.0 ** -8
    z, m = xd @ wd.T, xd.abs() @ wd.abs().T
    check(pre[:, both], z, (K + 4) * SUM * m + fp8_group_error(xd, wd), "preact")


def test_linear_rows_near_2_to_31():
    """A tile count, height and first row that leave 32 bits on the way: rows from both ends."""
    T, K, N = 2 ** 31 - 3001, 8, 8
    if torch.cuda.mem_get_info()[0] < 90 * 2 ** 30:
        pytest.skip("needs 70 GB")
    note("rows near 2^31")
    g = gen(3)
    part = randn((4096, K), torch.bfloat16, g)
    x = torch.empty((T, K), dtype=torch.bfloat16, device="cuda")
    whole = T // 4096 * 4096
    x[:whole].view(-1, 4096, K)[:] = part
    x[whole:] = part[:T - whole]
    w = randn((N, K), torch.bfloat16, g)
    out = torch.zeros((T, N), dtype=torch.bfloat16, device="cuda")
    B.ep_linear(x, w, out, B.EP_BF16)
    for at in (0, 4096 * 3, 2 ** 30 // 8 * 8, whole - 4096 * 2, T - 4096):
        xe = x[at:at + 4096].double()
        check(out[at:at + 4096], xe @ w.double().T, K * SUM * (xe.abs() @ w.double().abs().T), "rows at %d" % at)
    del x, out
    torch.cuda.empty_cache()


@pytest.mark.parametrize("name", ["bf16", "fp16"])
@pytest.mark.parametrize("a", ["relu", "gelu", "silu", "swiglu"])
@pytest.mark.parametrize("T", [8, 400])
def test_activations_over_the_whole_range(name, a, T):
    """Arguments from the type's smallest to its largest magnitudes, forward and back.  Exponentials
    past fp32's range end in 0 or infinity: up to 2^-80 absolute (|z| 2^-126 at |z| near 88)."""
    note("whole range", name, a, T)
    dtype, dt = TYPES[name]
    g = gen(T)
    N = 64
    e = (30.0 if name == "bf16" else 12.0) * torch.rand((T, width(N, a)), device="cuda", generator=g) - 15.0
    x = (torch.exp2(e) * torch.sign(torch.randn(e.shape, device="cuda", generator=g))).to(dt)
    x[:, :8] = torch.tensor([0.0, -0.0, 88.0, -88.0, -87.5, 104.0, -104.0, -20.0], device="cuda").to(dt)
    eye = torch.eye(width(N, a), device="cuda").to(dt)
    out, pre = torch.zeros((T, N), dtype=dt, device="cuda"), torch.zeros_like(x)
    B.ep_linear(x, eye, out, dtype, act=ACTS[a], preact=pre)
    assert torch.equal(pre, x)             # one product is not rounded
    z = x.double()
    tiny = 2.0 ** -80 * (1 + (z[:, N:].abs() if a == "swiglu" else 0))
    check(out, act(z, a), act_error(z, 0 * z, a) + tiny, "out")
    d = randn((T, N), dt, g)
    dz = torch.zeros_like(x)
    B.ep_act_grad(d, x, dz, dtype, ACTS[a])
    tiny = 2.0 ** -80 * (1 + z.abs().amax()) * d.double().abs().amax()
    check(dz, act_grad(d.double(), z, a), act_grad_error(d.double(), 0 * d.double(), z, a) + tiny, "dz")
