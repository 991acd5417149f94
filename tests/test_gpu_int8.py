"""8-bit integer rows and their products against the definition in 64 bits.

Codes and scales have to be equal.  A product: the integer sum is exact, its conversion and the two
scales' products are three roundings of 2^-24, and the bias one more; then as in products_ref."""
import math

import pytest
import torch

import block_ref as ref
from combine_moe_layout_amd import binding as B
from products_ref import ACTS, act, act_error, check, segments, used_rows, width

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def same_rows(q, s, x):
    wq, ws, _ = ref.int8_rows(x)
    assert torch.equal(q, wq), (q != wq).sum().item()
    assert torch.equal(torch.nan_to_num(s, nan=-1.0), torch.nan_to_num(ws, nan=-1.0))


@pytest.mark.parametrize("rows,n", [(1, 16), (5, 48), (300, 64), (7, 1024), (6, 1040), (3, 4096), (5, 7168), (2, 16384),
                                    (2, 16400), (1, 32768), (2, 65536), (5000, 80)])
@pytest.mark.parametrize("dt", [BF, torch.float16])
def test_rows(rows, n, dt):
    print("[gpu-int8]", rows, n, dt, flush=True)
    x = (torch.randn((rows, n), device="cuda", generator=gen(rows + n)) * 3).to(dt)
    q = torch.full((rows, n), 77, dtype=torch.int8, device="cuda")
    s = torch.full((rows,), 7.0, device="cuda")
    B.ep_quantize_int8(x, q, s, B.EP_BF16 if dt is BF else B.EP_F16)
    same_rows(q, s, x)


@pytest.mark.parametrize("dt", [BF, torch.float16])
def test_borders_between_codes(dt):
    """Scales of powers of two make exact ties; scales just beside them make quotients that fp32
    cannot tell from ties."""
    n = 256
    ties = torch.arange(-127, 127, device="cuda").float() + 0.5
    rows = []
    for top in (127.0, 126.0, 127.5, 126.5, 63.5, 100.0, 3.0, 1.0):
        row = torch.zeros(n, device="cuda")
        row[0] = top
        row[1:255] = (ties * (top / 127)).clamp(-top, top)
        rows.append(row)
    rows = torch.stack(rows)
    x = torch.cat([rows * 2.0 ** e for e in ((-14, -3, 0, 5, 8) if dt is torch.float16 else (-60, -3, 0, 5, 90))]).to(dt)
    # every 16-bit value of two binades under many maxima: quotients near every border
    bits = torch.arange(2 * 1024 if dt is torch.float16 else 2 * 128, device="cuda")
    base = torch.tensor([1.0], device="cuda").to(dt).view(torch.int16).long()
    values = (base + bits).short().view(dt)
    more = values[:240].repeat(900, 1) if dt is torch.float16 else values[:240].repeat(256, 1)
    top = (base + bits[:more.shape[0]]).short().view(dt)
    more = torch.cat([torch.zeros((more.shape[0], 16), dtype=dt, device="cuda"), more], 1)
    more[:, 0] = top.float().mul(8).to(dt)
    more[:, 1:16] = -more[:, 17:32]
    for v in (x, more.contiguous()):
        q = torch.empty(v.shape, dtype=torch.int8, device="cuda")
        s = torch.empty(v.shape[0], device="cuda")
        B.ep_quantize_int8(v, q, s, B.EP_BF16 if dt is BF else B.EP_F16)
        same_rows(q, s, v)


@pytest.mark.parametrize("dt", [BF, torch.float16])
def test_special_rows(dt):
    x = torch.randn((12, 1040), device="cuda", generator=gen(1)).to(dt)
    f = torch.finfo(dt)
    x[0], x[1] = 0, -0.0
    x[2, 700], x[3, 1039], x[4, 0] = math.nan, math.inf, -math.inf
    x[5], x[6] = f.max, f.smallest_normal
    x[7], x[7, 5] = 0, torch.tensor([1], dtype=torch.int16).view(dt).item()      # smallest subnormal
    x[8] = -1.0
    x[9, 3], x[9, 4] = math.nan, -math.inf
    x[10] = x[10] * 2.0 ** -14
    q = torch.full(x.shape, 77, dtype=torch.int8, device="cuda")
    s = torch.empty(12, device="cuda")
    B.ep_quantize_int8(x, q, s, B.EP_BF16 if dt is BF else B.EP_F16)
    same_rows(q, s, x)
    assert torch.isnan(s[[2, 3, 4, 9]]).all() and (q[[2, 3, 4, 9]] == 0).all()
    assert (q[0] == 0).all() and s[0] > 0


LAYOUTS = [(37, 3, 5, 0, 0.2), (50, 4, 8, 9, 0.0), (300, 1, 1, 0, 0.0), (1, 1, 3, 0, 0.0), (64, 8, 64, 3, 0.1),
           (700, 2, 6, 100, 0.1), (40, 2, 4, 16, 1.0)]


def layout(T, k, E, cap, masked, seed=0):
    g = gen(T + k + E + seed)
    idx = torch.rand((T, E), device="cuda", generator=g).topk(min(k, E), 1).indices
    if k > E:
        idx = torch.randint(0, E, (T, k), device="cuda", generator=g)
    idx = torch.where(torch.rand((T, k), device="cuda", generator=g) < masked, -1, idx)
    lay = B.EpLayout(T, k, E, 1, cap)
    B.ep_get_layout(idx, lay)
    return idx, lay


@pytest.mark.parametrize("T,k,E,cap,masked", LAYOUTS)
@pytest.mark.parametrize("H", [16, 208, 1024, 7168, 17408])
def test_dispatch(T, k, E, cap, masked, H):
    print("[gpu-int8] dispatch", T, k, E, cap, H, flush=True)
    idx, lay = layout(T, k, E, cap, masked)
    x = torch.randn((T, H), device="cuda", generator=gen(H)).to(BF)
    x[T // 2, H // 2] = math.nan
    R = lay.num_recv_rows
    wq, ws, _ = ref.int8_rows(x)
    want_q = torch.full((R, H), 77, dtype=torch.int8, device="cuda")
    want_s = torch.full((R,), 7.0, device="cuda")
    t, j = torch.nonzero(lay.slot_idx >= 0, as_tuple=True)
    want_q[lay.slot_idx[t, j].long()], want_s[lay.slot_idx[t, j].long()] = wq[t], ws[t]
    lay2 = B.EpLayout(T, k, E, 1, cap)
    for both in (False, True):
        q, s = torch.full_like(want_q, 77), torch.full_like(want_s, 7.0)
        if both:
            B.ep_layout_dispatch(idx, lay2, x, B.EP_INT8, q, s)
            assert torch.equal(lay2.slot_idx, lay.slot_idx)
        else:
            B.ep_dispatch(x, lay, B.EP_INT8, q, s)
        assert torch.equal(q, want_q)
        assert torch.equal(torch.nan_to_num(s, nan=-1.0), torch.nan_to_num(want_s, nan=-1.0))


@pytest.mark.parametrize("T,k,E,cap,masked", LAYOUTS)
def test_rows_of_a_layout(T, k, E, cap, masked):
    """Used rows are rounded, the others neither read (NaN) nor written."""
    _, lay = layout(T, k, E, cap, masked)
    R, n = lay.num_recv_rows, 272
    used = used_rows(lay)
    x = torch.randn((R, n), device="cuda", generator=gen(4)).to(BF)
    x[~used] = math.nan
    q, s = torch.full((R, n), 77, dtype=torch.int8, device="cuda"), torch.full((R,), 7.0, device="cuda")
    B.ep_quantize_int8(x, q, s, B.EP_BF16, layout=lay)
    same_rows(q[used], s[used], x[used])
    assert (q[~used] == 77).all() and (s[~used] == 7).all()


def exact_product(q, s, w, ws, bias):
    """z and how far it may be off before its activation."""
    z = (q.double() @ w.double().T) * s.double()[:, None] * ws.double()
    off = 3 * ref.STEP * z.abs()
    if bias is not None:
        z = z + bias.double()
        off = off + ref.STEP * (z.abs() + off)
    return z, off


def operands(E, W, K, rows, seed):
    g = gen(seed)
    q = torch.randint(-127, 128, (rows, K), device="cuda", generator=g, dtype=torch.int8)
    s = torch.rand(rows, device="cuda", generator=g) * (2.0 / 127 / 70) + 1e-5
    w = torch.randint(-128, 128, (E, W, K), device="cuda", generator=g, dtype=torch.int8)
    ws = torch.rand((E, W), device="cuda", generator=g) * (K ** -0.5 / 40) + 1e-5
    bias = (torch.randn((E, W), device="cuda", generator=g) * 0.1).to(BF)
    return q, s, w, ws, bias


EXPERTS = [(37, 3, 5, 0, 0.2, 16, 8), (50, 4, 8, 9, 0.0, 144, 72), (300, 1, 1, 0, 0.0, 128, 128), (1, 1, 3, 0, 0.0, 80, 264),
           (64, 8, 64, 3, 0.1, 384, 40), (700, 2, 6, 100, 0.1, 208, 136), (40, 2, 4, 16, 1.0, 64, 64),
           (1500, 2, 6, 0, 0.0, 1040, 520), (900, 2, 4, 500, 0.0, 256, 1032), (2000, 4, 7, 0, 0.1, 2064, 264),
           (130, 1, 2, 0, 0.0, 7168, 256), (2600, 2, 9, 0, 0.0, 96, 392)]


@pytest.mark.parametrize("T,k,E,cap,masked,K,N", EXPERTS)
@pytest.mark.parametrize("name", sorted(ACTS))
def test_experts(T, k, E, cap, masked, K, N, name):
    print("[gpu-int8] experts", T, k, E, cap, K, N, name, flush=True)
    _, lay = layout(T, k, E, cap, masked)
    R, W = lay.num_recv_rows, width(N, name)
    used = used_rows(lay)
    q, s, w, ws, bias = operands(E, W, K, R, K + N)
    s[~used] = math.nan
    bias = bias if (K + N) % 3 else None
    out, pre = torch.full((R, N), 7.0, dtype=BF, device="cuda"), torch.full((R, W), 7.0, dtype=BF, device="cuda")
    B.ep_expert_gemm(q, w, lay, out, B.EP_INT8, act=ACTS[name], x_scales=s, weight_scales=ws, bias=bias, preact=pre)
    for e, (b, n) in enumerate(segments(lay)):
        if not n:
            continue
        at = slice(b, b + n)
        z, off = exact_product(q[at], s[at], w[e], ws[e], None if bias is None else bias[e])
        check(pre[at], z, off, "preact of expert %d" % e)
        check(out[at], act(z, name), act_error(z, off, name), "out of expert %d" % e)
    assert (out[~used] == 7).all() and (pre[~used] == 7).all()
    again = torch.full_like(out, 7.0)
    B.ep_expert_gemm(q, w, lay, again, B.EP_INT8, act=ACTS[name], x_scales=s, weight_scales=ws, bias=bias)
    assert torch.equal(out, again)


LINEAR = [(1, 16, 8), (1, 7168, 4096), (3, 48, 24), (15, 1040, 200), (16, 640, 4096), (17, 128, 136), (33, 2064, 72),
          (64, 7168, 264), (65, 512, 512), (129, 400, 1000), (300, 1024, 2048), (1000, 272, 328), (2048, 384, 640), (40, 65536, 16),
          (5, 16, 65536)]


@pytest.mark.parametrize("T,K,N", LINEAR)
@pytest.mark.parametrize("name", ["none", "gelu", "swiglu"])
def test_linear(T, K, N, name):
    print("[gpu-int8] linear", T, K, N, name, flush=True)
    if 2 * N > 65536 and name == "swiglu":
        N = 32768
    q, s, w, ws, bias = operands(1, width(N, name), K, T, T + K + N)
    res = torch.randn((T, N), device="cuda", generator=gen(2)).to(BF)
    z, off = exact_product(q, s, w[0], ws[0], bias[0])
    a, aoff = act(z, name), act_error(z, off, name)
    out, pre = torch.full((T, N), 7.0, dtype=BF, device="cuda"), torch.full((T, z.shape[1]), 7.0, dtype=BF, device="cuda")
    B.ep_linear_int8(q, s, w[0], ws[0], out, act=ACTS[name], bias=bias[0], residual=res, preact=pre)
    check(pre, z, off, "preact")
    check(out, a + res.double(), aoff + ref.STEP * (a.abs() + aoff + res.double().abs()), "out")
    B.ep_linear_int8(q, s, w[0], ws[0], res, act=ACTS[name], bias=bias[0], residual=res)      # in place
    assert torch.equal(res, out)
    z, off = exact_product(q, s, w[0], ws[0], None)
    B.ep_linear_int8(q, s, w[0], ws[0], out, act=ACTS[name])
    check(out, act(z, name), act_error(z, off, name), "out alone")


@pytest.mark.parametrize("T,K,N", [(640, 1040, 4096), (1000, 400, 4096), (705, 208, 4096), (4000, 144, 1008), (300, 2048, 7168)])
@pytest.mark.parametrize("name", ["gelu", "swiglu"])
def test_one_tile_for_each_cu(T, K, N, name):
    """Sizes whose tiles of 128 x 128 number between half the CUs and all of them."""
    test_linear(T, K, N // 2 if name == "swiglu" else N, name)


@pytest.mark.parametrize("cap", [0, 150])
def test_one_tile_for_each_cu_of_experts(cap):
    test_experts(512, 2, 8, cap, 0.1, 336, 4096, "silu")
    test_experts(512, 2, 8, cap, 0.1, 272, 2048, "swiglu")


@pytest.mark.parametrize("T,K,N", [(3, 1040, 8192), (16, 400, 16384), (20, 1040, 8192), (32, 272, 12000), (50, 2064, 6144),
                                   (100, 400, 8192), (9, 16, 5008), (1, 16384, 4112)])
@pytest.mark.parametrize("name", ["gelu", "swiglu"])
def test_few_tiles(T, K, N, name):
    """Every height and width of the tiles that share out the reduction, with a part of a chunk at its end."""
    test_linear(T, K, N // 2 if name == "swiglu" else N, name)


@pytest.mark.parametrize("T,N", [(30, 512), (30, 1024), (60, 1024), (60, 2000), (120, 1024)])
def test_few_tiles_of_experts(T, N):
    test_experts(T, 2, 4, 0, 0.1, 400, N, "none")
    test_experts(T, 2, 4, 70, 0.0, 400, N // 2, "swiglu")


def test_largest_sums():
    """65,536 products of -128 and -128: 2^30, and its negative neighbours."""
    K = 65536
    for T in (3, 200):
        q = torch.full((T, K), -128, dtype=torch.int8, device="cuda")
        w = torch.full((24, K), -128, dtype=torch.int8, device="cuda")
        w[1], w[2] = 127, -127
        one_x, one_w = torch.full((T,), 2.0 ** -15, device="cuda"), torch.full((24,), 2.0 ** -15, device="cuda")
        out = torch.empty((T, 24), dtype=BF, device="cuda")
        B.ep_linear_int8(q, one_x, w, one_w, out)
        want = (q.double() @ w.double().T) * 2.0 ** -30
        assert (out.double() - want).abs().max() <= 2.0 ** -8 and out[0, 0] == 1.0


def test_nan_rows_give_nan_results():
    x = torch.randn((40, 256), device="cuda", generator=gen(8)).to(BF)
    x[7, 9], x[20, 0] = math.nan, math.inf
    q, s = torch.empty((40, 256), dtype=torch.int8, device="cuda"), torch.empty(40, device="cuda")
    B.ep_quantize_int8(x, q, s, B.EP_BF16)
    _, _, w, ws, _ = operands(1, 72, 256, 1, 3)
    out = torch.empty((40, 72), dtype=BF, device="cuda")
    B.ep_linear_int8(q, s, w[0], ws[0], out)
    bad = torch.isnan(out).all(1)
    assert bad.nonzero().flatten().tolist() == [7, 20] and torch.isfinite(out[~bad]).all()


def test_offsets_past_32_bits():
    """Rows, results and matrices of more than 2^32 bytes: the last of them come out as by themselves."""
    rows, K, N = 70_000, 65_536, 64
    x = torch.ones((rows, K), dtype=BF, device="cuda")
    x[-5:] = torch.randn((5, K), device="cuda", generator=gen(1)).to(BF)
    q, s = torch.empty((rows, K), dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    few_q, few_s = torch.empty_like(q[:5]), torch.empty_like(s[:5])
    B.ep_quantize_int8(x, q, s, 0)
    B.ep_quantize_int8(x[-5:].clone(), few_q, few_s, 0)
    assert torch.equal(q[-5:], few_q) and torch.equal(s[-5:], few_s)
    del x
    w, ws = few_q[:1].expand(N, K).contiguous(), torch.rand(N, device="cuda", generator=gen(3))
    out, few = torch.empty((rows, N), dtype=BF, device="cuda"), torch.empty((5, N), dtype=BF, device="cuda")
    B.ep_linear_int8(q, s, w, ws, out)
    B.ep_linear_int8(few_q, few_s, w, ws, few)
    assert torch.equal(out[-5:], few)
    # the rows' codes as a matrix of 70,000 columns, gates and ups 2.3e9 bytes apart
    W, rs = 35_000, torch.rand(70_000, device="cuda", generator=gen(4))
    for T in (3, 300):
        a, sa = q[-5:].repeat(T, 1)[:T], torch.rand(T, device="cuda", generator=gen(5))
        out, z = torch.empty((T, W), dtype=BF, device="cuda"), torch.empty((T, 2 * W), dtype=BF, device="cuda")
        few, few_z = torch.empty((T, 8), dtype=BF, device="cuda"), torch.empty((T, 16), dtype=BF, device="cuda")
        B.ep_linear_int8(a, sa, q, rs, out, act=B.EP_ACT_SWIGLU, preact=z)
        B.ep_linear_int8(a, sa, torch.cat([q[W - 8:W], q[-8:]]), torch.cat([rs[W - 8:W], rs[-8:]]), few,
                         act=B.EP_ACT_SWIGLU, preact=few_z)
        assert torch.equal(z[:, W - 8:W], few_z[:, :8]) and torch.equal(z[:, -8:], few_z[:, 8:])


def test_no_rows():
    e = lambda *s, dt=BF: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
    i8, f32 = torch.int8, torch.float32
    B.ep_quantize_int8(e(0, 64), e(0, 64, dt=i8), e(0, dt=f32), B.EP_BF16)
    B.ep_linear_int8(e(0, 64, dt=i8), e(0, dt=f32), e(8, 64, dt=i8), e(8, dt=f32), e(0, 8))
    torch.cuda.synchronize()
