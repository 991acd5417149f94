"""Refusals of the router's, the block norms' and the 8-bit integers' entry points, through the C ABI
with pointers that are never read: every call here fails validation, or has nothing to do, on the host."""
import ctypes

import pytest
import torch

from combine_moe_layout_amd import binding as B

P = 1 << 20                                # never read


@pytest.fixture(scope="module")
def L():
    return B.lib()


def lay(T=64, k=4, E=16, cap=0):
    s = B.ep_layout_t()
    assert B.lib().ep_layout_init(ctypes.byref(s), T, k, E, 1, cap) == 0
    s.num_tokens_per_expert = s.expert_offsets = s.num_tokens_per_group = s.slot_idx = s.error_flags = P
    return s


GOOD = dict(num_experts=64, num_topk=6, score=1, num_groups=8, topk_groups=4, group_top=2, renormalize=1, scale=1.0)
BAD = [dict(num_experts=0), dict(num_experts=1025), dict(num_experts=63), dict(num_topk=0), dict(num_topk=65, topk_groups=8),
       dict(num_topk=33), dict(num_groups=0), dict(num_groups=-8), dict(topk_groups=0), dict(topk_groups=9), dict(group_top=0),
       dict(group_top=3), dict(num_groups=64, topk_groups=8)]


def test_router_refusals(L):
    by = ctypes.byref

    def route(x=P, bias=None, T=4, r=None, dtype=B.EP_F32, idx=P, w=P, **kw):
        s = B.ep_router_t(**{**GOOD, **kw})
        return L.ep_route(x, bias, T, None if r is False else by(s), dtype, idx, w, None)

    def grad(dw=P, x=P, idx=P, T=4, r=None, dtype=B.EP_F32, d=P, **kw):
        s = B.ep_router_t(**{**GOOD, **kw})
        return L.ep_route_grad(dw, x, idx, T, None if r is False else by(s), dtype, d, None)

    for f in (route, grad):
        assert f(r=False) == -1 and f(x=None) == -1 and f(idx=None) == -1
        for kw in BAD + [dict(T=-1), dict(T=1 << 29)]:
            assert f(**kw) == -2, kw
        for kw in (dict(dtype=1), dict(dtype=3), dict(dtype=5), dict(dtype=6), dict(dtype=8), dict(dtype=-1),
                   dict(dtype=B.EP_F32 | B.EP_GRAD_F32), dict(score=2), dict(score=-1)):
            assert f(**kw) == -6, kw
        assert f(x=P + 8) == -3 and f(idx=P + 4) == -3
        assert f(T=0, x=None, idx=None) == 0
    assert route(w=None) == -1 and route(w=P + 2) == -3 and route(bias=P + 2) == -3
    assert grad(dw=None) == -1 and grad(d=None) == -1 and grad(dw=P + 2) == -3 and grad(d=P + 8) == -3
    with pytest.raises(B.EpError):
        B.EpRouter(64, 65)
    with pytest.raises(B.EpError):
        B.EpRouter(64, 4, num_groups=7)
    assert B.EpRouter(64, 4).num_topk == 4


def test_block_norm_refusals(L):
    def norm(y=P, post=None, gate=None, res=P, alpha=1.0, pre=P, rows=4, H=64, dtype=0, eps=1e-6, out=P, n=P):
        return L.ep_block_norm(y, post, gate, res, alpha, pre, rows, H, dtype, eps, out, n, None)

    for kw in (dict(rows=-1), dict(rows=1 << 31), dict(H=0), dict(H=12), dict(H=65544), dict(eps=0.0), dict(eps=-1.0),
               dict(eps=float("nan")), dict(eps=float("inf"))):
        assert norm(**kw) == -2, kw
    for d in (1, 2, 3, 5, 6, 7, B.EP_GRAD_F32, B.EP_GRAD_ACCUMULATE, B.EP_SCALES_MN_MAJOR):
        assert norm(dtype=d) == -6
    for kw in (dict(y=None, res=None), dict(y=None, post=P), dict(y=None, gate=P), dict(out=None, n=None, pre=None),
               dict(pre=None), dict(n=None)):
        assert norm(**kw) == -1, kw
    for kw in (dict(y=P + 8), dict(post=P + 8), dict(gate=P + 2), dict(res=P + 2), dict(pre=P + 4), dict(out=P + 8), dict(n=P + 8)):
        assert norm(**kw) == -3, kw
    assert norm(rows=0, y=None, res=None, out=None, n=None, pre=None) == 0

    need = L.ep_block_norm_grad_workspace_bytes(4, 64)
    assert need > 0 and need % 4 == 0 and L.ep_block_norm_grad_workspace_bytes(0, 64) == 0
    for rows, H in ((-1, 64), (4, 12), (4, 0), (4, 65544), (1 << 31, 64)):
        assert L.ep_block_norm_grad_workspace_bytes(rows, H) == 0

    def grad(do=P, dn=P, y=P, post=P, gate=P, res=P, alpha=1.0, pre=P, rows=4, H=64, dtype=0, eps=1e-6, dy=P, dres=P,
             dgate=P, dpost=P, dpre=P, ws=P, size=need):
        return L.ep_block_norm_grad(do, dn, y, post, gate, res, alpha, pre, rows, H, dtype, eps, dy, dres, dgate, dpost,
                                    dpre, ws, size, None)

    for kw in (dict(rows=-1), dict(H=12), dict(eps=0.0)):
        assert grad(**kw) == -2, kw
    for d in (1, 3, 6, B.EP_SCALES_MN_MAJOR, B.EP_READ_X_AHEAD, 0x1000):
        assert grad(dtype=d) == -6
    none = dict(dy=None, dres=None, dgate=None, dpost=None, dpre=None)
    for kw in (dict(do=None, dn=None, pre=None, dpre=None), dict(dn=None), dict(pre=None, dpre=None), dict(y=None),
               dict(res=None), dict(gate=None), dict(post=None), dict(ws=None), none,
               dict(y=None, post=None, gate=None, dgate=None, dpost=None)):
        assert grad(**kw) == -1, kw
    for kw in (dict(do=P + 8), dict(dn=P + 8), dict(dy=P + 8), dict(dgate=P + 2), dict(dpost=P + 4), dict(ws=P + 128)):
        assert grad(**kw) == -3, kw
    assert grad(size=need - 1) == -4 and grad(size=0) == -4
    assert grad(rows=0, **{**none, "do": None, "dn": None}) == 0


def test_int8_refusals(L):
    by = ctypes.byref
    s = lay()

    def rows(x=P, s=None, n=64, rows=8, dtype=0, q=P, sc=P):
        return L.ep_quantize_int8(x, by(s) if s else None, rows, n, dtype, q, sc, None)

    assert rows(rows=-1) == -2 and rows(rows=1 << 31) == -2 and rows(n=8) == -2 and rows(n=72) == -2 and rows(n=65552) == -2
    assert rows(s=s, rows=8) == -2 and rows(s=lay(T=0), rows=0, x=None, q=None, sc=None) == 0
    assert rows(dtype=6) == -6 and rows(dtype=1) == -6 and rows(dtype=7) == -6
    assert rows(x=None) == -1 and rows(q=None) == -1 and rows(sc=None) == -1
    assert rows(x=P + 8) == -3 and rows(q=P + 8) == -3 and rows(sc=P + 2) == -3
    assert rows(rows=0, x=None, q=None, sc=None) == 0
    bad = lay()
    bad.expert_offsets = None
    assert rows(s=bad, rows=256) == -1

    def dispatch(x=P, H=64, dtype=B.EP_INT8, q=P, sc=P):
        return L.ep_dispatch(x, by(s), H, dtype, q, sc, None)

    assert dispatch(sc=None) == -1 and dispatch(q=None) == -1 and dispatch(H=72) == -2 and dispatch(H=8) == -2
    assert dispatch(sc=P + 2) == -3 and dispatch(dtype=B.EP_INT8 | B.EP_SCALES_MN_MAJOR) == -6
    assert dispatch(dtype=B.EP_INT8 | B.EP_READ_X_AHEAD) == -6 and dispatch(dtype=7) == -6
    assert L.ep_scales_to_mn_major(P, 4, 128, B.EP_INT8, P + 4096, None) == -6

    def gemm(x=P, xs=P, w=P, ws=P, bias=None, K=64, N=64, dtype=B.EP_INT8, act=0, pre=None, out=P):
        return L.ep_expert_gemm(x, xs, w, ws, bias, by(s), K, N, dtype, act, pre, out, None)

    def linear(x=P, xs=P, w=P, ws=P, bias=None, res=None, rows=4, K=64, N=64, act=0, pre=None, out=P):
        return L.ep_linear_int8(x, xs, w, ws, bias, res, rows, K, N, act, pre, out, None)

    for f in (gemm, linear):
        for kw in (dict(x=None), dict(xs=None), dict(w=None), dict(ws=None), dict(out=None)):
            assert f(**kw) == -1, kw
        for kw in (dict(K=8), dict(K=72), dict(K=65552), dict(N=4), dict(N=65544), dict(N=12)):
            assert f(**kw) == -2, kw
        for kw in (dict(x=P + 8), dict(xs=P + 2), dict(w=P + 4), dict(ws=P + 1), dict(bias=P + 8), dict(pre=P + 8), dict(out=P + 2)):
            assert f(**kw) == -3, kw
        assert f(act=5) == -6
    assert linear(rows=-1) == -2 and linear(rows=1 << 31) == -2 and linear(res=P + 8) == -3
    assert linear(rows=0, x=None, xs=None, w=None, ws=None, out=None) == 0
    for flag in (B.EP_SCALES_MN_MAJOR, B.EP_READ_X_AHEAD, B.EP_GRAD_F32):
        assert gemm(dtype=B.EP_INT8 | flag) == -6
    for d in (B.EP_INT8, B.EP_F32):                # forward of 16 bits, and gradients, take neither
        assert L.ep_linear(P, P, None, None, 4, 64, 64, d, 0, None, P, None) == -6
        assert L.ep_expert_gemm_grad_x(P, P, by(s), 64, 64, d, 0, None, P, None) == -6
        assert L.ep_expert_gemm_grad_w(P, P, by(s), 64, 64, d, P, None, None) == -6
        assert L.ep_combine_grad(P, P, P, by(s), 64, d, P, P, None) == -6
    assert gemm(dtype=B.EP_F32) == -6


def test_binding_refuses_host_tensors():
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)  # noqa: E731
    r = B.EpRouter(8, 2)
    i8, f32 = torch.int8, torch.float32
    for call in (lambda: B.ep_route(z(4, 8), r, z(4, 2, dt=torch.int64), z(4, 2, dt=f32), 0),
                 lambda: B.ep_route_grad(z(4, 2, dt=f32), z(4, 8), z(4, 2, dt=torch.int64), r, z(4, 8), 0),
                 lambda: B.ep_block_norm(z(4, 8), None, z(4, 8), 0),
                 lambda: B.ep_block_norm_grad(z(4, 8), None, z(4, 8), None, 0, d_y=z(4, 8)),
                 lambda: B.ep_quantize_int8(z(4, 16), z(4, 16, dt=i8), z(4, dt=f32), 0),
                 lambda: B.ep_linear_int8(z(4, 16, dt=i8), z(4, dt=f32), z(8, 16, dt=i8), z(8, dt=f32), z(4, 8))):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
    for call in (lambda: B.ep_block_norm(None, None, z(4, 8), 0), lambda: B.ep_block_norm_grad(None, None, z(4, 8), None, 0)):
        with pytest.raises(ValueError, match="needed"):
            call()


@pytest.mark.gpu
def test_binding_refuses_wrong_tensors():
    """Shapes, types, strides and overlaps, before anything is enqueued."""
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    i8, f32, i64 = torch.int8, torch.float32, torch.int64
    r, lay_ = B.EpRouter(8, 2), B.EpLayout(4, 2, 3, 1)
    x, out = z(4, 16), z(4, 16)
    q, s, w, ws = z(4, 32, dt=i8), z(4, dt=f32), z(8, 32, dt=i8), z(8, dt=f32)
    pool = z(64, dt=f32)
    bwd = dict(post_weight=z(16), d_post_weight=z(16))
    cases = [lambda: B.ep_route(z(4, 7), r, z(4, 2, dt=i64), z(4, 2, dt=f32), 0),
             lambda: B.ep_route(z(4, 8), r, z(4, 2, dt=torch.int32), z(4, 2, dt=f32), 0),
             lambda: B.ep_route(z(4, 8), r, z(4, 2, dt=i64), z(4, 2, dt=f32), B.EP_F32),
             lambda: B.ep_route(z(4, 8), r, z(4, 3, dt=i64), z(4, 2, dt=f32), 0),
             lambda: B.ep_route(z(8, 4).T, r, z(4, 2, dt=i64), z(4, 2, dt=f32), 0),
             lambda: B.ep_route(z(4, 8), r, z(4, 2, dt=i64), z(4, 2, dt=f32), 0, bias=z(8)),
             lambda: B.ep_route(pool[:32].view(4, 8), r, z(4, 2, dt=i64), pool[24:32].view(4, 2), B.EP_F32),
             lambda: B.ep_route_grad(z(4, 2, dt=f32), x[:, :8].contiguous(), z(4, 2, dt=i64), r, z(4, 8, dt=f32), 0),
             lambda: B.ep_route_grad(pool[:8].view(4, 2), z(4, 8, dt=f32), z(4, 2, dt=i64), r, pool[:32].view(4, 8), B.EP_F32),
             lambda: B.ep_block_norm(x, z(3, 16), out, 0),
             lambda: B.ep_block_norm(x, None, out, 0, post_weight=z(8)),
             lambda: B.ep_block_norm(x, None, out, 0, gate=z(4)),
             lambda: B.ep_block_norm(x, None, out, B.EP_F16),
             lambda: B.ep_block_norm(x, None, out, 0, pre_weight=z(16), normed=out),
             lambda: B.ep_block_norm(z(5, 16)[:4], None, z(80)[8:72].view(4, 16).T.contiguous().T, 0),
             lambda: B.ep_block_norm_grad(x, None, out, None, 0, d_y=out),
             lambda: B.ep_block_norm_grad(x, None, out, None, 0, post_weight=z(16), d_post_weight=z(16, dt=f32)),
             lambda: B.ep_block_norm_grad(x, None, out, None, B.EP_GRAD_F32, z(2048, dt=torch.uint8), **bwd),
             lambda: B.ep_quantize_int8(x, z(4, 16), s, 0),
             lambda: B.ep_quantize_int8(x, z(4, 16, dt=i8), z(4, 1, dt=f32), 0),
             lambda: B.ep_quantize_int8(x, z(4, 16, dt=i8), s, 0, layout=lay_),
             lambda: B.ep_quantize_int8(x, x.view(torch.int8)[:, :16].contiguous().view(4, 16), s, B.EP_F16),
             lambda: B.ep_linear_int8(q, s, w, ws, z(4, 8, dt=torch.float16)),
             lambda: B.ep_linear_int8(q, s, w, ws, z(4, 16)),
             lambda: B.ep_linear_int8(q, z(3, dt=f32), w, ws, z(4, 8)),
             lambda: B.ep_linear_int8(q, s, w.view(torch.uint8), ws, z(4, 8)),
             lambda: B.ep_expert_gemm(z(8, 32, dt=i8), z(3, 8, 32, dt=i8), lay_, z(8, 8), B.EP_INT8, x_scales=z(8, dt=f32),
                                      weight_scales=z(3, 8, 1, dt=f32)),
             lambda: B.ep_dispatch(x, lay_, B.EP_INT8, z(8, 16, dt=torch.uint8), z(8, dt=f32)),
             lambda: B.ep_dispatch(x, lay_, B.EP_INT8, z(8, 16, dt=i8), z(8, 1, dt=f32))]
    for i, call in enumerate(cases):
        with pytest.raises(ValueError):
            call()
            raise AssertionError("case %d was accepted" % i)
