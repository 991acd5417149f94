"""Refusals of the matrix products' and gradients' entry points, through the C ABI with pointers
that are never read: every call here fails validation, or has nothing to do, on the host."""
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


def gemm(L, x=P, xs=None, w=P, ws=None, bias=None, s=None, K=64, N=64, dtype=0, act=0, pre=None, out=P):
    s = lay() if s is None else s
    return L.ep_expert_gemm(x, xs, w, ws, bias, ctypes.byref(s) if s else None, K, N, dtype, act, pre, out, None)


def test_expert_gemm_refusals(L):
    assert gemm(L, s=False) == -1
    bad = lay()
    bad.expert_offsets = None
    assert gemm(L, s=bad) == -1
    bad = lay()
    bad.num_recv_rows = 3
    assert gemm(L, s=bad) == -2
    for kw in (dict(x=None), dict(w=None), dict(out=None)):
        assert gemm(L, **kw) == -1, kw
    for kw in (dict(x=P + 8), dict(w=P + 8), dict(out=P + 2), dict(bias=P + 4), dict(pre=P + 8)):
        assert gemm(L, **kw) == -3, kw
    for kw in (dict(K=0), dict(K=60), dict(K=65544), dict(N=4), dict(N=-8), dict(N=65544)):
        assert gemm(L, **kw) == -2, kw
    for kw in (dict(dtype=5), dict(dtype=-1), dict(act=5), dict(act=-1), dict(dtype=B.EP_READ_X_AHEAD),
               dict(dtype=B.EP_SCALES_MN_MAJOR), dict(dtype=B.EP_GRAD_F32), dict(dtype=B.EP_F16 | B.EP_GRAD_ACCUMULATE),
               dict(dtype=B.EP_MXFP8_E4M3 | B.EP_SCALES_MN_MAJOR)):
        assert gemm(L, **kw) == -6, kw
    for d in (1, 2, 3):
        assert gemm(L, dtype=d, K=128, N=128, xs=P) == -1 and gemm(L, dtype=d, K=128, N=128, ws=P) == -1
        assert gemm(L, dtype=d, K=64, N=128, xs=P, ws=P) == -2 and gemm(L, dtype=d, K=128, N=64, xs=P, ws=P) == -2
        assert gemm(L, dtype=d, K=128, N=128, xs=P + 2, ws=P) == -3 and gemm(L, dtype=d, K=128, N=128, xs=P, ws=P + 1) == -3
    assert gemm(L, s=lay(T=0), x=None, w=None, out=None) == 0     # nothing to do


def test_gradient_refusals(L):
    by = ctypes.byref
    s, e = lay(), lay(T=0)

    def gx(dy=P, w=P, s=s, K=64, N=64, dtype=0, act=0, pre=None, dx=P):
        return L.ep_expert_gemm_grad_x(dy, w, by(s) if s else None, K, N, dtype, act, pre, dx, None)

    assert gx(s=None) == -1 and gx(dy=None) == -1 and gx(w=None) == -1 and gx(dx=None) == -1
    assert gx(act=4) == -1 and gx(act=1, pre=P + 2) == -3 and gx(act=7) == -6
    assert gx(dtype=1) == -6 and gx(dtype=B.EP_GRAD_F32) == -6 and gx(K=12) == -2 and gx(N=0) == -2
    assert gx(dy=P + 8) == -3 and gx(s=e, dy=None, w=None, dx=None) == 0

    def gw(dy=P, x=P, s=s, K=64, N=64, dtype=0, dw=P, db=None):
        return L.ep_expert_gemm_grad_w(dy, x, by(s) if s else None, K, N, dtype, dw, db, None)

    assert gw(s=None) == -1 and gw(dy=None) == -1 and gw(x=None) == -1 and gw(dw=None) == -1
    assert gw(dtype=3) == -6 and gw(dtype=B.EP_SCALES_MN_MAJOR) == -6 and gw(dtype=0x1000) == -6
    assert gw(K=4) == -2 and gw(N=100) == -2 and gw(dw=P + 8) == -3 and gw(db=P + 2) == -3


def test_linear_refusals(L):
    def lin(x=P, w=P, bias=None, res=None, rows=4, K=64, N=64, dtype=0, act=0, pre=None, out=P):
        return L.ep_linear(x, w, bias, res, rows, K, N, dtype, act, pre, out, None)

    assert lin(rows=-1) == -2 and lin(rows=1 << 31) == -2 and lin(K=7) == -2 and lin(N=12) == -2
    assert lin(dtype=1) == -6 and lin(dtype=3) == -6 and lin(dtype=B.EP_SCALES_MN_MAJOR) == -6 and lin(act=9) == -6
    assert lin(x=None) == -1 and lin(w=None) == -1 and lin(out=None) == -1
    assert lin(res=P + 4) == -3 and lin(bias=P + 2) == -3 and lin(out=P + 8) == -3
    assert lin(rows=0, x=None, w=None, out=None) == 0
    assert L.ep_linear_grad_x(P, P, -1, 64, 64, 0, 0, None, P, None) == -2
    assert L.ep_linear_grad_x(P, P, 4, 64, 64, 0, 2, None, P, None) == -1
    assert L.ep_linear_grad_x(None, None, 0, 64, 64, 0, 0, None, None, None) == 0
    assert L.ep_linear_grad_w(P, P, 4, 64, 60, 0, P, None, None) == -2
    assert L.ep_linear_grad_w(P, P, 4, 64, 64, 9, P, None, None) == -6
    assert L.ep_linear_grad_w(P, None, 4, 64, 64, 0, P, None, None) == -1
    assert L.ep_act_grad(P, P, 4, 64, 1, 0, P, None) == -6
    assert L.ep_act_grad(P, P, 4, 64, 0, 5, P, None) == -6
    assert L.ep_act_grad(P, P, -4, 64, 0, 1, P, None) == -2
    assert L.ep_act_grad(P, P, 4, 12, 0, 1, P, None) == -2
    assert L.ep_act_grad(P, None, 4, 64, 0, 1, P, None) == -1
    assert L.ep_act_grad(P, P + 8, 4, 64, 0, 1, P, None) == -3
    assert L.ep_act_grad(P, P + 64, 4, 64, 0, 4, P, None) == -2     # swiglu's dz is wider than dy
    assert L.ep_act_grad(None, None, 0, 64, 0, 1, None, None) == 0


def test_combine_grad_refusals(L):
    by = ctypes.byref
    s = lay()

    def cg(dout=P, y=P, w=P, s=s, H=64, dtype=0, dy=P, dw=P):
        return L.ep_combine_grad(dout, y, w, by(s) if s else None, H, dtype, dy, dw, None)

    assert cg(s=None) == -1 and cg(dout=None) == -1 and cg(w=None) == -1 and cg(dy=None) == -1 and cg(y=None) == -1
    assert cg(dtype=1) == -6 and cg(H=12) == -2 and cg(H=0) == -2 and cg(H=65544) == -2
    assert cg(dout=P + 8) == -3 and cg(y=P + 8) == -3 and cg(w=P + 2) == -3 and cg(dw=P + 1) == -3
    assert cg(s=lay(T=0), dout=None, y=None, w=None, dy=None, dw=None) == 0


def test_binding_refuses_host_tensors():
    lay_ = B.EpLayout(4, 1, 2, 1, device="cpu")
    t = torch.zeros((4, 8), dtype=torch.bfloat16)
    w = torch.zeros((2, 8, 8), dtype=torch.bfloat16)
    for call in (lambda: B.ep_expert_gemm(t, w, lay_, t, 0), lambda: B.ep_expert_gemm_grad_x(t, w, lay_, t, 0),
                 lambda: B.ep_expert_gemm_grad_w(t, t, lay_, w, 0), lambda: B.ep_linear(t, w[0], t, 0),
                 lambda: B.ep_linear_grad_x(t, w[0], t, 0), lambda: B.ep_linear_grad_w(t, t, w[0], 0),
                 lambda: B.ep_act_grad(t, t, t, 0, 1), lambda: B.ep_combine_grad(t, t, t, lay_, t, None, 0)):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()


@pytest.mark.gpu
def test_binding_refuses_wrong_tensors():
    """Shapes, types, strides, overlaps and layouts that do not fit, before anything is enqueued."""
    lay_ = B.EpLayout(4, 2, 3, 1)
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    x, w, out, wide = z(8, 16), z(3, 24, 16), z(8, 24), z(8, 16)
    cases = [lambda: B.ep_expert_gemm(x, w[:2].contiguous(), lay_, out, 0),
             lambda: B.ep_expert_gemm(z(7, 16), w, lay_, out, 0),
             lambda: B.ep_expert_gemm(x.half(), w, lay_, out, 0),
             lambda: B.ep_expert_gemm(x, w.transpose(1, 2), lay_, z(8, 16), 0),
             lambda: B.ep_expert_gemm(x, w, lay_, out, 0, act=B.EP_ACT_SWIGLU),
             lambda: B.ep_expert_gemm(x, w, lay_, out, 0, bias=z(24)),
             lambda: B.ep_expert_gemm(x, w, lay_, out, 0, preact=out),
             lambda: B.ep_expert_gemm(x, w, lay_, out, 0, x_scales=z(8, 1, dt=torch.float32)),
             lambda: B.ep_expert_gemm(z(8, 24)[:, :16], w, lay_, out, 0),
             lambda: B.ep_expert_gemm(z(16), w, lay_, out, 0),
             lambda: B.ep_expert_gemm_grad_x(out, w, lay_, x, 0, act=B.EP_ACT_SILU, preact=z(8, 8)),
             lambda: B.ep_expert_gemm_grad_x(out, w[0], lay_, x, 0),
             lambda: B.ep_expert_gemm_grad_w(out, x, lay_, w, B.EP_GRAD_F32),
             lambda: B.ep_expert_gemm_grad_w(out, x, lay_, w, 0, dbias=z(3, 16)),
             lambda: B.ep_linear(x, w[0], out, 0, residual=z(8, 16)),
             lambda: B.ep_linear(x, z(16, 16), x, 0),
             lambda: B.ep_linear(x, z(16, 16), x, 0, residual=x),   # may be the residual, not x too
             lambda: B.ep_act_grad(wide[:4], z(8, 32)[:4], wide[:4].view(2, 32), 0, B.EP_ACT_SWIGLU),
             lambda: B.ep_act_grad(wide[:4], wide.view(4, 32), wide.view(4, 32), 0, B.EP_ACT_SWIGLU),
             lambda: B.ep_linear_grad_w(out, z(7, 16), w[0], 0),
             lambda: B.ep_act_grad(x, x, out, 0, B.EP_ACT_SILU),
             lambda: B.ep_combine_grad(z(4, 16), x, z(4, 2), lay_, z(8, 16), None, 0),
             lambda: B.ep_combine_grad(z(4, 16), x, z(4, 2, dt=torch.float32), lay_, x, None, 0)]
    for i, call in enumerate(cases):
        with pytest.raises(ValueError):
            call()
            raise AssertionError("case %d was accepted" % i)
