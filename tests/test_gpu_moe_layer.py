"""A whole MoE layer from the entry points, as a training step and a serving step use them:
layout, dispatch, the experts' two products, combine, and the shared expert's products with the
combined rows as their residual; then every gradient back to the tokens, the weights and the
routing weights.  Against 64-bit autograd of the same layer; captured in a graph; on two streams."""
import pytest
import torch

from combine_moe_layout_amd import binding as B
from products_ref import sigmoid

pytestmark = pytest.mark.gpu
DT, BF = torch.bfloat16, B.EP_BF16


class Layer:
    """Buffers and calls of one layer: T tokens of H, E experts and a shared one of I."""

    def __init__(self, seed, T=203, H=136, E=6, k=2, I=72, cap=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        rn = lambda *s, scale=1.0: (torch.randn(s, device="cuda", generator=g) * scale).to(DT)  # noqa: E731
        self.T, self.H, self.E, self.k, self.I = T, H, E, k, I
        self.x = rn(T, H)
        idx = torch.rand((T, E), device="cuda", generator=g).topk(k, 1).indices
        idx[::17, 0] = -1
        self.idx = idx
        self.w = torch.rand((T, k), device="cuda", generator=g)
        self.w13, self.w2 = rn(E, 2 * I, H, scale=H ** -0.5), rn(E, H, I, scale=I ** -0.5)
        self.s13, self.s2 = rn(2 * I, H, scale=H ** -0.5), rn(H, I, scale=I ** -0.5)
        self.dout = rn(T, H)
        self.lay = B.EpLayout(T, k, E, 1, cap)
        R = self.lay.num_recv_rows
        z = lambda *s, dt=DT: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
        self.rx, self.pre, self.h, self.y = z(R, H), z(R, 2 * I), z(R, I), z(R, H)
        self.out0, self.spre, self.sh, self.out = z(T, H), z(T, 2 * I), z(T, I), z(T, H)
        self.dy, self.dw, self.dpre, self.drx = z(R, H), z(T, k, dt=torch.float32), z(R, 2 * I), z(R, H)
        self.dw13, self.dw2 = z(E, 2 * I, H, dt=torch.float32), z(E, H, I, dt=torch.float32)
        self.dspre, self.ds13, self.ds2 = z(T, 2 * I), z(2 * I, H, dt=torch.float32), z(H, I, dt=torch.float32)
        self.dx_routed, self.dx_shared = z(T, H), z(T, H)
        self.ones = torch.ones((T, k), device="cuda")

    def forward(self, stream=None):
        B.ep_layout_dispatch(self.idx, self.lay, self.x, BF, self.rx, stream=stream)
        B.ep_expert_gemm(self.rx, self.w13, self.lay, self.h, BF, act=B.EP_ACT_SWIGLU, preact=self.pre, stream=stream)
        B.ep_expert_gemm(self.h, self.w2, self.lay, self.y, BF, stream=stream)
        B.ep_combine(self.y, self.w, self.lay, self.out0, stream=stream)
        B.ep_linear(self.x, self.s13, self.sh, BF, act=B.EP_ACT_SWIGLU, preact=self.spre, stream=stream)
        B.ep_linear(self.sh, self.s2, self.out, BF, residual=self.out0, stream=stream)

    def backward(self, stream=None):
        F = BF | B.EP_GRAD_F32
        B.ep_linear_grad_x(self.dout, self.s2, self.dspre, BF, act=B.EP_ACT_SWIGLU, preact=self.spre, stream=stream)
        B.ep_linear_grad_w(self.dout, self.sh, self.ds2, F, stream=stream)
        B.ep_linear_grad_x(self.dspre, self.s13, self.dx_shared, BF, stream=stream)
        B.ep_linear_grad_w(self.dspre, self.x, self.ds13, F, stream=stream)
        B.ep_combine_grad(self.dout, self.y, self.w, self.lay, self.dy, self.dw, BF, stream=stream)
        B.ep_expert_gemm_grad_x(self.dy, self.w2, self.lay, self.dpre, BF, act=B.EP_ACT_SWIGLU, preact=self.pre,
                                stream=stream)
        B.ep_expert_gemm_grad_w(self.dy, self.h, self.lay, self.dw2, F, stream=stream)
        B.ep_expert_gemm_grad_x(self.dpre, self.w13, self.lay, self.drx, BF, stream=stream)
        B.ep_expert_gemm_grad_w(self.dpre, self.rx, self.lay, self.dw13, F, stream=stream)
        B.ep_combine(self.drx, self.ones, self.lay, self.dx_routed, stream=stream)   # dispatch's gradient

    def step(self, stream=None):
        self.forward(stream)
        self.backward(stream)

    def results(self):
        return [self.out, self.dx_routed, self.dx_shared, self.dw, self.dw13, self.dw2, self.ds13, self.ds2]

    def clear(self):
        for t in (self.rx, self.pre, self.h, self.y, self.out0, self.out, self.dy, self.drx, self.dpre, *self.results()):
            t.zero_()


def exact(L):
    """The layer in 64 bits, by autograd."""
    leaf = lambda t: t.double().requires_grad_(True)  # noqa: E731
    xr, xs, w, w13, w2, s13, s2 = map(leaf, (L.x, L.x, L.w, L.w13, L.w2, L.s13, L.s2))

    def ffn(v, a, b):
        z = v @ a.T
        return (z[:, :L.I] * sigmoid(z[:, :L.I]) * z[:, L.I:]) @ b.T

    out = ffn(xs, s13, s2)
    for e in range(L.E):
        for j in range(L.k):
            t = torch.nonzero((L.idx[:, j] == e) & (L.lay.slot_idx[:, j] >= 0))[:, 0]
            out = out.index_add(0, t, w[t, j, None] * ffn(xr[t], w13[e], w2[e]))
    out.backward(L.dout.double())
    return [out.detach(), xr.grad, xs.grad, w.grad, w13.grad, w2.grad, s13.grad, s2.grad]


@pytest.mark.parametrize("seed,kw", [(1, {}), (2, dict(T=64, H=256, E=4, k=3, I=128, cap=20)),
                                     (3, dict(T=1, H=64, E=3, k=1, I=16)), (4, dict(T=517, H=520, E=3, k=2, I=264))])
def test_layer_against_autograd(seed, kw):
    """On the way to a result at most six values are rounded to bf16 (rows, preact, h, y, dy, dpre):
    each by half a step, 2^-9 in the root mean square of values spread over a binade, and they are
    independent, so 2-norms stay within 6 * 2^-9 of the result's; twice that is allowed."""
    print("[gpu-moe-layer]", seed, kw, flush=True)
    L = Layer(seed, **kw)
    L.step()
    torch.cuda.synchronize()
    for name, got, ref in zip(("out", "dx routed", "dx shared", "dw", "dw13", "dw2", "ds13", "ds2"), L.results(), exact(L)):
        assert torch.isfinite(got).all(), name
        off, norm = (got.double() - ref).norm().item(), ref.norm().item()
        assert off <= 12 * 2.0 ** -9 * norm + 1e-12, (name, off / max(norm, 1e-30))


def test_layer_captured_and_replayed():
    """The whole training step in one graph, replayed between eager steps of another layer and with
    other inputs: every replay equals the eager step on its inputs, bit for bit."""
    L, other = Layer(11), Layer(12)
    wants = []
    for src in (L, other):
        src.step()
        torch.cuda.synchronize()
        wants.append([t.clone() for t in src.results()])
    mine = L.idx.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            L.step()
    torch.cuda.synchronize()
    for rep in range(4):
        print("[gpu-moe-layer] replay", rep, flush=True)
        L.clear()
        if rep == 3:                       # other tokens and routing through the same graph
            for dst, src in zip((L.x, L.idx, L.w, L.dout, L.w13, L.w2, L.s13, L.s2),
                                (other.x, other.idx, other.w, other.dout, other.w13, other.w2, other.s13, other.s2)):
                dst.copy_(src)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(L.results(), wants[1] if rep == 3 else wants[0]):
            assert torch.equal(got, want), rep
        other.step()                       # eager work between the replays
        torch.cuda.synchronize()
        for got, want in zip(other.results(), wants[1]):
            assert torch.equal(got, want)
    assert not torch.equal(mine, L.idx)    # the last replay did see another routing


def test_two_layers_on_two_streams():
    a, b = Layer(21, T=700, H=256, I=136), Layer(22, T=300, H=512, E=8, k=3)
    wants = []
    for src in (a, b):
        src.step()
        torch.cuda.synchronize()
        wants.append([t.clone() for t in src.results()])
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for rep in range(3):
        print("[gpu-moe-layer] two streams", rep, flush=True)
        a.clear()
        b.clear()
        torch.cuda.synchronize()
        a.step(sa)
        b.step(sb)
        torch.cuda.synchronize()
        for src, want in zip((a, b), wants):
            for got, w in zip(src.results(), want):
                assert torch.equal(got, w)
