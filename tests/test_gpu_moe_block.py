"""A whole mixture-of-experts block from its entry points: the norm before it, the router's logits
and choice, dispatch, the experts' products, combine, and the norm after it with gate and residual;
as a training step with every gradient against 64-bit autograd, and as a serving step in 8-bit
integers; captured in a graph; on two streams."""
import pytest
import torch

import block_ref as ref
from combine_moe_layout_amd import binding as B
from products_ref import segments, sigmoid

pytestmark = pytest.mark.gpu
DT, BF, F32 = torch.bfloat16, B.EP_BF16, torch.float32
EPS = 1e-6


class Block:
    """T tokens of H, E experts of I; out = residual + gate * norm(experts(norm(residual)))."""

    def __init__(self, seed, T=203, H=128, E=16, k=3, I=80, cap=0, score=B.EP_SCORE_SIGMOID):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        rn = lambda *s, scale=1.0: (torch.randn(s, device="cuda", generator=g) * scale).to(DT)  # noqa: E731
        z = lambda *s, dt=DT: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
        self.T, self.H, self.E, self.k, self.I = T, H, E, k, I
        self.router = B.EpRouter(E, k, score, num_groups=4, topk_groups=3, group_top=2, renormalize=True, scale=1.5)
        self.score = "sigmoid" if score == B.EP_SCORE_SIGMOID else "softmax"
        self.x, self.gate = rn(T, H), torch.rand(T, device="cuda", generator=g)
        self.n1, self.n2, self.n3 = (rn(H, scale=0.1) + 1 for _ in range(3))
        self.wr, self.bias = rn(E, H, scale=H ** -0.5), torch.randn(E, device="cuda", generator=g) * 0.05
        self.w13, self.w2 = rn(E, 2 * I, H, scale=H ** -0.5), rn(E, H, I, scale=I ** -0.5)
        self.q13, self.s13 = z(E, 2 * I, H, dt=torch.int8), z(E, 2 * I, dt=F32)
        self.q2, self.s2 = z(E, H, I, dt=torch.int8), z(E, H, dt=F32)
        B.ep_quantize_int8(self.w13.view(-1, H), self.q13.view(-1, H), self.s13.view(-1), BF)
        B.ep_quantize_int8(self.w2.view(-1, I), self.q2.view(-1, I), self.s2.view(-1), BF)
        self.dout, self.dnext = rn(T, H), rn(T, H)
        self.lay = B.EpLayout(T, k, E, 1, cap)
        R = self.lay.num_recv_rows
        self.u, self.logits, self.idx, self.w = z(T, H), z(T, E), z(T, k, dt=torch.int64), z(T, k, dt=F32)
        self.rx, self.pre, self.h, self.y = z(R, H), z(R, 2 * I), z(R, I), z(R, H)
        self.rq, self.rs, self.hq, self.hs = z(R, H, dt=torch.int8), z(R, dt=F32), z(R, I, dt=torch.int8), z(R, dt=F32)
        self.c, self.out, self.next = z(T, H), z(T, H), z(T, H)
        self.dc, self.dres, self.dgate = z(T, H), z(T, H), z(T, dt=F32)
        self.dn1, self.dn2, self.dn3 = (z(H, dt=F32) for _ in range(3))
        self.dy, self.dw, self.dpre, self.drx = z(R, H), z(T, k, dt=F32), z(R, 2 * I), z(R, H)
        self.dw13, self.dw2 = z(E, 2 * I, H, dt=F32), z(E, H, I, dt=F32)
        self.dlogits, self.dwr, self.du, self.du2, self.dx = z(T, E), z(E, H, dt=F32), z(T, H), z(T, H), z(T, H)
        self.ws = torch.empty(B.ep_block_norm_grad_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
        self.ones = torch.ones((T, k), device="cuda")

    def choose(self, stream=None):
        B.ep_block_norm(None, self.x, None, BF, EPS, pre_weight=self.n1, normed=self.u, stream=stream)
        B.ep_linear(self.u, self.wr, self.logits, BF, stream=stream)
        B.ep_route(self.logits, self.router, self.idx, self.w, BF, bias=self.bias, stream=stream)

    def close(self, stream=None):
        B.ep_combine(self.y, self.w, self.lay, self.c, stream=stream)
        B.ep_block_norm(self.c, self.x, self.out, BF, EPS, self.n2, self.gate, 1.0, self.n3, self.next, stream=stream)

    def forward(self, stream=None):
        self.choose(stream)
        B.ep_layout_dispatch(self.idx, self.lay, self.u, BF, self.rx, stream=stream)
        B.ep_expert_gemm(self.rx, self.w13, self.lay, self.h, BF, act=B.EP_ACT_SWIGLU, preact=self.pre, stream=stream)
        B.ep_expert_gemm(self.h, self.w2, self.lay, self.y, BF, stream=stream)
        self.close(stream)

    def serve(self, stream=None):
        self.choose(stream)
        B.ep_layout_dispatch(self.idx, self.lay, self.u, B.EP_INT8, self.rq, self.rs, stream=stream)
        B.ep_expert_gemm(self.rq, self.q13, self.lay, self.h, B.EP_INT8, act=B.EP_ACT_SWIGLU, x_scales=self.rs,
                         weight_scales=self.s13, stream=stream)
        B.ep_quantize_int8(self.h, self.hq, self.hs, BF, layout=self.lay, stream=stream)
        B.ep_expert_gemm(self.hq, self.q2, self.lay, self.y, B.EP_INT8, x_scales=self.hs, weight_scales=self.s2,
                         stream=stream)
        self.close(stream)

    def backward(self, stream=None):
        F = BF | B.EP_GRAD_F32
        B.ep_block_norm_grad(self.dout, self.dnext, self.c, self.x, F, self.ws, EPS, self.n2, self.gate, 1.0, self.n3,
                             d_y=self.dc, d_residual=self.dres, d_gate=self.dgate, d_post_weight=self.dn2,
                             d_pre_weight=self.dn3, stream=stream)
        B.ep_combine_grad(self.dc, self.y, self.w, self.lay, self.dy, self.dw, BF, stream=stream)
        B.ep_expert_gemm_grad_x(self.dy, self.w2, self.lay, self.dpre, BF, act=B.EP_ACT_SWIGLU, preact=self.pre,
                                stream=stream)
        B.ep_expert_gemm_grad_w(self.dy, self.h, self.lay, self.dw2, F, stream=stream)
        B.ep_expert_gemm_grad_x(self.dpre, self.w13, self.lay, self.drx, BF, stream=stream)
        B.ep_expert_gemm_grad_w(self.dpre, self.rx, self.lay, self.dw13, F, stream=stream)
        B.ep_combine(self.drx, self.ones, self.lay, self.du, stream=stream)       # dispatch's gradient
        B.ep_route_grad(self.dw, self.logits, self.idx, self.router, self.dlogits, BF, stream=stream)
        B.ep_linear_grad_x(self.dlogits, self.wr, self.du2, BF, stream=stream)
        B.ep_linear_grad_w(self.dlogits, self.u, self.dwr, F, stream=stream)
        B.ep_block_norm(self.du, self.du2, self.du, BF, EPS, stream=stream)        # their sum
        B.ep_block_norm_grad(self.dres, self.du, None, self.x, F, self.ws, EPS, pre_weight=self.n1, d_residual=self.dx,
                             d_pre_weight=self.dn1, stream=stream)

    def step(self, stream=None):
        self.forward(stream)
        self.backward(stream)

    NAMES = ("out", "next", "dx", "dgate", "dn1", "dn2", "dn3", "dwr", "dw13", "dw2")

    def results(self):
        return [getattr(self, n) for n in self.NAMES]

    def clear(self):
        for t in (self.u, self.logits, self.idx, self.w, self.rx, self.pre, self.h, self.y, self.rq, self.rs, self.hq,
                  self.hs, self.c, self.dc, self.dres, self.dy, self.dw, self.dpre, self.drx, self.dlogits, self.du,
                  self.du2, *self.results()):
            t.zero_()
        self.ws.fill_(0xFF)


def exact(L, w13=None, w2=None):
    """The block in 64 bits with the choice as it was made, by autograd."""
    leaf = lambda t: t.double().requires_grad_(True)  # noqa: E731
    x, gate, n1, n2, n3, wr = map(leaf, (L.x, L.gate, L.n1, L.n2, L.n3, L.wr))
    w13, w2 = leaf(L.w13 if w13 is None else w13), leaf(L.w2 if w2 is None else w2)
    u = ref.unit(x, EPS) * n1
    w = ref.weights(u @ wr.T, L.idx, L.score, True, 1.5)
    c = torch.zeros_like(x)
    for e in range(L.E):
        for j in range(L.k):
            t = torch.nonzero((L.idx[:, j] == e) & (L.lay.slot_idx[:, j] >= 0))[:, 0]
            z = u[t] @ w13[e].T
            c = c.index_add(0, t, w[t, j, None] * ((z[:, :L.I] * sigmoid(z[:, :L.I]) * z[:, L.I:]) @ w2[e].T))
    out, nxt = ref.block_norm(c, x, EPS, n2, gate, 1.0, n3)
    ((out * L.dout.double()).sum() + (nxt * L.dnext.double()).sum()).backward()
    return [out.detach(), nxt.detach(), x.grad, gate.grad, n1.grad, n2.grad, n3.grad, wr.grad, w13.grad, w2.grad]


def valid_choice(L):
    """The choice is that of the logits as they were rounded, whatever they are."""
    want = ref.choice(L.logits, L.bias, L.k, L.score, 4, 3, 2)
    assert torch.equal(L.idx, want)


@pytest.mark.parametrize("seed,kw", [(1, {}), (2, dict(T=64, H=256, E=8, k=2, I=128, cap=20)), (3, dict(T=1, H=64, E=8, k=1, I=16)),
                                     (4, dict(T=517, H=528, E=24, k=2, I=272, score=B.EP_SCORE_SOFTMAX))])
def test_training_step_against_autograd(seed, kw):
    """On the way to a result at most twelve values are rounded to bf16 (u, logits, rows, preact, h, y,
    c; dc, dy, dpre, drx, du): 2^-9 each in the root mean square, independent of each other; the
    norms' and the router's slopes hand on no more than they get, relative to the result.  So 2-norms
    stay within 12 * 2^-9 of the result's, and twice that is allowed; d_gate and the router's
    gradients are differences of values up to four times as large."""
    print("[gpu-moe-block]", seed, kw, flush=True)
    L = Block(seed, **kw)
    L.step()
    torch.cuda.synchronize()
    valid_choice(L)
    for name, got, want in zip(L.NAMES, L.results(), exact(L)):
        assert torch.isfinite(got).all(), name
        off, norm = (got.double() - want).norm().item(), want.norm().item()
        limit = 24 * 2.0 ** -9 * (4 if name in ("dgate", "dwr") else 1)
        assert off <= limit * norm + 1e-9, (name, off / max(norm, 1e-30))


@pytest.mark.parametrize("seed,kw", [(1, {}), (5, dict(T=40, H=256, E=8, k=2, I=128, cap=16)), (6, dict(T=1500, H=384, E=8, k=2, I=208))])
def test_serving_step_in_int8(seed, kw):
    """Against the block in 64 bits on the weights that the codes stand for.  Rounding rows to 8 bits is
    off by at most half a step of max / 127: 0.29 of a step in the root mean square, for rows whose
    maximum is at most 5 times theirs 0.29 * 5 / 127 = 2^-6.4; that happens twice, and ten roundings to
    bf16 add 10 * 2^-9: together below 2 * 2^-6.4 + 2^-5.6 = 0.045 of the block's own part."""
    print("[gpu-moe-block] serving", seed, kw, flush=True)
    L = Block(seed, **kw)
    L.serve()
    torch.cuda.synchronize()
    valid_choice(L)
    w13 = L.q13.double() * L.s13.double()[..., None]
    w2 = L.q2.double() * L.s2.double()[..., None]
    out, nxt = exact(L, w13, w2)[:2]
    x = L.x.double()
    assert (L.out.double() - out).norm() <= 0.045 * (out - x).norm() + 2.0 ** -9 * out.norm()
    assert (L.next.double() - nxt).norm() <= 0.045 * nxt.norm() + 2.0 ** -9 * nxt.norm()
    q, s, _ = ref.int8_rows(L.u)                       # the rows on the way, exactly
    t, j = torch.nonzero(L.lay.slot_idx >= 0, as_tuple=True)
    at = L.lay.slot_idx[t, j].long()
    assert torch.equal(L.rq[at], q[t]) and torch.equal(L.rs[at], s[t])
    for b, n in segments(L.lay):
        q, s, _ = ref.int8_rows(L.h[b:b + n])
        assert torch.equal(L.hq[b:b + n], q) and torch.equal(L.hs[b:b + n], s)


@pytest.mark.parametrize("what", ["step", "serve"])
def test_captured_and_replayed(what):
    """The whole step in one graph, replayed between eager steps of another block and with other
    inputs: every replay equals the eager step on its inputs, bit for bit.  (An eager step's results
    live on while the other is captured.)"""
    L, other = Block(11), Block(12)
    run = lambda b, *a: getattr(b, what)(*a)  # noqa: E731
    wants = []
    for src in (L, other):
        run(src)
        torch.cuda.synchronize()
        wants.append([t.clone() for t in src.results()])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            run(L)
    torch.cuda.synchronize()
    inputs = ("x", "gate", "n1", "n2", "n3", "wr", "bias", "w13", "w2", "q13", "s13", "q2", "s2", "dout", "dnext")
    for rep in range(4):
        print("[gpu-moe-block] replay", what, rep, flush=True)
        L.clear()
        if rep == 3:
            for n in inputs:
                getattr(L, n).copy_(getattr(other, n))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n, got, want in zip(L.NAMES, L.results(), wants[1] if rep == 3 else wants[0]):
            assert torch.equal(got, want), (rep, n)
        run(other)
        torch.cuda.synchronize()
        for got, want in zip(other.results(), wants[1]):
            assert torch.equal(got, want)


def test_two_blocks_on_two_streams():
    a, b = Block(21, T=700, H=256, I=144), Block(22, T=300, H=512, E=8, k=3)
    for what in ("step", "serve"):
        wants = []
        for src in (a, b):
            src.clear()
            getattr(src, what)()
            torch.cuda.synchronize()
            wants.append([t.clone() for t in src.results()])
        sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
        for rep in range(3):
            print("[gpu-moe-block] two streams", what, rep, flush=True)
            a.clear()
            b.clear()
            torch.cuda.synchronize()
            getattr(a, what)(sa)
            getattr(b, what)(sb)
            torch.cuda.synchronize()
            for src, want in zip((a, b), wants):
                for got, w in zip(src.results(), want):
                    assert torch.equal(got, w)
