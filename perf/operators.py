"""The operators between dispatch and combine, in plain torch and as the library's kernels.

  experts       the experts' products over a receive buffer, ragged by expert, with bias and
                activation in the epilogue (bf16, fp16, FP8 with fp32 scales, MXFP8)
  experts_grad  their backward pass: the rows' gradient through the activation that made the
                rows, and the weights' and biases' gradients
  linear        a dense product with bias, activation and residual (shared expert, router)
  linear_grad   its backward pass
  combine_grad  the backward pass of the weighted combine

With ``own`` false, ``run`` computes in elementary torch operations in fp32; with ``own`` true it
calls the library.  Rows of a receive buffer that no pair uses are neither read nor written.
"""
import math

import torch

own = False

_ELEM = {"bf16": torch.bfloat16, "fp16": torch.float16}
_BLOCK = 128                       # channels per fp32 scale, and rows per weight scale
_ACTS = ("none", "relu", "gelu", "silu", "swiglu")


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # a small layer's forward pass: latency of one call counts
        dict(name="experts_tiny_bf16", op="experts", dtype="bf16", T=128, H=256, E=8, k=2, cap=0,
             N=512, act="swiglu", bias=False, train=False, routing="uniform", masked=0),
        # a decode step: four rows per expert, so the weights' bytes are all that counts
        dict(name="experts_decode_mxfp8", op="experts", dtype="mxfp8", T=128, H=7168, E=256, k=8,
             cap=128, N=512, act="swiglu", bias=False, train=False, routing="uniform", masked=0),
        # serving prefill after an FP8 dispatch: 256 rows per expert on average
        dict(name="experts_prefill_fp8", op="experts", dtype="fp8", T=8192, H=7168, E=256, k=8,
             cap=0, N=2048, act="swiglu", bias=False, train=False, routing="uniform", masked=0),
        # training forward of a large batch with a shared expert: keeps the pre-activation
        dict(name="experts_large_bf16", op="experts", dtype="bf16", T=65536, H=4096, E=64, k=6,
             cap=0, N=1024, act="swiglu", bias=False, train=True, routing="shared", masked=0),
        # backward of the experts' second product under skewed routing, fp32 weight gradients
        dict(name="experts_grad_skewed_bf16", op="experts_grad", dtype="bf16", T=8192, H=2048,
             E=32, k=8, cap=0, N=4096, act="swiglu", bias=False, grad="f32", routing="skewed",
             masked=0),
        # small odd sizes with biases and unrouted pairs
        dict(name="experts_grad_odd_fp16", op="experts_grad", dtype="fp16", T=601, H=520, E=24,
             k=3, cap=0, N=392, act="gelu", bias=True, grad="elem", routing="uniform", masked=10),
        # the shared expert's first product in a decode step
        dict(name="linear_decode_bf16", op="linear", dtype="bf16", T=16, H=7168, N=2048,
             act="swiglu", bias=False, residual=False, train=False),
        # a dense layer of a prefill or training batch with everything in its epilogue
        dict(name="linear_prefill_bf16", op="linear", dtype="bf16", T=8192, H=7168, N=4096,
             act="gelu", bias=True, residual=True, train=True),
        # its backward pass
        dict(name="linear_grad_prefill_bf16", op="linear_grad", dtype="bf16", T=8192, H=7168,
             N=4096, act="gelu", bias=True, grad="elem"),
        dict(name="linear_grad_odd_fp16", op="linear_grad", dtype="fp16", T=777, H=1000, N=504,
             act="silu", bias=True, grad="f32"),
        # training backward of the combine at prefill size, and of a small padded batch
        dict(name="combine_grad_prefill_bf16", op="combine_grad", dtype="bf16", T=8192, H=7168,
             E=256, k=8, cap=0, routing="uniform", masked=0),
        dict(name="combine_grad_small_fp16", op="combine_grad", dtype="fp16", T=128, H=7168,
             E=256, k=8, cap=16, routing="uniform", masked=5),
    ]


def _log(rng, lo, hi, step=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(step, v // step * step)


def draw(rng):
    while True:                         # nothing that costs more than the largest listed case
        c = _draw(rng)
        w = work(c)
        if w["flops"] <= 6.5e12 and w["bytes"] <= 8e9:
            return c


def _draw(rng):
    op = rng.choice(["experts", "experts", "experts_grad", "linear", "linear_grad", "combine_grad"])
    train = rng.random() < 0.4
    dtype = rng.choice(["bf16", "fp16"])
    act = rng.choice(_ACTS)
    if op in ("linear", "linear_grad"):
        c = dict(op=op, dtype=dtype, T=_log(rng, 1, 16384), H=_log(rng, 64, 8192, 8),
                 N=_log(rng, 64, 8192, 8), act=act, bias=rng.random() < 0.5)
        if op == "linear":
            c.update(residual=rng.random() < 0.5, train=train)
        else:
            c.update(grad=rng.choice(["elem", "f32"]), act=rng.choice(_ACTS[:4]))
        return c
    E, k = _log(rng, 2, 256), rng.randint(1, 8)
    c = dict(op=op, dtype=dtype, T=_log(rng, 1, 16384), H=_log(rng, 64, 7168, 8), E=E,
             k=min(k, E), cap=0, routing=rng.choice(["uniform", "skewed"]),
             masked=rng.choice([0, 0, 10]))
    if rng.random() < 0.3:
        c["cap"] = max(1, int(c["T"] * c["k"] / E * rng.uniform(0.5, 4.0)))
    if op == "combine_grad":
        return c
    c.update(N=_log(rng, 64, 2048, 8), act=act, bias=rng.random() < 0.3)
    if op == "experts_grad":
        c.update(grad=rng.choice(["elem", "f32"]))
        return c
    c.update(dtype=rng.choice(["bf16", "fp16", "fp8", "mxfp8"]), train=train)
    if c["dtype"] in ("fp8", "mxfp8"):
        c.update(H=max(128, c["H"] // 128 * 128), N=max(128, c["N"] // 128 * 128))
    return c


# ------------------------------------------------------------------------------------ inputs
def _elem(case):
    return _ELEM.get(case["dtype"], torch.bfloat16)


def _width(n, act):
    """Rows of the weights that make n outputs: gate and up halves for swiglu."""
    return 2 * n if act == "swiglu" else n


def _route(case, g):
    """Top-k expert ids [T, k] (-1 for a masked pair)."""
    T, E, k = case["T"], case["E"], case["k"]
    score = torch.rand((T, E), device="cuda", generator=g)
    if case["routing"] == "skewed":     # Zipf(1.2) popularity, sampled without replacement
        p = -1.2 * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
        score = p - torch.log(-torch.log(score.clamp(1e-7, 1 - 1e-6)))
    elif case["routing"] == "shared":   # expert 0 takes every token
        score[:, 0] = 2.0
    idx = score.topk(k, dim=1).indices
    if case["masked"]:
        drop = torch.rand((T, k), device="cuda", generator=g) * 100 < case["masked"]
        idx = torch.where(drop, torch.full_like(idx, -1), idx)
    return idx


def _slots(case, idx):
    """The routing layout in plain torch: the first row of each expert, its rows, and the
    receive row of every pair (-1: none)."""
    E, cap = case["E"], case["cap"]
    flat = idx.reshape(-1)
    key = torch.where(flat < 0, torch.full_like(flat, E), flat)
    demand = torch.bincount(key, minlength=E + 1)[:E]
    order = torch.sort(key, stable=True).indices
    first = torch.cumsum(demand, 0) - demand
    rank = torch.empty_like(flat)
    rank[order] = torch.arange(flat.numel(), device=flat.device)
    ok = flat >= 0
    e = flat.clamp(min=0)
    rank = rank - first[e]
    if cap:
        begin, rows = torch.arange(E, device=flat.device) * cap, demand.clamp(max=cap)
        ok = ok & (rank < cap)
    else:
        begin, rows = first, demand
    slot = torch.where(ok, begin[e] + rank, torch.full_like(flat, -1)).reshape(idx.shape)
    return begin.tolist(), rows.tolist(), slot


def _rows(case):
    return case["E"] * case["cap"] if case["cap"] else case["T"] * case["k"]


def _randn(shape, scale, dtype, g):
    return torch.randn(shape, device="cuda", dtype=dtype, generator=g).mul_(scale)


def _quant_rows(x, mx):
    """E4M3 codes and scales of rows: one fp32 scale per 128 channels, or E8M0 per 32."""
    n = 32 if mx else _BLOCK
    b = x.float().reshape(x.shape[0], -1, n)
    a = b.abs().amax(-1)
    if mx:
        byte = (torch.floor(torch.log2(a.clamp(min=2.0 ** -100))) - 8).clamp(-127, 127) + 127
        s, keep = torch.exp2(byte - 127), byte.to(torch.uint8)
    else:
        s = keep = a.clamp(min=1e-4) / 448.0
    q = (b / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return q.reshape(x.shape), keep


def _quant_blocks(w):
    """E4M3 codes and one fp32 scale per 128 x 128 block of a weight matrix."""
    n, k = w.shape
    b = w.float().reshape(n // _BLOCK, _BLOCK, k // _BLOCK, _BLOCK)
    s = b.abs().amax((1, 3)).clamp(min=1e-4) / 448.0
    q = (b / s[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return q.reshape(n, k), s


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s, op, dt = {"case": case}, case["op"], _elem(case)
    H, T = case["H"], case["T"]
    if "E" in case:
        s["topk_idx"] = _route(case, g)
        s["begin"], s["rows"], s["slot"] = _slots(case, s["topk_idx"])
        R, E = _rows(case), case["E"]
    if op == "combine_grad":
        s["dout"] = _randn((T, H), 1.0, dt, g)
        s["y"] = _randn((R, H), 1.0, dt, g)
        s["w"] = torch.rand((T, case["k"]), device="cuda", generator=g)
        s["dy"] = torch.zeros((R, H), dtype=dt, device="cuda")
        s["dw"] = torch.zeros((T, case["k"]), device="cuda")
        return s
    N, act = case["N"], case["act"]
    wscale = 1.0 / math.sqrt(H)
    if op == "experts":
        Nw = _width(N, act)
        if case["dtype"] in _ELEM:
            s["x"] = _randn((R, H), 1.0, dt, g)
            s["weights"] = _randn((E, Nw, H), wscale, dt, g)
            s["x_scales"] = s["w_scales"] = None
        else:
            mx = case["dtype"] == "mxfp8"
            s["x"], s["x_scales"] = _quant_rows(_randn((R, H), 1.0, dt, g), mx)
            s["weights"] = torch.empty((E, Nw, H), dtype=torch.uint8, device="cuda")
            s["w_scales"] = torch.empty((E, Nw, H // 32) if mx else (E, Nw // _BLOCK, H // _BLOCK),
                                        dtype=torch.uint8 if mx else torch.float32, device="cuda")
            for e in range(E):
                w = _randn((Nw, H), wscale, torch.float32, g)
                s["weights"][e], s["w_scales"][e] = _quant_rows(w, True) if mx else _quant_blocks(w)
        s["bias"] = _randn((E, Nw), 0.1, dt, g) if case["bias"] else None
        s["out"] = torch.zeros((R, N), dtype=dt, device="cuda")
        s["preact"] = torch.zeros((R, Nw), dtype=dt, device="cuda") if case["train"] else None
    elif op == "experts_grad":
        # a product of [rows, H] with [E, N, H] whose rows came out of `act`
        s["x"] = _randn((R, H), 1.0, dt, g)
        s["preact"] = _randn((R, _width(H, act)), 1.0, dt, g) if act != "none" else None
        s["weights"] = _randn((E, N, H), wscale, dt, g)
        s["dy"] = _randn((R, N), 1.0, dt, g)
        s["dx"] = torch.zeros((R, _width(H, act)), dtype=dt, device="cuda")
        gt = torch.float32 if case["grad"] == "f32" else dt
        s["dweights"] = torch.zeros((E, N, H), dtype=gt, device="cuda")
        s["dbias"] = torch.zeros((E, N), dtype=gt, device="cuda") if case["bias"] else None
    elif op == "linear":
        Nw = _width(N, act)
        s["x"] = _randn((T, H), 1.0, dt, g)
        s["weights"] = _randn((Nw, H), wscale, dt, g)
        s["bias"] = _randn((Nw,), 0.1, dt, g) if case["bias"] else None
        s["residual"] = _randn((T, N), 1.0, dt, g) if case["residual"] else None
        s["out"] = torch.zeros((T, N), dtype=dt, device="cuda")
        s["preact"] = torch.zeros((T, Nw), dtype=dt, device="cuda") if case["train"] else None
    else:                               # linear_grad: y = act(x W^T + b)
        s["x"] = _randn((T, H), 1.0, dt, g)
        s["weights"] = _randn((N, H), wscale, dt, g)
        s["preact"] = _randn((T, N), 1.0, dt, g)
        s["dy"] = _randn((T, N), 1.0, dt, g)
        s["dz"] = torch.zeros((T, N), dtype=dt, device="cuda")
        s["dx"] = torch.zeros((T, H), dtype=dt, device="cuda")
        gt = torch.float32 if case["grad"] == "f32" else dt
        s["dweights"] = torch.zeros((N, H), dtype=gt, device="cuda")
        s["dbias"] = torch.zeros((N,), dtype=gt, device="cuda") if case["bias"] else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:                             # the handle that dispatch and combine also take
        from combine_moe_layout_amd import binding as B
        if "E" in case:
            s["layout"] = B.EpLayout(case["T"], case["k"], case["E"], 1, case["cap"])
            B.ep_get_layout(s["topk_idx"], s["layout"])
        s["dtype"] = {"bf16": B.EP_BF16, "fp16": B.EP_F16, "fp8": B.EP_FP8_E4M3,
                      "mxfp8": B.EP_MXFP8_E4M3}[case["dtype"]]
        if "act" in case:
            s["act"] = {"none": B.EP_ACT_NONE, "relu": B.EP_ACT_RELU, "gelu": B.EP_ACT_GELU,
                        "silu": B.EP_ACT_SILU, "swiglu": B.EP_ACT_SWIGLU}[case["act"]]
        s["grad"] = B.EP_GRAD_F32 if case.get("grad") == "f32" else 0
    return s


# -------------------------------------------------------------------------------- plain forms
def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "swiglu":
        gate, up = z.chunk(2, dim=-1)
        return gate / (1 + torch.exp(-gate)) * up
    return z


def _act_grad(d, z, act):
    """d act(z) / dz times d; z is [.., 2n] for swiglu."""
    if act == "relu":
        return torch.where(z > 0, d, torch.zeros_like(d))
    if act == "gelu":
        return d * (0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
                    + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi))
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return d * p * (1 + z * (1 - p))
    if act == "swiglu":
        gate, up = z.chunk(2, dim=-1)
        p = 1 / (1 + torch.exp(-gate))
        return torch.cat([d * up * p * (1 + gate * (1 - p)), d * gate * p], dim=-1)
    return d


def _decode(q, scales, dtype):
    """fp32 values of a [rows, channels] operand."""
    if dtype in _ELEM:
        return q.float()
    v = q.view(torch.float8_e4m3fn).float()
    if dtype == "mxfp8":
        return v * torch.exp2(scales.float() - 127).repeat_interleave(32, dim=1)
    s = scales.repeat_interleave(_BLOCK, dim=1)
    return v * (s if s.shape[0] == v.shape[0] else s.repeat_interleave(_BLOCK, dim=0))


def _plain_experts(s):
    c = s["case"]
    # one product per expert: the rows of each are another matrix's
    for e, (b, n) in enumerate(zip(s["begin"], s["rows"])):
        if not n:
            continue
        fp8 = s["x_scales"] is not None
        x = _decode(s["x"][b:b + n], s["x_scales"][b:b + n] if fp8 else None, c["dtype"])
        w = _decode(s["weights"][e], s["w_scales"][e] if fp8 else None, c["dtype"])
        z = x @ w.T
        if s["bias"] is not None:
            z = z + s["bias"][e].float()
        if s["preact"] is not None:
            s["preact"][b:b + n] = z.to(s["preact"].dtype)
        s["out"][b:b + n] = _act(z, c["act"]).to(s["out"].dtype)
    return s["out"], s["preact"]


def _plain_experts_grad(s):
    c = s["case"]
    for e, (b, n) in enumerate(zip(s["begin"], s["rows"])):
        dy = s["dy"][b:b + n].float()
        d = dy @ s["weights"][e].float()
        if c["act"] != "none":
            d = _act_grad(d, s["preact"][b:b + n].float(), c["act"])
        s["dx"][b:b + n] = d.to(s["dx"].dtype)
        s["dweights"][e] = (dy.T @ s["x"][b:b + n].float()).to(s["dweights"].dtype)
        if s["dbias"] is not None:
            s["dbias"][e] = dy.sum(0).to(s["dbias"].dtype)
    return s["dx"], s["dweights"], s["dbias"]


def _plain_linear(s):
    z = s["x"].float() @ s["weights"].float().T
    if s["bias"] is not None:
        z = z + s["bias"].float()
    if s["preact"] is not None:
        s["preact"].copy_(z)
    a = _act(z, s["case"]["act"])
    if s["residual"] is not None:
        a = a + s["residual"].float()
    s["out"].copy_(a)
    return s["out"], s["preact"]


def _plain_linear_grad(s):
    c = s["case"]
    s["dz"].copy_(_act_grad(s["dy"].float(), s["preact"].float(), c["act"]))
    d = s["dz"].float()
    s["dx"].copy_(d @ s["weights"].float())
    s["dweights"].copy_(d.T @ s["x"].float())
    if s["dbias"] is not None:
        s["dbias"].copy_(d.sum(0))
    return s["dz"], s["dx"], s["dweights"], s["dbias"]


def _plain_combine_grad(s):
    slot = s["slot"].reshape(-1)
    pair = torch.nonzero(slot >= 0).reshape(-1)
    row, token = slot[pair], pair // s["case"]["k"]
    d = s["dout"].float()[token]
    s["dy"][row] = (d * s["w"].reshape(-1)[pair, None]).to(s["dy"].dtype)
    dw = torch.zeros(slot.numel(), device=slot.device)
    dw[pair] = (d * s["y"][row].float()).sum(-1)
    s["dw"].copy_(dw.reshape(s["dw"].shape))
    return s["dy"], s["dw"]


# ------------------------------------------------------------------------- the library's calls
def _own_experts(s):
    from combine_moe_layout_amd import binding as B
    B.ep_expert_gemm(s["x"], s["weights"], s["layout"], s["out"], s["dtype"], act=s["act"],
                     x_scales=s["x_scales"], weight_scales=s["w_scales"], bias=s["bias"],
                     preact=s["preact"])
    return s["out"], s["preact"]


def _own_experts_grad(s):
    from combine_moe_layout_amd import binding as B
    B.ep_expert_gemm_grad_x(s["dy"], s["weights"], s["layout"], s["dx"], s["dtype"], act=s["act"],
                            preact=s["preact"])
    B.ep_expert_gemm_grad_w(s["dy"], s["x"], s["layout"], s["dweights"], s["dtype"] | s["grad"],
                            dbias=s["dbias"])
    return s["dx"], s["dweights"], s["dbias"]


def _own_linear(s):
    from combine_moe_layout_amd import binding as B
    B.ep_linear(s["x"], s["weights"], s["out"], s["dtype"], act=s["act"], bias=s["bias"],
                residual=s["residual"], preact=s["preact"])
    return s["out"], s["preact"]


def _own_linear_grad(s):
    from combine_moe_layout_amd import binding as B
    B.ep_act_grad(s["dy"], s["preact"], s["dz"], s["dtype"], s["act"])
    B.ep_linear_grad_x(s["dz"], s["weights"], s["dx"], s["dtype"])
    B.ep_linear_grad_w(s["dz"], s["x"], s["dweights"], s["dtype"] | s["grad"], dbias=s["dbias"])
    return s["dz"], s["dx"], s["dweights"], s["dbias"]


def _own_combine_grad(s):
    from combine_moe_layout_amd import binding as B
    B.ep_combine_grad(s["dout"], s["y"], s["w"], s["layout"], s["dy"], s["dw"], s["dtype"])
    return s["dy"], s["dw"]


_PLAIN = {"experts": _plain_experts, "experts_grad": _plain_experts_grad, "linear": _plain_linear,
          "linear_grad": _plain_linear_grad, "combine_grad": _plain_combine_grad}
_OWN = {"experts": _own_experts, "experts_grad": _own_experts_grad, "linear": _own_linear,
        "linear_grad": _own_linear_grad, "combine_grad": _own_combine_grad}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------------------------ floor and truth
def _touched(case):
    """Pairs with a row, and experts with at least one (their expectation)."""
    E = case["E"]
    pairs = case["T"] * case["k"] * (100 - case["masked"]) / 100
    if case["routing"] == "skewed":
        p = [(e + 1) ** -1.2 for e in range(E)]
        q = [min(1.0, x * case["k"] / sum(p)) for x in p]
    else:
        q = [case["k"] / E] * E
    if case["cap"]:
        pairs = sum(min(case["cap"], pairs * x / sum(q)) for x in q)
    return pairs, sum(1 - (1 - x) ** case["T"] for x in q)


def work(case):
    H, T, op = case["H"], case["T"], case["op"]
    if "E" in case:
        P, used = _touched(case)
    if op == "combine_grad":
        return {"bytes": 2 * T * H + 4 * P * H + 12 * T * case["k"], "flops": 3 * P * H}
    N, act = case["N"], case["act"]
    if op == "experts":
        Nw = _width(N, act)
        per = {"bf16": 2.0, "fp16": 2.0, "fp8": 1 + 4 / 128, "mxfp8": 1 + 1 / 32}[case["dtype"]]
        wper = 1 + 4 / _BLOCK ** 2 if case["dtype"] == "fp8" else per
        b = P * H * per + used * Nw * H * wper + 2 * P * (N + (Nw if case["train"] else 0))
        return {"bytes": b + (2 * used * Nw if case["bias"] else 0), "flops": 2 * P * H * Nw}
    if op == "experts_grad":
        Hw, g = _width(H, act), 4 if case["grad"] == "f32" else 2
        b = 2 * P * (N + H + Hw + (Hw if act != "none" else 0)) + 2 * used * N * H
        return {"bytes": b + g * case["E"] * N * (H + case["bias"]), "flops": 4 * P * H * N}
    if op == "linear":
        Nw = _width(N, act)
        b = 2 * (T * H + Nw * H + T * N * (1 + case["residual"]) + (T * Nw if case["train"] else 0))
        return {"bytes": b + (2 * Nw if case["bias"] else 0), "flops": 2 * T * H * Nw}
    g = 4 if case["grad"] == "f32" else 2
    b = 2 * (3 * T * N + 2 * T * H + N * H) + g * N * (H + case["bias"])
    return {"bytes": b, "flops": 4 * T * H * N}


def _f64(q, scales, dtype):
    v = q.view(torch.float8_e4m3fn).double() if dtype in ("fp8", "mxfp8") else q.double()
    if dtype == "mxfp8":
        n, k = v.shape
        return (v.view(n, k // 32, 32) * (2.0 ** (scales.double() - 127)).unsqueeze(2)).view(n, k)
    if dtype == "fp8":
        rows = v.shape[0] // scales.shape[0]
        n, k = scales.shape
        return (v.view(n, rows, k, _BLOCK) * scales.double().view(n, 1, k, 1)).reshape(v.shape)
    return v


def _f64_act(z, act):
    """(act(z), act'(z)) from the definitions in 64 bits."""
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    if act == "gelu":
        phi = torch.special.ndtr(z)
        return z * phi, phi + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "silu":
        p = torch.special.expit(z)
        return z * p, p + z * p * torch.special.expit(-z)
    return z, torch.ones_like(z)


def exact(case, seed):
    s = _inputs(case, seed)
    op, H = case["op"], case["H"]
    act, N = case.get("act"), case.get("N")
    if op == "combine_grad":
        dy, dw = s["dy"].double(), s["dw"].double()
        for j in range(case["k"]):      # one choice of every token at a time
            t = torch.nonzero(s["slot"][:, j] >= 0)[:, 0]
            r = s["slot"][t, j]
            d = s["dout"][t].double()
            dy[r] = s["w"][t, j].double()[:, None] * d
            dw[t, j] = torch.einsum("th,th->t", d, s["y"][r].double())
        return dy, dw
    if op == "linear":
        z = s["x"].double() @ s["weights"].double().T
        z = z if s["bias"] is None else z + s["bias"].double()
        a = _f64_act(z[:, :N], "silu")[0] * z[:, N:] if act == "swiglu" else _f64_act(z, act)[0]
        a = a if s["residual"] is None else a + s["residual"].double()
        return a, None if s["preact"] is None else z
    if op == "linear_grad":
        d = s["dy"].double() * _f64_act(s["preact"].double(), act)[1]
        # the later products take the rounded gradient, as both sides hand it over
        r = d.to(s["dz"].dtype).double()
        return (d, r @ s["weights"].double(), r.T @ s["x"].double(),
                None if s["dbias"] is None else r.sum(0))
    if op == "experts":
        out = s["out"].double()
        pre = None if s["preact"] is None else s["preact"].double()
        for e in range(case["E"]):
            if not s["rows"][e]:
                continue
            at = slice(s["begin"][e], s["begin"][e] + s["rows"][e])
            fp8 = s["x_scales"] is not None
            z = torch.mm(_f64(s["x"][at], s["x_scales"][at] if fp8 else None, case["dtype"]),
                         _f64(s["weights"][e], s["w_scales"][e] if fp8 else None, case["dtype"]).T)
            z = z if s["bias"] is None else z + s["bias"][e].double()
            if pre is not None:
                pre[at] = z
            out[at] = (_f64_act(z[:, :N], "silu")[0] * z[:, N:] if act == "swiglu"
                       else _f64_act(z, act)[0])
        return out, pre
    dx, dw = s["dx"].double(), s["dweights"].double()
    db = None if s["dbias"] is None else s["dbias"].double()
    for e in range(case["E"]):
        at = slice(s["begin"][e], s["begin"][e] + s["rows"][e])
        dy = s["dy"][at].double()
        d = dy @ s["weights"][e].double()
        z = s["preact"][at].double() if act != "none" else None
        if act == "swiglu":
            v, v1 = _f64_act(z[:, :H], "silu")
            dx[at] = torch.cat([d * z[:, H:] * v1, d * v], 1)
        else:
            dx[at] = d if act == "none" else d * _f64_act(z, act)[1]
        dw[e] = dy.T @ s["x"][at].double()
        if db is not None:
            db[e] = dy.sum(0)
    return dx, dw, db
