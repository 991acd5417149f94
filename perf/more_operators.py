"""The operators at the two ends of a mixture-of-experts block and its products in 8-bit integers,
in plain torch and as the library's kernels.

  route         the router's choice: softmax or sigmoid scores, a bias for balance, groups, top-k,
                renormalised weights; with ``train`` its gradient by the logits too
  norm          the norm after a block with its gate and residual scale, and the norm before the
                next one; with ``train`` their gradients too
  experts_int8  the experts' products in int8 with a scale for each token and channel, from the
                tokens (dispatch rounds them) or from the rows that a first product left
  linear_int8   a dense product of the same kind, its rows rounded within the call

With ``own`` false, ``run`` computes in elementary torch operations; with ``own`` true it calls the
library.  Rows of a receive buffer that no pair uses are neither read nor written.
"""
import math

import torch

own = False

_ELEM = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_ACTS = ("none", "relu", "gelu", "silu", "swiglu")
_MOST = 3.4028234663852886e38       # +inf logits count as the largest fp32 value
_EPS = 1e-6


# ------------------------------------------------------------------------------------- cases
def listed():
    v3 = dict(op="route", E=256, k=8, score="sigmoid", bias=True, groups=8, topk_groups=4,
              group_top=2, renorm=True, scale=2.5, masked=0)
    return [
        # a decode step's routing: latency of one call counts
        dict(v3, name="route_decode_bf16", T=16, dtype="bf16", train=False),
        # the routing of a serving prefill, by groups, with fp32 logits
        dict(v3, name="route_prefill_fp32", T=8192, dtype="fp32", train=False),
        # a large training batch with softmax scores, there and back
        dict(name="route_train_large_fp32", op="route", T=65536, E=64, k=6, dtype="fp32",
             score="softmax", bias=False, groups=1, topk_groups=1, group_top=1, renorm=True,
             scale=1.0, masked=0, train=True),
        # the end of one block and the start of the next in a decode step
        dict(name="norm_decode_bf16", op="norm", T=16, H=7168, dtype="bf16", post=True, gate=True,
             pre=True, alpha=1.0, train=False, grad="elem"),
        # the same at prefill size
        dict(name="norm_prefill_bf16", op="norm", T=8192, H=7168, dtype="bf16", post=True,
             gate=True, pre=True, alpha=0.7, train=False, grad="elem"),
        # a large training batch, there and back, fp32 gradients of the weights
        dict(name="norm_train_bf16", op="norm", T=16384, H=4096, dtype="bf16", post=True, gate=True,
             pre=True, alpha=1.0, train=True, grad="f32"),
        # small odd sizes without a norm after the block
        dict(name="norm_train_odd_fp16", op="norm", T=601, H=1000, dtype="fp16", post=False,
             gate=False, pre=True, alpha=1.0, train=True, grad="elem"),
        # a decode step: four rows per expert, so the weights' bytes are all that counts
        dict(name="experts_int8_decode", op="experts_int8", T=128, H=7168, E=256, k=8, cap=128,
             N=512, act="swiglu", bias=False, source="tokens", routing="uniform", masked=0),
        # serving prefill: 256 rows per expert on average
        dict(name="experts_int8_prefill", op="experts_int8", T=8192, H=7168, E=256, k=8, cap=0,
             N=2048, act="swiglu", bias=False, source="tokens", routing="uniform", masked=0),
        # its second product under skewed routing, from the activated rows of the first
        dict(name="experts_int8_second", op="experts_int8", T=8192, H=2048, E=32, k=8, cap=0,
             N=4096, act="none", bias=True, source="rows", routing="skewed", masked=0),
        # the shared expert's first product in a decode step
        dict(name="linear_int8_decode", op="linear_int8", T=16, H=7168, N=2048, act="swiglu",
             bias=False, residual=False),
        # a dense layer of a prefill with everything in its epilogue
        dict(name="linear_int8_prefill", op="linear_int8", T=8192, H=7168, N=4096, act="gelu",
             bias=True, residual=True),
    ]


def _log(rng, lo, hi, step=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(step, v // step * step)


def draw(rng):
    while True:                         # nothing that costs more than the largest listed case
        c = _draw(rng)
        w = work(c)
        if w["flops"] <= 3.8e12 and w["bytes"] <= 4.5e9:
            return c


def _draw(rng):
    op = rng.choice(["route", "norm", "experts_int8", "experts_int8", "linear_int8"])
    if op == "route":
        E, dtype = _log(rng, 2, 1024), rng.choice(["fp32", "fp32", "bf16", "fp16"])
        groups = rng.choice([g for g in (1, 1, 2, 4, 8) if E % g == 0])
        topk_groups = rng.randint(1, groups)
        k = rng.randint(1, min(16, E // groups * topk_groups))
        return dict(op=op, T=_log(rng, 1, 65536 if E <= 256 else 16384), E=E, k=k, dtype=dtype,
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups,
                    topk_groups=topk_groups, group_top=rng.choice([1, 2]) if E > groups else 1,
                    renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]),
                    masked=rng.choice([0, 0, 20]), train=rng.random() < 0.5)
    if op == "norm":
        post, pre = rng.choice([(True, True), (True, True), (False, True), (True, False)])
        return dict(op=op, T=_log(rng, 1, 16384), H=_log(rng, 8, 16384, 8),
                    dtype=rng.choice(["bf16", "fp16"]), post=post, gate=rng.random() < 0.5, pre=pre,
                    alpha=rng.choice([1.0, 0.5]), train=rng.random() < 0.5,
                    grad=rng.choice(["elem", "f32"]))
    if op == "linear_int8":
        return dict(op=op, T=_log(rng, 1, 16384), H=_log(rng, 64, 8192, 16), N=_log(rng, 64, 8192, 8),
                    act=rng.choice(_ACTS), bias=rng.random() < 0.5, residual=rng.random() < 0.5)
    E = _log(rng, 2, 256)
    c = dict(op=op, T=_log(rng, 1, 16384), H=_log(rng, 64, 7168, 16), E=E, k=min(rng.randint(1, 8), E),
             cap=0, N=_log(rng, 64, 2048, 8), act=rng.choice(_ACTS), bias=rng.random() < 0.3,
             source=rng.choice(["tokens", "rows"]), routing=rng.choice(["uniform", "skewed"]),
             masked=rng.choice([0, 0, 10]))
    if rng.random() < 0.3:
        c["cap"] = max(1, int(c["T"] * c["k"] / E * rng.uniform(0.5, 4.0)))
    return c


# ------------------------------------------------------------------------------------ inputs
def _width(n, act):
    """Rows of the weights that make n outputs: gate and up halves for swiglu."""
    return 2 * n if act == "swiglu" else n


def _topk(case, g):
    """Top-k expert ids [T, k] (-1 for a masked pair)."""
    T, E, k = case["T"], case["E"], case["k"]
    score = torch.rand((T, E), device="cuda", generator=g)
    if case["routing"] == "skewed":     # Zipf(1.2) popularity, sampled without replacement
        p = -1.2 * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
        score = p - torch.log(-torch.log(score.clamp(1e-7, 1 - 1e-6)))
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


def _randn(shape, scale, dtype, g):
    return torch.randn(shape, device="cuda", dtype=dtype, generator=g).mul_(scale)


def _channels(shape, scale, g):
    """A matrix of int8 codes, rounded from normal values by its rows, and the rows' scales."""
    q = torch.empty(shape, dtype=torch.int8, device="cuda")
    s = torch.empty(shape[:-1], device="cuda")
    for e in range(shape[0] if len(shape) == 3 else 1):
        at = e if len(shape) == 3 else slice(None)
        w = _randn(shape[-2:], scale, torch.float32, g)
        s[at] = w.abs().amax(-1) / 127
        q[at] = torch.round(w / s[at][:, None]).to(torch.int8)
    return q, s


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s, op, T = {"case": case}, case["op"], case["T"]
    zeros = lambda *shape, dt=torch.float32: torch.zeros(shape, dtype=dt, device="cuda")  # noqa: E731
    if op == "route":
        E, k, dt = case["E"], case["k"], _ELEM[case["dtype"]]
        s["logits"] = _randn((T, E), 1.0, torch.float32, g)
        if case["masked"]:              # experts that a token may not go to; every 16th row has none
            dead = torch.rand((T, E), device="cuda", generator=g) * 100 < case["masked"]
            dead[::16] = True
            s["logits"].masked_fill_(dead, -math.inf)
        s["logits"] = s["logits"].to(dt)
        s["bias"] = _randn((E,), 0.05, torch.float32, g) if case["bias"] else None
        s["idx"], s["w"] = zeros(T, k, dt=torch.int64), zeros(T, k)
        if case["train"]:
            s["dw"], s["dlogits"] = _randn((T, k), 1.0, torch.float32, g), zeros(T, E, dt=dt)
        return s
    H = case["H"]
    if op == "norm":
        dt = _ELEM[case["dtype"]]
        s["y"], s["residual"] = _randn((T, H), 1.0, dt, g), _randn((T, H), 1.0, dt, g)
        s["post"] = _randn((H,), 0.1, dt, g).add_(1) if case["post"] else None
        s["gate"] = torch.rand((T,), device="cuda", generator=g) if case["gate"] else None
        s["pre"] = _randn((H,), 0.1, dt, g).add_(1) if case["pre"] else None
        s["out"] = zeros(T, H, dt=dt)
        s["normed"] = zeros(T, H, dt=dt) if case["pre"] else None
        if case["train"]:
            gt = torch.float32 if case["grad"] == "f32" else dt
            s["dout"] = _randn((T, H), 1.0, dt, g)
            s["dnormed"] = _randn((T, H), 1.0, dt, g) if case["pre"] else None
            s["dy"], s["dresidual"] = zeros(T, H, dt=dt), zeros(T, H, dt=dt)
            s["dgate"] = zeros(T) if case["gate"] else None
            s["dpost"] = zeros(H, dt=gt) if case["post"] else None
            s["dpre"] = zeros(H, dt=gt) if case["pre"] else None
        return s
    bf, N = torch.bfloat16, case["N"]
    Nw, wscale = _width(N, case["act"]), 1.0 / math.sqrt(H)
    if op == "linear_int8":
        s["x"] = _randn((T, H), 1.0, bf, g)
        s["q"], s["s"] = zeros(T, H, dt=torch.int8), zeros(T)
        s["weights"], s["ws"] = _channels((Nw, H), wscale, g)
        s["bias"] = _randn((Nw,), 0.1, bf, g) if case["bias"] else None
        s["residual"] = _randn((T, N), 1.0, bf, g) if case["residual"] else None
        s["out"] = zeros(T, N, dt=bf)
        return s
    E = case["E"]
    R = E * case["cap"] if case["cap"] else T * case["k"]
    s["topk_idx"] = _topk(case, g)
    s["begin"], s["rows"], s["slot"] = _slots(case, s["topk_idx"])
    s["x"] = _randn((T if case["source"] == "tokens" else R, H), 1.0, bf, g)
    s["q"], s["s"] = zeros(R, H, dt=torch.int8), zeros(R)
    s["weights"], s["ws"] = _channels((E, Nw, H), wscale, g)
    s["bias"] = _randn((E, Nw), 0.1, bf, g) if case["bias"] else None
    s["out"] = zeros(R, N, dt=bf)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:                             # the handles that a program keeps, and a workspace
        from combine_moe_layout_amd import binding as B
        s["dtype"] = {"bf16": B.EP_BF16, "fp16": B.EP_F16, "fp32": B.EP_F32}[case.get("dtype", "bf16")]
        if "act" in case:
            s["act"] = {"none": B.EP_ACT_NONE, "relu": B.EP_ACT_RELU, "gelu": B.EP_ACT_GELU,
                        "silu": B.EP_ACT_SILU, "swiglu": B.EP_ACT_SWIGLU}[case["act"]]
        if case["op"] == "route":
            s["router"] = B.EpRouter(
                case["E"], case["k"], B.EP_SCORE_SOFTMAX if case["score"] == "softmax" else B.EP_SCORE_SIGMOID,
                num_groups=case["groups"], topk_groups=case["topk_groups"],
                group_top=case["group_top"], renormalize=case["renorm"], scale=case["scale"])
        if case["op"] == "norm" and case["train"]:
            s["grad"] = B.EP_GRAD_F32 if case["grad"] == "f32" else 0
            s["workspace"] = torch.empty(B.ep_block_norm_grad_workspace_bytes(case["T"], case["H"]),
                                         dtype=torch.uint8, device="cuda")
        if "E" in case and case["op"] != "route":
            s["layout"] = B.EpLayout(case["T"], case["k"], case["E"], 1, case["cap"])
            B.ep_get_layout(s["topk_idx"], s["layout"])
    return s


# -------------------------------------------------------------------------------- plain forms
def _plain_keys(s):
    """What the choice goes by, in 64 bits (keys may lie closer than 32 bits can tell), and
    which experts can be chosen at all."""
    c = s["case"]
    l = s["logits"].double().clamp(max=_MOST)
    live = l > -math.inf
    if c["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-l))
    else:
        top = torch.where(live, l, -_MOST).amax(1, keepdim=True)
        p = torch.where(live, torch.exp(l - top), 0.0)
        score = p / p.sum(1, keepdim=True).clamp(min=1e-300)
    biased = score if s["bias"] is None else score + s["bias"].double()
    key = l if s["bias"] is None else biased    # a score rises with its logit
    return torch.where(live, key, -math.inf), torch.where(live, biased, -math.inf)


def _plain_route(s):
    c = s["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    key, biased = _plain_keys(s)
    if c["topk_groups"] < G:
        best = torch.sort(biased.reshape(T, G, E // G), dim=2, descending=True).values
        of_group = best[:, :, 0]
        if c["group_top"] == 2:
            of_group = of_group + torch.where(best[:, :, 1] > -math.inf, best[:, :, 1], 0.0)
        elif s["bias"] is None:
            of_group = key.reshape(T, G, E // G).amax(2)
        order = torch.sort(of_group, dim=1, descending=True, stable=True).indices
        keep = torch.zeros((T, G), dtype=torch.bool, device=key.device)
        keep.scatter_(1, order[:, :c["topk_groups"]], True)
        key = torch.where(keep.repeat_interleave(E // G, 1), key, -math.inf)
    value, idx = torch.sort(key, dim=1, descending=True, stable=True)
    none = value[:, :k] == -math.inf
    idx = idx[:, :k]
    l = s["logits"].float().clamp(max=_MOST)
    chosen = l.gather(1, idx)
    if c["score"] == "softmax":
        over = chosen if c["renorm"] else torch.where(l > -math.inf, l, -math.inf)
        over = torch.where(none, -math.inf, over) if c["renorm"] else over
        top = over.amax(1, keepdim=True).clamp(min=-_MOST)
        w = torch.exp(chosen - top) / torch.exp(over - top).sum(1, keepdim=True)
    else:
        w = 1 / (1 + torch.exp(-chosen))
        if c["renorm"]:
            w = torch.where(none, 0.0, w)
            w = w / w.sum(1, keepdim=True)
    w = torch.where(none, 0.0, w)           # before the scale
    s["idx"].copy_(torch.where(none, -1, idx))
    s["w"].copy_(w * c["scale"])
    if not c["train"]:
        return s["idx"], s["w"]
    # a choice that is missing has weight 0 and adds nothing
    at, dw = s["idx"].clamp(min=0), torch.where(none, 0.0, s["dw"] * c["scale"])
    if c["score"] == "softmax" and not c["renorm"]:
        p = torch.where(l > -math.inf, torch.exp(l - top) / torch.exp(over - top).sum(1, keepdim=True), 0.0)
        d = (-p * (dw * w).sum(1, keepdim=True)).scatter_add(1, at, dw * w)
    else:
        # sum_i w_i (dw_j - dw_i): exactly 0 where one choice has all the weight
        d = w * ((dw[:, :, None] - dw[:, None, :]) * w[:, None, :]).sum(2) if c["renorm"] else dw * w
        if c["score"] == "sigmoid":
            d = d / (1 + torch.exp(chosen))
        d = torch.zeros_like(l).scatter_add(1, at, torch.where(none, 0.0, d))
    s["dlogits"].copy_(d)
    return s["idx"], s["w"], s["dlogits"]


def _plain_norm(s):
    c = s["case"]
    y, res = s["y"].float(), s["residual"].float()
    inv = 1 / torch.sqrt((y * y).mean(1, keepdim=True) + _EPS)
    b = y * inv * s["post"].float() if c["post"] else y
    x = c["alpha"] * res + (b * s["gate"][:, None] if c["gate"] else b)
    s["out"].copy_(x)
    if c["pre"]:
        s["normed"].copy_(x / torch.sqrt((x * x).mean(1, keepdim=True) + _EPS) * s["pre"].float())
    if not c["train"]:
        return s["out"], s["normed"]
    dx = s["dout"].float()
    if c["pre"]:
        dn = s["dnormed"].float()
        r = 1 / torch.sqrt((x * x).mean(1, keepdim=True) + _EPS)
        a = dn * s["pre"].float()
        s["dpre"].copy_((dn * x * r).sum(0))
        dx = dx + r * a - x * r ** 3 * (a * x).mean(1, keepdim=True)
    s["dresidual"].copy_(c["alpha"] * dx)
    if c["gate"]:
        s["dgate"].copy_((dx * b).sum(1))
    db = dx * s["gate"][:, None] if c["gate"] else dx
    if c["post"]:
        s["dpost"].copy_((db * y * inv).sum(0))
        a = db * s["post"].float()
        db = inv * a - y * inv ** 3 * (a * y).mean(1, keepdim=True)
    s["dy"].copy_(db)
    return tuple(s[n] for n in ("out", "normed", "dy", "dresidual", "dgate", "dpost", "dpre"))


def _round_rows(x):
    """Codes and scales of rows: the quotients are rounded in 64 bits, where a border is a border."""
    x = x.double()
    a = x.abs().amax(1).clamp(min=2.0 ** -100)
    scale = (a / torch.full_like(a, 127)).float()   # a true quotient, rounded once
    return torch.round(x / scale.double()[:, None]).float(), scale


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


def _plain_experts(s):
    c = s["case"]
    if c["source"] == "tokens":
        q, scale = _round_rows(s["x"])
        slot = s["slot"].reshape(-1)
        pair = torch.nonzero(slot >= 0).reshape(-1)
        s["q"][slot[pair]] = q.to(torch.int8)[pair // c["k"]]
        s["s"][slot[pair]] = scale[pair // c["k"]]
    # one product per expert: the rows of each are another matrix's
    for e, (b, n) in enumerate(zip(s["begin"], s["rows"])):
        if not n:
            continue
        q, scale = (s["q"][b:b + n].float(), s["s"][b:b + n]) if c["source"] == "tokens" else _round_rows(s["x"][b:b + n])
        z = (q @ s["weights"][e].float().T) * scale[:, None] * s["ws"][e]
        if s["bias"] is not None:
            z = z + s["bias"][e].float()
        s["out"][b:b + n] = _act(z, c["act"]).to(s["out"].dtype)
    return s["out"]


def _plain_linear(s):
    q, scale = _round_rows(s["x"])
    z = (q @ s["weights"].float().T) * scale[:, None] * s["ws"]
    if s["bias"] is not None:
        z = z + s["bias"].float()
    a = _act(z, s["case"]["act"])
    if s["residual"] is not None:
        a = a + s["residual"].float()
    s["out"].copy_(a)
    return s["out"]


# ------------------------------------------------------------------------- the library's calls
def _own_route(s):
    from combine_moe_layout_amd import binding as B
    B.ep_route(s["logits"], s["router"], s["idx"], s["w"], s["dtype"], bias=s["bias"])
    if not s["case"]["train"]:
        return s["idx"], s["w"]
    B.ep_route_grad(s["dw"], s["logits"], s["idx"], s["router"], s["dlogits"], s["dtype"])
    return s["idx"], s["w"], s["dlogits"]


def _own_norm(s):
    from combine_moe_layout_amd import binding as B
    c = s["case"]
    B.ep_block_norm(s["y"], s["residual"], s["out"], s["dtype"], eps=_EPS, post_weight=s["post"],
                    gate=s["gate"], residual_scale=c["alpha"], pre_weight=s["pre"], normed=s["normed"])
    if not c["train"]:
        return s["out"], s["normed"]
    B.ep_block_norm_grad(s["dout"], s["dnormed"], s["y"], s["residual"], s["dtype"] | s["grad"],
                         s["workspace"], eps=_EPS, post_weight=s["post"], gate=s["gate"],
                         residual_scale=c["alpha"], pre_weight=s["pre"], d_y=s["dy"],
                         d_residual=s["dresidual"], d_gate=s["dgate"], d_post_weight=s["dpost"],
                         d_pre_weight=s["dpre"])
    return tuple(s[n] for n in ("out", "normed", "dy", "dresidual", "dgate", "dpost", "dpre"))


def _own_experts(s):
    from combine_moe_layout_amd import binding as B
    if s["case"]["source"] == "tokens":
        B.ep_dispatch(s["x"], s["layout"], B.EP_INT8, s["q"], s["s"])
    else:
        B.ep_quantize_int8(s["x"], s["q"], s["s"], s["dtype"], layout=s["layout"])
    B.ep_expert_gemm(s["q"], s["weights"], s["layout"], s["out"], B.EP_INT8, act=s["act"],
                     x_scales=s["s"], weight_scales=s["ws"], bias=s["bias"])
    return s["out"]


def _own_linear(s):
    from combine_moe_layout_amd import binding as B
    B.ep_quantize_int8(s["x"], s["q"], s["s"], s["dtype"])
    B.ep_linear_int8(s["q"], s["s"], s["weights"], s["ws"], s["out"], act=s["act"], bias=s["bias"],
                     residual=s["residual"])
    return s["out"]


_PLAIN = {"route": _plain_route, "norm": _plain_norm, "experts_int8": _plain_experts,
          "linear_int8": _plain_linear}
_OWN = {"route": _own_route, "norm": _own_norm, "experts_int8": _own_experts,
        "linear_int8": _own_linear}


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
    op, T = case["op"], case["T"]
    if op == "route":
        b = T * case["E"] * (4 if case["dtype"] == "fp32" else 2)
        small = 12 * T * case["k"] + (4 * case["E"] if case["bias"] else 0)
        train = b + 4 * T * case["k"] if case["train"] else 0
        return {"bytes": b + small + train, "flops": T * case["E"] * (20 if case["train"] else 10)}
    H = case["H"]
    if op == "norm":
        rows = 3 + case["pre"]                               # y, residual, out, normed
        grads = (3 + case["pre"]) if case["train"] else 0    # dout, dnormed, dy, dresidual
        b = 2 * T * H * (rows + grads) + 4 * T * case["gate"] * (1 + case["train"])
        weights = (case["post"] + case["pre"]) * H * (2 + (4 * case["train"] if case["grad"] == "f32" else 2 * case["train"]))
        return {"bytes": b + weights, "flops": T * H * (24 if case["train"] else 8)}
    N = case["N"]
    Nw = _width(N, case["act"])
    if op == "linear_int8":
        b = 2 * T * H + Nw * (H + 4) + 2 * T * N * (1 + case["residual"]) + (2 * Nw if case["bias"] else 0)
        return {"bytes": b, "flops": 2 * T * H * Nw}
    P, used = _touched(case)
    rows = min(T, P) if case["source"] == "tokens" else P
    b = 2 * rows * H + used * Nw * (H + 4) + 2 * P * N + (2 * used * Nw if case["bias"] else 0)
    return {"bytes": b, "flops": 2 * P * H * Nw}


def _exact_route(s):
    c = s["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    l = s["logits"].double()
    dead = torch.isnan(l) | torch.isneginf(l)
    l = torch.where(torch.isposinf(l), torch.full_like(l, _MOST), l)
    empty = dead.all(1, keepdim=True)
    if c["score"] == "sigmoid":
        log_s = torch.nn.functional.logsigmoid(l)
    else:
        log_s = l - torch.logsumexp(l.masked_fill(dead, -math.inf).masked_fill(empty, 0.0), 1, keepdim=True)
    score = torch.special.expit(l) if c["score"] == "sigmoid" else torch.exp(log_s)
    key = score + s["bias"].double() if s["bias"] is not None else score
    rank_by = (key if s["bias"] is not None else l).masked_fill(dead, -math.inf)
    if c["topk_groups"] < G:
        if c["group_top"] == 1:
            of_group = rank_by.view(T, G, -1).max(2).values
        else:
            two = key.masked_fill(dead, -math.inf).view(T, G, -1).topk(2, dim=2).values
            of_group = two[..., 0] + two[..., 1].masked_fill(torch.isneginf(two[..., 1]), 0.0)
        # a group's place: the groups ahead of it (better ones, and equal ones before it)
        a, b = of_group[:, :, None], of_group[:, None, :]
        before = torch.ones((G, G), dtype=torch.bool, device=l.device).tril(-1)
        place = ((b > a) | ((b == a) & before)).sum(2)
        rank_by = rank_by.masked_fill((place >= c["topk_groups"]).repeat_interleave(E // G, dim=1), -math.inf)
    left, idx, live = rank_by.clone(), [], []
    for _ in range(k):                  # the largest, the first of equals, one at a time
        best = left.amax(1, keepdim=True)
        one = (left == best).to(torch.uint8).argmax(1, keepdim=True)
        idx.append(one)
        live.append(best > -math.inf)
        left.scatter_(1, one, -math.inf)
    idx, live = torch.cat(idx, 1), torch.cat(live, 1)
    log_c = log_s.gather(1, idx).masked_fill(~live, -math.inf)
    if c["renorm"]:
        none = ~live.any(1, keepdim=True)
        w = torch.softmax(log_c.masked_fill(none, 0.0), 1).masked_fill(none, 0.0)
    else:
        w = torch.exp(log_c)
    w = w * c["scale"]
    out_idx = idx.masked_fill(~live, -1)
    if not c["train"]:
        return out_idx, w
    # by the chain rule over the scores' logarithms
    dlog = s["dw"].double().masked_fill(~live, 0.0) * w
    if c["renorm"]:
        dlog = dlog - w / c["scale"] * dlog.sum(1, keepdim=True)
    d = torch.zeros_like(l)
    if c["score"] == "sigmoid":
        d.scatter_add_(1, idx, dlog * torch.special.expit(-l).gather(1, idx))
    else:
        d.scatter_add_(1, idx, dlog)
        d = d - score.masked_fill(dead, 0.0) * dlog.sum(1, keepdim=True)
    return out_idx, w, d.masked_fill(dead, 0.0)


def _exact_norm(s):
    c = s["case"]
    y, res = s["y"].double(), s["residual"].double()
    unit = lambda v: v * torch.rsqrt(v.square().mean(1, keepdim=True) + _EPS)  # noqa: E731
    gate = s["gate"].double()[:, None] if c["gate"] else 1.0
    branch = unit(y) * s["post"].double() if c["post"] else y
    x = c["alpha"] * res + gate * branch
    normed = unit(x) * s["pre"].double() if c["pre"] else None
    if not c["train"]:
        return x, normed

    def back(d, v):                     # gradient of sum(d * unit(v))
        inv = torch.rsqrt(v.square().mean(1, keepdim=True) + _EPS)
        u = v * inv
        return inv * (d - u * (d * u).mean(1, keepdim=True))

    dx, dpre, dpost = s["dout"].double(), None, None
    if c["pre"]:
        dn = s["dnormed"].double()
        dx = dx + back(dn * s["pre"].double(), x)
        dpre = (dn * unit(x)).sum(0)
    db = gate * dx
    if c["post"]:
        dpost = (db * unit(y)).sum(0)
        dy = back(db * s["post"].double(), y)
    else:
        dy = db
    dgate = (dx * branch).sum(1) if c["gate"] else None
    return x, normed, dy, c["alpha"] * dx, dgate, dpost, dpre


def _exact_product(x, w, ws, bias, case):
    x = x.double()
    scale = (x.abs().max(1).values.clamp_min(2.0 ** -100) / 127).float().double()
    z = torch.mm(torch.round(x / scale[:, None]), w.double().T) * (scale[:, None] * ws.double()[None, :])
    z = z if bias is None else z + bias.double()
    act, N = case["act"], case["N"]
    if act == "swiglu":
        return z[:, :N] * torch.special.expit(z[:, :N]) * z[:, N:]
    return {"none": lambda: z, "relu": lambda: z.clamp(min=0), "gelu": lambda: z * torch.special.ndtr(z),
            "silu": lambda: z * torch.special.expit(z)}[act]()


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "route":
        return _exact_route(s)
    if case["op"] == "norm":
        return _exact_norm(s)
    if case["op"] == "linear_int8":
        a = _exact_product(s["x"], s["weights"], s["ws"], s["bias"], case)
        return a if s["residual"] is None else a + s["residual"].double()
    x, out = s["x"], s["out"].double()
    if case["source"] == "tokens":      # the token of every receive row
        token = torch.zeros(out.shape[0], dtype=torch.int64, device="cuda")
        t, j = torch.nonzero(s["slot"] >= 0, as_tuple=True)
        token[s["slot"][t, j]] = t
    for e in range(case["E"]):
        at = slice(s["begin"][e], s["begin"][e] + s["rows"][e])
        if s["rows"][e]:
            rows = x[token[at]] if case["source"] == "tokens" else x[at]
            out[at] = _exact_product(rows, s["weights"][e], s["ws"][e],
                                     None if s["bias"] is None else s["bias"][e], case)
    return out
