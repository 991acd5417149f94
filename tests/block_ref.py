"""The router, the block norms and the 8-bit integer rows in 64 bits, from their definitions."""
import math

import torch

STEP = 2.0 ** -24                    # half a step of fp32, relative
MOST = torch.finfo(torch.float32).max


def usable(logits):
    """Logits in 64 bits, +inf as the largest fp32 value, and which experts can be chosen."""
    l = logits.double()
    dead = torch.isnan(l) | (l == -math.inf)
    return torch.where(dead, -math.inf, l.clamp(max=MOST)), ~dead


def scores(logits, score):
    l, live = usable(logits)
    if score == "sigmoid":
        return torch.where(live, 1 / (1 + torch.exp(-l)), 0.0)
    top = l.amax(1, keepdim=True).clamp(min=-MOST)
    p = torch.where(live, torch.exp(l - top), 0.0)
    return p / p.sum(1, keepdim=True).clamp(min=1e-300)


def choice(logits, bias, k, score, groups=1, topk_groups=1, group_top=1):
    """The chosen experts [T, k], -1 where there is none: one token and one choice at a time, by
    Python's own comparisons of (key, -index)."""
    l, live = usable(logits)
    s = scores(logits, score)
    key = l if bias is None else s + bias.double()
    of = key if bias is not None or group_top == 1 else s
    T, E = l.shape
    key = torch.where(live & (key > -math.inf), key, -math.inf).tolist()
    of = torch.where(live & (of > -math.inf), of, -math.inf).tolist()
    n, out = E // groups, []
    for t in range(T):
        keep = range(groups)
        if topk_groups < groups:
            value = []
            for g in range(groups):
                best = sorted(of[t][g * n:(g + 1) * n], reverse=True)[:group_top]
                value.append(sum(b for b in best if b > -math.inf) if best[0] > -math.inf else -math.inf)
            keep = sorted(range(groups), key=lambda g: (-value[g], g))[:topk_groups]
        can = [e for g in keep for e in range(g * n, (g + 1) * n) if key[t][e] > -math.inf]
        can = sorted(can, key=lambda e: (-key[t][e], e))[:k]
        out.append(can + [-1] * (k - len(can)))
    return torch.tensor(out, dtype=torch.int64, device=logits.device).reshape(T, k)


def log_scores(logits, idx, score):
    """ln of the chosen scores (-inf for a missing choice): differentiable in logits."""
    pick = logits.gather(1, idx.clamp(min=0))
    if score == "sigmoid":
        v = torch.nn.functional.logsigmoid(pick)
    else:
        v = pick - torch.logsumexp(logits, 1, keepdim=True)
    return torch.where(idx >= 0, v, -math.inf)


def weights(logits, idx, score, renormalize, scale):
    """topk_weights of a choice, in 64 bits; a row without any choice gets zeros."""
    empty = (idx < 0).all(1, keepdim=True)
    v = log_scores(logits, idx, score)
    if renormalize:
        v = torch.where(empty, 0.0, v)
        w = torch.exp(v - v.amax(1, keepdim=True))
        w = w / w.sum(1, keepdim=True)
    else:
        w = torch.exp(v)
    return torch.where(idx >= 0, w, 0.0) * scale


def unit(v, eps):
    return v / torch.sqrt((v * v).mean(1, keepdim=True) + eps)


def block_norm(y, residual, eps, post=None, gate=None, alpha=1.0, pre=None):
    """(x, normed) in 64 bits, differentiable; tensors in 64 bits or None."""
    x = 0.0
    if y is not None:
        x = y if post is None else unit(y, eps) * post
        x = x if gate is None else x * gate[:, None]
    if residual is not None:
        x = x + alpha * residual
    return x, None if pre is None else unit(x, eps) * pre


def int8_rows(x):
    """(codes, scales, values) of rows."""
    v = x.double()
    bad = ~torch.isfinite(v).all(1)
    a = torch.where(bad[:, None], 0.0, v).abs().amax(1).clamp(min=2.0 ** -100)
    scale = (a / torch.full_like(a, 127)).float()   # (torch divides by a number by its rounded reciprocal)
    q = torch.round(torch.where(bad[:, None], 0.0, v) / scale.double()[:, None])   # ties to even
    return q.to(torch.int8), torch.where(bad, math.nan, scale), q * scale.double()[:, None]
