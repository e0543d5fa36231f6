"""The router, the experts' products, the weighted combine and their gradients
in 64 bits on the host, written from their definitions for the tests."""
from __future__ import annotations

import math

import torch

INF = math.inf


def half_step(dtype) -> float:
    """Largest relative error of one rounding to nearest."""
    return torch.finfo(dtype).eps / 2


# ------------------------------------------------------------------ router
def scores(z, sigmoid):
    """s of one token's float64 logits; None for a token that has NaN weights."""
    if torch.isnan(z).any() or (not sigmoid and (z == INF).any()):
        return None
    if sigmoid:
        return torch.where(z == -INF, 0.0, 1 / (1 + torch.exp(-z)))
    m = z.max()
    if m == -INF:
        return torch.zeros_like(z)
    e = torch.exp(z - m)
    return e / e.sum()


def route(logits, sigmoid, bias, groups, topk_groups, group_top, k, renorm, scale):
    """ids [T, k] (int32) and weights [T, k] (float64) of float64 logits [T, E]."""
    T, E = logits.shape
    ids = torch.zeros((T, k), dtype=torch.int32)
    weights = torch.full((T, k), math.nan, dtype=torch.float64)
    for t in range(T):
        z = logits[t]
        s = scores(z, sigmoid)
        if s is None:
            ids[t] = torch.arange(k)
            continue
        c = s + (0 if bias is None else bias.double())
        c = torch.where((z == -INF) | torch.isnan(c), -INF, c).tolist()
        zl, per = z.tolist(), E // groups
        best = lambda es: sorted(es, key=lambda e: (-c[e], -zl[e], e))  # noqa: E731
        score = []
        for g in range(groups):
            top = [c[e] for e in best(range(g * per, (g + 1) * per))[:group_top]]
            v = sum(top)
            score.append(-INF if math.isnan(v) else v)
        kept = sorted(range(groups), key=lambda g: (-score[g], g))[:topk_groups]
        chosen = best([e for e in range(E) if e // per in kept])[:k]
        ids[t] = torch.tensor(chosen, dtype=torch.int32)
        w = s[chosen]
        if renorm:
            w = w / w.sum() if w.sum() > 0 else torch.zeros_like(w)
        weights[t] = w * scale
    return ids, weights


def route_weights(logits, ids, sigmoid, renorm, scale):
    """The weights of given ids, differentiable in the float64 logits [T, E]."""
    s = 1 / (1 + torch.exp(-logits)) if sigmoid else torch.softmax(logits, -1)
    w = s.gather(-1, ids.long())
    if renorm:
        w = w / w.sum(-1, keepdim=True)
    return w * scale


def route_grad(logits, ids, d_weights, sigmoid, renorm, scale):
    """d_logits [T, E], the formula; finite logits."""
    s = 1 / (1 + torch.exp(-logits)) if sigmoid else torch.softmax(logits, -1)
    sj, g = s.gather(-1, ids.long()), d_weights * scale
    if renorm:
        S = sj.sum(-1, keepdim=True)
        g = (g - (g * sj).sum(-1, keepdim=True) / S) / S
    d = torch.zeros_like(logits)
    for j in range(ids.shape[1]):
        d.scatter_add_(-1, ids[:, j:j + 1].long(), g[:, j:j + 1])
    if sigmoid:
        return s * (1 - s) * d
    # with renorm the sum of g * s is 0: sum_j s_j (g_j - sum g s / S) / S
    return s * (d - (0 if renorm else (g * sj).sum(-1, keepdim=True)))


# ------------------------------------------------------------------ experts
def activate(act, h):
    if act == "relu":
        return torch.where(h < 0, torch.zeros_like(h), h)
    if act == "gelu":
        return 0.5 * h * torch.erfc(-h / math.sqrt(2))
    if act == "silu":
        return h / (1 + torch.exp(-h))
    if act == "swiglu":
        g, u = h.chunk(2, -1)
        return g / (1 + torch.exp(-g)) * u
    return h


def activate_grad(act, h, d):
    if act == "relu":
        return torch.where(h <= 0, torch.zeros_like(d), d)
    if act == "gelu":
        pdf = torch.exp(-0.5 * h * h) / math.sqrt(2 * math.pi)
        return d * (0.5 * torch.erfc(-h / math.sqrt(2)) + h * pdf)
    if act == "silu":
        s = 1 / (1 + torch.exp(-h))
        return d * s * (1 + h * (1 - s))
    if act == "swiglu":
        g, u = h.chunk(2, -1)
        s = 1 / (1 + torch.exp(-g))
        return torch.cat([d * u * s * (1 + g * (1 - s)), d * g * s], -1)
    return d
