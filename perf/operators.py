"""Timing cases of the operators that make the MoE exchange a trainable layer: the router in front of
the dispatch and its gradient, the experts' products on the rows the dispatch delivers and theirs, and
the gradient of the weighted combine.

``run`` makes one pass. With ``own`` it makes the library's calls; without, it computes the same outputs
from elementary torch operations in 32 bits (the router's selection keys in 64, since two scores next to
each other decide a whole number), rounded once at the end. ``exact`` gives the values in 64 bits.
"""
import math

import numpy as np
import torch

own = False

F16 = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ACTS = ("none", "relu", "gelu", "silu", "swiglu")


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoded token: sigmoid scores, a balance bias, 4 of 8 groups by their two best, top 8 of 256
        dict(name="route token", op="route", W=1, T=1, E=256, k=8, type="fp32", score="sigmoid", bias=True,
             groups=8, topk_groups=4, group_top=2, renorm=True, scale=2.5),
        # the dispatch workload's routing: 8 ranks of 8192 tokens, top 8 of 256 experts, softmax scores
        dict(name="route batch", op="route", W=8, T=8192, E=256, k=8, type="fp32", score="softmax", bias=False,
             groups=1, topk_groups=1, group_top=1, renorm=True, scale=1.0),
        # the same batch balanced by a bias and limited to groups, from a bf16 router
        dict(name="route groups bf16", op="route", W=8, T=4096, E=256, k=8, type="bf16", score="sigmoid", bias=True,
             groups=8, topk_groups=4, group_top=2, renorm=True, scale=2.5),
        # training through scores that are not renormalised: every logit has a gradient
        dict(name="route grad", op="route_grad", W=8, T=8192, E=256, k=8, type="fp32", score="softmax", renorm=False,
             scale=1.0),
        # a small model's odd expert count and token count
        dict(name="route grad odd bf16", op="route_grad", W=1, T=1021, E=60, k=4, type="bf16", score="sigmoid",
             renorm=True, scale=1.0),
        # the combine's gradient read and written at the owners, at the dispatch workload's width
        dict(name="combine grad owners", op="combine_grad", W=8, T=1024, E=256, k=8, H=7168, layout=1),
        # the same over a returned buffer: an odd batch with a width that is no power of two
        dict(name="combine grad odd", op="combine_grad", W=2, T=129, E=16, k=3, H=1000, layout=-1),
        # one rank's 32 experts, gate and up products of a training batch, pre-activations kept
        dict(name="experts up", op="experts", W=1, P=32, rows=16384, K=7168, N=2048, type="bf16", act="swiglu",
             bias=False, residual=False, pre=True),
        # one decoded token's eight experts: the weights are what has to be read
        dict(name="experts up token", op="experts", W=1, P=32, rows=8, K=7168, N=2048, type="bf16", act="swiglu",
             bias=False, residual=False, pre=False),
        # small experts with a bias and a residual, ragged sizes on two ranks
        dict(name="experts odd fp16", op="experts", W=2, P=5, rows=777, K=1000, N=712, type="fp16", act="gelu",
             bias=True, residual=True, pre=True),
        # the gradient of the first: input, weight and pre-activation gradients
        dict(name="experts up grad", op="experts_grad", W=1, P=32, rows=8192, K=7168, N=2048, type="bf16",
             act="swiglu", bias=False),
        # the small experts' gradient, bias included
        dict(name="experts odd grad fp16", op="experts_grad", W=2, P=6, rows=555, K=520, N=264, type="fp16",
             act="gelu", bias=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_grad", "combine_grad", "experts", "experts_grad"])
    if op in ("route", "route_grad"):
        W = rng.choice([1, 2, 4, 8])
        groups = rng.choice([1, 1, 2, 4, 8]) if op == "route" else 1
        per = _log(rng, 2, 256 // groups)
        E = W * groups * per if W * groups * per <= 512 else groups * per
        W = W if E % W == 0 else 1
        topk_groups = rng.randint(1, groups)
        k = rng.randint(1, min(16, topk_groups * (E // groups)))
        T = min(_log(rng, 1, 8192), max(1, (8 * 8192 * 256) // (W * E)))
        c = dict(op=op, W=W, T=T, E=E, k=k, type=rng.choice(["fp32", "bf16", "fp16"]),
                 score=rng.choice(["softmax", "sigmoid"]), renorm=rng.random() < 0.6,
                 scale=rng.choice([1.0, 2.5]))
        if op == "route":
            c.update(bias=rng.random() < 0.5, groups=groups, topk_groups=topk_groups,
                     group_top=rng.choice([1, 2]) if E // groups >= 2 else 1)
        return c
    if op == "combine_grad":
        W = rng.choice([1, 2, 4, 8])
        E = W * _log(rng, 1, 32)
        k = rng.randint(1, min(8, E))
        H = _log(rng, 16, 8192)
        T = min(_log(rng, 1, 4096), max(1, (1024 * 8 * 8 * 7168) // (W * k * H)))
        return dict(op=op, W=W, T=T, E=E, k=k, H=H, layout=rng.choice([-1, 0, 1]))
    W, P = rng.choice([1, 2, 4]), _log(rng, 1, 16)
    K, N = _log(rng, 32, 4096), _log(rng, 32, 2048)
    if rng.random() < 0.8:
        K, N = K // 8 * 8, N // 8 * 8
    c = dict(op=op, W=W, P=P, rows=_log(rng, 1, 8192), K=K, N=N, type=rng.choice(["bf16", "fp16"]),
             act=rng.choice(ACTS), bias=rng.random() < 0.5)
    if op == "experts":
        c.update(residual=rng.random() < 0.5, pre=rng.random() < 0.5)
    return c


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _logits(c, g):
    """Router logits: N(0, 1) around an expert popularity of its own."""
    z = _randn(g, c["W"], c["T"], c["E"]) + 0.5 * _randn(g, c["E"])
    return z.to(F16[c["type"]])


def _expert_rows(c, seed):
    """Rows of each (rank, expert), lognormal popularity, every rank's total within its share."""
    r = np.random.default_rng(int(seed))
    W, P = c["W"], c["P"]
    share = [c["rows"] // W + (1 if d < c["rows"] % W else 0) for d in range(W)]
    out = np.zeros((W, P), dtype=np.int64)
    for d in range(W):
        p = np.exp(0.5 * r.standard_normal(P))
        out[d] = r.multinomial(share[d], p / p.sum())
    return out


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    W = c["W"]
    s = {"c": c, "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    if c["op"] in ("route", "route_grad"):
        T, E, k = c["T"], c["E"], c["k"]
        s["logits"] = _logits(c, g)
        if c["op"] == "route":
            s["bias"] = 0.1 * _randn(g, E) if c["bias"] else None
            s["ids"] = torch.empty((W, T, k), dtype=torch.int32, device="cuda")
            s["weights"] = torch.empty((W, T, k), device="cuda")
        else:
            z = s["logits"].double()
            p = torch.softmax(z, -1) if c["score"] == "softmax" else torch.sigmoid(z)
            w, ids = torch.topk(p, k, -1)
            if c["renorm"]:
                w = w / w.sum(-1, keepdim=True)
            s["ids"], s["weights"] = ids.to(torch.int32), (w * c["scale"]).float()
            s["d_weights"] = _randn(g, W, T, k)
            s["d_logits"] = torch.empty_like(s["logits"])
        return s
    if c["op"] == "combine_grad":
        T, E, k, H = c["T"], c["E"], c["k"], c["H"]
        Q = T * k
        ids = torch.topk(_randn(g, W, T, E) + 0.5 * _randn(g, E), k, -1).indices.reshape(W, Q)
        perm = torch.argsort(torch.argsort(ids, dim=1, stable=True), dim=1)
        src = torch.arange(W, device="cuda")[:, None]
        if c["layout"] < 0:  # pack order of each rank
            s["row_of"] = perm + src * Q
            cut = [Q] * W
        else:  # rows at their owners, source-major (0) or expert-major (1)
            order = ids if c["layout"] == 1 else ((ids // (E // W)) * W + src) * E + ids
            s["row_of"] = torch.argsort(torch.argsort(order.reshape(-1), stable=True)).reshape(W, Q)
            cut = torch.bincount(ids.reshape(-1) // (E // W), minlength=W).tolist()
        s["counts"] = (ids[:, :, None] == torch.arange(E, device="cuda")).sum(1) if W * Q * E < 1 << 28 else \
            torch.stack([torch.bincount(x, minlength=E) for x in ids])
        s["ids"], s["perm"], s["cut"] = ids.to(torch.int32), perm, cut
        s["rows"] = _randn(g, W * Q, H).to(torch.bfloat16)
        s["d_out"] = _randn(g, W, T, H).to(torch.bfloat16)
        s["weights"] = torch.softmax(_randn(g, W, T, k), -1)
        s["d_rows"] = torch.empty_like(s["rows"])
        s["d_weights"] = torch.empty((W, T, k), device="cuda")
        return s
    t, P, K, N = F16[c["type"]], c["P"], c["K"], c["N"]
    NW = 2 * N if c["act"] == "swiglu" else N
    per = _expert_rows(c, seed)
    R = int(per.sum())
    s["per"] = per.reshape(-1).tolist()
    s["cut"] = per.sum(1).tolist()
    s["offsets"] = torch.from_numpy(np.concatenate([np.zeros((W, 1), np.int64), per.cumsum(1)], 1)).cuda()
    s["x"] = _randn(g, R, K).to(t)
    s["weight"] = torch.empty((W * P, NW, K), dtype=t, device="cuda")
    for e in range(W * P):
        s["weight"][e] = _randn(g, NW, K) / math.sqrt(K)
    s["bias"] = (0.5 * _randn(g, W * P, NW)).to(t) if c["bias"] else None
    if c["op"] == "experts":
        s["residual"] = _randn(g, R, N).to(t) if c["residual"] else None
        s["out"] = torch.empty((R, N), dtype=t, device="cuda")
        s["pre"] = torch.empty((R, NW), dtype=t, device="cuda") if c["pre"] else None
    else:
        s["pre"] = _randn(g, R, NW).to(t) if c["act"] != "none" else None
        s["d_out"] = _randn(g, R, N).to(t)
        s["d_pre"] = torch.empty((R, NW), dtype=t, device="cuda") if c["act"] != "none" else None
        s["d_x"] = torch.empty_like(s["x"])
        s["d_weight"] = torch.empty_like(s["weight"])
        s["d_bias"] = torch.empty_like(s["bias"]) if c["bias"] else None
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["c"]["op"]
    if own:
        return {"route": _own_route, "route_grad": _own_route_grad, "combine_grad": _own_combine_grad,
                "experts": _own_experts, "experts_grad": _own_experts_grad}[op](state)
    return {"route": _route, "route_grad": _route_grad, "combine_grad": _combine_grad,
            "experts": _experts, "experts_grad": _experts_grad}[op](state)


def _ranks(x, W):
    return [None if x is None else x[r] for r in range(W)]


def _cut(x, cut):
    return None if x is None else list(torch.split(x, cut))


def _own_route(s):
    from embeddings_a2av_virtual_amd import _binding as B
    c, W = s["c"], s["c"]["W"]
    B.moe_route(W, c["T"], c["k"], c["E"], B.SCORE_SOFTMAX if c["score"] == "softmax" else B.SCORE_SIGMOID,
                _ranks(s["logits"], W), s["bias"], c["groups"], c["topk_groups"], c["group_top"], c["renorm"],
                c["scale"], _ranks(s["ids"], W), _ranks(s["weights"], W), s["status"])
    return {"ids": s["ids"], "weights": s["weights"]}


def _own_route_grad(s):
    from embeddings_a2av_virtual_amd import _binding as B
    c, W = s["c"], s["c"]["W"]
    B.moe_route_backward(W, c["T"], c["k"], c["E"], B.SCORE_SOFTMAX if c["score"] == "softmax" else B.SCORE_SIGMOID,
                         _ranks(s["logits"], W), _ranks(s["ids"], W), _ranks(s["weights"], W), c["renorm"],
                         c["scale"], _ranks(s["d_weights"], W), _ranks(s["d_logits"], W), s["status"])
    return {"d_logits": s["d_logits"]}


def _workspace(s, size):
    """Kept between passes, as a program keeps it between steps."""
    if "workspace" not in s:
        s["workspace"] = torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")
    return s["workspace"]


def _own_combine_grad(s):
    from embeddings_a2av_virtual_amd import _binding as B
    c, W, cut = s["c"], s["c"]["W"], s["cut"]
    if c["layout"] < 0:
        ws = _workspace(s, B.moe_combine_backward_workspace_bytes(W, c["T"], c["k"]))
        B.moe_combine_backward(W, c["T"], c["k"], c["H"], _cut(s["rows"], cut), _ranks(s["perm"], W),
                               _ranks(s["weights"], W), _ranks(s["d_out"], W), _cut(s["d_rows"], cut),
                               _ranks(s["d_weights"], W), ws, s["status"])
    else:
        ws = _workspace(s, B.moe_combine_return_backward_workspace_bytes(W, c["T"], c["k"], c["E"]))
        B.moe_combine_return_backward(W, c["T"], c["k"], c["E"], c["H"], s["counts"], _ranks(s["ids"], W),
                                      _ranks(s["perm"], W), _cut(s["rows"], cut), cut, _ranks(s["weights"], W),
                                      _ranks(s["d_out"], W), _cut(s["d_rows"], cut), _ranks(s["d_weights"], W),
                                      c["layout"], ws, s["status"])
    return {"d_rows": s["d_rows"], "d_weights": s["d_weights"]}


def _act_code(B, act):
    return {"none": B.ACT_NONE, "relu": B.ACT_RELU, "gelu": B.ACT_GELU, "silu": B.ACT_SILU, "swiglu": B.ACT_SWIGLU}[act]


def _experts_of(x, W, P):
    return None if x is None else [x[d * P:(d + 1) * P] for d in range(W)]


def _own_experts(s):
    from embeddings_a2av_virtual_amd import _binding as B
    c, W, P, cut = s["c"], s["c"]["W"], s["c"]["P"], s["cut"]
    act = _act_code(B, c["act"])
    ws = _workspace(s, B.moe_expert_linear_workspace_bytes(W, P, c["K"], c["N"], act, cut))
    B.moe_expert_linear(W, P, c["K"], c["N"], act, _cut(s["x"], cut), cut, s["offsets"],
                        _experts_of(s["weight"], W, P), _experts_of(s["bias"], W, P), _cut(s["residual"], cut),
                        _cut(s["out"], cut), _cut(s["pre"], cut), ws, s["status"])
    return {"out": s["out"], "pre": s["pre"]}


def _own_experts_grad(s):
    from embeddings_a2av_virtual_amd import _binding as B
    c, W, P, cut = s["c"], s["c"]["W"], s["c"]["P"], s["cut"]
    act = _act_code(B, c["act"])
    ws = _workspace(s, B.moe_expert_linear_backward_workspace_bytes(W, P, c["K"], c["N"], act, cut))
    B.moe_expert_linear_backward(W, P, c["K"], c["N"], act, _cut(s["x"], cut), cut, s["offsets"],
                                 _experts_of(s["weight"], W, P), _cut(s["pre"], cut), _cut(s["d_out"], cut),
                                 _cut(s["d_pre"], cut), _cut(s["d_x"], cut), _experts_of(s["d_weight"], W, P),
                                 _experts_of(s["d_bias"], W, P), ws, s["status"])
    return {"d_pre": s["d_pre"], "d_x": s["d_x"], "d_weight": s["d_weight"], "d_bias": s["d_bias"]}


# ------------------------------------------------------------------ the plain forms
def _route(s):
    c, z = s["c"], s["logits"].double()
    if c["score"] == "softmax":
        e = torch.exp(z - z.amax(-1, keepdim=True))
        p = e / e.sum(-1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-z))
    key = p if s["bias"] is None else p + s["bias"].double()
    G = c["groups"]
    if G > 1:
        by = key.reshape(*key.shape[:-1], G, -1)
        score = by.sort(dim=-1, descending=True).values[..., :c["group_top"]].sum(-1)
        kept = score.sort(dim=-1, descending=True, stable=True).indices[..., :c["topk_groups"]]
        live = torch.zeros(score.shape, dtype=torch.bool, device=z.device).scatter_(-1, kept, True)
        key = torch.where(live[..., None], by, -math.inf).reshape(key.shape)
    ids = key.sort(dim=-1, descending=True, stable=True).indices[..., :c["k"]]
    w = p.gather(-1, ids).float()
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    return {"ids": ids.to(torch.int32), "weights": w * c["scale"]}


def _route_grad(s):
    c, z, ids = s["c"], s["logits"].float(), s["ids"].long()
    if c["score"] == "softmax":
        e = torch.exp(z - z.amax(-1, keepdim=True))
        p = e / e.sum(-1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-z))
    g, ps = s["d_weights"] * c["scale"], p.gather(-1, ids)
    if c["renorm"]:
        S = ps.sum(-1, keepdim=True)
        g = (g - (g * ps).sum(-1, keepdim=True) / S) / S
    d = torch.zeros_like(z).scatter_add_(-1, ids, g)
    if c["score"] == "softmax":
        d = p * (d - (g * ps).sum(-1, keepdim=True))
    else:
        d = p * (1 - p) * d
    return {"d_logits": d.to(s["logits"].dtype)}


def _combine_grad(s):
    c, row_of = s["c"], s["row_of"].reshape(s["c"]["W"], s["c"]["T"], s["c"]["k"])
    d = s["d_out"].float()[:, :, None, :]
    d_rows = torch.empty_like(s["rows"])
    d_rows[row_of] = (s["weights"][..., None] * d).to(torch.bfloat16)
    return {"d_rows": d_rows, "d_weights": (s["rows"][row_of].float() * d).sum(-1)}


def _activate(act, h):
    if act == "relu":
        return torch.clamp(h, min=0)
    if act == "gelu":
        return h * 0.5 * (1 + torch.erf(h * math.sqrt(0.5)))
    if act == "silu":
        return h / (1 + torch.exp(-h))
    if act == "swiglu":
        gate, up = h.chunk(2, -1)
        return gate / (1 + torch.exp(-gate)) * up
    return h


def _activate_grad(act, h, d):
    if act == "relu":
        return d * (h > 0)
    if act == "gelu":
        return d * (0.5 * (1 + torch.erf(h * math.sqrt(0.5))) + h * torch.exp(-0.5 * h * h) / math.sqrt(2 * math.pi))
    if act == "silu":
        p = 1 / (1 + torch.exp(-h))
        return d * p * (1 + h * (1 - p))
    if act == "swiglu":
        gate, up = h.chunk(2, -1)
        p = 1 / (1 + torch.exp(-gate))
        return torch.cat([d * up * p * (1 + gate * (1 - p)), d * gate * p], -1)
    return d


# One product for each expert that has rows: a padded batch of them would do several times the work.
def _experts(s):
    c, x = s["c"], s["x"]
    out = torch.empty_like(s["out"])
    pre = None if s["pre"] is None else torch.empty_like(s["pre"])
    at = 0
    for e, n in enumerate(s["per"]):
        if n:
            rows = slice(at, at + n)
            h = x[rows].float() @ s["weight"][e].float().t()
            if s["bias"] is not None:
                h = h + s["bias"][e].float()
            if pre is not None:
                pre[rows] = h.to(x.dtype)
            y = _activate(c["act"], h)
            if s["residual"] is not None:
                y = y + s["residual"][rows].float()
            out[rows] = y.to(x.dtype)
            at += n
    return {"out": out, "pre": pre}


def _experts_grad(s):
    c, x = s["c"], s["x"]
    h = _activate_grad(c["act"], None if s["pre"] is None else s["pre"].float(), s["d_out"].float())
    d_x, d_weight = torch.empty_like(x), torch.zeros_like(s["weight"])
    d_bias = None if s["bias"] is None else torch.zeros_like(s["bias"])
    at = 0
    for e, n in enumerate(s["per"]):
        if n:
            rows = slice(at, at + n)
            d_x[rows] = (h[rows] @ s["weight"][e].float()).to(x.dtype)
            d_weight[e] = (h[rows].t() @ x[rows].float()).to(x.dtype)
            if d_bias is not None:
                d_bias[e] = h[rows].sum(0).to(x.dtype)
            at += n
    return {"d_pre": None if s["pre"] is None else h.to(x.dtype), "d_x": d_x, "d_weight": d_weight, "d_bias": d_bias}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c, W = case, case["W"]
    if c["op"] in ("route", "route_grad"):
        n, b = W * c["T"], 4 if c["type"] == "fp32" else 2
        if c["op"] == "route":
            return {"bytes": n * (c["E"] * b + c["k"] * 8) + (4 * c["E"] if c["bias"] else 0), "flops": 8 * n * c["E"]}
        # a renormalised softmax needs no logit, a renormalised sigmoid the selected ones
        read = c["E"] if not c["renorm"] and c["score"] == "softmax" else c["k"] if c["score"] == "sigmoid" else 0
        return {"bytes": n * (c["E"] * b + read * b + c["k"] * 12), "flops": 6 * n * max(read, c["k"])}
    if c["op"] == "combine_grad":
        q = W * c["T"] * c["k"]
        index = 16 if c["layout"] < 0 else 20  # perm, weight and its gradient; the expert id at the owners
        return {"bytes": 2 * q * c["H"] * 2 + W * c["T"] * c["H"] * 2 + q * index, "flops": 3 * q * c["H"]}
    NW = 2 * c["N"] if c["act"] == "swiglu" else c["N"]
    R, K, N, P = c["rows"], c["K"], c["N"], c["P"]
    busy = min(R, W * P)  # experts that can have rows
    if c["op"] == "experts":
        b = R * K + busy * NW * K + R * N * (2 if c["residual"] else 1) + (R * NW if c["pre"] else 0)
        return {"bytes": 2 * (b + (busy * NW if c["bias"] else 0)), "flops": 2 * R * NW * K}
    b = 2 * R * K + busy * NW * K + W * P * NW * K + R * N + (2 * R * NW if c["act"] != "none" else 0)
    return {"bytes": 2 * (b + (W * P * NW if c["bias"] else 0)), "flops": 4 * R * NW * K}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "route_grad": _exact_route_grad, "combine_grad": _exact_combine_grad,
            "experts": _exact_experts, "experts_grad": _exact_experts_grad}[case["op"]](s)


def _exact_scores(c, z):
    if c["score"] == "softmax":
        return torch.exp(z - torch.logsumexp(z, -1, keepdim=True))
    return 0.5 * (1 + torch.tanh(0.5 * z))


def _largest(key, count):
    """The places of the `count` largest values of the last axis, one after the other, the lowest of equals first."""
    key, at = key.clone(), torch.arange(key.shape[-1], device=key.device)
    found = []
    for _ in range(count):
        top = key.amax(-1, keepdim=True)
        found.append(torch.where(key == top, at, key.shape[-1]).amin(-1, keepdim=True))
        key.scatter_(-1, found[-1], -math.inf)
    return torch.cat(found, -1)


def _exact_route(s):
    c, z = s["c"], s["logits"].double()
    # the keys as they are defined; the weights from another form of the scores
    key = torch.sigmoid(z) if c["score"] == "sigmoid" else torch.softmax(z, -1)
    if s["bias"] is not None:
        key = key + s["bias"].double()
    if c["groups"] > 1:
        width = c["E"] // c["groups"]
        by = key.unflatten(-1, (c["groups"], width))
        score = by.gather(-1, _largest(by, c["group_top"])).sum(-1)
        chosen = _largest(score, c["topk_groups"])
        live = (torch.arange(c["E"], device=z.device) // width == chosen[..., None]).any(-2)
        key = key.masked_fill(~live, -math.inf)
    ids = _largest(key, c["k"])
    w = torch.take_along_dim(_exact_scores(c, z), ids, -1)
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    return {"ids": ids.to(torch.int32), "weights": w * c["scale"]}


def _exact_route_grad(s):
    """The Jacobian's products written out: dw_j/dz_e through the chosen scores."""
    c, z, ids = s["c"], s["logits"].double(), s["ids"].long()
    p = _exact_scores(c, z)
    chosen, g = torch.take_along_dim(p, ids, -1), c["scale"] * s["d_weights"].double()
    if c["renorm"]:
        total = chosen.sum(-1, keepdim=True)
        g = g / total - (g * chosen).sum(-1, keepdim=True) / total.square()
    d = torch.zeros_like(z)
    for j in range(c["k"]):
        e, pj, gj = ids[..., j:j + 1], chosen[..., j:j + 1], g[..., j:j + 1]
        if c["score"] == "softmax":
            d -= gj * pj * p
            d.scatter_add_(-1, e, gj * pj)
        else:
            d.scatter_add_(-1, e, gj * pj * (1 - pj))
    return {"d_logits": d}


def _exact_combine_grad(s):
    c = s["c"]
    d_rows = torch.empty(s["rows"].shape, dtype=torch.float64, device="cuda")
    d_weights = torch.empty((c["W"], c["T"], c["k"]), dtype=torch.float64, device="cuda")
    row_of = s["row_of"].reshape(c["W"], c["T"], c["k"])
    for r in range(c["W"]):
        d = s["d_out"][r].double()
        for j in range(c["k"]):
            at = row_of[r, :, j]
            d_rows[at] = d * s["weights"][r, :, j:j + 1].double()
            d_weights[r, :, j] = (s["rows"][at].double() * d).sum(-1)
    return {"d_rows": d_rows, "d_weights": d_weights}


def _exact_act(act, h):
    if act == "relu":
        return torch.maximum(h, torch.zeros_like(h))
    if act == "gelu":
        return h * 0.5 * torch.erfc(-h / math.sqrt(2))
    if act == "silu":
        return h * torch.sigmoid(h)
    if act == "swiglu":
        n = h.shape[-1] // 2
        return h[..., :n] * torch.sigmoid(h[..., :n]) * h[..., n:]
    return h


def _exact_experts(s):
    c = s["c"]
    out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
    pre = None if s["pre"] is None else torch.empty(s["pre"].shape, dtype=torch.float64, device="cuda")
    ends = np.cumsum(s["per"])
    for e, end in enumerate(ends):
        rows = slice(int(end) - s["per"][e], int(end))
        h = s["x"][rows].double() @ s["weight"][e].double().t()
        if s["bias"] is not None:
            h += s["bias"][e].double()
        if pre is not None:
            pre[rows] = h
        out[rows] = _exact_act(c["act"], h)
    if s["residual"] is not None:
        out += s["residual"].double()
    return {"out": out, "pre": pre}


def _exact_experts_grad(s):
    """The activation's derivative by automatic differentiation in 64 bits, then the products."""
    c = s["c"]
    d_pre = s["d_out"].double()
    if s["pre"] is not None:
        h = s["pre"].double().requires_grad_(True)
        d_pre, = torch.autograd.grad(_exact_act(c["act"], h), h, d_pre)
    d_x = torch.empty(s["x"].shape, dtype=torch.float64, device="cuda")
    d_weight = torch.empty(s["weight"].shape, dtype=torch.float64, device="cuda")
    d_bias = None if s["bias"] is None else torch.empty(s["bias"].shape, dtype=torch.float64, device="cuda")
    ends = np.cumsum(s["per"])
    for e, end in enumerate(ends):
        rows = slice(int(end) - s["per"][e], int(end))
        d_x[rows] = d_pre[rows] @ s["weight"][e].double()
        d_weight[e] = d_pre[rows].t() @ s["x"][rows].double()
        if d_bias is not None:
            d_bias[e] = d_pre[rows].sum(0)
    return {"d_pre": None if s["pre"] is None else d_pre, "d_x": d_x, "d_weight": d_weight, "d_bias": d_bias}
