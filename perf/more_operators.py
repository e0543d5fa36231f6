"""Timing cases of the operators that put a MoE layer on microscaled rows: the root-mean-square norm in
front of the router (with the residual's addition, and rows in 8 bits ready for the dispatch) and its
gradient, the conversion of rows and weights to and from 8- and 4-bit blocks, and the experts' products
on such rows with 4-bit weights.

A microscaled row of width H holds H elements padded with zeros to a multiple of 256 (e4m3: a byte each;
e2m1: two a byte, the even one in the low half), then a scale byte (2^(byte - 127)) for every 32 of them,
and fills up to a multiple of 128 bytes. A block's scale is 2^(floor(log2(largest magnitude)) - 8) for
e4m3 and - 2 for e2m1, its elements are rounded to nearest even and stop at 448 and 6.

``run`` makes one pass. With ``own`` it makes the library's calls; without, it computes the same outputs
from elementary torch operations in 32 bits (what is rounded to 8 bits or fewer in 64, since values next to
a rounding border decide an element), rounded once at the end. ``exact`` gives the values in 64 bits. Eight-bit
elements and their scales are returned as the floating types that they are; four-bit ones go back to values by
the library's own call.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ACTS = ("none", "relu", "gelu", "silu", "swiglu")
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoded token: residual added, normed, and ready for the dispatch in 8 bits
        dict(name="norm token", op="norm", W=1, T=1, H=7168, type="bf16", residual=True, out=False, rows=True),
        # a prompt's batch on 8 ranks at the dispatch workload's width, the same way
        dict(name="norm batch", op="norm", W=8, T=2048, H=7168, type="bf16", residual=True, out=False, rows=True),
        # a width that is no multiple of a vector or a block: the normed rows in 16 and in 8 bits
        dict(name="norm odd fp16", op="norm", W=2, T=333, H=1003, type="fp16", residual=False, out=True, rows=True),
        # training: the gradient through the norm and past it, with the weight's
        dict(name="norm grad", op="norm_grad", W=8, T=2048, H=7168, type="bf16", d_sum=True),
        # the same in full precision at an odd size
        dict(name="norm grad odd fp32", op="norm_grad", W=1, T=1021, H=1111, type="fp32", d_sum=False),
        # tokens to 8 bits in front of the dispatch, where no norm does it
        dict(name="mx rows", op="mx", W=8, rows=2048, H=7168, type="bf16", format="fp8", back=False),
        # eight experts' up weights to 4 bits, and what they then stand for
        dict(name="mx weights back", op="mx", W=1, rows=8 * 4096, H=7168, type="bf16", format="fp4", back=True),
        # received rows back to values for products in 16 bits and their gradients: odd sizes
        dict(name="mx odd back fp32", op="mx", W=2, rows=389, H=1003, type="fp32", format="fp8", back=True),
        # one rank's 32 experts, gate and up products of a batch: 8-bit rows in, 8-bit rows out
        dict(name="experts mx up", op="experts", W=1, P=32, rows=16384, K=7168, N=2048, format="fp8", act="swiglu",
             bias=False, out="fp8"),
        # one decoded token's eight experts: the 4-bit weights are what has to be read
        dict(name="experts mx up token", op="experts", W=1, P=32, rows=8, K=7168, N=2048, format="fp8", act="swiglu",
             bias=False, out="fp8"),
        # the down products on 4-bit rows, out in the type that the combine reads
        dict(name="experts mx down fp4", op="experts", W=1, P=32, rows=16384, K=2048, N=7168, format="fp4",
             act="none", bias=False, out="bf16"),
        # small experts with a bias, ragged sizes on two ranks
        dict(name="experts mx odd fp16", op="experts", W=2, P=5, rows=777, K=1000, N=711, format="fp8", act="gelu",
             bias=True, out="fp16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "mx", "experts", "experts"])
    if op != "experts":
        W, H = rng.choice([1, 2, 4, 8]), _log(rng, 16, 16384)
        if rng.random() < 0.7:
            H = H // 16 * 16
        n = min(_log(rng, 1, 4096), max(1, 8 * 2048 * 7168 // (W * H)))
        c = dict(op=op, W=W, H=H, type=rng.choice(list(TYPES)))
        if op == "norm":
            rows = rng.random() < 0.7
            c.update(T=n, residual=rng.random() < 0.6, out=not rows or rng.random() < 0.4, rows=rows)
        elif op == "norm_grad":
            c.update(T=n, d_sum=rng.random() < 0.6)
        else:
            form = rng.choice(["fp8", "fp4"])
            c.update(rows=n, format=form, back=form == "fp4" or rng.random() < 0.4)
        return c
    W, P = rng.choice([1, 2, 4]), _log(rng, 1, 16)
    K, N = _log(rng, 32, 7168), _log(rng, 32, 2048)
    if rng.random() < 0.8:
        K, N = K // 8 * 8, N // 8 * 8
    return dict(op=op, W=W, P=P, rows=_log(rng, 1, 8192), K=K, N=N, format=rng.choice(["fp8", "fp4"]),
                act=rng.choice(ACTS), bias=rng.random() < 0.5, out=rng.choice(["bf16", "fp16", "fp8"]))


# ------------------------------------------------------------------ the microscaled rows' bytes
def _padded(H):
    return -(-H // 256) * 256


def _element_bytes(form, H):
    return _padded(H) if form == "fp8" else _padded(H) // 2


def _row_bytes(form, H):
    return -(-(_element_bytes(form, H) + _padded(H) // 32) // 128) * 128


def _blocks(v):
    """[..., H] as [..., blocks, 32], zeros behind the end."""
    blocks = -(-v.shape[-1] // 32)
    v = torch.nn.functional.pad(v, (0, blocks * 32 - v.shape[-1]))
    return v.reshape(*v.shape[:-1], blocks, 32)


def _power(exponent):
    """2^exponent in 64 bits without a rounding, from the bits of the number."""
    return ((exponent.long() + 1023) << 52).view(torch.float64)


def _quantize(v, form):
    """Elements [..., H] and scale exponents [..., blocks] of values. What is between two elements goes to the
    nearest by rounding in units of the value's own last place."""
    top, low, bits, most = (8, -6, 3, 448.0) if form == "fp8" else (2, 0, 1, 6.0)
    b = _blocks(v.double())
    exponent = torch.frexp(b.abs().amax(-1)).exponent - 1 - top
    exponent = torch.where(b.abs().amax(-1) == 0, -127, exponent).clamp(min=-127)
    s = b * _power(-exponent)[..., None]
    unit = (torch.frexp(s).exponent - 1).clamp(min=low) - bits
    s = (torch.round(s * _power(-unit)) * _power(unit)).clamp(-most, most)
    return s.flatten(-2)[..., :v.shape[-1]], exponent


def _table(form):
    """The magnitudes of the 4- or 8-bit elements in the order of their codes."""
    if form == "fp4":
        return torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device="cuda", dtype=torch.float64)
    m = torch.arange(127, device="cuda", dtype=torch.int64)
    e, f = m >> 3, (m & 7).double()
    return torch.where(e == 0, f * 2.0 ** -9, (1 + f / 8) * _power(e - 7))


def _to_bytes(v, form):
    """Microscaled rows [R, row_bytes] of values [R, H]."""
    H = v.shape[-1]
    s, exponent = _quantize(v, form)
    out = torch.zeros((v.shape[0], _row_bytes(form, H)), dtype=torch.uint8, device=v.device)
    n = _element_bytes(form, H)
    if form == "fp8":
        out[:, :H] = s.to(E4M3).view(torch.uint8)
    else:
        code = torch.bucketize(s.abs(), _table("fp4")).to(torch.uint8) + 8 * (s < 0).to(torch.uint8)
        code = torch.nn.functional.pad(code, (0, H % 2))
        out[:, :code.shape[-1] // 2] = code[:, ::2] + 16 * code[:, 1::2]
    out[:, n:n + exponent.shape[-1]] = (exponent + 127).to(torch.uint8)
    return out


def _values(rows, form, H, dtype=torch.float32):
    """The values [R, H] that microscaled rows stand for."""
    n, blocks = _element_bytes(form, H), -(-H // 32)
    if form == "fp8":
        v = rows[:, :H].view(E4M3).to(dtype)
    else:
        code = rows[:, :-(-H // 2)]
        code = torch.stack([code & 15, code >> 4], -1).flatten(1)[:, :H].long()
        v = torch.cat([_table("fp4"), -_table("fp4")]).to(dtype)[code]
    scale = _power(rows[:, n:n + blocks].long() - 127).to(dtype)
    return (_blocks(v) * scale[..., None]).flatten(-2)[:, :H]


def _eight_bits(rows, H):
    """The elements and scales of 8-bit rows as the types they are, where they lie."""
    n = _element_bytes("fp8", H)
    return {"elements": rows[:, :H].view(E4M3), "scales": rows[:, n:n + -(-H // 32)].view(E8M0)}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _tokens(g, W, T, H):
    """Hidden states: tokens and channels of different sizes."""
    return _randn(g, W, T, H) * torch.exp(0.5 * _randn(g, W, T, 1)) * torch.exp(0.5 * _randn(g, H))


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
    if c["op"] == "norm":
        t, T, H = TYPES[c["type"]], c["T"], c["H"]
        s["x"] = _tokens(g, W, T, H).to(t)
        s["residual"] = _tokens(g, W, T, H).to(t) if c["residual"] else None
        s["weight"] = (1 + 0.1 * _randn(g, H)).to(t)
        s["sum"] = torch.empty_like(s["x"]) if c["residual"] else None
        s["out"] = torch.empty_like(s["x"]) if c["out"] else None
        s["rows"] = torch.empty((W * T, _row_bytes("fp8", H)), dtype=torch.uint8, device="cuda") if c["rows"] else None
        return s
    if c["op"] == "norm_grad":
        t, T, H = TYPES[c["type"]], c["T"], c["H"]
        s["x"] = _tokens(g, W, T, H).to(t)
        s["weight"] = (1 + 0.1 * _randn(g, H)).to(t)
        s["d_out"] = _randn(g, W, T, H).to(t)
        s["d_sum"] = _randn(g, W, T, H).to(t) if c["d_sum"] else None
        s["d_x"] = torch.empty_like(s["x"])
        s["d_weight"] = torch.empty(H, device="cuda")
        return s
    if c["op"] == "mx":
        s["x"] = _tokens(g, W, c["rows"], c["H"]).to(TYPES[c["type"]])
        s["rows"] = torch.empty((W * c["rows"], _row_bytes(c["format"], c["H"])), dtype=torch.uint8, device="cuda")
        s["back"] = torch.empty_like(s["x"]) if c["back"] else None
        return s
    P, K, N = c["P"], c["K"], c["N"]
    NW = 2 * N if c["act"] == "swiglu" else N
    per = _expert_rows(c, seed)
    R = int(per.sum())
    s["per"] = per.reshape(-1).tolist()
    s["cut"] = per.sum(1).tolist()
    s["offsets"] = torch.from_numpy(np.concatenate([np.zeros((W, 1), np.int64), per.cumsum(1)], 1)).cuda()
    s["x"] = _to_bytes(_randn(g, R, K), c["format"])
    s["weight"] = torch.empty((W * P, NW, _row_bytes("fp4", K)), dtype=torch.uint8, device="cuda")
    for e in range(W * P):
        s["weight"][e] = _to_bytes(_randn(g, NW, K) / math.sqrt(K), "fp4")
    s["bias"] = 0.5 * _randn(g, W * P, NW) if c["bias"] else None
    s["out"] = torch.empty((R, _row_bytes("fp8", N)), dtype=torch.uint8, device="cuda") if c["out"] == "fp8" else \
        torch.empty((R, N), dtype=TYPES[c["out"]], device="cuda")
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["c"]["op"]
    if own:
        return {"norm": _own_norm, "norm_grad": _own_norm_grad, "mx": _own_mx, "experts": _own_experts}[op](state)
    return {"norm": _norm, "norm_grad": _norm_grad, "mx": _mx, "experts": _experts}[op](state)


def _ranks(x, W):
    return None if x is None else list(x.chunk(W))


def _cut(x, cut):
    return None if x is None else list(torch.split(x, cut))


def _workspace(s, size):
    """Kept between passes, as a program keeps it between steps."""
    if "workspace" not in s:
        s["workspace"] = torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")
    return s["workspace"]


def _own_norm(s):
    from embeddings_a2av_virtual_amd import _binding as B
    c, W = s["c"], s["c"]["W"]
    B.moe_rms_norm(W, c["T"], c["H"], EPS, _ranks(s["x"], W), _ranks(s["residual"], W), s["weight"],
                   _ranks(s["sum"], W), _ranks(s["out"], W), _ranks(s["rows"], W), B.MX_FP8, s["status"])
    return {"sum": s["sum"], "out": s["out"], "rows": None if s["rows"] is None else _eight_bits(s["rows"], c["H"])}


def _own_norm_grad(s):
    from embeddings_a2av_virtual_amd import _binding as B
    c, W = s["c"], s["c"]["W"]
    ws = _workspace(s, B.moe_rms_norm_backward_workspace_bytes(W, c["T"], c["H"]))
    B.moe_rms_norm_backward(W, c["T"], c["H"], EPS, _ranks(s["x"], W), s["weight"], _ranks(s["d_out"], W),
                            _ranks(s["d_sum"], W), _ranks(s["d_x"], W), s["d_weight"], ws, s["status"])
    return {"d_x": s["d_x"], "d_weight": s["d_weight"]}


def _own_mx(s):
    from embeddings_a2av_virtual_amd import _binding as B
    c, W = s["c"], s["c"]["W"]
    form, n = B.MX_FP8 if c["format"] == "fp8" else B.MX_FP4, [c["rows"]] * W
    B.moe_mx_quantize(W, c["H"], form, _ranks(s["x"], W), n, _ranks(s["rows"], W), s["status"])
    if not c["back"]:
        return _eight_bits(s["rows"], c["H"])
    B.moe_mx_dequantize(W, c["H"], form, _ranks(s["rows"], W), n, _ranks(s["back"], W), s["status"])
    return {"back": s["back"]}


def _own_experts(s):
    from embeddings_a2av_virtual_amd import _binding as B
    c, W, P, cut = s["c"], s["c"]["W"], s["c"]["P"], s["cut"]
    form = B.MX_FP8 if c["format"] == "fp8" else B.MX_FP4
    act = {"none": B.ACT_NONE, "relu": B.ACT_RELU, "gelu": B.ACT_GELU, "silu": B.ACT_SILU,
           "swiglu": B.ACT_SWIGLU}[c["act"]]
    ws = _workspace(s, B.moe_expert_linear_mx_workspace_bytes(W, P, c["K"], c["N"], act, cut))
    B.moe_expert_linear_mx(W, P, c["K"], c["N"], form, act, _cut(s["x"], cut), cut, s["offsets"],
                           _ranks(s["weight"], W), _ranks(s["bias"], W), _cut(s["out"], cut), ws, s["status"])
    return _eight_bits(s["out"], c["N"]) if c["out"] == "fp8" else {"out": s["out"]}


# ------------------------------------------------------------------ the plain forms
def _plain_eight_bits(v):
    elements, exponent = _quantize(v.flatten(0, -2), "fp8")
    return {"elements": elements.to(E4M3), "scales": (exponent + 127).to(torch.uint8).view(E8M0)}


def _norm(s):
    c, h = s["c"], s["x"]
    if s["residual"] is not None:
        h = (h.float() + s["residual"].float()).to(h.dtype)
    got = {"sum": h if c["residual"] else None, "out": None, "rows": None}
    if c["out"]:
        v = h.float()
        v = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * s["weight"].float()
        got["out"] = v.to(h.dtype)
    if c["rows"]:
        v = h.double()
        got["rows"] = _plain_eight_bits(v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * s["weight"].double())
    return got


def _norm_grad(s):
    x, g = s["x"].float(), s["d_out"].float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    x = x * r
    d_weight = (g * x).sum((0, 1))
    g = g * s["weight"].float()
    d = r * (g - x * (g * x).mean(-1, keepdim=True))
    if s["d_sum"] is not None:
        d = d + s["d_sum"].float()
    return {"d_x": d.to(s["x"].dtype), "d_weight": d_weight}


def _mx(s):
    c, x = s["c"], s["x"]
    if not c["back"]:
        return _plain_eight_bits(x)
    elements, exponent = _quantize(x, c["format"])
    v = (_blocks(elements) * _power(exponent)[..., None]).flatten(-2)[..., :c["H"]]
    return {"back": v.to(s["x"].dtype)}


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


# One product for each expert that has rows: a padded batch of them would do several times the work.
def _experts(s):
    c = s["c"]
    x = _values(s["x"], c["format"], c["K"])
    y = torch.empty((x.shape[0], c["N"]), device=x.device)
    at = 0
    for e, n in enumerate(s["per"]):
        if n:
            h = x[at:at + n] @ _values(s["weight"][e], "fp4", c["K"]).t()
            if s["bias"] is not None:
                h = h + s["bias"][e]
            y[at:at + n] = _activate(c["act"], h)
            at += n
    return _plain_eight_bits(y) if c["out"] == "fp8" else {"out": y.to(s["out"].dtype)}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c, W = case, case["W"]
    if c["op"] == "experts":
        NW = 2 * c["N"] if c["act"] == "swiglu" else c["N"]
        R, K, N, P = c["rows"], c["K"], c["N"], c["P"]
        busy = min(R, W * P)  # experts that can have rows
        bits = lambda form, n: n if form == "fp8" else n / 2  # noqa: E731
        b = R * (bits(c["format"], K) + K / 32) + busy * NW * (K / 2 + K / 32) + (4 * busy * NW if c["bias"] else 0)
        return {"bytes": b + R * (N + N / 32 if c["out"] == "fp8" else 2 * N), "flops": 2 * R * NW * K}
    size = 4 if c["type"] == "fp32" else 2
    n = W * (c["rows"] if c["op"] == "mx" else c["T"]) * c["H"]
    if c["op"] == "mx":
        e = (1 if c["format"] == "fp8" else 0.5) + 1 / 32  # written, and read again on the way back
        return {"bytes": n * (size + e) + (n * (size + e) if c["back"] else 0), "flops": 4 * n}
    if c["op"] == "norm":
        arrays = 1 + 2 * c["residual"] + c["out"]
        return {"bytes": n * (arrays * size + (1 + 1 / 32 if c["rows"] else 0)) + size * c["H"], "flops": 4 * n}
    return {"bytes": n * size * (3 + c["d_sum"]) + (size + 4) * c["H"], "flops": 10 * n}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "norm_grad": _exact_norm_grad, "mx": _exact_mx, "experts": _exact_experts}[case["op"]](s)


def _exact_quantize(v, form):
    """Elements and scales by searches in the tables of what can be represented."""
    H, top = v.shape[-1], 8 if form == "fp8" else 2
    powers = torch.tensor([2.0 ** k for k in range(-400, 400)], dtype=torch.float64, device=v.device)
    b = torch.cat([v, v.new_zeros(*v.shape[:-1], -H % 32)], -1).unflatten(-1, ((H + 31) // 32, 32))
    k = torch.searchsorted(powers, b.abs().amax(-1), right=True) - 401 - top  # -401 - top or less for a block of zeros
    scale = powers[k.clamp(min=-127) + 400]
    a, t = (b / scale[..., None]).abs(), _table(form)
    half = (t[1:] + t[:-1]) / 2
    at = torch.searchsorted(half, a)
    tie = (at < len(half)) & (a == half[at.clamp(max=len(half) - 1)])
    at = at + (tie & (at % 2 == 1))
    return (torch.sign(b) * t[at]).flatten(-2)[..., :H], scale


def _exact_eight_bits(v):
    elements, scales = _exact_quantize(v.flatten(0, -2), "fp8")
    return {"elements": elements, "scales": scales}


def _exact_norm(s):
    c, h = s["c"], s["x"].double()
    if s["residual"] is not None:
        h = (h + s["residual"].double()).to(s["x"].dtype).double()
    y = h / torch.sqrt(torch.linalg.vector_norm(h, dim=-1, keepdim=True) ** 2 / c["H"] + EPS) * s["weight"].double()
    return {"sum": h if c["residual"] else None, "out": y if c["out"] else None,
            "rows": _exact_eight_bits(y) if c["rows"] else None}


def _exact_norm_grad(s):
    """By automatic differentiation in 64 bits, a few rows at a time."""
    c, w = s["c"], s["weight"].double().requires_grad_(True)
    x, g = s["x"].flatten(0, 1), s["d_out"].flatten(0, 1)
    d_x, d_weight = torch.empty(x.shape, dtype=torch.float64, device=x.device), torch.zeros_like(w)
    for at in range(0, x.shape[0], 4096):
        v = x[at:at + 4096].double().requires_grad_(True)
        y = v / torch.sqrt(v.square().mean(-1, keepdim=True) + EPS) * w
        d, dw = torch.autograd.grad(y, (v, w), g[at:at + 4096].double())
        d_x[at:at + 4096] = d
        d_weight = d_weight + dw
    if s["d_sum"] is not None:
        d_x += s["d_sum"].flatten(0, 1).double()
    return {"d_x": d_x.reshape(s["x"].shape), "d_weight": d_weight.detach()}


def _exact_mx(s):
    c = s["c"]
    if not c["back"]:
        return _exact_eight_bits(s["x"].double())
    elements, scales = _exact_quantize(s["x"].double(), c["format"])
    return {"back": elements * scales.repeat_interleave(32, -1)[..., :c["H"]]}


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
    y = torch.empty((len(s["x"]), c["N"]), dtype=torch.float64, device="cuda")
    ends = np.cumsum(s["per"])
    for e, end in enumerate(ends):
        rows = slice(int(end) - s["per"][e], int(end))
        h = _values(s["x"][rows], c["format"], c["K"], torch.float64) @ _values(s["weight"][e], "fp4", c["K"],
                                                                                torch.float64).t()
        if s["bias"] is not None:
            h += s["bias"][e].double()
        y[rows] = _exact_act(c["act"], h)
    return _exact_eight_bits(y) if c["out"] == "fp8" else {"out": y}
