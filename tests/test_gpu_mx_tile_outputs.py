"""Every kind of output of the microscaled products from every tile: 8-bit rows from both
formats (from e4m3 by two sums), fp16 and bf16, each activation and gate weights that are
not zero. The tile is computed by the library's rule; sums are whole numbers of a unit
that fp32 holds, over scales of two sizes and e4m3 elements on both sides of 2, so that
8-bit outputs are known to the bit but where an activation lies within 1e-9 of a
border. Products and 64-bit values on the GPU."""
import math

import pytest
import torch

import layer_ref as R
import mx_ref as M
from embeddings_a2av_virtual_amd import _binding as B
from gpu_util import SENT

pytestmark = pytest.mark.gpu

FORMATS = {"fp8": M.FP8, "fp4": M.FP4}
OUTS = {"fp8": torch.uint8, "fp16": torch.float16, "bf16": torch.bfloat16}
ACTS = {"none": B.ACT_NONE, "relu": B.ACT_RELU, "gelu": B.ACT_GELU, "silu": B.ACT_SILU, "swiglu": B.ACT_SWIGLU}
ROWS, COLS = (256, 128, 64), (256, 128, 128)
FEW = 3


def tile_of(rows, experts, N, gated, form, out):
    """The library's choice; the padding of 8-bit outputs has columns too, and from e4m3
    rows they leave no room for tiles of 256."""
    if rows <= 12 * experts:
        return FEW
    n, two = (M.padded(N) if out == "fp8" else N), form == M.FP8 and out == "fp8"
    cols = (n + 15) // 16 * 32 if gated else n
    for i in range(2 if rows <= 64 * experts else 1 if rows <= 128 * experts or two else 0, 2):
        tiles = rows // ROWS[i] + (experts // 2 if rows % (experts * ROWS[i]) else 0)
        if tiles * -(-cols // COLS[i]) >= 200:
            return i
    return 2


def power(e):
    """2^e in 64 bits from the number's bits (the GPU's pow is off by a place)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def quantize(v):
    """8-bit rows [R, used_bytes] of values [R, N], as M.quantize on the GPU."""
    b = torch.nn.functional.pad(v, (0, M.padded(v.shape[1]) - v.shape[1])).unflatten(1, (-1, 32))
    m = b.abs().amax(-1)
    byte = torch.where(m == 0, 0, (torch.frexp(m).exponent - 1 + 119).clamp(0, 254))
    s, t = b * power(127 - byte)[..., None], M.table(M.FP8).cuda()
    half = (t[1:] + t[:-1]) / 2
    code = torch.searchsorted(half, s.abs())
    code += (code % 2 == 1) & (s.abs() == half[code.clamp(max=len(half) - 1)])
    return torch.cat([(code + 128 * torch.signbit(s)).flatten(1), byte], 1).to(torch.uint8)


def whole(n, K, form, scale, g):
    """Rows of e2m1 elements, or of e4m3 ones of 0.25 to 14, with scales of `scale` and its double, and their values."""
    at = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device="cuda")  # noqa: E731
    code = at(0, 8, n, K) if form == M.FP4 else at(39, 87, n, K)
    if form == M.FP8:
        code = torch.where(code == 39, 0, code)
    table = M.table(form).cuda()
    sign = at(0, 2, n, K)
    byte = at(0, 2, n, M.padded(K) // 32) + 127 + scale
    v = table[code] * (1 - 2 * sign) * power(byte - 127).repeat_interleave(32, 1)[:, :K]
    code = torch.nn.functional.pad(code + sign * (8 if form == M.FP4 else 128), (0, M.padded(K) - K))
    if form == M.FP4:
        code = code[:, ::2] + 16 * code[:, 1::2]
    rows = torch.full((n, M.row_bytes(form, K)), 255, dtype=torch.uint8, device="cuda")
    rows[:, :code.shape[1]] = code.to(torch.uint8)
    rows[:, code.shape[1]:M.used_bytes(form, K)] = byte.to(torch.uint8)
    return rows, v


def activate(act, h):
    if act == "relu":
        return h.clamp(min=0)
    if act == "gelu":
        return 0.5 * h * torch.special.erfc(-h / math.sqrt(2))
    if act == "none":
        return h
    n = h.shape[1] // 2
    return h / (1 + torch.exp(-h)) if act == "silu" else h[:, :n] / (1 + torch.exp(-h[:, :n])) * h[:, n:]


def run(per, K, N, form, act, out, want):
    P, T, gated = len(per), sum(per), act == "swiglu"
    form, NW = FORMATS[form], 2 * N if gated else N
    assert tile_of(T, P, N, gated, form, out) == want
    g = torch.Generator(device="cuda").manual_seed(T + K + N)
    # activations of h of standard deviation about 4: elements and weights are about 8 and 4
    scale = 0 if act in ("none", "relu") else round(math.log2(4 / (32 * math.sqrt(K))))
    x, xv = whole(T, K, form, 0, g)
    w, wv = whole(P * NW, K, M.FP4, scale, g)
    wv = wv.reshape(P, NW, K)
    bias = torch.randint(-30, 31, (P, NW), generator=g, device="cuda") * 2.0 ** scale
    off = torch.tensor([[0] + torch.tensor(per).cumsum(0).tolist()], dtype=torch.int64, device="cuda")
    width = M.row_bytes(M.FP8, N) if out == "fp8" else 2 * N
    got = torch.full((T + 1, width), SENT, dtype=torch.uint8, device="cuda")
    ws = torch.empty(B.moe_expert_linear_mx_workspace_bytes(1, P, K, N, ACTS[act], [T]), dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.moe_expert_linear_mx(1, P, K, N, form, ACTS[act], [x], [T], off, [w], [bias.float()], [got.view(OUTS[out])], ws, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and (got[T] == SENT).all()
    at, unit = 0, 2.0 ** (scale - 6)
    for e, n in enumerate(per):
        if n == 0:
            continue
        xe, we, be = xv[at:at + n], wv[e], bias[e].double()
        assert ((xe.abs() @ we.t().abs() + be.abs()) / unit).max() < 2 ** 24
        h = xe @ we.t() + be
        y, o = activate(act, h), got[at:at + n]
        at += n
        if out == "fp8":
            used, pad = M.used_bytes(M.FP8, N), M.padded(N)
            assert (o[:, used:] == SENT).all()
            bad = torch.ones(n, pad // 32, dtype=torch.bool, device="cuda")
            for f in (0.0,) if act in ("none", "relu") else (0.0, -1e-9, 1e-9):
                d = o[:, :used] != quantize(y * (1 + f))
                bad &= d[:, :pad].reshape(n, pad // 32, 32).any(-1) | d[:, pad:]
        elif act in ("none", "relu"):
            bad = o.view(OUTS[out]) != y.to(OUTS[out])
        else:
            # fp32 steps of the activation, then the type's half a step
            err = (h[:, :N] * h[:, N:]).abs() * (h[:, :N].abs() + 16) if gated else h.abs() * (h.abs() + 16)
            half = R.half_step(OUTS[out])
            bad = (o.view(OUTS[out]).double() - y).abs() > err * 2.0 ** -23 + y.abs() * half * 1.01 + torch.finfo(
                OUTS[out]).smallest_normal * half * 2
        assert not bad.any(), (e, n, bad.nonzero()[:4].tolist(), int(bad.sum()))


# row tiles that end with 1, 64, 65, 128, 129 and 256 rows, and experts of fewer
LARGE = [257, 320, 321, 384, 385, 512, 1, 0, 63]
MIDDLE = [129, 192, 193, 256, 1, 0, 64]
SMALL = [65, 32, 33, 64, 1, 0, 128]


@pytest.mark.parametrize("macros", [1, 2, 3, 4, 5, 8, 9])
def test_largest_tiles_to_8_bits(macros):
    run(LARGE, macros * 256 - 5, 6008, "fp4", "none", "fp8", 0)
    run([300, 256, 40, 513, 0, 100], macros * 256, 4000, "fp4", "swiglu", "fp8", 0)


@pytest.mark.parametrize("form", FORMATS)
@pytest.mark.parametrize("macros", [1, 2, 3, 4, 5, 8, 9])
def test_middle_tiles_to_8_bits(form, macros):
    run(MIDDLE, macros * 256 - 7, 3300, form, "none", "fp8", 1)
    run([129, 60, 200], macros * 256 - 7, 3500, form, "swiglu", "fp8", 1)


@pytest.mark.parametrize("macros", [1, 2, 3, 5])
def test_many_rows_by_two_sums(macros):
    """What takes tiles of 256 with one sum."""
    run(LARGE, macros * 256, 6008, "fp8", "relu", "fp8", 1)
    run([300, 256, 40, 513, 0, 100], macros * 256, 4000, "fp8", "swiglu", "fp8", 1)


@pytest.mark.parametrize("form", FORMATS)
@pytest.mark.parametrize("macros", [1, 2, 3, 4, 5, 8, 9])
def test_smallest_tiles_to_8_bits(form, macros):
    run(SMALL, macros * 256 - 9, 330, form, "none", "fp8", 2)
    run([70, 60, 3], macros * 256 - 9, 250, form, "swiglu", "fp8", 2)


@pytest.mark.parametrize("form", FORMATS)
@pytest.mark.parametrize("act", ACTS)
def test_activations_to_8_bits(form, act):
    run(LARGE, 700, 6008, form, act, "fp8", 0 if form == "fp4" else 1)
    run(MIDDLE, 700, 3300, form, act, "fp8", 1)
    run([12, 0, 17, 3], 700, 300, form, act, "fp8", FEW)


@pytest.mark.parametrize("form", FORMATS)
@pytest.mark.parametrize("out", ["fp16", "bf16"])
@pytest.mark.parametrize("act", ACTS)
def test_activations_to_16_bits(form, out, act):
    run(LARGE, 1020, 6008, form, act, out, 0)
    run(MIDDLE, 1020, 3299, form, act, out, 1)
    run(SMALL, 1020, 330, form, act, out, 2)
    run([12, 0, 17, 3], 1020, 300, form, act, out, FEW)


def test_quantize():
    """The oracle on the GPU is the one on the host."""
    g = torch.Generator().manual_seed(1)
    v = torch.randn(40, 1000, generator=g).double() * torch.exp(2 * torch.randn(40, 1, generator=g))
    v[1:3], v[3, ::2], v[4] = torch.randint(-5000, 5000, (2, 1000), generator=g) / 4.0, 2.0 ** -130, 0
    assert torch.equal(quantize(v.cuda()).cpu(), M.quantize(v, M.FP8))
