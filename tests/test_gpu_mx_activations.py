"""Outputs of moe_expert_linear_mx in 8 bits, element by element: on sums that fp32
holds exactly the activations' values are those of 64 bits to 1e-9, so that only
elements that far from a border of two may be otherwise; few rows and tiles."""
import math

import pytest
import torch

import mx_ref as M
from embeddings_a2av_virtual_amd import _binding as B
from test_gpu_mx_tiles import whole

pytestmark = pytest.mark.gpu

FORMATS = {"fp8": B.MX_FP8, "fp4": B.MX_FP4}


def silu(h):
    return h / (1 + torch.exp(-h))


ACTS = {"none": (B.ACT_NONE, lambda h: h), "relu": (B.ACT_RELU, lambda h: h.clamp(min=0)),
        "gelu": (B.ACT_GELU, lambda h: 0.5 * h * torch.special.erfc(-h / math.sqrt(2))), "silu": (B.ACT_SILU, silu),
        "swiglu": (B.ACT_SWIGLU, lambda h: silu(h[:, :h.shape[1] // 2]) * h[:, h.shape[1] // 2:])}


@pytest.mark.parametrize("rows", [9, 300])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("form", FORMATS)
@pytest.mark.parametrize("scale", [118, 121, 125])
def test_elements(form, act, rows, scale):
    """h of standard deviation about 0.4, 3 and 50."""
    g = torch.Generator(device="cuda").manual_seed(rows + scale)
    K, N, (code, f) = 512, 328, ACTS[act]
    NW = 2 * N if act == "swiglu" else N
    x, xv = whole(rows, K, FORMATS[form], g)
    w, wv = whole(NW, K, M.FP4, g)
    w[:, K // 2:K // 2 + K // 32] = scale
    bias = torch.randint(-30, 31, (1, NW), generator=g, device="cuda") * 2.0 ** (scale - 127)
    h = xv @ wv.t() * 2.0 ** (scale - 127) + bias.double()
    assert torch.equal(h.float().double(), h)
    out = torch.zeros(rows, M.row_bytes(M.FP8, N), dtype=torch.uint8, device="cuda")
    ws = torch.empty(B.moe_expert_linear_mx_workspace_bytes(1, 1, K, N, code, [rows]), dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    off = torch.tensor([[0, rows]], dtype=torch.int64, device="cuda")
    B.moe_expert_linear_mx(1, 1, K, N, FORMATS[form], code, [x], [rows], off, [w], [bias.float()], [out], ws, st)
    assert int(st.item()) == 0
    y, got, n = f(h).cpu(), out.cpu(), M.padded(N)
    near = [M.quantize(y * (1 + e), M.FP8) for e in (0.0, -1e-9, 1e-9)]
    bad = torch.ones(rows, n // 32, dtype=torch.bool)
    for want in near:
        off = got[:, :want.shape[1]] != want
        bad &= off[:, :n].reshape(rows, n // 32, 32).any(-1) | off[:, n:]
    assert not bad.any(), bad.nonzero()[:4].tolist()


@pytest.mark.parametrize("act", ACTS)
def test_far_values(act):
    """h from -2^100 to 2^100, infinite and NaN, by the bias alone."""
    code, f = ACTS[act]
    mags = torch.tensor([0, 2.0 ** -100, 1e-3, 0.5, 4, 8, 12, 18, 25, 60, 87, 90, 104, 200, 1e4, 2.0 ** 100], dtype=torch.float64)
    h = torch.cat([mags, -mags]).repeat_interleave(32)
    if act != "gelu":
        special = torch.tensor([math.inf, math.nan], dtype=torch.float64)
        h = torch.cat([h, special.repeat_interleave(32)])
    N = len(h)
    bias = (torch.cat([h, torch.ones(N, dtype=torch.float64)]) if act == "swiglu" else h).float()[None].cuda()
    NW, K = bias.shape[1], 32
    x = torch.zeros(1, M.row_bytes(M.FP8, K), dtype=torch.uint8, device="cuda")
    w = torch.zeros(NW, M.row_bytes(M.FP4, K), dtype=torch.uint8, device="cuda")
    out = torch.zeros(1, M.row_bytes(M.FP8, N), dtype=torch.uint8, device="cuda")
    ws = torch.empty(B.moe_expert_linear_mx_workspace_bytes(1, 1, K, N, code, [1]), dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    off = torch.tensor([[0, 1]], dtype=torch.int64, device="cuda")
    B.moe_expert_linear_mx(1, 1, K, N, M.FP8, code, [x], [1], off, [w], [bias], [out], ws, st)
    assert int(st.item()) == 0
    used = M.used_bytes(M.FP8, N)
    h = h + 0.0  # the products' sum is +0, and so is its sum with -0
    full = torch.cat([h, torch.ones(N, dtype=torch.float64)]) if act == "swiglu" else h
    y, got, n = f(full[None]), out.cpu()[:, :used], M.padded(N)
    same = torch.zeros(1, n // 32, dtype=torch.bool)
    for e in (0.0, -1e-9, 1e-9):
        off = got != M.quantize(y * (1 + e), M.FP8)
        same |= ~(off[:, :n].reshape(1, n // 32, 32).any(-1) | off[:, n:])
    assert same.all(), same.logical_not().nonzero().tolist()
