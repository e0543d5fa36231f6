"""Microscaled rows on the GPU: both directions bit for bit against the tables
of what can be represented, at sizes and bases that are no multiples of
anything, with zeros, infinities, NaN, the smallest and the largest values and
every tie between two elements."""
import math

import pytest
import torch

import mx_ref as M
from embeddings_a2av_virtual_amd import _binding as B
from gpu_util import GuardedBuffer, SENT

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
FORMATS = {"fp8": B.MX_FP8, "fp4": B.MX_FP4}


def _array(x, pad):
    b = GuardedBuffer(x.numel() * x.element_size(), pad=pad)
    v = b.view.view(x.dtype).reshape(x.shape)
    v.copy_(x)
    return b, v


def quantize(xs, form, pad=0, status=0):
    """Rows of every rank, all of their bytes, behind a check of the guards."""
    H = xs[0].shape[1]
    wide = B.moe_mx_row_bytes(form, H)
    bufs = [GuardedBuffer(len(x) * wide) for x in xs]
    st = torch.full((1,), status, dtype=torch.int32, device="cuda")
    B.moe_mx_quantize(len(xs), H, form, [_array(x, pad)[1] for x in xs], [len(x) for x in xs],
                      [b.view for b in bufs], st)
    torch.cuda.synchronize()
    assert int(st.item()) == status and all(b.guards_intact() for b in bufs)
    return [b.view.cpu().reshape(len(x), wide) for b, x in zip(bufs, xs)]


def dequantize(rows, form, H, dtype, pad=0):
    bufs = [GuardedBuffer(len(r) * H * dtype.itemsize, pad=pad) for r in rows]
    out = [b.view.view(dtype).reshape(len(r), H) for b, r in zip(bufs, rows)]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.moe_mx_dequantize(len(rows), H, form, [_array(r, 0)[1] for r in rows], [len(r) for r in rows], out, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and all(b.guards_intact() for b in bufs)
    return [x.cpu() for x in out]


def check(xs, form, pad=0):
    H = xs[0].shape[1]
    for x, got in zip(xs, quantize(xs, form, pad)):
        want = M.quantize(x.double(), form)
        n = M.used_bytes(form, H)
        assert torch.equal(got[:, :n], want), (got[:, :n] != want).nonzero()[:4].tolist()
        assert (got[:, n:] == SENT).all()


@pytest.mark.parametrize("form", FORMATS)
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("H", [1, 7, 32, 33, 248, 256, 257, 1000, 1003, 4104])
def test_quantize(form, kind, H):
    g = torch.Generator().manual_seed(H)
    xs = [(torch.randn(n, H, generator=g) * torch.exp(2 * torch.randn(n, 1, generator=g))).to(TYPES[kind])
          for n in (5, 0, 1, 17)]
    check(xs, FORMATS[form])
    check(xs, FORMATS[form], pad=TYPES[kind].itemsize)


@pytest.mark.parametrize("form", FORMATS)
@pytest.mark.parametrize("kind", TYPES)
def test_special_values(form, kind):
    t, f = TYPES[kind], FORMATS[form]
    top, tiny = torch.finfo(t).max, torch.finfo(t).tiny
    g = torch.Generator().manual_seed(7)
    rows = [torch.zeros(64), -torch.zeros(64), torch.full((64,), top), torch.full((64,), -top), torch.full((64,), tiny),
            torch.full((64,), tiny / 8), torch.randn(64, generator=g) * tiny, torch.randn(64, generator=g) * top / 8]
    for bad in (math.inf, -math.inf, math.nan):
        x = torch.randn(64, generator=g)
        x[5] = bad
        rows.append(x)
    # every element, every middle of two and their neighbours, beside the largest
    e = M.table(f).float()
    near = torch.cat([e, (e[1:] + e[:-1]) / 2])
    near = near.to(t)
    near = torch.cat([near, torch.nextafter(near, near * 2 + 1), torch.nextafter(near, near * 0 - 1)])
    for sign in (1, -1):
        for k in (-3, 0, 2):
            x = torch.zeros(-(-len(near) // 31), 32)
            x[:, 0] = e[-1]
            flat = torch.zeros(x.shape[0] * 31)
            flat[:len(near)] = near.float()
            x[:, 1:] = flat.reshape(-1, 31)
            x = sign * x * 2.0 ** k
            rows += list(torch.nn.functional.pad(x, (0, 32)))
    x = torch.stack(rows).to(t)
    check([x], f)


@pytest.mark.parametrize("form", FORMATS)
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("H", [1, 8, 33, 256, 1003])
def test_dequantize(form, kind, H):
    g = torch.Generator().manual_seed(H)
    f, t = FORMATS[form], TYPES[kind]
    rows = []
    for n in (3, 0, 11):
        r = torch.randint(0, 256, (n, M.row_bytes(f, H)), generator=g).to(torch.uint8)
        at = M.padded(H) // (1 if f == M.FP8 else 2)
        r[:, at:] = torch.randint(100, 150, r[:, at:].shape, generator=g).to(torch.uint8)
        if n == 11:  # the smallest and largest scales, and NaN
            r[0, at:], r[1, at:], r[2, at:], r[3, at:] = 0, 254, 255, 1
        rows.append(r)
    for pad in (0, t.itemsize):
        for r, got in zip(rows, dequantize(rows, f, H, t, pad)):
            want = M.values(r, f, H).to(t)  # at most four bits of mantissa: one rounding, if any
            nan = torch.isnan(want)
            assert torch.equal(torch.isnan(got), nan) and torch.equal(got[~nan], want[~nan])


def test_a_set_status_stops_both():
    x = torch.randn(3, 64)
    assert all((r == SENT).all() for r in quantize([x], B.MX_FP8, status=1))
    out = torch.full((3, 64), 5.0, device="cuda")
    st = torch.ones(1, dtype=torch.int32, device="cuda")
    B.moe_mx_dequantize(1, 64, B.MX_FP8, [torch.zeros(3, 384, dtype=torch.uint8, device="cuda")], [3], [out], st)
    torch.cuda.synchronize()
    assert (out == 5).all()


def test_refusals():
    x, rows = torch.zeros(4, 64, device="cuda"), torch.zeros(4, 384, dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for args in ((1, 64, 7, [x], [4], [rows]), (1, 64, B.MX_FP8, [x], [5], [rows]), (2, 64, B.MX_FP8, [x], [4], [rows]),
                 (1, 64, B.MX_FP8, [x.double()], [4], [rows]), (1, 64, B.MX_FP8, [x.cpu()], [4], [rows]),
                 (1, 64, B.MX_FP8, [x.t()], [4], [rows]), (1, 64, B.MX_FP8, [x], [4], [rows.float()]),
                 (1, 64, B.MX_FP8, [x], [4], [rows[:3]])):
        with pytest.raises((ValueError, B.A2avError)):
            B.moe_mx_quantize(*args, st)
    with pytest.raises(B.A2avError):
        B.moe_mx_dequantize(1, 64, B.MX_FP4, [rows.flatten()[4:4 + 3 * 256]], [3], [x], st)


@pytest.mark.parametrize("grid", [1, 3])
def test_small_grids(grid, monkeypatch):
    monkeypatch.setenv("A2AV_MAX_GRID", str(grid))
    g = torch.Generator().manual_seed(grid)
    xs = [torch.randn(n, 600, generator=g).to(torch.bfloat16) for n in (70, 9)]
    check(xs, B.MX_FP4)
    rows = [torch.nn.functional.pad(M.quantize(x.double(), M.FP8), (0, M.row_bytes(M.FP8, 600) - M.used_bytes(M.FP8, 600)))
            for x in xs]
    for r, got in zip(rows, dequantize(rows, B.MX_FP8, 600, torch.float32)):
        assert torch.equal(got, M.values(r, M.FP8, 600).float())
