"""Microscaled rows, the root-mean-square norm and its gradient in 64 bits on
the host, written from their definitions for the tests."""
from __future__ import annotations

import math

import torch

FP8, FP4 = 3, 4
TOP = {FP8: 8, FP4: 2}


def table(form):
    """The magnitudes of the elements in the order of their codes."""
    if form == FP4:
        return torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)
    return torch.tensor([m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                         for e in range(16) for m in range(8)][:127], dtype=torch.float64)


def padded(H):
    return -(-H // 256) * 256


def used_bytes(form, H):
    """Bytes of a row that are written: elements and scales."""
    return padded(H) // (1 if form == FP8 else 2) + padded(H) // 32


def row_bytes(form, H):
    return -(-used_bytes(form, H) // 128) * 128


def quantize(v, form):
    """Rows [R, used_bytes] of float64 values [R, H]."""
    R, H = v.shape
    b = torch.zeros((R, padded(H)), dtype=torch.float64)
    b[:, :H] = v
    b = b.reshape(R, padded(H) // 32, 32)
    m = b.abs().amax(-1)
    bad = ~torch.isfinite(b).all(-1)
    powers = torch.tensor([2.0 ** k for k in range(-1074, 1024)], dtype=torch.float64)
    k = torch.searchsorted(powers, torch.where(bad, 1.0, m), right=True) - 1 - 1074  # floor(log2 m)
    byte = torch.where(m == 0, 0, (k + 127 - TOP[form]).clamp(0, 254))
    s = torch.where(bad[..., None], 0.0, b) * torch.pow(torch.tensor(2.0, dtype=torch.float64), 127 - byte)[..., None]
    t = table(form)
    half = (t[1:] + t[:-1]) / 2
    code = torch.searchsorted(half, s.abs())
    tie = (code < len(half)) & (s.abs() == half[code.clamp(max=len(half) - 1)])
    code = code + (tie & (code % 2 == 1))
    code = (code + torch.signbit(s) * (128 if form == FP8 else 8)).flatten(1)
    if form == FP4:
        code = code[:, ::2] + 16 * code[:, 1::2]
    return torch.cat([code, torch.where(bad, 255, byte)], 1).to(torch.uint8)


def values(rows, form, H):
    """The float64 values [R, H] that rows stand for (at least their used bytes)."""
    n, t = padded(H) // (1 if form == FP8 else 2), table(form)
    code = rows[:, :n].long()
    if form == FP4:
        code = torch.stack([code & 15, code >> 4], -1).flatten(1)
        v = torch.cat([t, -t])[code]
    else:
        nan = torch.tensor([math.nan], dtype=torch.float64)
        v = torch.cat([t, nan, -t, nan])[code]
    b = rows[:, n:n + padded(H) // 32].long()
    scale = torch.where(b == 255, math.nan, torch.pow(torch.tensor(2.0, dtype=torch.float64), b - 127))
    return (v.reshape(len(rows), padded(H) // 32, 32) * scale[..., None]).flatten(1)[:, :H]


def add(x, residual):
    """h, as it is rounded: in fp32 and then to the type."""
    return x if residual is None else (x.float() + residual.float()).to(x.dtype)


def norm(h, weight, eps):
    """y in float64 of rows h [R, H]."""
    v = h.double()
    return v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps) * weight.double()


def norm_grad(h, weight, eps, d_out, d_sum):
    """d_x [R, H] and d_weight [H] by the formula."""
    v, w, g = h.double(), weight.double(), d_out.double()
    r = 1 / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)
    d = r * (g * w - v * r * r * (g * w * v).mean(-1, keepdim=True))
    return d if d_sum is None else d + d_sum.double(), (g * v * r).sum(0)
