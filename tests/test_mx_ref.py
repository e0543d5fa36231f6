"""The 64-bit references of the microscaled rows and the norm, pinned against
torch's own 8-bit type, automatic differentiation and differences (no GPU)."""
import math

import pytest
import torch

import mx_ref as M


def test_e4m3_table_is_torchs():
    t = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    assert torch.equal(t, M.table(M.FP8))


def test_elements_are_torchs_casts():
    g = torch.Generator().manual_seed(0)
    v = torch.randn(64, 512, generator=g)
    rows = M.quantize(v.double(), M.FP8)
    scale = torch.pow(2.0, rows[:, 512:].double() - 127).repeat_interleave(32, 1)
    want = (v / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(rows[:, :512], want)


@pytest.mark.parametrize("form", [M.FP8, M.FP4])
def test_values_that_fit_come_back(form):
    t = M.table(form)
    t = torch.cat([t, -t[1:]])
    for k in (-100, 0, 60):
        v = torch.zeros(len(t), 32, dtype=torch.float64)
        v[:, 0] = M.table(form)[-1] * 2.0 ** k
        v[:, 1] = t * 2.0 ** k
        rows = M.quantize(v, form)
        assert torch.equal(M.values(rows, form, 32), v)
        assert (rows[:, -8] == k + 127).all() and (rows[:, -7:] == 0).all()


@pytest.mark.parametrize("form", [M.FP8, M.FP4])
def test_rounding_and_scales(form):
    top = M.TOP[form]
    for m in (1.0, 1.999, 2.0, 3.7, 2.0 ** -120, 2.0 ** 100):
        rows = M.quantize(torch.tensor([[m] + [0.0] * 31], dtype=torch.float64), form)
        assert int(rows[0, -8]) == max(0, math.floor(math.log2(m)) + 127 - top)
        got = float(M.values(rows, form, 1)[0, 0])
        assert abs(got - m) <= m / 4  # past the largest element it stops there
    for bad in (math.inf, -math.inf, math.nan):
        rows = M.quantize(torch.tensor([[1.0, bad] + [0.0] * 62], dtype=torch.float64), form)
        assert int(rows[0, -8]) == 255 and int(rows[0, -7]) == 0 and (rows[0, :16] == 0).all()
        assert torch.isnan(M.values(rows, form, 32)).all()


def test_norm_gradient():
    g = torch.Generator().manual_seed(1)
    h, w = torch.randn(3, 10, generator=g).double(), torch.randn(10, generator=g).double()
    d, ds = torch.randn(3, 10, generator=g).double(), torch.randn(3, 10, generator=g).double()
    x, v = h.clone().requires_grad_(True), w.clone().requires_grad_(True)
    ((M.norm(x, v, 1e-3) * d).sum() + (x * ds).sum()).backward()
    dx, dw = M.norm_grad(h, w, 1e-3, d, ds)
    assert torch.allclose(dx, x.grad, rtol=1e-12) and torch.allclose(dw, v.grad, rtol=1e-12)
    f = lambda a, b: float((M.norm(a, b, 1e-3) * d).sum() + (a * ds).sum())  # noqa: E731
    step = 1e-6
    for at in ((0, 0), (2, 7)):
        e = torch.zeros_like(h)
        e[at] = step
        assert abs((f(h + e, w) - f(h - e, w)) / (2 * step) - float(dx[at])) < 1e-7
    e = torch.zeros_like(w)
    e[4] = step
    assert abs((f(h, w + e) - f(h, w - e)) / (2 * step) - float(dw[4])) < 1e-7
