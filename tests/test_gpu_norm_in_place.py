"""The norm and its gradient over their own inputs where a workgroup has several rows and
several waves a row, and where rows are read twice."""
import pytest
import torch

import mx_ref as M
from test_gpu_norm import TYPES, _rows, check, check_grad

pytestmark = pytest.mark.gpu

WIDTHS = [512, 1032, 2056, 5003, 9000, 16384, 16392]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("place", [("x", ""), ("", "x"), ("x", "r"), ("r", "x")])
def test_norm(H, kind, place, monkeypatch):
    monkeypatch.setenv("A2AV_MAX_GRID", "6")
    g = torch.Generator().manual_seed(H)
    t = TYPES[kind]
    weight = (1 + 0.2 * torch.randn(H, generator=g)).to(t)
    check(_rows(g, 2, 11, H, t), _rows(g, 2, 11, H, t), weight, M.FP8, place=place)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("place", ["x", "d_out", "d_sum"])
def test_gradient(H, kind, place, monkeypatch):
    monkeypatch.setenv("A2AV_MAX_GRID", "6")
    g = torch.Generator().manual_seed(H)
    t = TYPES[kind]
    weight = (1 + 0.2 * torch.randn(H, generator=g)).to(t)
    hs, gs, ds = (_rows(g, 2, 11, H, t) for _ in range(3))
    check_grad(hs, weight, gs, ds, place=place)
