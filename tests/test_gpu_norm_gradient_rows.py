"""The gradient of rows of 1025 to 2048 elements on both sides of the count from which
they take a wave each."""
import pytest
import torch

from test_gpu_norm import TYPES, _rows, check_grad

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("H", [1025, 1032, 1111, 1536, 2047, 2048])
@pytest.mark.parametrize("T", [1, 256, 257, 300])
def test_wide_waves(T, H, kind):
    g = torch.Generator().manual_seed(T + H)
    t = TYPES[kind]
    weight = (1 + 0.2 * torch.randn(H, generator=g)).to(t)
    hs, gs, ds = (_rows(g, 2, T, H, t) for _ in range(3))
    check_grad(hs, weight, gs, ds)
    check_grad(hs, weight, gs, None, want_w=False)


@pytest.mark.parametrize("H", [1025, 2048])
def test_one_workgroup(H, monkeypatch):
    monkeypatch.setenv("A2AV_MAX_GRID", "1")
    g = torch.Generator().manual_seed(H)
    hs, gs, ds = (_rows(g, 1, 520, H, torch.bfloat16) for _ in range(3))
    check_grad(hs, torch.ones(H, dtype=torch.bfloat16), gs, ds)
