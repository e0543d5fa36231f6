"""The 64-bit definitions the layer's GPU tests compare with: their gradients
against finite differences of their forward formulas (no GPU)."""
import pytest
import torch

import layer_ref as R


def _differences(f, x, d, eps=1e-6):
    """d . df/dx by central differences."""
    g = torch.zeros_like(x)
    flat, out = x.reshape(-1), g.reshape(-1)
    for i in range(flat.numel()):
        keep = flat[i].item()
        flat[i] = keep + eps
        hi = (f(x) * d).sum()
        flat[i] = keep - eps
        lo = (f(x) * d).sum()
        flat[i] = keep
        out[i] = (hi - lo) / (2 * eps)
    return g


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_is_the_difference_quotient(sigmoid, renorm):
    torch.manual_seed(3)
    T, E, k = 5, 9, 3
    z = torch.randn(T, E, dtype=torch.float64)
    ids, w = R.route(z, sigmoid, None, 1, 1, 1, k, renorm, 1.5)
    assert torch.allclose(w, R.route_weights(z, ids, sigmoid, renorm, 1.5), rtol=1e-12, atol=0)
    d = torch.randn(T, k, dtype=torch.float64)
    want = _differences(lambda x: R.route_weights(x, ids, sigmoid, renorm, 1.5), z, d)
    got = R.route_grad(z, ids, d, sigmoid, renorm, 1.5)
    # central differences of eps = 1e-6: truncation about 1e-12, rounding about 1e-16 / 1e-6
    assert (got - want).abs().max() < 1e-8


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu", "swiglu"])
def test_activation_gradient_is_the_difference_quotient(act):
    torch.manual_seed(4)
    h = torch.randn(6, 8, dtype=torch.float64)
    d = torch.randn(6, 4 if act == "swiglu" else 8, dtype=torch.float64)
    want = _differences(lambda x: R.activate(act, x), h, d)
    assert (R.activate_grad(act, h, d) - want).abs().max() < 1e-8


def test_route_rules():
    """Ties, masks and groups by hand."""
    z = torch.tensor([[1.0, 3.0, 3.0, 2.0, 0.0, 3.0]], dtype=torch.float64)
    assert R.route(z, False, None, 1, 1, 1, 4, True, 1.0)[0].tolist() == [[1, 2, 5, 3]]
    # three groups of two by their best: {1, 3}, {3, 2}, {0, 3} tie; two kept: the first two
    assert R.route(z, False, None, 3, 2, 1, 3, True, 1.0)[0].tolist() == [[1, 2, 3]]
    # by the sum of their two best the last group's 0 loses to 1 and 2
    bias = torch.tensor([0.0, 0.0, 0.0, 0.0, 0.0, 0.1])
    assert R.route(z, True, bias, 3, 1, 2, 1, False, 1.0)[0].tolist() == [[2]]
    z = torch.full((1, 4), -R.INF, dtype=torch.float64)
    ids, w = R.route(z, False, None, 2, 1, 2, 2, True, 1.0)
    assert ids.tolist() == [[0, 1]] and w.tolist() == [[0.0, 0.0]]
