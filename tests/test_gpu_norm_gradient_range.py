"""The gradient of the norm at the ends of what it is defined for, in the kernels of rows
in registers and of wider ones: rows of magnitude 2^-120 to 2^120 and d_out * weight
from 2^-110 to next to 2^128."""
import pytest
import torch

from test_gpu_norm import TYPES, check_grad

pytestmark = pytest.mark.gpu


def _scaled(g, n, H, e, t):
    return (torch.randn(n, H, generator=g).double() * 2.0 ** e).to(t)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("H", [64, 264, 1003, 2056, 9000, 16392])
@pytest.mark.parametrize("rows,weights,d_out", [(120, 20, 0), (120, 60, 60), (-120, -110, 0), (-100, 0, 5), (0, 115, -115),
                                                (0, -115, 110), (0, -50, -50), (20, 60, 60), (60, -40, 110),
                                                (-60, 30, -110), (115, 0, 0)])
def test_magnitudes(H, kind, rows, weights, d_out):
    g = torch.Generator().manual_seed(H + rows + weights)
    t = TYPES[kind]
    h, d, w = (_scaled(g, n, H, e, t) for n, e in ((3, rows), (3, d_out), (1, weights)))
    check_grad([h], w[0], [d], None, eps=0.0)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("H", [64, 1003, 9000, 16392])
def test_one_large_product(H, kind):
    """A single column whose product is 2^127, over rows of large elements."""
    g = torch.Generator().manual_seed(H)
    h, d, w = (_scaled(g, n, H, e, TYPES[kind]) for n, e in ((3, 40), (3, 0), (1, 0)))
    d[1, 3], w[0, 3] = 2.0 ** 63, 2.0 ** 64
    check_grad([h], w[0], [d], None, eps=0.0)
