"""The gradient of the norm where d_out is infinite or NaN in a row's last elements,
which lanes behind the row read again: infinities and NaN are those of the formula
in 64 bits, whatever the width."""
import math

import pytest
import torch

import mx_ref as M
from test_gpu_norm import EPS, TYPES, grad

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("H", [8, 40, 512, 520, 1003, 1024, 2056, 5003, 7168, 9000, 16384, 16392])
@pytest.mark.parametrize("last", [math.inf, -math.inf, math.nan])
def test_last_elements(kind, H, last):
    g = torch.Generator().manual_seed(H)
    t = TYPES[kind]
    h, d = (torch.randn(3, H, generator=g).to(t) for _ in range(2))
    weight = (1 + 0.2 * torch.randn(H, generator=g)).to(t)
    h[h == 0] = 1
    d[1, H - 1] = last
    got, got_w = grad([h], weight, [d], None)
    want, want_w = M.norm_grad(h, weight, EPS, d, None)
    for a, b in ((got[0].double(), want), (got_w.double(), want_w)):
        assert torch.equal(torch.isnan(a), torch.isnan(b))
        assert torch.equal(torch.where(torch.isinf(a), a, 0), torch.where(torch.isinf(b), b, 0))
