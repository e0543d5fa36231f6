"""The norm of rows and weights that are not finite: where y is NaN its block of a
microscaled row is, infinities under weights of zero and infinite weights over
zeros among them, for every way that a row is spread over threads."""
import math

import pytest
import torch

import mx_ref as M
from test_gpu_norm import EPS, TYPES, check, norm

pytestmark = pytest.mark.gpu

# a wave a row, whole and odd, workgroups of two sizes, rows that are read twice
WIDTHS = [64, 1003, 2056, 5003, 9000, 16392]


def exactly(x, weight, form, r=None):
    """Where y is NaN, out is and every block that holds one; the rest within the norm's own tolerance."""
    check([x], None if r is None else [r], weight, form)
    got = norm([x], None if r is None else [r], weight, form)
    y = M.norm(M.add(x, r), weight, EPS)
    assert torch.equal(torch.isnan(got["out"][0]), torch.isnan(y))
    H = x.shape[1]
    bad = torch.nn.functional.pad(~torch.isfinite(y), (0, M.padded(H) - H)).reshape(len(x), -1, 32).any(-1)
    n = M.padded(H) // (1 if form == M.FP8 else 2)
    assert torch.equal(got["rows"][0][:, n:M.used_bytes(form, H)] == 255, bad)
    return bad


@pytest.mark.parametrize("form", [M.FP8, M.FP4])
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("H", WIDTHS)
def test_infinities_under_weights_of_zero(kind, H, form):
    g = torch.Generator().manual_seed(H)
    at = [5, H // 2, H - 1]
    x, weight = torch.randn(5, H, generator=g), 1 + 0.2 * torch.randn(H, generator=g)
    weight[at] = 0
    x[1, 5], x[2, H // 2], x[3, at], x[4, 7] = math.inf, -math.inf, math.inf, -math.inf
    bad = exactly(x.to(TYPES[kind]), weight.to(TYPES[kind]), form)
    assert bad.sum(-1).tolist()[:2] == [0, 1] and bad[4].sum() == 1


@pytest.mark.parametrize("form", [M.FP8, M.FP4])
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("H", WIDTHS)
def test_infinite_weights_over_zeros(kind, H, form):
    g = torch.Generator().manual_seed(H + 1)
    x, weight = torch.randn(4, H, generator=g), 1 + 0.2 * torch.randn(H, generator=g)
    weight[3], weight[H // 2], weight[H - 1] = math.inf, -math.inf, math.inf
    x[0, 3] = x[1, H // 2] = x[2, H - 1] = 0
    x[3] = 0
    exactly(x.to(TYPES[kind]), weight.to(TYPES[kind]), form)


@pytest.mark.parametrize("H", WIDTHS)
def test_a_sum_that_overflows_under_a_weight_of_zero(H):
    g = torch.Generator().manual_seed(H + 2)
    x, r = (torch.randn(3, H, generator=g).half() for _ in range(2))
    weight = torch.ones(H).half()
    x[1, H - 2], r[1, H - 2], weight[H - 2] = 60000, 40000, 0
    assert exactly(x, weight, M.FP8, r).sum().item() == 1
