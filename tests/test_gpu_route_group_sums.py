"""Groups of moe_route whose two best keys cancel: biases of both signs far
larger than the scores, so that a group's sum is small beside what it adds up
and fp32 loses more of it than its own size says. The ids are those of the sums
in double."""
import math
import zlib

import pytest
import torch

import layer_ref as R
from test_gpu_route import TYPES, check_route

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [1.0, 10.0, 100.0, 1000.0, 1e6])
@pytest.mark.parametrize("E,groups,topk_groups", [(16, 4, 2), (60, 4, 1), (256, 8, 4), (512, 16, 5)], ids=str)
def test_groups_of_cancelling_keys(E, groups, topk_groups, size, sigmoid):
    """One expert of a group has a bias of +size, one of -size, the others less:
    the group's sum is that of two scores, which differ between the groups by
    about what one rounding of a key loses."""
    g = torch.Generator().manual_seed(zlib.crc32(repr((E, groups, size, sigmoid)).encode()))
    T, per = 64, E // groups
    bias = torch.full((groups, per), -4.0 * size)
    bias[:, 0], bias[:, per - 1] = size, -size
    z = 0.5 + size * 2.0 ** -22 * torch.randn(T, E, generator=g) * (1 if sigmoid else E)
    check_route([z], sigmoid, bias.reshape(-1), groups, topk_groups, 2, min(4, per), True, 1.0)
    # every magnitude in one row: groups whose sums are far apart beside some that are not
    bias = bias * torch.logspace(-3, 0, groups).reshape(-1, 1)
    check_route([z], sigmoid, bias.reshape(-1), groups, topk_groups, 2, min(4, per), False, 1.0)


@pytest.mark.parametrize("kind", list(TYPES))
def test_sums_that_fp32_orders_the_other_way(kind):
    """Double: 1.18349914 and 1.18349596; in fp32 1.1834946 and 1.1835022."""
    z = torch.tensor([[0.578125, 0.171875, -0.140625, 0.9375]]).to(TYPES[kind])
    bias = torch.tensor([100.0, -100.0, 100.0, -100.0])
    ids, _ = check_route([z], True, bias, 2, 1, 2, 1, True, 1.0)
    assert ids[0].tolist() == [[0]]


@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
def test_infinite_and_overflowing_sums(sigmoid):
    """Sums that fp32 cannot hold and double can, and infinities of both signs."""
    g = torch.Generator().manual_seed(3)
    T, E, groups = 24, 32, 8
    z = torch.randn(T, E, generator=g)
    top = float(torch.finfo(torch.float32).max)
    edits = [
        {0: top, 1: top, 4: top, 5: top * 0.5, 8: top, 9: top},                       # sums past fp32's range
        {e: -top for e in range(0, 20)},                                              # and below it
        {0: top, 1: -top, 4: top, 5: -top, 12: math.inf, 16: -math.inf},
        {0: math.inf, 1: -math.inf, 2: -math.inf, 3: -math.inf, 4: math.inf, 8: math.inf},
        {e: -math.inf for e in range(0, 28)},
    ]
    for edit in edits:
        bias = 0.1 * torch.randn(E, generator=g)
        for e, v in edit.items():
            bias[e] = v
        for topk_groups in (1, 3, 6):
            check_route([z], sigmoid, bias, groups, topk_groups, 2, 3, True, 1.0)


def test_definition_of_the_planted_row():
    """The reference's own sums of the row above."""
    z = torch.tensor([[0.578125, 0.171875, -0.140625, 0.9375]], dtype=torch.float64)
    s = R.scores(z[0], True) + torch.tensor([100.0, -100.0, 100.0, -100.0], dtype=torch.float64)
    assert float(s[0] + s[1]) > float(s[2] + s[3]) > 1.18
