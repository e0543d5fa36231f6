"""The norm of rows and weights of every magnitude of their type: rows whose elements
times the weight lie outside fp32's range while y does not, and weights of very
different magnitudes side by side."""
import pytest
import torch

import mx_ref as M
from test_gpu_norm import check, norm

pytestmark = pytest.mark.gpu


def _scaled(g, n, H, e, t):
    return (torch.randn(n, H, generator=g).double() * torch.pow(torch.tensor(2.0, dtype=torch.float64), e)).to(t)


@pytest.mark.parametrize("H", [64, 1003, 2056, 9000, 16392])
@pytest.mark.parametrize("rows,weights", [(0, 110), (10, 122), (20, 100), (30, 90), (38, 86), (100, 20), (60, 66),
                                          (120, -120), (-100, -20), (-30, -90), (-20, -105), (-28, 118), (0, -120),
                                          (-120, 100), (-125, -5), (15, 17), (-17, -15)])
def test_bf16(H, rows, weights):
    g = torch.Generator().manual_seed(H + rows)
    t = torch.bfloat16
    x, w = _scaled(g, 3, H, rows, t), _scaled(g, 1, H, weights, t)[0]
    check([x], None, w, M.FP8, eps=0.0)
    check([x], None, w, M.FP4, eps=0.0, want_out=False)


@pytest.mark.parametrize("H", [64, 1003, 16392])
@pytest.mark.parametrize("rows,weights", [(-20, -20), (-20, 14), (12, -20), (12, 2), (-6, 14)])
def test_fp16(H, rows, weights):
    g = torch.Generator().manual_seed(H + rows)
    t = torch.float16
    x, w = _scaled(g, 3, H, rows, t), _scaled(g, 1, H, weights, t)[0]
    check([x], None, w, M.FP8, eps=0.0, want_out=False)
    # y from 65520 is infinite in fp16; it is off by fp32's two roundings before that
    y, out = M.norm(x, w, 0.0), norm([x], None, w, eps=0.0)["out"][0].double()
    near = (y.abs() - 65520).abs() <= 65520 * 2.0 ** -23
    err = y.abs() * (2.0 ** -11 + 2.0 ** -23) + 2.0 ** -25
    ok = torch.where(y.abs() > 65520, out == torch.sign(y) * torch.inf, (out - y).abs() <= err)
    assert (ok | near).all(), (~ok).nonzero()[:4].tolist()


@pytest.mark.parametrize("H", [64, 1003, 2056, 9000, 16392])
def test_weights_of_all_magnitudes(H):
    g = torch.Generator().manual_seed(H)
    t = torch.bfloat16
    x = _scaled(g, 4, H, torch.tensor([[0], [40], [-40], [14]]), t)
    near = torch.randint(-100, 112, ((H + 31) // 32,), generator=g).repeat_interleave(32)[:H]
    check([x], None, _scaled(g, 1, H, near, t)[0], M.FP8, eps=0.0)
    check([x], None, _scaled(g, 1, H, torch.randint(-80, 112, (H,), generator=g), t)[0], M.FP4, eps=0.0, want_out=False)


@pytest.mark.parametrize("H", [64, 1003, 9000, 16392])
def test_next_to_the_end(H):
    """|h|, weights and y of 2^127: half of bf16's largest, a fourth of what overflows."""
    g = torch.Generator().manual_seed(H)
    sign = lambda n: 1 - 2 * torch.randint(0, 2, (n, H), generator=g)  # noqa: E731
    x, w = (sign(3) * 2.0 ** 127).bfloat16(), (sign(1)[0] * 2.0 ** 127).bfloat16()
    check([x], None, w, M.FP8, eps=0.0)
    check([(x.double() / 2.0 ** 254).bfloat16()], None, w, M.FP4, eps=0.0)
