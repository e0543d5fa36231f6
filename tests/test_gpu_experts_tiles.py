"""The experts' products on every tile shape that the library chooses by size,
with contractions of one step to many: the largest tiles of each product (256 x
256) beside the middle and the small ones. Which shape a call takes is computed
here by the library's rule, so that a changed rule cannot leave one untested."""
import zlib

import pytest
import torch

from test_gpu_experts import Experts

pytestmark = pytest.mark.gpu

TILE = (256, 128, 64)


def shape_of(R, n, M, C):
    """Edge of the largest tile of which a product of n experts with R rows has
    at least 200 (M: the rows of each product, or 0 for the experts' own)."""
    for t in TILE[:2]:
        if M:
            tiles = n * -(-M // t)
        else:
            tiles = R if R <= n else R // t + (n // 2 if R % (n * t) else 0)
        if tiles * -(-C // t) >= 200:
            return t
    return 64


def d_weight_shape(R, n, M, C):
    t = shape_of(R, n, M, C)
    return 128 if t == 256 and R < 384 * n else t


def _seed(*what):
    return zlib.crc32(repr(what).encode())


def _sizes(e):
    return sum(e.tot) + e.spare * e.W, e.W * e.P


# tiles with all rows, with a quarter, half and one of them, experts without any
ROWS = [[256, 1, 300, 0, 512, 130, 383, 64, 600, 65]]


@pytest.mark.parametrize("steps", [1, 2, 5, 6, 7, 13])
@pytest.mark.parametrize("kind,act", [("bf16", "none"), ("fp16", "gelu"), ("bf16", "swiglu"), ("fp16", "swiglu")])
def test_forward_on_the_largest_tiles(steps, kind, act):
    """Contractions of 64 * steps and, from two steps on, of 56 less."""
    K = 64 * steps - (56 if steps > 1 else 0)
    N = 1800 if act == "swiglu" else 3592
    e = Experts(ROWS, K, N, kind, act, _seed("fwd", steps, kind, act))
    R, n = _sizes(e)
    assert shape_of(R, n, 0, e.NW) == 256
    e.check_forward()


@pytest.mark.parametrize("steps", [1, 2, 5, 6, 7, 13])
@pytest.mark.parametrize("kind,act", [("bf16", "none"), ("fp16", "gelu"), ("bf16", "swiglu"), ("fp16", "swiglu")])
def test_row_gradients_on_the_largest_tiles(steps, kind, act):
    NW = 64 * steps - (48 if steps > 1 else 0)
    N = NW // 2 if act == "swiglu" else NW
    e = Experts(ROWS, 3592, N, kind, act, _seed("dx", steps, kind, act))
    R, n = _sizes(e)
    assert shape_of(R, n, 0, e.K) == 256
    e.check_backward(("d_x", "d_bias"))


# 1 to 17 steps of 64 rows, with and without a ragged last one, and an expert without rows
LONG = [[1000, 0, 63, 385, 700], [129, 1, 1088, 768, 512]]


@pytest.mark.parametrize("kind,act", [("bf16", "none"), ("fp16", "none"), ("bf16", "swiglu"), ("fp16", "swiglu"),
                                      ("bf16", "silu"), ("fp16", "gelu")])
@pytest.mark.parametrize("K,N", [(1224, 648), (1536, 512)], ids=str)
def test_weight_gradients_on_the_largest_tiles(K, N, kind, act):
    N = N if act == "swiglu" else 2 * N
    e = Experts(LONG, K, N, kind, act, _seed("dw", K, N, kind, act))
    R, n = _sizes(e)
    assert R >= 384 * n and d_weight_shape(R, n, e.NW, K) == 256
    e.check_backward()


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_weight_gradients_of_few_rows_take_the_middle_tiles(kind):
    e = Experts([[200, 0, 321, 64, 97, 300, 31, 33, 512, 1]], 1224, 1296, kind, "silu", _seed("dw mid", kind))
    R, n = _sizes(e)
    assert shape_of(R, n, e.NW, e.K) == 256 and d_weight_shape(R, n, e.NW, e.K) == 128
    e.check_backward()


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_largest_tiles_give_the_same_bits_every_time(kind):
    e = Experts(LONG, 1224, 648, kind, "swiglu", _seed("again", kind))
    f, b = e.forward(), e.backward()
    for _ in range(3):
        f2, b2 = e.forward(), e.backward()
        assert all(torch.equal(x.view(torch.int16), y.view(torch.int16)) for x, y in zip(f[1] + f[2], f2[1] + f2[2]))
        for k in b[1]:
            assert all(torch.equal(x.view(torch.int16), y.view(torch.int16)) for x, y in zip(b[1][k], b2[1][k])), k
