"""Expert products of more tiles than one launch of the tile kernels can have:
4096 experts, nearly all without rows, and products of 262152 columns. The
ranks share one weight, which is only read."""
import pytest
import torch

from embeddings_a2av_virtual_amd import _binding as B

pytestmark = pytest.mark.gpu

W, P, WIDE = 64, 64, 262152
BF = torch.bfloat16


def _rows(n):
    """One row of rank 0's expert 3, n - 1 of its last."""
    off = torch.zeros((W, P + 1), dtype=torch.int64)
    if n:
        off[0, 4:] = 1
        off[0, P] = n
    return off.cuda(), [n] + [0] * (W - 1)


@pytest.mark.parametrize("n", [0, 2])
def test_wide_products(n):
    g = torch.Generator(device="cuda").manual_seed(n)
    K = 8
    w = torch.randn((P, WIDE, K), generator=g, device="cuda").to(BF)
    x = torch.randn((max(n, 1), K), generator=g, device="cuda").to(BF)
    off, rows = _rows(n)
    out, st = torch.full((max(n, 1), WIDE), 7.0, dtype=BF, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(B.moe_expert_linear_workspace_bytes(W, P, K, WIDE, B.ACT_NONE, rows), dtype=torch.uint8, device="cuda")
    none = [None] * (W - 1)
    B.moe_expert_linear(W, P, K, WIDE, B.ACT_NONE, [x] + none, rows, off, [w] * W, None, None, [out] + none, None, ws, st)
    assert int(st.item()) == 0
    for i, e in enumerate((3, P - 1)[:n]):
        y = w[e].double() @ x[i].double()
        # 8 products in fp32, then half a step of bf16
        tol = y.abs() * 2.0 ** -8 + (w[e].double().abs() @ x[i].double().abs()) * 24 * 2.0 ** -24
        assert ((out[i].double() - y).abs() <= tol).all()
    assert n or (out == 7.0).all()


@pytest.mark.parametrize("n", [0, 2])
def test_wide_gradients(n):
    g = torch.Generator(device="cuda").manual_seed(n)
    N = 8
    w = torch.randn((P, N, WIDE), generator=g, device="cuda").to(BF)
    x = torch.randn((max(n, 1), WIDE), generator=g, device="cuda").to(BF)
    d_out = torch.randn((max(n, 1), N), generator=g, device="cuda").to(BF)
    off, rows = _rows(n)
    d_x, st = torch.full((max(n, 1), WIDE), 7.0, dtype=BF, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    d_bias = [torch.full((P, N), 7.0, dtype=BF, device="cuda") for _ in range(W)]
    ws = torch.empty(B.moe_expert_linear_backward_workspace_bytes(W, P, WIDE, N, B.ACT_NONE, rows), dtype=torch.uint8,
                     device="cuda")
    none = [None] * (W - 1)
    B.moe_expert_linear_backward(W, P, WIDE, N, B.ACT_NONE, [x] + none, rows, off, [w] * W, None, [d_out] + none, None,
                                 [d_x] + none, None, d_bias, ws, st)
    assert int(st.item()) == 0
    for i, e in enumerate((3, P - 1)[:n]):
        y = d_out[i].double() @ w[e].double()
        tol = y.abs() * 2.0 ** -8 + (d_out[i].double().abs() @ w[e].double().abs()) * 24 * 2.0 ** -24
        assert ((d_x[i].double() - y).abs() <= tol).all()
        assert torch.equal(d_bias[0][e], d_out[i])
    assert n or (d_x == 7.0).all()
    assert all((b == 0).all() for b in d_bias[1:])


def test_few_rows_of_many_experts_and_long_weights():
    """Two rows and weights long enough for the few-rows kernel, whose tiles of
    16 columns would be too many for 4096 experts."""
    g = torch.Generator(device="cuda").manual_seed(5)
    K, N, n = 4096, 16424, 2
    w = torch.empty((P, N, K), dtype=BF, device="cuda").normal_(std=K ** -0.5, generator=g)
    x = torch.randn((n, K), generator=g, device="cuda").to(BF)
    off, rows = _rows(n)
    out, st = torch.full((n, N), 7.0, dtype=BF, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(B.moe_expert_linear_workspace_bytes(W, P, K, N, B.ACT_NONE, rows), dtype=torch.uint8, device="cuda")
    none = [None] * (W - 1)
    B.moe_expert_linear(W, P, K, N, B.ACT_NONE, [x] + none, rows, off, [w] * W, None, None, [out] + none, None, ws, st)
    assert int(st.item()) == 0
    for i, e in enumerate((3, P - 1)):
        y = w[e].double() @ x[i].double()
        # the fp32 sum of K products in any order, then half a step of bf16
        tol = y.abs() * 2.0 ** -8 * 1.01 + (w[e].double().abs() @ x[i].double().abs()) * (2 * K + 8) * 2.0 ** -24
        assert ((out[i].double() - y).abs() <= tol).all()
