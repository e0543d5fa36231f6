"""Sums of the microscaled products past fp32's range, in few rows and in tiles of
them alike: an infinite sum is infinite, and with ReLU a negative one gives 0."""
import pytest
import torch

import mx_ref as M
from embeddings_a2av_virtual_amd import _binding as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out_type", [torch.uint8, torch.bfloat16])
@pytest.mark.parametrize("form", [M.FP8, M.FP4])
@pytest.mark.parametrize("rows", [1, 40])
def test_infinite_sums(rows, form, out_type):
    K, N = 64, 96
    x = torch.zeros(rows, M.row_bytes(form, K), dtype=torch.uint8, device="cuda")
    at = M.padded(K) // (1 if form == M.FP8 else 2)
    x[:, :K if form == M.FP8 else K // 2] = 0x7E if form == M.FP8 else 0x77  # 448, or 6 and 6
    x[:, at:at + 2] = 254
    w = torch.zeros(N, M.row_bytes(M.FP4, K), dtype=torch.uint8, device="cuda")
    w[5, :K // 2], w[40, :K // 2], w[70, :K // 2] = 0xFF, 0x77, 0x22  # -6, 6, 1
    w[:, 128:130] = 250
    w[70, 128:130] = 0  # 2^-127 each
    off = torch.tensor([[0, rows]], dtype=torch.int64, device="cuda")
    wide = M.row_bytes(M.FP8, N) if out_type == torch.uint8 else N
    for act in (B.ACT_RELU, B.ACT_NONE):
        out = torch.zeros(rows, wide, dtype=out_type, device="cuda")
        ws = torch.empty(B.moe_expert_linear_mx_workspace_bytes(1, 1, K, N, act, [rows]), dtype=torch.uint8, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        B.moe_expert_linear_mx(1, 1, K, N, form, act, [x], [rows], off, [w], None, [out], ws, st)
        assert int(st.item()) == 0
        y = torch.zeros(rows, N, dtype=torch.float64)
        y[:, 5], y[:, 40], y[:, 70] = 0 if act == B.ACT_RELU else -torch.inf, torch.inf, K * (448 if form == M.FP8 else 6)
        if out_type == torch.uint8:
            assert torch.equal(out.cpu()[:, :M.used_bytes(M.FP8, N)], M.quantize(y, M.FP8)), act
        else:
            assert torch.equal(out.cpu(), y.to(out_type)), act
