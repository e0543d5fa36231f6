"""The microscaled layer's calls with as many ranks as there may be, each with rows
of its own (some without any), on a stream given as an argument."""
import pytest
import torch

import mx_ref as M
from embeddings_a2av_virtual_amd import _binding as B
from test_gpu_mx_tiles import whole

pytestmark = pytest.mark.gpu

W = B.MAX_W


def test_norm_and_its_gradient():
    T, H = 3, 520
    g = torch.Generator().manual_seed(1)
    x, d = ([torch.randn(T, H, generator=g).to(torch.bfloat16) for _ in range(W)] for _ in range(2))
    w = (1 + 0.2 * torch.randn(H, generator=g)).to(torch.bfloat16)
    cu = lambda ts: [t.cuda() for t in ts]  # noqa: E731
    rows = [torch.zeros(T, M.row_bytes(M.FP4, H), dtype=torch.uint8, device="cuda") for _ in range(W)]
    d_x, d_w = cu(d), torch.empty(H, device="cuda")
    xs, ds, wc = cu(x), cu(d), w.cuda()
    ws = torch.empty(B.moe_rms_norm_backward_workspace_bytes(W, T, H), dtype=torch.uint8, device="cuda")
    st, side = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.cuda.Stream()
    torch.cuda.synchronize()
    B.moe_rms_norm(W, T, H, 1e-6, xs, None, wc, None, None, rows, M.FP4, st, stream=side)
    B.moe_rms_norm_backward(W, T, H, 1e-6, xs, wc, ds, None, d_x, d_w, ws, st, stream=side)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    sums = torch.zeros(H, dtype=torch.float64)
    for r in range(W):
        want = M.quantize(M.norm(x[r], w, 1e-6), M.FP4)
        assert torch.equal(rows[r].cpu()[:, :want.shape[1]], want), r
        dx, dw = M.norm_grad(x[r], w, 1e-6, d[r], None)
        # half a step of bf16, and fp32 steps of terms that cancel
        assert ((d_x[r].cpu().double() - dx).abs() <= dx.abs() * 2.0 ** -8 + 2.0 ** -18).all(), r
        sums += dw
    # 192 terms of at most about 16, an fp32 step of the running sum for each
    assert ((d_w.cpu().double() - sums).abs() < 192 * 64 * 2.0 ** -23).all()


def test_rows():
    H, n = 300, [r % 5 for r in range(W)]
    g = torch.Generator().manual_seed(2)
    x = [torch.randn(k, H, generator=g) for k in n]
    xs, used = [t.cuda() for t in x], M.used_bytes(M.FP8, H)
    rows = [torch.zeros(k, M.row_bytes(M.FP8, H), dtype=torch.uint8, device="cuda") for k in n]
    back = [torch.zeros(k, H, device="cuda") for k in n]
    st, side = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.cuda.Stream()
    torch.cuda.synchronize()
    B.moe_mx_quantize(W, H, M.FP8, xs, n, rows, st, stream=side)
    B.moe_mx_dequantize(W, H, M.FP8, rows, n, back, st, stream=side)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for r in range(W):
        want = M.quantize(x[r].double(), M.FP8)
        assert torch.equal(rows[r].cpu()[:, :used], want)
        assert torch.equal(back[r].cpu(), M.values(want, M.FP8, H).float())


@pytest.mark.parametrize("most", [3, 40])
def test_products(most):
    K, N, P = 300, 40, 2
    g = torch.Generator(device="cuda").manual_seed(most)
    per = [[(7 * r + 3 * j) % (most + 1) for j in range(P)] for r in range(W)]
    n = [sum(p) for p in per]
    x, xv = zip(*[whole(k, K, M.FP8, g) for k in n])
    w, wv = zip(*[whole(P * N, K, M.FP4, g) for _ in n])
    off = torch.tensor([[0, p[0], p[0] + p[1]] for p in per], dtype=torch.int64, device="cuda")
    out = [torch.full((k + 1, N), 7.0, dtype=torch.bfloat16, device="cuda") for k in n]
    ws = torch.empty(B.moe_expert_linear_mx_workspace_bytes(W, P, K, N, B.ACT_NONE, n), dtype=torch.uint8, device="cuda")
    st, side = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.cuda.Stream()
    torch.cuda.synchronize()
    B.moe_expert_linear_mx(W, P, K, N, M.FP8, B.ACT_NONE, list(x), n, off, list(w), None, out, ws, st, stream=side)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for r in range(W):
        a = per[r][0]
        want = torch.cat([xv[r][:a] @ wv[r][:N].t(), xv[r][a:] @ wv[r][N:].t()])
        assert torch.equal(out[r][:-1], want.float().to(torch.bfloat16)), r
        assert (out[r][-1] == 7).all()
