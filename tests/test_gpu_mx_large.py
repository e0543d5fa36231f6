"""The microscaled layer's calls where byte offsets pass 32 bits: values, rows
and weights over 4 GiB, zero but for the last rows, whose results are those of
a call on these rows alone."""
import pytest
import torch

import mx_ref as M
from embeddings_a2av_virtual_amd import _binding as B
from test_gpu_mx_tiles import whole

pytestmark = pytest.mark.gpu

H, LAST = 4096, 2500
T = (1 << 32) // H + 60_000  # rows of a byte an element pass 4 GiB too


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _last(seed, dtype=torch.bfloat16):
    """T rows, and the last of them on their own."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    own = torch.randn(LAST, H, generator=g, device="cuda").to(dtype)
    x = torch.zeros(T, H, dtype=dtype, device="cuda")
    x[-LAST:] = own
    return x, own


@pytest.mark.parametrize("form", [M.FP8, M.FP4])
def test_blocks_past_4_gib(form):
    x, own = _last(1)
    st, used = _status(), M.used_bytes(form, H)
    rows = torch.zeros(T, M.row_bytes(form, H), dtype=torch.uint8, device="cuda")
    B.moe_mx_quantize(1, H, form, [x], [T], [rows], st)
    assert torch.equal(rows[-60:, :used].cpu(), M.quantize(own[-60:].double().cpu(), form))
    assert not rows[-LAST - 1].any()
    x.fill_(7)
    B.moe_mx_dequantize(1, H, form, [rows], [T], [x], st)
    assert int(st.item()) == 0 and not x[-LAST - 1].any()
    assert torch.equal(x[-60:].cpu(), M.values(rows[-60:].cpu(), form, H).to(torch.bfloat16))


def test_norm_past_4_gib():
    x, own = _last(2)
    r, own_r = _last(3)
    st, w = _status(), torch.randn(H, device="cuda").to(torch.bfloat16)
    stride = M.row_bytes(M.FP8, H)
    got = []
    for n, a, b in ((T, x, r), (LAST, own, own_r)):
        s, o = torch.empty_like(a), torch.empty_like(a)
        rows = torch.zeros(n, stride, dtype=torch.uint8, device="cuda")
        B.moe_rms_norm(1, n, H, 1e-6, [a], [b], w, [s], [o], [rows], M.FP8, st)
        got.append((s, o, rows))
    assert int(st.item()) == 0
    for a, b in zip(*got):
        assert torch.equal(a[-LAST:], b)
    del got, r
    d, own_d = _last(4)
    dw, own_dw = torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
    for n, a, b, out in ((T, x, d, dw), (LAST, own, own_d, own_dw)):
        ws = torch.empty(B.moe_rms_norm_backward_workspace_bytes(1, n, H), dtype=torch.uint8, device="cuda")
        B.moe_rms_norm_backward(1, n, H, 1e-6, [a], w, [b], [b], [b], out, ws, st)
    assert int(st.item()) == 0 and torch.equal(d[-LAST:], own_d)
    # the other rows add nothing; the sums of 2500 terms of order 1 in other orders
    assert (dw - own_dw).abs().max() < 2500 * 16 * 2.0 ** -23


def _product(K, N, x, w, per, out_rows):
    st = _status()
    off = torch.tensor([[0] + torch.tensor(per).cumsum(0).tolist()], dtype=torch.int64, device="cuda")
    ws = torch.empty(B.moe_expert_linear_mx_workspace_bytes(1, len(per), K, N, B.ACT_NONE, [len(x)]), dtype=torch.uint8,
                     device="cuda")
    out = torch.full((out_rows, N), 7.0, dtype=torch.bfloat16, device="cuda")
    B.moe_expert_linear_mx(1, len(per), K, N, M.FP4, B.ACT_NONE, [x], [len(x)], off, [w], None, [out], ws, st)
    assert int(st.item()) == 0
    return out


def test_rows_past_4_gib():
    """Two experts, the second one's rows behind 4 GiB; then its outputs too."""
    g = torch.Generator(device="cuda").manual_seed(5)
    K, n, last = 4096, 2_100_000, 700
    own, xv = whole(last, K, M.FP4, g)
    x = torch.zeros(n, own.shape[1], dtype=torch.uint8, device="cuda")
    assert (n - last) * x.shape[1] > 1 << 32
    x[-last:] = own
    for N in (40, 1100):
        w, wv = whole(2 * N, K, M.FP4, g)
        out = _product(K, N, x, w, [n - last, last], n)
        assert torch.equal(out[-last:], (xv @ wv[N:].t()).float().to(torch.bfloat16))
        assert not out[-last - 1].any()


@pytest.mark.parametrize("rows", [3, 40, 500])
def test_weights_past_4_gib(rows):
    g = torch.Generator(device="cuda").manual_seed(rows)
    K, N, last = 8192, 1 << 20, 600
    x, xv = whole(rows, K, M.FP4, g)
    own, wv = whole(last, K, M.FP4, g)
    w = torch.zeros(N, own.shape[1], dtype=torch.uint8, device="cuda")
    assert (N - last) * w.shape[1] > 1 << 32
    w[-last:] = own
    out = _product(K, N, x, w, [rows], rows)
    assert torch.equal(out[:, -last:], (xv @ wv.t()).float().to(torch.bfloat16))
    assert not out[:, :-last].any()
