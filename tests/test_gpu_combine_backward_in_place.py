"""The combine's gradient written over the rows it reads (d_back at back,
d_recv at recv): the same bits as in buffers of their own."""
import zlib

import pytest
import torch

from embeddings_a2av_virtual_amd import _binding as B
from test_gpu_combine_backward import Trip

pytestmark = pytest.mark.gpu


def _same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


@pytest.mark.parametrize("case", [(2, 33, 3, 1000), (1, 5, 8, 7168), (1, 17, 5, 129), (3, 9, 2, 20000)], ids=str)
def test_over_the_returned_buffer(case):
    W, T, k, H = case
    g = torch.Generator().manual_seed(zlib.crc32(repr(case).encode()))
    back = [torch.randn(T * k, H, generator=g).to(torch.bfloat16).cuda() for _ in range(W)]
    d_out = [torch.randn(T, H, generator=g).to(torch.bfloat16).cuda() for _ in range(W)]
    perm = [torch.randperm(T * k, generator=g).cuda() for _ in range(W)]
    w = [torch.randn(T, k, generator=g).cuda() for _ in range(W)]
    apart, st = [torch.empty_like(x) for x in back], torch.zeros(1, dtype=torch.int32, device="cuda")
    dw, dw2 = ([torch.empty_like(x) for x in w] for _ in range(2))
    ws = torch.empty(B.moe_combine_backward_workspace_bytes(W, T, k), dtype=torch.uint8, device="cuda")
    B.moe_combine_backward(W, T, k, H, back, perm, w, d_out, apart, dw, ws, st)
    B.moe_combine_backward(W, T, k, H, back, perm, w, d_out, back, dw2, ws, st)
    assert int(st.item()) == 0 and _same(apart, back) and _same(dw, dw2)


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("case", [(2, 33, 3, 8, 24), (4, 20, 8, 32, 7168), (3, 40, 2, 6, 1001)], ids=str)
def test_over_the_owners_rows(case, layout):
    W, T, k, E, H = case
    t = Trip(*case, layout, seed=sum(case))
    assert t.run() == 0
    apart, dw = [x.clone() for x in t.dv], [x.clone() for x in t.dw]
    t.dv = t.rv
    assert t.run() == 0
    assert _same([x[:c] for x, c in zip(apart, t.cap)], [x[:c] for x, c in zip(t.rv, t.cap)]) and _same(dw, t.dw)
    for x, rows, c in zip(t.rv, t.rows, t.cap):  # rows past the total stay
        assert _same([x[c:].cpu()], [rows[c:]])
