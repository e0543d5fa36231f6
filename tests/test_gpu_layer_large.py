"""The layer's calls where byte offsets pass 32 bits (logits, rows and weights
over 4 GiB), on a stream given as an argument, and with grids capped so that
every loop makes later passes."""
import os

import pytest
import torch

import layer_ref as R
from embeddings_a2av_virtual_amd import _binding as B
from test_gpu_combine_backward import Trip, expected, same_bits
from test_gpu_route import check_route, check_route_grad

pytestmark = pytest.mark.gpu


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def test_router_past_4_gib():
    """9 M tokens of 256 bf16 logits: the last rows are 4.6 GB into the array."""
    T, E, k = 9_000_001, 256, 4
    z = torch.empty((T, E), dtype=torch.bfloat16, device="cuda").normal_()
    ids, w = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    st = _status()
    B.moe_route(1, T, k, E, B.SCORE_SOFTMAX, [z], None, 1, 1, 1, True, 1.0, [ids], [w], st)
    d, dz = torch.empty_like(w).normal_(), torch.empty_like(z)
    B.moe_route_backward(1, T, k, E, B.SCORE_SOFTMAX, [z], [ids], [w], True, 1.0, [d], [dz], st)
    assert int(st.item()) == 0
    for at in (slice(0, 20), slice(T - 20, T)):
        x = z[at].cpu().double()
        rid, rw = R.route(x, False, None, 1, 1, 1, k, True, 1.0)
        assert torch.equal(ids[at].cpu(), rid)
        assert ((w[at].cpu().double() - rw).abs() <= rw * 1e-5).all()
        want = R.route_grad(x, rid, d[at].cpu().double(), False, True, 1.0)
        got = dz[at].cpu().double()
        # half a step of bf16, and the fp32 steps of terms that cancel
        assert ((got - want).abs() <= want.abs() * 2.0 ** -8 + 1e-5 * d[at].abs().max().item()).all()


def test_expert_rows_and_weights_past_4_gib():
    """330000 rows of 7168 (4.7 GB) over two experts, then 80 experts' weights
    of 2 x 2048 x 7168 (4.7 GB) for one row each."""
    bf = torch.bfloat16
    K, N = 7168, 64
    per = [40_000, 290_000]
    x = torch.empty((sum(per), K), dtype=bf, device="cuda").normal_()
    w = (torch.randn(2, N, K, device="cuda") / K ** 0.5).to(bf)
    off = torch.tensor([[0, per[0], sum(per)]], device="cuda")
    out, st = torch.empty((sum(per), N), dtype=bf, device="cuda"), _status()
    ws = torch.empty(B.moe_expert_linear_backward_workspace_bytes(1, 2, K, N, B.ACT_NONE, [sum(per)]), dtype=torch.uint8,
                     device="cuda")
    B.moe_expert_linear(1, 2, K, N, B.ACT_NONE, [x], [sum(per)], off, [w], None, None, [out], None, ws, st)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    B.moe_expert_linear_backward(1, 2, K, N, B.ACT_NONE, [x], [sum(per)], off, [w], None, [out], None, [dx], [dw], None,
                                 ws, st)
    assert int(st.item()) == 0
    for at, e in ((slice(0, 40), 0), (slice(sum(per) - 40, sum(per)), 1)):
        xs, ww = x[at].cpu().double(), w[e].cpu().double()
        y = xs @ ww.t()
        assert ((out[at].cpu().double() - y).abs() <= y.abs() * 2.0 ** -8 * 1.01 + xs.abs() @ ww.abs().t() * K * 2.0 ** -22).all()
        g = out[at].cpu().double()
        v = g @ ww
        assert ((dx[at].cpu().double() - v).abs() <= v.abs() * 2.0 ** -8 * 1.01 + g.abs() @ ww.abs() * N * 2.0 ** -22).all()
    # one corner of the second expert's weight gradient, its sums in 64 bits
    rows = slice(per[0], sum(per))
    g, xs = out[rows, :4].double(), x[rows, -4:].double()
    v, mag = g.t() @ xs, g.abs().t() @ xs.abs()
    # the fp32 sum of 290000 terms: the bound of a random walk of half steps, ten times over
    tol = v.abs() * 2.0 ** -8 * 1.01 + 10 * mag * 2.0 ** -24 * per[1] ** 0.5
    assert ((dw[1, :4, -4:].double() - v).abs() <= tol).all()
    del x, dx, out
    P, N = 80, 2048
    w = torch.empty((P, 2 * N, K), dtype=bf, device="cuda").normal_(std=K ** -0.5)
    x = torch.randn(P, K, device="cuda").to(bf)
    off = torch.arange(P + 1, device="cuda").reshape(1, -1)
    out = torch.empty((P, N), dtype=bf, device="cuda")
    ws = torch.empty(B.moe_expert_linear_workspace_bytes(1, P, K, N, B.ACT_SWIGLU, [P]), dtype=torch.uint8, device="cuda")
    B.moe_expert_linear(1, P, K, N, B.ACT_SWIGLU, [x], [P], off, [w], None, None, [out], None, ws, st)
    assert int(st.item()) == 0
    for e in (0, P - 1):
        h = w[e].cpu().double() @ x[e].cpu().double()
        y = R.activate("swiglu", h)
        assert ((out[e].cpu().double() - y).abs() <= y.abs() * 2.0 ** -8 * 1.01 + 0.01 * 2.0 ** -8).all()


def test_on_a_stream_given_as_an_argument():
    """Every call enqueued on a stream of its own, behind work that is still
    running there."""
    t = Trip(2, 60, 2, 8, 512, 1, seed=31)
    s = torch.cuda.Stream()
    w, d_out = [x.cuda() for x in t.w], [x.cuda() for x in t.d_out]
    ws = torch.empty(B.moe_combine_return_backward_workspace_bytes(2, 60, 2, 8), dtype=torch.uint8, device="cuda")
    z = torch.randn(500, 64)
    zc, ids = torch.empty((500, 64), device="cuda"), torch.empty((500, 4), dtype=torch.int32, device="cuda")
    gates, zh = torch.empty((500, 4), device="cuda"), z.pin_memory()
    big = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(10):
            big.add_(1)
        zc.copy_(zh, non_blocking=True)
    B.moe_route(1, 500, 4, 64, B.SCORE_SIGMOID, [zc], None, 1, 1, 1, True, 1.0, [ids], [gates], t.status, s)
    B.moe_combine_return_backward(2, 60, 2, 8, 512, t.counts, t.cids, t.perm, list(t.rv), t.recv_rows, w, d_out,
                                  list(t.dv), t.dw, 1, ws, t.status, s)
    s.synchronize()
    assert int(t.status.item()) == 0
    assert torch.equal(ids.cpu(), R.route(z.double(), True, None, 1, 1, 1, 4, True, 1.0)[0])
    place = t.place()
    rows = torch.stack([t.rows[d][i] for d, i in place[0]])
    got = torch.stack([t.dv[d].cpu()[i] for d, i in place[0]])
    assert same_bits(got, expected(rows, t.d_out[0], t.w[0], 2)[0])


@pytest.mark.parametrize("cap", ["1", "3"])
def test_capped_grids(cap, monkeypatch):
    monkeypatch.setenv("A2AV_MAX_GRID", cap)
    g = torch.Generator().manual_seed(5)
    z = [torch.randn(90, 96, generator=g) for _ in range(2)]
    ids, w = check_route(z, False, 0.1 * torch.randn(96, generator=g), 4, 2, 2, 5, True, 1.0)
    check_route_grad(z, ids, w, [torch.randn(90, 5, generator=g) for _ in z], False, True, 1.0)
    big = [torch.randn(9, 1100, generator=g)]
    ids, w = check_route(big, True, None, 1, 1, 1, 5, False, 1.0)
    check_route_grad(big, ids, w, [torch.randn(9, 5, generator=g)], True, False, 1.0)
    t = Trip(2, 30, 3, 8, 136, 0, seed=32)
    assert t.run() == 0
    rows = torch.stack([t.rows[d][i] for d, i in t.place()[1]])
    got = torch.stack([t.dv[d].cpu()[i] for d, i in t.place()[1]])
    assert same_bits(got, expected(rows, t.d_out[1], t.w[1], 3)[0])
    assert os.environ["A2AV_MAX_GRID"] == cap
