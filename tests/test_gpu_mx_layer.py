"""A MoE layer on microscaled rows as a server runs it: the residual's addition
and the norm with 8-bit rows, the router, the pack and dispatch of those rows,
the up and down products with 4-bit weights, and the combine at the owners,
against the same steps in 64 bits; captured and replayed, on two streams, and
with a failing dispatch. Then a training step with 8-bit rows on the wire:
received rows back to values, the products in 16 bits and their gradients, and
the norm's."""
import pytest
import torch

import layer_ref as R
import mx_ref as M
from embeddings_a2av_virtual_amd import _binding as B

pytestmark = pytest.mark.gpu

EPS = 1e-6


class Served:
    """Weights, inputs and every buffer of one layer; ``step`` enqueues the
    forward pass and allocates nothing."""

    def __init__(self, W, T, k, E, H, F, form, seed):
        self.W, self.T, self.k, self.E, self.H, self.F, self.form = W, T, k, E, H, F, form
        P = self.P = E // W
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s, scale=1.0: scale * torch.randn(*s, generator=g)  # noqa: E731
        bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        i64 = lambda *s: torch.zeros(*s, dtype=torch.int64, device="cuda")  # noqa: E731
        u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
        self.x = [rnd(T, H).to(torch.bfloat16).cuda() for _ in range(W)]
        self.residual = [rnd(T, H).to(torch.bfloat16).cuda() for _ in range(W)]
        self.norm_w = (1 + rnd(H, scale=0.1)).to(torch.bfloat16).cuda()
        self.router = rnd(E, H, scale=H ** -0.5).cuda()
        self.up_v = [rnd(P * 2 * F, H, scale=H ** -0.5) for _ in range(W)]
        self.down_v = [rnd(P * H, F, scale=F ** -0.5) for _ in range(W)]
        self.bias = [rnd(P, H, scale=0.1).cuda() for _ in range(W)]
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.up = [u8(P * 2 * F, B.moe_mx_row_bytes(B.MX_FP4, H)) for _ in range(W)]
        self.down = [u8(P * H, B.moe_mx_row_bytes(B.MX_FP4, F)) for _ in range(W)]
        for v, w, n, K in ((self.up_v, self.up, P * 2 * F, H), (self.down_v, self.down, P * H, F)):
            B.moe_mx_quantize(W, K, B.MX_FP4, [a.cuda() for a in v], [n] * W, w, self.status)
        cap = self.cap = [W * T * k] * W
        self.wide = B.moe_mx_row_bytes(form, H)
        self.sum, self.normed, self.rows = [bf(T, H) for _ in range(W)], [bf(T, H) for _ in range(W)], \
            [u8(T, self.wide) for _ in range(W)]
        self.logits = [torch.zeros(T, E, device="cuda") for _ in range(W)]
        self.ids = [torch.zeros((T, k), dtype=torch.int32, device="cuda") for _ in range(W)]
        self.w = [torch.zeros((T, k), device="cuda") for _ in range(W)]
        self.perm, self.S, self.counts, self.off = [i64(T * k) for _ in range(W)], i64(W, W), i64(W, E), i64(W, P + 1)
        self.recv = [u8(c, self.wide) for c in cap]
        self.mid = [u8(c, B.moe_mx_row_bytes(B.MX_FP8, F)) for c in cap]
        self.back, self.out = [bf(c, H) for c in cap], [bf(T, H) for _ in range(W)]
        self.ws = u8(max(B.moe_pack_dispatch_workspace_bytes(W, T, k, E), B.moe_combine_return_workspace_bytes(W, T, k, E),
                         B.moe_expert_linear_mx_workspace_bytes(W, P, H, F, B.ACT_SWIGLU, cap),
                         B.moe_expert_linear_mx_workspace_bytes(W, P, F, H, B.ACT_NONE, cap)))

    def step(self):
        W, T, k, E, H, F, P, st, ws, cap = (self.W, self.T, self.k, self.E, self.H, self.F, self.P, self.status,
                                            self.ws, self.cap)
        B.moe_rms_norm(W, T, H, EPS, self.x, self.residual, self.norm_w, self.sum, self.normed, self.rows, self.form, st)
        for a, z in zip(self.normed, self.logits):
            torch.mm(a.float(), self.router.t(), out=z)
        B.moe_route(W, T, k, E, B.SCORE_SOFTMAX, self.logits, None, 1, 1, 1, True, 1.0, self.ids, self.w, st)
        B.moe_pack_dispatch(W, T, k, E, self.wide, self.rows, self.ids, self.recv, cap, self.perm, self.S, self.counts,
                            self.off, 1, ws, st)
        B.moe_expert_linear_mx(W, P, H, F, self.form, B.ACT_SWIGLU, self.recv, cap, self.off, self.up, None, self.mid,
                               ws, st)
        B.moe_expert_linear_mx(W, P, F, H, B.MX_FP8, B.ACT_NONE, self.mid, cap, self.off, self.down, self.bias,
                               self.back, ws, st)
        B.moe_combine_return(W, T, k, E, H, self.counts, self.ids, self.perm, self.back, cap, self.w, self.out, 1, ws,
                             st)

    def results(self):
        return self.sum + self.normed + self.w + self.ids + self.out

    def reference(self):
        """The layer in 64 bits from the rows that the norm wrote."""
        W, T, k, P, H, F = self.W, self.T, self.k, self.P, self.H, self.F
        up = [M.values(M.quantize(v.double(), M.FP4), M.FP4, H).reshape(P, 2 * F, H) for v in self.up_v]
        down = [M.values(M.quantize(v.double(), M.FP4), M.FP4, F).reshape(P, H, F) for v in self.down_v]
        outs = []
        for s in range(W):
            h = M.add(self.x[s].cpu(), self.residual[s].cpu())
            assert torch.equal(self.sum[s].cpu(), h)
            rows = M.quantize(M.norm(h, self.norm_w.cpu(), EPS), self.form)
            assert torch.equal(self.rows[s].cpu()[:, :rows.shape[1]], rows)
            v = M.values(rows, self.form, H)
            y = torch.zeros(T, H, dtype=torch.float64)
            for t in range(T):
                for j in range(k):
                    e = int(self.ids[s][t, j])
                    m = R.activate("swiglu", up[e // P][e % P] @ v[t])
                    m = M.values(M.quantize(m[None], M.FP8), M.FP8, F)[0]
                    y[t] += float(self.w[s][t, j]) * (down[e // P][e % P] @ m + self.bias[e // P][e % P].cpu().double())
            outs.append(y)
        return outs


CASES = [(2, 24, 3, 8, 64, 48, B.MX_FP8), (4, 9, 2, 4, 320, 264, B.MX_FP4), (1, 1, 4, 16, 4352, 64, B.MX_FP8),
         (2, 200, 2, 4, 257, 100, B.MX_FP8)]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_served_step(case):
    m = Served(*case, seed=sum(case))
    m.step()
    torch.cuda.synchronize()
    assert int(m.status.item()) == 0
    got, want = torch.cat([x.cpu().double() for x in m.out]), torch.cat(m.reference())
    # back and out are rounded to bf16 once each; an element of mid next to a border may
    # be its neighbour's (1/16 of itself, seldom), which a fourth of a rounding covers
    rel = float((got - want).norm() / want.norm())
    assert rel <= 2.25 * R.half_step(torch.bfloat16), rel


def test_step_captured_and_replayed():
    args = (2, 40, 4, 16, 320, 96, B.MX_FP8)
    m = Served(*args, seed=5)
    m.step()
    torch.cuda.synchronize()
    want = [x.clone() for x in m.results()]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.step()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            m.step()
    for i in range(4):
        for x in m.results() + m.rows + m.mid:
            x.zero_()
        m.ws.random_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert int(m.status.item()) == 0
        assert all(torch.equal(a, b) for a, b in zip(m.results(), want)), i
        (torch.randn(1 << 18, device="cuda") * 2).sum().item()
    other = Served(*args, seed=6)
    other.step()
    inputs = lambda q: q.x + q.residual + [q.norm_w, q.router] + q.up + q.down + q.bias  # noqa: E731
    for a, b in zip(inputs(m), inputs(other)):
        a.copy_(b)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(m.results(), other.results()))


def test_two_layers_on_two_streams():
    layers = [Served(2, 40, 4, 16, 320, 96, B.MX_FP8, seed=7), Served(1, 90, 2, 8, 256, 128, B.MX_FP4, seed=8)]
    want = []
    for m in layers:
        m.step()
        torch.cuda.synchronize()
        want.append([x.clone() for x in m.results()])
        for x in m.results():
            x.zero_()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(4):
        for m, s in zip(layers, streams):
            with torch.cuda.stream(s):
                m.step()
    torch.cuda.synchronize()
    for m, w in zip(layers, want):
        assert int(m.status.item()) == 0 and all(torch.equal(a, b) for a, b in zip(m.results(), w))


def test_a_failed_dispatch_stops_the_step():
    m = Served(2, 24, 3, 8, 64, 48, B.MX_FP8, seed=9)
    m.cap = [3, 3]
    for x in m.mid + m.back + m.out:
        x.fill_(7)
    m.step()
    torch.cuda.synchronize()
    assert int(m.status.item()) == B.ST_RECV_OVERFLOW
    assert all((x == 7).all() for x in m.mid + m.back + m.out)


class Trained:
    """Norm, 8-bit dispatch, products in 16 bits, combine, and the way back to
    the hidden states: the dispatch's conversion passes its gradient through."""

    def __init__(self, W, T, k, E, H, F, seed):
        self.W, self.T, self.k, self.E, self.H, self.F = W, T, k, E, H, F
        P = self.P = E // W
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s, scale=1.0: (scale * torch.randn(*s, generator=g)).to(torch.bfloat16).cuda()  # noqa: E731
        bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        i64 = lambda *s: torch.zeros(*s, dtype=torch.int64, device="cuda")  # noqa: E731
        u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
        self.x, self.residual = [rnd(T, H) for _ in range(W)], [rnd(T, H) for _ in range(W)]
        self.norm_w = (1 + rnd(H, scale=0.1).float()).to(torch.bfloat16)
        self.experts = [rnd(P, F, H, scale=H ** -0.5) for _ in range(W)]
        self.d_out, self.d_sum = [rnd(T, F) for _ in range(W)], [rnd(T, H) for _ in range(W)]
        self.ids = [torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32).cuda()
                    for _ in range(W)]
        self.w = [torch.softmax(torch.randn(T, k, generator=g), -1).cuda() for _ in range(W)]
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        cap = self.cap = [W * T * k] * W
        self.wide = B.moe_mx_row_bytes(B.MX_FP8, H)
        self.sum, self.rows = [bf(T, H) for _ in range(W)], [u8(T, self.wide) for _ in range(W)]
        self.perm, self.S, self.counts, self.off = [i64(T * k) for _ in range(W)], i64(W, W), i64(W, E), i64(W, P + 1)
        self.recv, self.values = [u8(c, self.wide) for c in cap], [bf(c, H) for c in cap]
        self.back, self.d_back, self.d_recv = [bf(c, F) for c in cap], [bf(c, F) for c in cap], [bf(c, H) for c in cap]
        self.out, self.d_w = [bf(T, F) for _ in range(W)], [torch.zeros(T, k, device="cuda") for _ in range(W)]
        self.d_y, self.d_x = [bf(T, H) for _ in range(W)], [bf(T, H) for _ in range(W)]
        self.ones = [torch.ones(T, k, device="cuda") for _ in range(W)]
        self.d_experts, self.d_norm = [torch.zeros_like(e) for e in self.experts], torch.zeros(H, device="cuda")
        self.ws = u8(max(B.moe_pack_dispatch_workspace_bytes(W, T, k, E),
                         B.moe_combine_return_backward_workspace_bytes(W, T, k, E),
                         B.moe_expert_linear_backward_workspace_bytes(W, P, H, F, B.ACT_NONE, cap),
                         B.moe_rms_norm_backward_workspace_bytes(W, T, H)))

    def step(self):
        W, T, k, E, H, F, P, st, ws, cap = (self.W, self.T, self.k, self.E, self.H, self.F, self.P, self.status,
                                            self.ws, self.cap)
        B.moe_rms_norm(W, T, H, EPS, self.x, self.residual, self.norm_w, self.sum, None, self.rows, B.MX_FP8, st)
        B.moe_pack_dispatch(W, T, k, E, self.wide, self.rows, self.ids, self.recv, cap, self.perm, self.S, self.counts,
                            self.off, 1, ws, st)
        B.moe_mx_dequantize(W, H, B.MX_FP8, self.recv, cap, self.values, st)
        B.moe_expert_linear(W, P, H, F, B.ACT_NONE, self.values, cap, self.off, self.experts, None, None, self.back,
                            None, ws, st)
        B.moe_combine_return(W, T, k, E, F, self.counts, self.ids, self.perm, self.back, cap, self.w, self.out, 1, ws,
                             st)
        B.moe_combine_return_backward(W, T, k, E, F, self.counts, self.ids, self.perm, self.back, cap, self.w,
                                      self.d_out, self.d_back, self.d_w, 1, ws, st)
        B.moe_expert_linear_backward(W, P, H, F, B.ACT_NONE, self.values, cap, self.off, self.experts, None, self.d_back,
                                     None, self.d_recv, self.d_experts, None, ws, st)
        B.moe_combine_return(W, T, k, E, H, self.counts, self.ids, self.perm, self.d_recv, cap, self.ones, self.d_y, 1,
                             ws, st)
        B.moe_rms_norm_backward(W, T, H, EPS, self.sum, self.norm_w, self.d_y, self.d_sum, self.d_x, self.d_norm, ws, st)

    def results(self):
        return self.out + self.d_x + self.d_w + self.d_experts + [self.d_norm]

    def reference(self):
        """By automatic differentiation in 64 bits, the conversion's error a constant."""
        W, T, k, P = self.W, self.T, self.k, self.P
        x = [M.add(a.cpu(), b.cpu()).double().requires_grad_(True) for a, b in zip(self.x, self.residual)]
        nw = self.norm_w.cpu().double().requires_grad_(True)
        ex = [e.cpu().double().requires_grad_(True) for e in self.experts]
        w = [v.cpu().double().requires_grad_(True) for v in self.w]
        outs = []
        for s in range(W):
            y = M.norm(x[s], nw, EPS)
            v = M.values(M.quantize(y.detach(), M.FP8), M.FP8, self.H)
            y = y + (v - y).detach()
            outs.append(torch.stack([sum(w[s][t, j] * (ex[e // P][e % P] @ y[t]) for j, e in
                                         enumerate(self.ids[s][t].tolist())) for t in range(T)]))
        loss = sum((o * d.cpu().double()).sum() for o, d in zip(outs, self.d_out))
        loss = loss + sum((a * d.cpu().double()).sum() for a, d in zip(x, self.d_sum))
        g = torch.autograd.grad(loss, x + ex + w + [nw])
        return [o.detach() for o in outs], g[:W], g[W:2 * W], g[2 * W:3 * W], g[3 * W:]


def _close(got, want, roundings):
    """Each stage rounds its rows to bf16 once, half a step of their norm."""
    g, w = torch.cat([x.cpu().double().reshape(-1) for x in got]), torch.cat([x.reshape(-1) for x in want])
    assert float((g - w).norm() / w.norm()) <= 2 * roundings * R.half_step(torch.bfloat16)


@pytest.mark.parametrize("case", [(2, 24, 3, 8, 64, 48), (1, 33, 2, 4, 264, 40), (4, 5, 1, 4, 40, 72)], ids=str)
def test_training_step(case):
    m = Trained(*case, seed=sum(case))
    m.step()
    torch.cuda.synchronize()
    assert int(m.status.item()) == 0
    out, d_x, d_experts, d_w, d_norm = m.reference()
    # roundings on the way: back, out; then d_back, d_recv, d_y, d_x
    _close(m.out, out, 2)
    _close(m.d_w, d_w, 1)
    _close(m.d_experts, d_experts, 2)
    _close(m.d_x, d_x, 4)
    _close([m.d_norm], d_norm, 3)


def test_training_step_captured_beside_an_eager_one():
    m = Trained(2, 40, 2, 8, 264, 96, seed=3)
    m.step()
    torch.cuda.synchronize()
    want = [x.clone() for x in m.results()]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            m.step()
    for i in range(4):
        for x in m.results():
            x.zero_()
        m.ws.random_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert int(m.status.item()) == 0 and all(torch.equal(a, b) for a, b in zip(m.results(), want)), i
        m.step()  # the eager step between the replays
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(m.results(), want)), i
