"""A whole MoE layer on the library, as a training step runs it: route, pack
and dispatch, the experts' up and down products, the combine at the owners, and
the gradients of all of them back to the tokens, the weights and the router's
logits. Against the same layer in 64 bits with automatic differentiation, then
captured into a graph and replayed, and from two streams at once."""
import pytest
import torch

import layer_ref as R
from embeddings_a2av_virtual_amd import _binding as B

pytestmark = pytest.mark.gpu


class Layer:
    """Weights, inputs and every buffer of one layer; ``step`` enqueues the
    forward and backward pass and allocates nothing."""

    def __init__(self, W, T, k, E, H, F, seed, sigmoid=True):
        self.W, self.T, self.k, self.E, self.H, self.F, self.sigmoid = W, T, k, E, H, F, sigmoid
        P = self.P = E // W
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s, scale=1.0: (scale * torch.randn(*s, generator=g)).to(torch.bfloat16).cuda()  # noqa: E731
        self.tokens = [rnd(T, H) for _ in range(W)]
        self.logits = [torch.randn(T, E, generator=g).cuda() for _ in range(W)]
        self.bias = (0.1 * torch.randn(E, generator=g)).cuda()
        self.up = [rnd(P, 2 * F, H, scale=H ** -0.5) for _ in range(W)]
        self.down = [rnd(P, H, F, scale=F ** -0.5) for _ in range(W)]
        self.down_bias = [rnd(P, H, scale=0.1) for _ in range(W)]
        self.d_out = [rnd(T, H) for _ in range(W)]
        cap = self.cap = [W * T * k] * W
        f32 = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
        i64 = lambda *s: torch.zeros(*s, dtype=torch.int64, device="cuda")  # noqa: E731
        bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.ids = [torch.zeros((T, k), dtype=torch.int32, device="cuda") for _ in range(W)]
        self.w, self.d_w = [f32(T, k) for _ in range(W)], [f32(T, k) for _ in range(W)]
        self.ones = [torch.ones((T, k), device="cuda") for _ in range(W)]
        self.perm, self.S, self.counts = [i64(T * k) for _ in range(W)], i64(W, W), i64(W, E)
        self.off = i64(W, P + 1)
        rows = lambda n: [bf(c, n) for c in cap]  # noqa: E731
        self.recv, self.pre, self.mid, self.back = rows(H), rows(2 * F), rows(F), rows(H)
        self.d_back, self.d_mid, self.d_pre, self.d_recv = rows(H), rows(F), rows(2 * F), rows(H)
        self.out, self.d_tokens = [bf(T, H) for _ in range(W)], [bf(T, H) for _ in range(W)]
        self.d_logits = [f32(T, E) for _ in range(W)]
        self.d_up, self.d_down = [torch.zeros_like(x) for x in self.up], [torch.zeros_like(x) for x in self.down]
        self.d_down_bias = [torch.zeros_like(x) for x in self.down_bias]
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        size = max(B.moe_pack_dispatch_workspace_bytes(W, T, k, E),
                   B.moe_combine_return_backward_workspace_bytes(W, T, k, E),
                   B.moe_expert_linear_backward_workspace_bytes(W, P, H, F, B.ACT_SWIGLU, cap),
                   B.moe_expert_linear_backward_workspace_bytes(W, P, F, H, B.ACT_NONE, cap))
        self.ws = torch.empty(size, dtype=torch.uint8, device="cuda")

    def step(self):
        W, T, k, E, H, F, P, st, ws, cap = (self.W, self.T, self.k, self.E, self.H, self.F, self.P, self.status,
                                            self.ws, self.cap)
        score = B.SCORE_SIGMOID if self.sigmoid else B.SCORE_SOFTMAX
        B.moe_route(W, T, k, E, score, self.logits, self.bias, 1, 1, 1, True, 1.0, self.ids, self.w, st)
        B.moe_pack_dispatch(W, T, k, E, 2 * H, self.tokens, self.ids, self.recv, cap, self.perm, self.S, self.counts,
                            self.off, 1, ws, st)
        B.moe_expert_linear(W, P, H, F, B.ACT_SWIGLU, self.recv, cap, self.off, self.up, None, None, self.mid,
                            self.pre, ws, st)
        B.moe_expert_linear(W, P, F, H, B.ACT_NONE, self.mid, cap, self.off, self.down, self.down_bias, None,
                            self.back, None, ws, st)
        B.moe_combine_return(W, T, k, E, H, self.counts, self.ids, self.perm, self.back, cap, self.w, self.out, 1, ws,
                             st)
        B.moe_combine_return_backward(W, T, k, E, H, self.counts, self.ids, self.perm, self.back, cap, self.w,
                                      self.d_out, self.d_back, self.d_w, 1, ws, st)
        B.moe_expert_linear_backward(W, P, F, H, B.ACT_NONE, self.mid, cap, self.off, self.down, None, self.d_back,
                                     None, self.d_mid, self.d_down, self.d_down_bias, ws, st)
        B.moe_expert_linear_backward(W, P, H, F, B.ACT_SWIGLU, self.recv, cap, self.off, self.up, self.pre, self.d_mid,
                                     self.d_pre, self.d_recv, self.d_up, None, ws, st)
        # the tokens' gradient: their slots' rows added up
        B.moe_combine_return(W, T, k, E, H, self.counts, self.ids, self.perm, self.d_recv, cap, self.ones,
                             self.d_tokens, 1, ws, st)
        B.moe_route_backward(W, T, k, E, score, self.logits, self.ids, self.w, True, 1.0, self.d_w, self.d_logits, st)

    def results(self):
        return (self.out + self.d_tokens + self.d_logits + self.d_up + self.d_down + self.d_down_bias + self.w +
                self.ids)

    def reference(self):
        """The layer in 64 bits on the host: outputs and gradients, rank by rank."""
        W, T, k, P = self.W, self.T, self.k, self.P
        d64 = lambda xs: [x.cpu().double().requires_grad_(True) for x in xs]  # noqa: E731
        tokens, logits, up, down, bias = (d64(x) for x in (self.tokens, self.logits, self.up, self.down,
                                                           self.down_bias))
        outs, all_ids = [], []
        for s in range(W):
            ids, _ = R.route(logits[s].detach(), self.sigmoid, self.bias.cpu(), 1, 1, 1, k, True, 1.0)
            w = R.route_weights(logits[s], ids, self.sigmoid, True, 1.0)
            all_ids.append(ids)
            rows = []
            for t in range(T):
                y = 0
                for j in range(k):
                    e = int(ids[t, j])
                    h = R.activate("swiglu", up[e // P][e % P] @ tokens[s][t])
                    y = y + w[t, j] * (down[e // P][e % P] @ h + bias[e // P][e % P])
                rows.append(y)
            outs.append(torch.stack(rows))
        loss = sum((o * d.cpu().double()).sum() for o, d in zip(outs, self.d_out))
        leaves = tokens + logits + up + down + bias
        g = iter(torch.autograd.grad(loss, leaves))
        take = lambda n: [next(g) for _ in range(n)]  # noqa: E731
        return all_ids, [o.detach() for o in outs], *(take(W) for _ in range(5))


def _close(got, want, roundings, what):
    """Every stage rounds its rows to bf16 once, which moves a row by at most
    half a step of its norm; the products are with near-isometries, SwiGLU at
    most doubles a relative error, so the errors of the stages add up, doubled."""
    g, w = torch.cat([x.cpu().double().reshape(-1) for x in got]), torch.cat([x.reshape(-1) for x in want])
    rel = float((g - w).norm() / w.norm())
    assert rel <= 2 * roundings * R.half_step(torch.bfloat16), (what, rel)


@pytest.mark.parametrize("case", [(2, 24, 3, 8, 64, 48), (4, 9, 2, 4, 40, 24), (1, 1, 4, 16, 128, 64)], ids=str)
@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
def test_training_step(case, sigmoid):
    m = Layer(*case, seed=sum(case), sigmoid=sigmoid)
    m.step()
    torch.cuda.synchronize()
    assert int(m.status.item()) == 0
    ids, out, d_tokens, d_logits, d_up, d_down, d_bias = m.reference()
    for s in range(m.W):
        assert torch.equal(m.ids[s].cpu(), ids[s])
    # roundings on the way: mid, rows, out; then d_rows, d_mid, d_pre, d_row, the sum (and pre, which the way back reads)
    _close(m.out, out, 3, "out")
    _close(m.d_logits, d_logits, 3, "d_logits")
    _close(m.d_down, d_down, 3, "d_down")
    _close(m.d_down_bias, d_bias, 2, "d_down_bias")
    _close(m.d_up, d_up, 5, "d_up")
    _close(m.d_tokens, d_tokens, 6, "d_tokens")


def test_step_captured_and_replayed():
    m = Layer(2, 40, 4, 16, 128, 64, seed=5)
    m.step()
    torch.cuda.synchronize()
    want = [x.clone() for x in m.results()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        m.step()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            m.step()
    torch.cuda.synchronize()
    for i in range(5):
        for x in m.results():
            x.zero_()
        m.ws.random_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert int(m.status.item()) == 0
        for a, b in zip(m.results(), want):
            assert torch.equal(a, b), i
        x = torch.randn(1 << 20, device="cuda")
        (x * 2).sum().item()
    # new inputs through the captured step against an eager one
    other = Layer(2, 40, 4, 16, 128, 64, seed=6)
    other.step()
    for a, b in zip(m.tokens + m.logits + m.up + m.down + m.down_bias + m.d_out + [m.bias],
                    other.tokens + other.logits + other.up + other.down + other.down_bias + other.d_out + [other.bias]):
        a.copy_(b)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(m.results(), other.results()):
        assert torch.equal(a, b)


def test_two_layers_on_two_streams():
    """Calls on disjoint buffers from two streams at once."""
    a, b = Layer(2, 40, 4, 16, 128, 64, seed=7), Layer(1, 90, 2, 8, 256, 128, seed=8)
    want = []
    for m in (a, b):
        m.step()
        torch.cuda.synchronize()
        want.append([x.clone() for x in m.results()])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for m in (a, b):
        for x in m.results():
            x.zero_()
    torch.cuda.synchronize()
    for _ in range(4):
        for m, s in ((a, streams[0]), (b, streams[1])):
            with torch.cuda.stream(s):
                m.step()
    torch.cuda.synchronize()
    for m, w in ((a, want[0]), (b, want[1])):
        assert int(m.status.item()) == 0 and all(torch.equal(x, y) for x, y in zip(m.results(), w))


def test_a_failed_call_stops_the_step():
    """A receiver too small: the status word carries the dispatch's failure and
    no later call writes anything."""
    m = Layer(2, 24, 3, 8, 64, 48, seed=9)
    m.cap = [3, 3]
    for x in m.results():
        x.fill_(7)
    m.step()
    torch.cuda.synchronize()
    assert int(m.status.item()) == B.ST_RECV_OVERFLOW
    kept = m.out + m.d_tokens + m.d_logits + m.d_up + m.d_down + m.d_down_bias
    assert all((x == 7).all() for x in kept)
