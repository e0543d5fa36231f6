"""The weighted combine's gradient over a returned buffer
(moe_combine_backward) and at the owners (moe_combine_return_backward): the
rows' gradient bit for bit (one fp32 product, one rounding), the weights'
within the rounding of an fp32 sum, refusals, and rows past the totals."""
import zlib

import numpy as np
import pytest
import torch

from embeddings_a2av_virtual_amd import _binding as B
from embeddings_a2av_virtual_amd import inputs as I
from gpu_util import GuardedBuffer, SENT

pytestmark = pytest.mark.gpu


def _bf16(g, *shape):
    return torch.randn(*shape, generator=g).to(torch.bfloat16)


def _buffer(x, pad=0, extra=0):
    """x on the device behind `pad` bytes, with `extra` rows more."""
    rows = x.shape[0] + extra
    b = GuardedBuffer(rows * x.shape[1] * 2, pad=pad)
    v = b.view.view(torch.bfloat16).reshape(rows, x.shape[1])
    v[: x.shape[0]].copy_(x)
    return b, v


def _empty(rows, H, pad=0):
    b = GuardedBuffer(rows * H * 2, pad=pad)
    return b, b.view.view(torch.bfloat16).reshape(rows, H)


def expected(rows, d_out, w, k):
    """d_rows and d_weights of the slots' rows [Q, H] (host), in slot order."""
    d = d_out.repeat_interleave(k, 0)
    d_rows = (w.reshape(-1, 1) * d.float()).to(torch.bfloat16)
    prod = rows.double() * d.double()
    # a chain of H / 64 fused multiply-adds per lane (8 a step), then a tree of 6 adds
    tol = (rows.shape[1] / 64 + 24) * 2.0 ** -24 * prod.abs().sum(-1)
    return d_rows, prod.sum(-1), tol


def same_bits(got, want):
    return torch.equal(got.view(torch.int16), want.view(torch.int16)) or (
        torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(got[~torch.isnan(got)], want[~torch.isnan(want)]))


def run_pack(W, T, k, H, rows, perm, w, d_out, pad=0, status=0):
    rb, rv = zip(*[_buffer(x, pad) for x in rows])
    gb, gv = zip(*[_buffer(x, pad) for x in d_out])
    db, dv = zip(*[_empty(T * k, H, pad) for _ in range(W)])
    dw = [torch.full((T, k), -7.0, device="cuda") for _ in range(W)]
    st = torch.full((1,), status, dtype=torch.int32, device="cuda")
    ws = torch.empty(B.moe_combine_backward_workspace_bytes(W, T, k), dtype=torch.uint8, device="cuda")
    B.moe_combine_backward(W, T, k, H, list(rv), [p.cuda() for p in perm], [x.cuda() for x in w], list(gv),
                           list(dv), dw, ws, st)
    torch.cuda.synchronize()
    assert all(b.guards_intact() for b in rb + gb + db)
    return int(st.item()), [x.cpu() for x in dv], [x.cpu() for x in dw]


@pytest.mark.parametrize("case", [(1, 1, 1, 8), (1, 1, 8, 7168), (2, 129, 3, 1000), (3, 17, 5, 129),
                                  (1, 40, 64, 72), (4, 33, 8, 512), (1, 5, 2, 1), (2, 9, 4, 4100),
                                  (1, 3, 9, 20000)], ids=str)
@pytest.mark.parametrize("pad", [0, 2, 16])
def test_over_a_returned_buffer(case, pad):
    W, T, k, H = case
    g = torch.Generator().manual_seed(zlib.crc32(repr(case).encode()))
    rows, d_out = [_bf16(g, T * k, H) for _ in range(W)], [_bf16(g, T, H) for _ in range(W)]
    perm = [torch.randperm(T * k, generator=g) for _ in range(W)]
    w = [torch.randn(T, k, generator=g) for _ in range(W)]
    st, d_rows, d_w = run_pack(W, T, k, H, rows, perm, w, d_out, pad)
    assert st == 0
    for r in range(W):
        want, ww, tol = expected(rows[r][perm[r]], d_out[r], w[r], k)
        assert same_bits(d_rows[r][perm[r]], want), r
        assert ((d_w[r].reshape(-1).double() - ww).abs() <= tol).all()


def test_infinities_nan_and_zero_weights():
    g = torch.Generator().manual_seed(5)
    W, T, k, H = 1, 12, 4, 64
    rows, d_out = [_bf16(g, T * k, H)], [_bf16(g, T, H)]
    perm, w = [torch.randperm(T * k, generator=g)], [torch.randn(T, k, generator=g)]
    d_out[0][1, 3], d_out[0][2, 5], rows[0][7, 1] = float("nan"), float("inf"), float("inf")
    w[0][3], w[0][4, 0], w[0][5, 1] = 0.0, float("inf"), 1e-39
    st, d_rows, d_w = run_pack(W, T, k, H, rows, perm, w, d_out)
    want, ww, _ = expected(rows[0][perm[0]], d_out[0], w[0], k)
    assert st == 0 and same_bits(d_rows[0][perm[0]], want)
    assert torch.equal(torch.isfinite(d_w[0].reshape(-1)), torch.isfinite(ww))


@pytest.mark.parametrize("bad", ["negative", "past", "twice"])
def test_refuses_bad_permutations(bad):
    g = torch.Generator().manual_seed(6)
    W, T, k, H = 2, 300, 2, 16
    rows, d_out = [_bf16(g, T * k, H)] * W, [_bf16(g, T, H)] * W
    perm = [torch.randperm(T * k, generator=g) for _ in range(W)]
    perm[1][77] = {"negative": -1, "past": T * k, "twice": perm[1][500]}[bad]
    st, d_rows, d_w = run_pack(W, T, k, H, rows, perm, [torch.ones(T, k)] * W, d_out)
    assert st == B.ST_BAD_PERM
    assert all((x.view(torch.uint8) == SENT).all() for x in d_rows) and all((x == -7).all() for x in d_w)


def test_poisoned_status_and_no_tokens():
    g = torch.Generator().manual_seed(7)
    st, d_rows, _ = run_pack(1, 4, 2, 8, [_bf16(g, 8, 8)], [torch.arange(8)], [torch.ones(4, 2)], [_bf16(g, 4, 8)],
                             status=2)
    assert st == 2 and (d_rows[0].view(torch.uint8) == SENT).all()
    assert run_pack(1, 0, 2, 8, [_bf16(g, 0, 8)], [torch.arange(0)], [torch.ones(0, 2)], [_bf16(g, 0, 8)])[0] == 0


# ------------------------------------------------------------------ at the owners
class Trip:
    """Routing of W ranks, packed and dispatched by the library."""

    def __init__(self, W, T, k, E, H, layout, seed, repeats=False, spare=3, pad=0):
        self.W, self.T, self.k, self.E, self.H, self.layout = W, T, k, E, H, layout
        g = I.rng(seed)
        gen = torch.Generator().manual_seed(seed)
        self.ids = [torch.from_numpy(np.ascontiguousarray(
            I.uniform_ids(g, T, k, E) if repeats else I.topk_ids(g, T, k, E))).reshape(T, k) for _ in range(W)]
        self.d_out = [_bf16(gen, T, H) for _ in range(W)]
        self.w = [torch.randn(T, k, generator=gen) for _ in range(W)]
        Q, P = T * k, E // W
        flat = torch.cat([x.reshape(-1) for x in self.ids]).long() if Q else torch.zeros(0, dtype=torch.long)
        self.cap = [int((flat // P == d).sum()) for d in range(W)]
        z = dict(dtype=torch.int64, device="cuda")
        self.perm = [torch.zeros(Q, **z) for _ in range(W)]
        self.S, self.counts = torch.zeros((W, W), **z), torch.zeros((W, E), **z)
        self.off = torch.zeros((W, (P if layout else W) + 1), **z)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.cids = [x.cuda() for x in self.ids]
        toks = [torch.zeros((T, H), dtype=torch.bfloat16, device="cuda") for _ in range(W)]
        recv = [torch.zeros((max(c, 1), H), dtype=torch.bfloat16, device="cuda") for c in self.cap]
        ws = torch.empty(B.moe_pack_dispatch_workspace_bytes(W, T, k, E), dtype=torch.uint8, device="cuda")
        B.moe_pack_dispatch(W, T, k, E, 2 * H, toks, self.cids, recv, self.cap, self.perm, self.S, self.counts,
                            self.off, layout, ws, self.status)
        assert int(self.status.item()) == 0
        # owner rows of random values, `spare` rows past the total
        self.rows = [_bf16(gen, c + spare, H) for c in self.cap]
        self.rb, self.rv = zip(*[_buffer(x, pad) for x in self.rows])
        self.db, self.dv = zip(*[_empty(c + spare, H, pad) for c in self.cap])
        self.dw = [torch.full((T, k), -7.0, device="cuda") for _ in range(W)]
        self.recv_rows = [c + spare for c in self.cap]

    def place(self):
        """(owner, row) of every slot of every source, from the definition of the layouts."""
        P, out = self.E // self.W, []
        keys = []
        for s in range(self.W):
            for q, e in enumerate(self.ids[s].reshape(-1).tolist()):
                keys.append(((e // P, s, e, q) if self.layout == 0 else (e // P, e, s, q), s, q))
        at, seen = {}, {}
        for key, s, q in sorted(keys):
            at[(s, q)] = (key[0], seen.get(key[0], 0))
            seen[key[0]] = seen.get(key[0], 0) + 1
        for s in range(self.W):
            out.append([at[(s, q)] for q in range(self.T * self.k)])
        return out

    def run(self, counts=None, perm=None, ids=None, recv_rows=None, status=0):
        self.status.fill_(status)
        ws = torch.empty(B.moe_combine_return_backward_workspace_bytes(self.W, self.T, self.k, self.E),
                         dtype=torch.uint8, device="cuda").random_()
        B.moe_combine_return_backward(
            self.W, self.T, self.k, self.E, self.H, self.counts if counts is None else counts,
            self.cids if ids is None else ids, self.perm if perm is None else perm, list(self.rv),
            self.recv_rows if recv_rows is None else recv_rows, [x.cuda() for x in self.w],
            [x.cuda() for x in self.d_out], list(self.dv), self.dw, self.layout, ws, self.status)
        torch.cuda.synchronize()
        assert all(b.guards_intact() for b in self.rb + self.db)
        return int(self.status.item())

    def untouched(self):
        return all((x.view(torch.uint8) == SENT).all() for x in self.dv) and all((x == -7).all() for x in self.dw)


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("case", [(1, 1, 1, 1, 8), (2, 33, 3, 8, 24), (4, 20, 8, 32, 7168), (8, 11, 4, 64, 130),
                                  (3, 40, 2, 6, 1000), (2, 0, 2, 4, 16)], ids=str)
def test_at_the_owners(case, layout):
    t = Trip(*case, layout, seed=sum(case), repeats=case[2] < case[3] and layout == 0)
    assert t.run() == 0
    place = t.place()
    d_rows = [x.cpu() for x in t.dv]
    for s in range(t.W):
        if t.T == 0:
            continue
        rows = torch.stack([t.rows[d][i] for d, i in place[s]])
        want, ww, tol = expected(rows, t.d_out[s], t.w[s], t.k)
        got = torch.stack([d_rows[d][i] for d, i in place[s]])
        assert same_bits(got, want)
        assert ((t.dw[s].cpu().reshape(-1).double() - ww).abs() <= tol).all()
    for d in range(t.W):  # the rows past the total
        assert (d_rows[d][t.cap[d]:].view(torch.uint8) == SENT).all()


def test_at_the_owners_unaligned():
    t = Trip(2, 21, 3, 8, 40, 1, seed=9, pad=2)
    assert t.run() == 0
    rows = torch.stack([t.rows[d][i] for d, i in t.place()[1]])
    got = torch.stack([t.dv[d].cpu()[i] for d, i in t.place()[1]])
    assert same_bits(got, expected(rows, t.d_out[1], t.w[1], t.k)[0])


@pytest.mark.parametrize("layout", [0, 1])
def test_at_the_owners_refusals(layout):
    t = Trip(2, 30, 2, 8, 16, layout, seed=10)
    counts = t.counts.clone()
    counts[0, 3] = -1
    assert t.run(counts=counts) == B.ST_BAD_SPLIT and t.untouched()
    ids = [x.clone() for x in t.cids]
    ids[1][3, 1] = 8
    assert t.run(ids=ids) & B.ST_BAD_EXPERT and t.untouched()
    assert t.run(recv_rows=[t.cap[0] - 1, t.recv_rows[1]]) == B.ST_SEND_OVERRUN and t.untouched()
    perm = [x.clone() for x in t.perm]
    perm[0][5] = 60
    assert t.run(perm=perm) == B.ST_BAD_PERM and t.untouched()
    # the same row twice, inside its expert's block
    e = int(t.ids[0].reshape(-1)[0])
    q = [i for i, x in enumerate(t.ids[0].reshape(-1).tolist()) if x == e]
    if len(q) > 1:
        perm = [x.clone() for x in t.perm]
        perm[0][q[1]] = perm[0][q[0]]
        assert t.run(perm=perm) == B.ST_BAD_PERM and t.untouched()
    # counts that promise more rows than there are slots
    counts = t.counts.clone()
    counts[:, 0] += 1000
    assert t.run(counts=counts, recv_rows=t.recv_rows) != 0 and t.untouched()
    assert t.run(status=16) == 16 and t.untouched()
    assert t.run() == 0 and not t.untouched()


def test_argument_checks():
    t = Trip(2, 6, 2, 4, 16, 1, seed=11)
    st, ws = t.status, torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    a = [list(t.rv), t.perm, [x.cuda() for x in t.w], [x.cuda() for x in t.d_out], list(t.dv), t.dw]
    for i, x in ((0, [v.half() for v in a[0]]), (1, [p.int() for p in a[1]]), (3, a[3][:1]), (5, [d[:2] for d in a[5]])):
        b = list(a)
        b[i] = x
        with pytest.raises(ValueError):
            B.moe_combine_backward(2, 6, 2, 16, *b, ws, st)
    with pytest.raises(B.A2avError):
        B.moe_combine_return_backward(2, 6, 2, 4, 16, t.counts, t.cids, t.perm, a[0], t.recv_rows, a[2], a[3], a[4],
                                      a[5], 2, ws, st)
    with pytest.raises(B.A2avError):
        B.moe_combine_return_backward(2, 6, 2, 4, 16, t.counts, t.cids, t.perm, a[0], t.recv_rows, a[2], a[3], a[4],
                                      a[5], 1, ws[:256], st)
