"""The experts' products (moe_expert_linear) and their gradients against 64
bits: every activation and type, row counts from none to many tiles, sizes and
bases that are no 16-byte multiples, infinities and NaN in rows that belong to
other experts or to nobody, refusals, and rows past the totals."""
import itertools
import zlib

import pytest
import torch

import layer_ref as R
from embeddings_a2av_virtual_amd import _binding as B
from gpu_util import GuardedBuffer, SENT

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
ACTS = {"none": B.ACT_NONE, "relu": B.ACT_RELU, "gelu": B.ACT_GELU, "silu": B.ACT_SILU, "swiglu": B.ACT_SWIGLU}


def _buffer(shape, dtype, pad=0, of=None):
    n = 1
    for s in shape:
        n *= s
    b = GuardedBuffer(n * 2, pad=pad)
    v = b.view.view(dtype).reshape(shape)
    if of is not None:
        v.copy_(of)
    return b, v


class Experts:
    """W ranks of P experts with the given rows each, and `spare` rows of NaN
    behind every rank's last one."""

    def __init__(self, per, K, N, kind, act, seed, bias=True, residual=True, pre=True, spare=2, pad=0):
        self.W, self.P, self.K, self.N, self.act, self.pad = len(per), len(per[0]), K, N, act, pad
        self.NW, self.t, self.spare = (2 * N if act == "swiglu" else N), TYPES[kind], spare
        self.per = per
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g).to(self.t)  # noqa: E731
        tot = self.tot = [sum(p) for p in per]
        self.x = [torch.cat([rnd(n, K), torch.full((spare, K), float("nan")).to(self.t)]) for n in tot]
        self.weight = [(torch.randn(self.P, self.NW, K, generator=g) / K ** 0.5).to(self.t) for _ in per]
        self.bias = [rnd(self.P, self.NW) for _ in per] if bias else None
        self.residual = [rnd(n + spare, N) for n in tot] if residual else None
        self.d_out = [torch.cat([rnd(n, N), torch.full((spare, N), float("nan")).to(self.t)]) for n in tot]
        self.h = [rnd(n + spare, self.NW) for n in tot]
        self.want_pre = pre
        self.offsets = torch.tensor([[0] + list(itertools.accumulate(p)) for p in per], dtype=torch.int64)

    def _dev(self, xs):
        return None if xs is None else [_buffer(x.shape, self.t, self.pad, x)[1] for x in xs]

    def forward(self, offsets=None, x_rows=None, status=0, in_place=False):
        rows = x_rows or [n + self.spare for n in self.tot]
        ob, out = zip(*[_buffer((n + self.spare, self.N), self.t, self.pad) for n in self.tot])
        pb, pre = zip(*[_buffer((n + self.spare, self.NW), self.t, self.pad) for n in self.tot])
        res = self._dev(self.residual)
        if in_place:
            for o, r in zip(out, res):
                o.copy_(r)
            res = list(out)
        st = torch.full((1,), status, dtype=torch.int32, device="cuda")
        act = ACTS[self.act]
        ws = torch.empty(B.moe_expert_linear_workspace_bytes(self.W, self.P, self.K, self.N, act, rows),
                         dtype=torch.uint8, device="cuda").random_()
        B.moe_expert_linear(self.W, self.P, self.K, self.N, act, self._dev(self.x), rows,
                            (self.offsets if offsets is None else offsets).cuda(), self._dev(self.weight),
                            self._dev(self.bias), res, list(out), list(pre) if self.want_pre else None, ws, st)
        torch.cuda.synchronize()
        assert all(b.guards_intact() for b in ob + pb)
        return int(st.item()), [x.cpu() for x in out], [x.cpu() for x in pre]

    def backward(self, offsets=None, want=("d_x", "d_weight", "d_bias"), status=0, in_place=False):
        rows = [n + self.spare for n in self.tot]
        none = self.act == "none"
        bufs = {"d_pre": [(n + self.spare, self.NW) for n in self.tot], "d_x": [x.shape for x in self.x],
                "d_weight": [w.shape for w in self.weight], "d_bias": [(self.P, self.NW)] * self.W}
        made = {k: [_buffer(s, self.t, self.pad) for s in v] for k, v in bufs.items()}
        arg = {k: [v for _, v in x] for k, x in made.items()}
        st = torch.full((1,), status, dtype=torch.int32, device="cuda")
        act = ACTS[self.act]
        h = None if none else self._dev(self.h)
        if in_place:
            arg["d_pre"] = h
        ws = torch.empty(B.moe_expert_linear_backward_workspace_bytes(self.W, self.P, self.K, self.N, act, rows),
                         dtype=torch.uint8, device="cuda").random_()
        B.moe_expert_linear_backward(self.W, self.P, self.K, self.N, act, self._dev(self.x), rows,
                                     (self.offsets if offsets is None else offsets).cuda(), self._dev(self.weight),
                                     h, self._dev(self.d_out),
                                     None if none else arg["d_pre"],
                                     *[arg[k] if k in want else None for k in ("d_x", "d_weight", "d_bias")], ws, st)
        torch.cuda.synchronize()
        assert all(b.guards_intact() for v in made.values() for b, _ in v)
        return int(st.item()), {k: [x.cpu() for x in v] for k, v in arg.items()}

    def spans(self, d):
        at = 0
        for j, n in enumerate(self.per[d]):
            yield j, slice(at, at + n)
            at += n

    # a sum of L products in fp32, in any order: half a step of the running sum
    # for each term and one more for each product the matrix cores add at once
    def _gamma(self, L):
        return (2 * L + 8) * 2.0 ** -24

    def check_forward(self, **kw):
        st, out, pre = self.forward(**kw)
        assert st == 0
        half = R.half_step(self.t)
        tiny = torch.finfo(self.t).smallest_normal * half * 2
        for d in range(self.W):
            for j, s in self.spans(d):
                x, w = self.x[d][s].double(), self.weight[d][j].double()
                h, mag = x @ w.t(), x.abs() @ w.t().abs()
                if self.bias:
                    h, mag = h + self.bias[d][j].double(), mag + self.bias[d][j].double().abs()
                err = mag * self._gamma(self.K)
                if self.want_pre:
                    assert ((pre[d][s].double() - h).abs() <= err + h.abs() * half * 1.01 + tiny).all()
                y = R.activate(self.act, h)
                # slopes: |silu'|, |gelu'| < 1.13, |relu'| <= 1; fp32 steps of the activation itself
                if self.act == "swiglu":
                    g, u = h.chunk(2, -1)
                    eg, eu = err.chunk(2, -1)
                    err = 1.13 * eg * u.abs() + g.abs() * eu + 1.13 * eg * eu + (g * u).abs() * (g.abs() + 16) * 2.0 ** -23
                elif self.act != "none":
                    err = 1.13 * err + h.abs() * (h.abs() + 16) * 2.0 ** -23
                if self.residual:
                    y = y + self.residual[d][s].double()
                    err = err + (y.abs() + self.residual[d][s].double().abs()) * 2.0 ** -23
                far = (out[d][s].double() - y).abs() > err + y.abs() * half * 1.01 + tiny
                assert not far.any(), (d, j, far.nonzero()[:4].tolist(), int(far.sum()), far.numel())
            n = self.tot[d]
            if not kw.get("in_place"):
                assert (out[d][n:].view(torch.uint8) == SENT).all()
            assert (pre[d][n if self.want_pre else 0:].view(torch.uint8) == SENT).all()

    def check_backward(self, want=("d_x", "d_weight", "d_bias")):
        st, got = self.backward(want=want)
        assert st == 0
        half = R.half_step(self.t)
        tiny = torch.finfo(self.t).smallest_normal * half * 2
        for d in range(self.W):
            for j, s in self.spans(d):
                g = self.d_out[d][s].double()
                if self.act == "none":
                    d_pre = exact = g
                    err = torch.zeros_like(g)
                else:
                    h = self.h[d][s].double()
                    exact = R.activate_grad(self.act, h, g)
                    # the fp32 steps of act'(h): about 8 half steps and one for each unit of |h|, of the largest term
                    hm = h[:, : self.N] if self.act == "swiglu" else h
                    up = (1 + h[:, self.N:].abs()) if self.act == "swiglu" else 1
                    err = g.abs() * up * (1 + hm.abs()) * (hm.abs() + 8) * 2.0 ** -23
                    if self.act == "swiglu":
                        err = torch.cat([err, err], -1)
                    d_pre = got["d_pre"][d][s].double()
                    far = (d_pre - exact).abs() > err + exact.abs() * half * 1.01 + tiny
                    assert not far.any(), ("d_pre", d, j, far.nonzero()[:4].tolist())
                n = d_pre.shape[0]
                x, w = self.x[d][s].double(), self.weight[d][j].double()
                for name, v, mag, L in (("d_x", d_pre @ w, d_pre.abs() @ w.abs(), self.NW),
                                        ("d_weight", d_pre.t() @ x, d_pre.abs().t() @ x.abs(), n),
                                        ("d_bias", exact.sum(0), exact.abs().sum(0), n)):
                    if name not in want:
                        continue
                    y = got[name][d][s] if name == "d_x" else got[name][d][j]
                    tol = mag * self._gamma(L) + v.abs() * half * 1.01 + tiny
                    if name == "d_bias":
                        tol = tol + err.sum(0)
                    far = (y.double() - v).abs() > tol
                    assert not far.any(), (name, d, j, far.nonzero()[:4].tolist(), int(far.sum()), far.numel())
            for name in ("d_pre", "d_x"):
                used = self.tot[d] if name in want or (name == "d_pre" and self.act != "none") else 0
                assert (got[name][d][used:].view(torch.uint8) == SENT).all()
            for name in ("d_weight", "d_bias"):
                if name not in want:
                    assert (got[name][d].view(torch.uint8) == SENT).all()


SHAPES = [
    # rows per (rank, expert), K, N
    ([[1]], 64, 64),
    ([[0, 1, 0]], 32, 16),
    ([[5, 0, 70, 16], [0, 0, 0, 0], [64, 65, 1, 129]], 128, 96),
    ([[300, 3]], 520, 264),
    ([[33, 150]], 1000, 200),
    ([[17, 0, 9]], 7, 5),
    ([[40, 129]], 65, 67),
    ([[2, 1, 0, 3, 1, 1, 0, 2]], 256, 128),
    ([[513]], 192, 320),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}x{s[1]}x{s[2]}".replace(" ", ""))
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("act", list(ACTS))
def test_forward(shape, kind, act):
    per, K, N = shape
    seed = zlib.crc32(repr((shape, kind, act)).encode())
    Experts(per, K, N, kind, act, seed).check_forward()
    Experts(per, K, N, kind, act, seed, bias=False, residual=False, pre=False).check_forward()


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}x{s[1]}x{s[2]}".replace(" ", ""))
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("act", list(ACTS))
def test_backward(shape, kind, act):
    per, K, N = shape
    Experts(per, K, N, kind, act, zlib.crc32(repr((shape, kind, act)).encode())).check_backward()


# enough tiles of 256 x 256 and of 128 x 128 to fill the compute units
LARGE = [([[257, 300, 30, 0, 512] + [260] * 35], 640, 648), ([[130] * 20, [1, 127] * 10], 200, 1000)]


@pytest.mark.parametrize("shape", LARGE, ids=["256", "128"])
@pytest.mark.parametrize("kind,act", [("bf16", "swiglu"), ("fp16", "gelu"), ("fp16", "swiglu"), ("bf16", "none")])
def test_large_tiles(shape, kind, act):
    per, K, N = shape
    seed = zlib.crc32(repr((shape, kind, act)).encode())
    Experts(per, K, N, kind, act, seed).check_forward()
    Experts(per, K, N, kind, act, seed, bias=False, residual=False, pre=False).check_forward()
    Experts(per, K, N, kind, act, seed + 1).check_backward()


@pytest.mark.parametrize("per,K,N", [([[1, 0, 3, 1, 0, 2, 1, 5]], 4104, 72), ([[1]], 7168, 16),
                                     ([[20, 0, 0, 0, 0, 0, 0, 1], [0, 0, 16, 0, 0, 0, 0, 0]], 4096, 40),
                                     ([[0, 17, 0, 0, 1, 2, 3, 4]], 5000, 264)], ids=str)
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("act", list(ACTS))
def test_few_rows_of_long_weights(per, K, N, kind, act):
    seed = zlib.crc32(repr((per, K, N, kind, act)).encode())
    Experts(per, K, N, kind, act, seed).check_forward()
    Experts(per, K, N, kind, act, seed, bias=False, residual=False, pre=False).check_forward()


@pytest.mark.parametrize("want", [("d_x",), ("d_weight",), ("d_bias",), ()], ids=str)
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_backward_of_some(want, act):
    Experts([[20, 70]], 64, 32, "bf16", act, 5).check_backward(want)


@pytest.mark.parametrize("pad", [2, 8, 16])
def test_bases_of_other_alignments(pad):
    e = Experts([[20, 0, 70]], 64, 48, "fp16", "swiglu", 6, pad=pad)
    e.check_forward()
    e.check_backward()


def test_residual_in_place():
    Experts([[20, 70]], 64, 48, "bf16", "gelu", 7).check_forward(in_place=True)


@pytest.mark.parametrize("act", ["gelu", "swiglu"])
@pytest.mark.parametrize("K,N", [(64, 48), (33, 31)])
def test_gradient_of_pre_in_place(K, N, act):
    e = Experts([[20, 70, 0, 150]], K, N, "bf16", act, 8)
    st, apart = e.backward()
    st2, there = e.backward(in_place=True)
    assert st == st2 == 0
    n = e.tot[0]
    for k in apart:
        a, b = apart[k][0], there[k][0]
        if k in ("d_pre", "d_x"):
            a, b = a[:n], b[:n]
        assert torch.equal(a.view(torch.int16), b.view(torch.int16)), k


@pytest.mark.parametrize("K,N", [(64, 64), (72, 40), (33, 31), (1024, 512), (4096, 24)])
def test_other_experts_infinities_stay_out(K, N):
    """An expert whose rows and weights are infinite or NaN leaves its
    neighbours' results as they are."""
    for kind in TYPES:
        e = Experts([[9, 40, 70]], K, N, kind, "none", 8, residual=False)
        clean_f, clean_b = e.forward(), e.backward()
        e.x[0][9:49], e.weight[0][1] = float("inf"), float("nan")
        e.d_out[0][9:49], e.h[0][9:49] = float("nan"), float("nan")
        f, b = e.forward(), e.backward()
        for x, y in ((clean_f[1][0], f[1][0]), (clean_f[2][0], f[2][0]), (clean_b[1]["d_x"][0], b[1]["d_x"][0])):
            assert torch.equal(x[:9].view(torch.int16), y[:9].view(torch.int16))
            assert torch.equal(x[49:].view(torch.int16), y[49:].view(torch.int16))
        for j in (0, 2):
            assert torch.equal(clean_b[1]["d_weight"][0][j], b[1]["d_weight"][0][j])
            assert torch.equal(clean_b[1]["d_bias"][0][j], b[1]["d_bias"][0][j])


def test_same_result_every_time():
    e = Experts([[130, 40, 0, 7]], 200, 96, "bf16", "swiglu", 9)
    f, b = e.forward(), e.backward()
    for _ in range(3):
        f2, b2 = e.forward(), e.backward()
        assert all(torch.equal(x.view(torch.int16), y.view(torch.int16)) for x, y in zip(f[1] + f[2], f2[1] + f2[2]))
        for k in b[1]:
            assert all(torch.equal(x.view(torch.int16), y.view(torch.int16)) for x, y in zip(b[1][k], b2[1][k]))


def test_many_experts():
    """4096 experts in all, most without rows, one with most of them."""
    W, P = 2, 2048
    per = [[(i * 7 + d) % 3 if i % 5 == 0 else 0 for i in range(P)] for d in range(W)]
    per[1][77] = 700
    e = Experts(per, 24, 16, "bf16", "silu", 10)
    e.check_forward()
    e.check_backward()


@pytest.mark.parametrize("back", [False, True])
def test_refuses_bad_offsets(back):
    e = Experts([[5, 3], [2, 9]], 32, 16, "bf16", "relu", 11)

    def status(edit, x_rows=None):
        off = e.offsets.clone()
        edit(off)
        if back:
            st, got = e.backward(offsets=off)
            assert all((x.view(torch.uint8) == SENT).all() for v in got.values() for x in v)
        else:
            st, out, pre = e.forward(offsets=off)
            assert all((x.view(torch.uint8) == SENT).all() for x in out + pre)
        return st

    def edit(i, j, v):
        def f(off):
            off[i, j] = v
        return f

    assert status(edit(0, 0, 1)) == B.ST_BAD_OFFSETS
    assert status(edit(0, 0, -1)) == B.ST_BAD_OFFSETS
    assert status(edit(1, 1, 12)) == B.ST_BAD_OFFSETS        # above the next one
    assert status(edit(1, 1, -(1 << 62))) == B.ST_BAD_OFFSETS
    assert status(edit(1, 1, 1 << 62)) == B.ST_BAD_OFFSETS
    assert status(edit(1, 2, 14)) == B.ST_SEND_OVERRUN       # 13 rows are there
    assert status(edit(0, 2, 1 << 62)) == B.ST_SEND_OVERRUN
    st = e.backward(status=8)[0] if back else e.forward(status=8)[0]
    assert st == 8


def test_no_rows_at_all():
    e = Experts([[0, 0]], 32, 16, "bf16", "silu", 12, spare=0)
    assert e.forward()[0] == 0
    st, got = e.backward()
    assert st == 0 and (got["d_weight"][0] == 0).all() and (got["d_bias"][0] == 0).all()


def test_argument_checks():
    e = Experts([[5, 3]], 32, 16, "bf16", "silu", 13)
    x, w, off = [e.x[0].cuda()], [e.weight[0].cuda()], e.offsets.cuda()
    out, ws = [torch.empty((10, 16), dtype=torch.bfloat16, device="cuda")], torch.empty(4096, dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(x=x, rows=(10,), w=w, out=out, off=off, ws=ws, act=B.ACT_SILU, K=32, N=16, P=2, bias=None):
        B.moe_expert_linear(1, P, K, N, act, x, list(rows), off, w, bias, None, out, None, ws, st)

    call()
    for kw in (dict(x=[x[0].half()]), dict(rows=(11,)), dict(w=[w[0].float()]), dict(out=[out[0][:9]]),
               dict(off=off.int()), dict(K=33), dict(rows=(10, 10)), dict(bias=[w[0][0, 0, 1:]]), dict(x=[x[0].cpu()])):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(ws=ws[:64]), dict(act=5), dict(act=-1), dict(rows=(-1,)), dict(K=0), dict(P=0)):
        with pytest.raises(B.A2avError):
            call(**kw)
