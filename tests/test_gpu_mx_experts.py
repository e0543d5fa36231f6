"""The experts' products on microscaled rows (moe_expert_linear_mx) against 64
bits: both row formats, every activation and output type, row counts from none
to many tiles, sizes that are no multiples of anything, sums that fp32 holds
exactly, NaN blocks in rows of other experts or of nobody, and refusals."""
import itertools
import zlib

import pytest
import torch

import layer_ref as R
import mx_ref as M
from embeddings_a2av_virtual_amd import _binding as B
from gpu_util import GuardedBuffer, SENT

pytestmark = pytest.mark.gpu

ACTS = {"none": B.ACT_NONE, "relu": B.ACT_RELU, "gelu": B.ACT_GELU, "silu": B.ACT_SILU, "swiglu": B.ACT_SWIGLU}
FORMATS = {"fp8": B.MX_FP8, "fp4": B.MX_FP4}
OUTS = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp8": torch.uint8}


def _full(rows, form, H):
    """Whole rows, the unused bytes all ones."""
    return torch.nn.functional.pad(rows, (0, M.row_bytes(form, H) - rows.shape[1]), value=255)


class Experts:
    """W ranks of P experts with the given rows each, and `spare` rows of NaN
    behind every rank's last one. whole: small integers with scales of 1, whose
    sums fp32 holds exactly."""

    def __init__(self, per, K, N, form, act, out, seed, bias=True, spare=2, pad=0, whole=False):
        self.W, self.P, self.K, self.N, self.act, self.pad = len(per), len(per[0]), K, N, act, pad
        self.NW, self.form, self.out, self.spare = (2 * N if act == "swiglu" else N), FORMATS[form], OUTS[out], spare
        self.per, self.whole = per, whole
        self.tot = [sum(p) for p in per]
        g = torch.Generator().manual_seed(seed)
        values = lambda n, f: M.table(f)[torch.randint(0, 8, (n, K), generator=g)] * (  # noqa: E731
            1 - 2 * torch.randint(0, 2, (n, K), generator=g)) if whole else torch.randn(n, K, generator=g).double()
        self.x, self.weight, self.xv, self.wv = [], [], [], []
        for n in self.tot:
            v = values(n, M.FP4)  # e2m1 values are e4m3 ones too
            if whole and K > 1:
                v[:, ::32] = 6 if self.form == M.FP4 else 448
            rows = M.quantize(v, self.form)
            self.xv.append(M.values(rows, self.form, K))
            nan = torch.full((spare, rows.shape[1]), 255, dtype=torch.uint8)
            self.x.append(_full(torch.cat([rows, nan]), self.form, K))
            v = values(self.P * self.NW, M.FP4) / (1 if whole else K ** 0.5)
            if whole and K > 1:
                v[:, 1::32] = 6
            rows = M.quantize(v, M.FP4)
            self.wv.append(M.values(rows, M.FP4, K).reshape(self.P, self.NW, K))
            self.weight.append(_full(rows, M.FP4, K))
        self.bias = [torch.randint(-3, 4, (self.P, self.NW), generator=g).float() if whole else
                     torch.randn(self.P, self.NW, generator=g) for _ in per] if bias else None
        self.offsets = torch.tensor([[0] + list(itertools.accumulate(p)) for p in per], dtype=torch.int64)

    def forward(self, offsets=None, x_rows=None, status=0, x=None):
        rows = x_rows or [n + self.spare for n in self.tot]
        if self.out == torch.uint8:
            bufs = [GuardedBuffer((n + self.spare) * M.row_bytes(M.FP8, self.N)) for n in self.tot]
            out = [b.view.reshape(n + self.spare, -1) for b, n in zip(bufs, self.tot)]
        else:
            bufs = [GuardedBuffer((n + self.spare) * self.N * 2, pad=self.pad) for n in self.tot]
            out = [b.view.view(self.out).reshape(n + self.spare, self.N) for b, n in zip(bufs, self.tot)]
        st = torch.full((1,), status, dtype=torch.int32, device="cuda")
        act = ACTS[self.act]
        ws = torch.empty(B.moe_expert_linear_mx_workspace_bytes(self.W, self.P, self.K, self.N, act, rows),
                         dtype=torch.uint8, device="cuda").random_()
        B.moe_expert_linear_mx(self.W, self.P, self.K, self.N, self.form, act, [v.cuda() for v in x or self.x], rows,
                               (self.offsets if offsets is None else offsets).cuda(), [w.cuda() for w in self.weight],
                               None if self.bias is None else [b.cuda() for b in self.bias], out, ws, st)
        torch.cuda.synchronize()
        assert all(b.guards_intact() for b in bufs)
        return int(st.item()), [v.cpu() for v in out]

    def spans(self, d):
        at = 0
        for j, n in enumerate(self.per[d]):
            yield j, slice(at, at + n)
            at += n

    def check(self, **kw):
        st, out = self.forward(**kw)
        assert st == 0
        for d in range(self.W):
            for j, s in self.spans(d):
                if s.start == s.stop:
                    continue
                x, w = self.xv[d][s], self.wv[d][j]
                h, mag = x @ w.t(), x.abs() @ w.t().abs()
                if self.bias:
                    h, mag = h + self.bias[d][j].double(), mag + self.bias[d][j].double().abs()
                # a sum of K products in fp32 in any order, one step of the running sum for
                # each; whole numbers below 2^24 have none
                if self.whole:
                    assert mag.max() < 2 ** 23
                err = mag * 0 if self.whole else mag * (2 * self.K + 8) * 2.0 ** -24
                y = R.activate(self.act, h)
                # slopes: |silu'|, |gelu'| < 1.13, |relu'| <= 1; fp32 steps of the activation itself
                if self.act == "swiglu":
                    g, u = h.chunk(2, -1)
                    eg, eu = err.chunk(2, -1)
                    err = 1.13 * eg * u.abs() + g.abs() * eu + 1.13 * eg * eu + (g * u).abs() * (g.abs() + 16) * 2.0 ** -23
                elif self.act in ("gelu", "silu"):
                    err = 1.13 * err + h.abs() * (h.abs() + 16) * 2.0 ** -23
                self.compare(out[d][s], y, err, (d, j))
            assert (out[d][self.tot[d]:].view(torch.uint8) == SENT).all()
        return out

    def compare(self, got, y, err, at):
        if self.out != torch.uint8:
            half = R.half_step(self.out)
            tiny = torch.finfo(self.out).smallest_normal * half * 2
            far = (got.double() - y).abs() > err + y.abs() * half * (1.01 if not self.whole else 1) + tiny
            assert not far.any(), (at, far.nonzero()[:4].tolist(), int(far.sum()), far.numel())
            return
        n = M.used_bytes(M.FP8, self.N)
        assert (got[:, n:] == SENT).all()
        if not err.any():
            want = M.quantize(y, M.FP8)
            assert torch.equal(got[:, :n], want), (at, (got[:, :n] != want).nonzero()[:4].tolist())
            return
        # what is off by err may land on the next element, or have the next scale: elements
        # between those of y - err and y + err under the scale that was written
        assert not got[:, M.padded(self.N) + -(-self.N // 32):n].any()
        assert not got[:, self.N:M.padded(self.N)].any()
        pad = M.padded(self.N) - self.N
        b = lambda v: torch.nn.functional.pad(v, (0, pad)).reshape(len(y), M.padded(self.N) // 32, 32)  # noqa: E731
        byte = got[:, M.padded(self.N):n].double()
        top = b(y).abs()
        k = lambda m: torch.floor(torch.log2(m.clamp(min=1e-300))).clamp(min=-119) + 119  # noqa: E731
        assert (byte >= k((top - b(err)).clamp(min=0).amax(-1))).all() and (byte <= k((top + b(err)).amax(-1))).all()
        unit = torch.pow(torch.tensor(2.0, dtype=torch.float64), byte - 127)[..., None]
        v = b(M.values(got, M.FP8, self.N)) / unit
        lo, hi = ((b(y) + e * b(err)) / unit for e in (-1, 1))
        # half a step of e4m3 around both ends: 2^-4 of the value, 2^-10 below 2^-6
        off = lambda u: torch.maximum(u.abs() / 16, torch.tensor(2.0 ** -10, dtype=torch.float64)) * (1 + 1e-9)  # noqa: E731
        lo, hi = lo - off(lo), hi + off(hi)
        far = (v < lo.clamp(max=448)) | (v > hi.clamp(min=-448))
        assert not far.any(), (at, far.nonzero()[:4].tolist(), int(far.sum()))


def _seed(*a):
    return zlib.crc32(repr(a).encode())


@pytest.mark.parametrize("out", OUTS)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("form", FORMATS)
def test_products(form, act, out):
    Experts([[3, 0, 70, 130], [1, 65, 0, 0]], 520, 200, form, act, out, _seed(form, act, out)).check()


@pytest.mark.parametrize("K,N", [(1, 1), (31, 5), (32, 33), (256, 256), (257, 264), (1000, 711), (2304, 100), (640, 1030)])
@pytest.mark.parametrize("form", FORMATS)
def test_sizes(form, K, N):
    for act, out in (("none", "bf16"), ("swiglu", "fp8"), ("swiglu", "fp16")):
        Experts([[5, 0, 33], [0, 17, 1]], K, N, form, act, out, _seed(form, K, N, act)).check()


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 31, 64, 65, 129, 257, 700])
@pytest.mark.parametrize("form", FORMATS)
def test_whole_numbers(form, rows):
    """Sums without a rounding: every product has to be there, once."""
    for K, N, act, out in ((1300, 264, "none", "bf16"), (300, 130, "relu", "fp8"), (513, 1000, "none", "fp16"),
                           (4096, 96, "relu", "fp8"), (4608, 40, "none", "bf16")):
        Experts([[rows, 3]], K, N, form, act, out, _seed(form, rows, K), whole=True).check()


@pytest.mark.parametrize("form", FORMATS)
@pytest.mark.parametrize("steps", range(1, 15))
def test_contraction_steps(form, steps):
    """1 to 14 steps of 256 elements, on tiles of every size."""
    for per in ([[300, 270]], [[150, 90]], [[20, 0, 7]]):
        Experts(per, steps * 256 - 3, 520, form, "none", "bf16", _seed(form, steps), whole=True).check()


@pytest.mark.parametrize("form", FORMATS)
def test_one_token(form):
    """A decoded token's experts, long rows, rows of a rank without any."""
    per = [[0] * 16, [0] * 16]
    for e in (0, 3, 7, 15):
        per[0][e] = 1
    per[1][5] = 2
    for act, out in (("swiglu", "fp8"), ("gelu", "bf16"), ("none", "fp16")):
        Experts(per, 4500, 200, form, act, out, _seed(form, act)).check()
        Experts(per, 7168, 96, form, act, out, _seed(form, act, 1), bias=False, spare=0).check()
    Experts(per, 4500, 203, form, "none", "bf16", _seed(form), whole=True).check()


def test_odd_bases():
    for out in ("bf16", "fp16"):
        Experts([[40, 3], [0, 90]], 300, 200, "fp8", "silu", out, 5, pad=2).check()


@pytest.mark.parametrize("form", FORMATS)
def test_nan_blocks_stay_where_they_are(form):
    e = Experts([[4, 40, 3]], 600, 96, form, "none", "bf16", 11)
    x = e.x[0].clone()
    at = M.padded(600) // (1 if e.form == M.FP8 else 2)
    x[7, at + 2] = 255            # a block of one row of expert 1
    e.weight[0][96 * 2 + 5, M.padded(600) // 2 + 18] = 255  # one of a row of expert 2's weights
    st, out = e.forward(x=[x])
    assert st == 0
    want = torch.zeros(47, 96, dtype=torch.bool)
    want[7], want[44:, 5] = True, True
    assert torch.equal(torch.isnan(out[0][:47].float()), want)
    if e.form == M.FP8:           # an element that is NaN
        e = Experts([[2, 3]], 64, 40, form, "relu", "fp8", 12, bias=False)
        e.x[0][3, 63] = 127
        st, out = e.forward()
        assert st == 0 and [bool((r[256:258] == 255).all()) for r in out[0][:5]] == [False, False, False, True, False]


def test_infinite_sums():
    """fp32 sums past its range, and outputs past fp16's."""
    e = Experts([[3]], 64, 32, "fp8", "none", "fp8", 13, bias=False)
    e.x[0][1, 256:258] = 254
    e.x[0][1, :64] = 0x7E
    e.weight[0][:, :32] = 0x77
    e.weight[0][:, 128:130] = 250
    st, out = e.forward()
    assert st == 0 and int(out[0][1, 256]) == 255 and not (out[0][1, :32]).any()
    e = Experts([[2]], 32, 8, "fp4", "none", "fp16", 14, bias=False, whole=True)
    e.weight[0][:, 128] = 160
    st, out = e.forward()
    assert st == 0 and torch.isinf(out[0][:2]).any()


def test_bad_offsets_and_a_set_status():
    e = Experts([[4, 40, 3], [2, 0, 1]], 300, 64, "fp8", "none", "bf16", 21)
    off = e.offsets.clone()
    for at, v, want in (((0, 0), 1, B.ST_BAD_OFFSETS), ((1, 1), 3, B.ST_BAD_OFFSETS), ((0, 3), 60, B.ST_SEND_OVERRUN),
                        ((1, 2), -1, B.ST_BAD_OFFSETS)):
        o = off.clone()
        o[at] = v
        st, out = e.forward(offsets=o)
        assert st == want and all((x.view(torch.uint8) == SENT).all() for x in out)
    st, out = e.forward(status=B.ST_BAD_PERM)
    assert st == B.ST_BAD_PERM and all((x.view(torch.uint8) == SENT).all() for x in out)


def test_many_experts():
    per = [[(7 * i) % 5 for i in range(1024)], [(3 * i) % 4 for i in range(1024)]]
    Experts(per, 100, 24, "fp8", "none", "bf16", 31, whole=True).check()


def test_refusals():
    e = Experts([[4, 3]], 300, 64, "fp8", "none", "bf16", 41, bias=False, spare=0)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    x, w, off = e.x[0].cuda(), e.weight[0].cuda(), e.offsets.cuda()
    out = torch.zeros(7, 64, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(B.moe_expert_linear_mx_workspace_bytes(1, 2, 300, 64, 0, [7]), dtype=torch.uint8, device="cuda")
    ok = dict(W=1, P=2, K=300, N=64, x_format=B.MX_FP8, act=0, x=[x], x_rows=[7], expert_offsets=off, weight=[w],
              bias=None, out=[out], workspace=ws, status=st)
    for kw in (dict(x_format=1), dict(x=[x[:6]]), dict(x=[x.float()]), dict(x_rows=[8]), dict(x_rows=[7, 7]),
               dict(P=3), dict(K=600), dict(N=65), dict(act=7), dict(weight=[w[:100]]), dict(weight=[w.float()]),
               dict(bias=[torch.zeros(2, 64, device="cuda").half()]), dict(bias=[torch.zeros(2, 63, device="cuda")]),
               dict(out=[out.float()]), dict(out=[out[:6]]), dict(workspace=ws[:-1]), dict(expert_offsets=off.int()),
               dict(out=[x], N=200), dict(x=[x.cpu()])):
        with pytest.raises((ValueError, B.A2avError)):
            B.moe_expert_linear_mx(**{**ok, **kw})
    B.moe_expert_linear_mx(**ok)
    torch.cuda.synchronize()
    assert int(st.item()) == 0


@pytest.mark.parametrize("form", FORMATS)
@pytest.mark.parametrize("K", [8192, 8193, 8448, 16384, 20000, 24600])
def test_long_contractions_of_few_rows(form, K):
    """More scales of a row than one filling of LDS takes, up to four fillings."""
    Experts([[3, 0, 16, 1], [0, 2, 0, 17]], K, 40, form, "none", "bf16", _seed(form, K), whole=True).check()
    Experts([[1, 0], [2, 5]], K, 24, form, "swiglu", "fp8", _seed(form, K)).check()


def test_offsets_are_checked_without_rows():
    e = Experts([[0, 0], [0, 0]], 300, 64, "fp8", "none", "bf16", 22)
    assert e.forward(x_rows=[0, 0])[0] == 0
    for at, v, want in (((0, 0), 1, B.ST_BAD_OFFSETS), ((1, 2), 1, B.ST_SEND_OVERRUN), ((1, 1), -1, B.ST_BAD_OFFSETS)):
        o = e.offsets.clone()
        o[at] = v
        st, out = e.forward(offsets=o, x_rows=[0, 0])
        assert st == want and all((x.view(torch.uint8) == SENT).all() for x in out)
