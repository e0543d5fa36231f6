"""The router (moe_route) and its gradient (moe_route_backward) against their
definitions in 64 bits: ids equal, weights and gradients within the rounding
of the fp32 steps they take."""
import math
import zlib

import pytest
import torch

import layer_ref as R
from embeddings_a2av_virtual_amd import _binding as B
from gpu_util import GuardedBuffer

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def _guarded(shape, dtype):
    n = math.prod(shape) * torch.empty(0, dtype=dtype).element_size()
    b = GuardedBuffer(n)
    return b, b.view.view(dtype).reshape(shape)


def gpu_route(z, sigmoid, bias, groups, topk_groups, group_top, k, renorm, scale, status=0, stream=None):
    """z: list of [T, E] host tensors."""
    W, (T, E) = len(z), z[0].shape
    ib, ids = zip(*[_guarded((T, k), torch.int32) for _ in range(W)])
    wb, w = zip(*[_guarded((T, k), torch.float32) for _ in range(W)])
    st = torch.full((1,), status, dtype=torch.int32, device="cuda")
    B.moe_route(W, T, k, E, B.SCORE_SIGMOID if sigmoid else B.SCORE_SOFTMAX, [x.cuda() for x in z],
                None if bias is None else bias.cuda(), groups, topk_groups, group_top, renorm, scale,
                list(ids), list(w), st, stream)
    torch.cuda.synchronize()
    assert all(b.guards_intact() for b in ib + wb)
    return int(st.item()), [x.cpu() for x in ids], [x.cpu() for x in w]


def weight_rtol(z, E):
    """Relative error of an fp32 weight: z - max and the exponential's argument
    are off by up to |z - max| half steps each, the exponential, the sums (at
    most E / 16 terms in a row, then a tree), a reciprocal and two products by
    a few steps more."""
    span = float((z[torch.isfinite(z)].max() - z[torch.isfinite(z)].min()).item()) if torch.isfinite(z).any() else 0
    span = max(span, float(z[torch.isfinite(z)].abs().max().item())) if torch.isfinite(z).any() else 0
    return (4 * span + E / 8 + 32) * 2.0 ** -24


def check_route(z, sigmoid, bias, groups, topk_groups, group_top, k, renorm, scale):
    st, ids, w = gpu_route(z, sigmoid, bias, groups, topk_groups, group_top, k, renorm, scale)
    assert st == 0
    for r, x in enumerate(z):
        rid, rw = R.route(x.double(), sigmoid, bias, groups, topk_groups, group_top, k, renorm, scale)
        bad = (ids[r] != rid).any(-1).nonzero().reshape(-1)
        assert bad.numel() == 0, f"rank {r}: token {int(bad[0])}: {ids[r][bad[0]]} != {rid[bad[0]]}"
        assert torch.equal(torch.isnan(w[r]), torch.isnan(rw))
        fine = ~torch.isnan(rw)
        # weights below fp32's normal range are held to its smallest step
        tol = rw[fine].abs() * weight_rtol(x.double(), x.shape[1]) + 2.0 ** -125 * abs(scale)
        assert ((w[r].double()[fine] - rw[fine]).abs() <= tol).all()
    return ids, w


CASES = [
    # W, T, E, k, groups, topk_groups, group_top
    (1, 1, 256, 8, 8, 4, 2),
    (2, 67, 256, 8, 1, 1, 1),
    (1, 33, 256, 8, 8, 4, 1),
    (3, 41, 60, 4, 1, 1, 1),
    (1, 19, 60, 6, 4, 2, 2),
    (1, 7, 1, 1, 1, 1, 1),
    (1, 9, 2, 2, 2, 2, 1),
    (1, 23, 17, 5, 1, 1, 1),
    (1, 11, 63, 9, 9, 3, 2),
    (2, 5, 64, 64, 1, 1, 1),
    (1, 13, 300, 10, 3, 2, 2),
    (1, 6, 1024, 64, 64, 9, 2),
    (1, 5, 1025, 7, 1, 1, 1),
    (1, 3, 4096, 16, 16, 5, 2),
    (1, 21, 8, 2, 1, 1, 1),
    (1, 29, 128, 1, 1, 1, 1),
]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
def test_route_matches_definition(case, sigmoid, kind):
    W, T, E, k, groups, topk_groups, group_top = case
    g = torch.Generator().manual_seed(zlib.crc32(repr((case, sigmoid, kind)).encode()))
    for bias, renorm, scale in ((None, True, 1.0), (0.1 * torch.randn(E, generator=g), True, 2.5),
                                (0.1 * torch.randn(E, generator=g), False, 1.0), (None, False, 0.5)):
        z = [(1.5 * torch.randn(T, E, generator=g)).to(TYPES[kind]) for _ in range(W)]
        check_route(z, sigmoid, bias, groups, topk_groups, group_top, k, renorm, scale)


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [None, "zero", "steps"])
@pytest.mark.parametrize("groups", [(1, 1, 1), (8, 3, 2), (8, 3, 1)], ids=str)
def test_route_ties_go_to_the_lowest_id(kind, sigmoid, bias, groups):
    """Few distinct logits, so that equal scores decide most choices."""
    g = torch.Generator().manual_seed(11)
    T, E = 50, 256
    z = torch.randint(-2, 3, (T, E), generator=g).to(TYPES[kind])
    z[0] = 0
    b = {None: None, "zero": torch.zeros(E), "steps": 0.125 * torch.randint(0, 2, (E,), generator=g)}[bias]
    check_route([z], sigmoid, b, *groups, 8, True, 1.0)


def test_route_neighbouring_values():
    """Keys one fp32 step apart, and logits that differ in their last bit."""
    g = torch.Generator().manual_seed(12)
    T, E = 64, 256
    base = torch.randn(T, 1, generator=g)
    z = base + torch.randint(0, 5, (T, E), generator=g) * 2.0 ** -23 * base.abs()
    check_route([z], False, None, 1, 1, 1, 8, True, 1.0)
    check_route([z], True, 0.01 * torch.randint(0, 2, (E,), generator=g), 8, 4, 2, 8, True, 1.0)
    b = 1e-7 * torch.randn(E, generator=g)
    check_route([z], True, b, 1, 1, 1, 8, False, 1.0)


@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [(1, 1, 1), (4, 2, 2)], ids=str)
@pytest.mark.parametrize("E", [64, 60, 1028])
def test_route_masks_infinities_and_nan(sigmoid, groups, E):
    g = torch.Generator().manual_seed(13)
    T, k = 24, 6
    z = torch.randn(T, E, generator=g)
    z[0] = -math.inf                               # nothing left
    z[1, 5:] = -math.inf                           # fewer than k left
    z[2, torch.randperm(E, generator=g)[: E // 2]] = -math.inf
    z[3, 7] = math.nan
    z[4, 3] = math.inf
    z[5] = torch.finfo(torch.float32).min          # the type's lowest value
    z[6, ::2] = torch.finfo(torch.float32).min
    z[7] *= 40                                     # saturated sigmoids
    z[8] = -200.0                                  # scores under fp32's range
    z[9] = -math.inf
    z[9, E - 1] = 0.0
    bias = 0.1 * torch.randn(E, generator=g)
    for b in (None, bias):
        for renorm in (True, False):
            check_route([z], sigmoid, b, *groups, k, renorm, 1.0)
    bias[2], bias[9], bias[11] = -math.inf, math.nan, math.inf
    check_route([z], sigmoid, bias, *groups, k, True, 1.0)


@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("E", [32, 256, 512])
def test_route_groups_whose_best_scores_are_equal_in_double(E, kind, sigmoid):
    """Groups by their best expert, whose logits differ where the scores do not:
    the lowest group is kept, not the one with the larger logit."""
    g = torch.Generator().manual_seed(14)
    T, groups = 16, 8
    per = E // groups
    z = torch.randn(T, E, generator=g).clamp(-2, 2)
    best = torch.zeros(T, groups)
    best[0] = 40.0 + torch.arange(groups)          # sigmoid 1
    best[1] = 6.0
    best[2] = torch.tensor([5, 6, 7, 8, 6, 7, 5, 6.0])
    best[3] = torch.tensor([36, 50, 3, 37, 60, 38, 2, 40.0])
    z[4] = z[5] = z[6] = -1000.0
    best[4] = -900.0 + torch.arange(groups)        # sigmoid 0
    best[5] = -800.0 - 10 * torch.arange(groups)
    best[5, 6] = 5.0                               # softmax 0 beside it
    best[6] = -5e-7 * torch.arange(groups)
    z[7:10] = -3.0
    best[7] = 1e-7 * torch.arange(groups)          # about 1 / 2
    best[8] = torch.tensor([0, 6e-8, 0, 1.2e-7, 1e-3, 0, 2e-7, 0])
    best[9] = torch.tensor([-math.inf, 1, -math.inf, 0, -math.inf, -math.inf, -math.inf, -math.inf])
    z[9].view(groups, per)[[0, 2, 4, 5, 6, 7]] = -math.inf
    best[10] = 16.0 + 2.0 ** -6 * torch.arange(groups)
    best[11] = 30.0 + 2.0 ** -5 * torch.arange(groups)
    best[12] = 2.5 + 2.0 ** -6 * torch.arange(groups)
    best[13] = torch.tensor([3, 3, 90, 3, 3, 80, 3, 3.0])
    best[14] = 700.0 * torch.arange(groups).flip(0)
    best[15] = 20.0
    z.view(T, groups, per)[:, :, 1] = best
    z = z.to(TYPES[kind])
    for topk_groups in (1, 3, 6):
        k = min(5, topk_groups * per)
        check_route([z], sigmoid, None, groups, topk_groups, 1, k, True, 1.0)
        check_route([z], sigmoid, torch.zeros(E), groups, topk_groups, 2, k, True, 1.0)


def test_route_poisoned_status_writes_nothing():
    z = torch.randn(4, 16)
    st, ids, w = gpu_route([z], False, None, 1, 1, 1, 2, True, 1.0, status=64)
    assert st == 64 and (ids[0].view(torch.uint8) == 0xA5).all() and (w[0].view(torch.uint8) == 0xA5).all()


def test_route_no_tokens():
    assert gpu_route([torch.zeros(0, 16)], False, None, 1, 1, 1, 2, True, 1.0)[0] == 0


def test_route_unaligned_rows():
    """Logits one element past an aligned base."""
    g = torch.Generator().manual_seed(14)
    for kind in TYPES.values():
        z = torch.randn(9 * 64 + 1, generator=g).to(kind)
        view = z.cuda()[1:].reshape(9, 64)
        ids = torch.empty((9, 4), dtype=torch.int32, device="cuda")
        w = torch.empty((9, 4), device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        B.moe_route(1, 9, 4, 64, B.SCORE_SOFTMAX, [view], None, 1, 1, 1, True, 1.0, [ids], [w], st)
        d = torch.zeros(9 * 64 + 1, dtype=kind, device="cuda")
        B.moe_route_backward(1, 9, 4, 64, B.SCORE_SOFTMAX, [view], [ids], [w], False, 1.0,
                             [torch.ones_like(w)], [d[1:].reshape(9, 64)], st)
        rid, rw = R.route(z[1:].reshape(9, 64).double(), False, None, 1, 1, 1, 4, True, 1.0)
        assert int(st.item()) == 0 and torch.equal(ids.cpu(), rid)
        assert ((w.cpu().double() - rw).abs() <= rw * weight_rtol(z.double(), 64)).all()
        assert d[0].item() == 0


# ------------------------------------------------------------------ gradient
def gpu_route_grad(z, ids, w, d, sigmoid, renorm, scale, status=0):
    W, (T, E), k = len(z), z[0].shape, ids[0].shape[1]
    buf, out = zip(*[_guarded((T, E), z[0].dtype) for _ in range(W)])
    st = torch.full((1,), status, dtype=torch.int32, device="cuda")
    B.moe_route_backward(W, T, k, E, B.SCORE_SIGMOID if sigmoid else B.SCORE_SOFTMAX, [x.cuda() for x in z],
                         [x.cuda() for x in ids], [x.cuda() for x in w], renorm, scale, [x.cuda() for x in d],
                         list(out), st)
    torch.cuda.synchronize()
    assert all(b.guards_intact() for b in buf)
    return int(st.item()), [x.cpu() for x in out]


def check_route_grad(z, ids, w, d, sigmoid, renorm, scale):
    st, got = gpu_route_grad(z, ids, w, d, sigmoid, renorm, scale)
    assert st == 0
    for r, x in enumerate(z):
        T, E = x.shape
        x64, d64, s = x.double(), d[r].double(), None
        want = R.route_grad(x64, ids[r], d64, sigmoid, renorm, scale)
        # each of the terms that the formula adds up, at its own rounding
        s = torch.sigmoid(x64) if sigmoid else torch.softmax(x64, -1)
        sj = s.gather(-1, ids[r].long())
        S = sj.sum(-1, keepdim=True) if renorm else 1.0
        g = (scale * d64).abs() / S
        g = g + ((g * sj).sum(-1, keepdim=True) / S if renorm else 0)
        size = torch.zeros_like(x64).scatter_add_(-1, ids[r].long(), g)
        if not sigmoid and not renorm:
            size = size + (g * sj).sum(-1, keepdim=True)
        tol = s * size * (weight_rtol(x64, E) + (2 * ids[r].shape[1] + 16) * 2.0 ** -24)
        tol = tol + want.abs() * R.half_step(x.dtype) + torch.finfo(x.dtype).smallest_normal * R.half_step(x.dtype) * 2
        far = (got[r].double() - want).abs() > tol
        assert not far.any(), (r, far.nonzero()[0], got[r][far][0], want[far][0], tol[far][0])


@pytest.mark.parametrize("case", [c[:4] for c in CASES], ids=str)
@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
def test_route_gradient_matches_definition(case, sigmoid, kind):
    W, T, E, k = case
    g = torch.Generator().manual_seed(zlib.crc32(repr((case, sigmoid, kind)).encode()))
    for renorm, scale in ((True, 1.0), (False, 1.0), (True, 2.5), (False, 0.5)):
        z = [(1.5 * torch.randn(T, E, generator=g)).to(TYPES[kind]) for _ in range(W)]
        ids = [torch.rand(T, E, generator=g).topk(k, -1).indices.to(torch.int32) for _ in range(W)]
        w = [R.route_weights(x.double(), i, sigmoid, renorm, scale).float() for x, i in zip(z, ids)]
        d = [torch.randn(T, k, generator=g) for _ in range(W)]
        check_route_grad(z, ids, w, d, sigmoid, renorm, scale)


@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
def test_route_gradient_of_repeated_ids_adds_up(sigmoid):
    g = torch.Generator().manual_seed(21)
    z = [torch.randn(40, 24, generator=g)]
    ids = [torch.randint(0, 5, (40, 6), generator=g).to(torch.int32)]
    for renorm in (True, False):
        w = [R.route_weights(z[0].double(), ids[0], sigmoid, renorm, 1.0).float()]
        check_route_grad(z, ids, w, [torch.randn(40, 6, generator=g)], sigmoid, renorm, 1.0)


def test_route_gradient_of_masked_rows():
    """-inf logits have no gradient; rows with nothing left have none at all."""
    g = torch.Generator().manual_seed(22)
    z = torch.randn(6, 64, generator=g)
    z[0] = -math.inf
    z[1, 3:] = -math.inf
    z[2, ::2] = -math.inf
    for sigmoid in (False, True):
        for renorm in (True, False):
            _, ids, w = gpu_route([z], sigmoid, None, 1, 1, 1, 5, renorm, 1.0)
            st, (got,) = gpu_route_grad([z], ids, w, [torch.randn(6, 5, generator=g)], sigmoid, renorm, 1.0)
            assert st == 0 and (got[0] == 0).all() and (got[z == -math.inf] == 0).all()
            assert torch.isfinite(got).all() and (got[2] != 0).any()


def test_route_gradient_refuses_bad_ids():
    z, d = [torch.randn(9, 16)] * 2, [torch.randn(9, 2)] * 2
    for bad in (-1, 16, 1 << 30):
        ids = [torch.zeros(9, 2, dtype=torch.int32), torch.zeros(9, 2, dtype=torch.int32)]
        ids[1][8, 1] = bad
        st, out = gpu_route_grad(z, ids, [torch.ones(9, 2)] * 2, d, False, True, 1.0)
        assert st == B.ST_BAD_EXPERT and all((x.view(torch.uint8) == 0xA5).all() for x in out)
    assert gpu_route_grad(z, [torch.zeros(9, 2, dtype=torch.int32)] * 2, [torch.ones(9, 2)] * 2, d, False, True,
                          1.0, status=4)[0] == 4


def test_route_argument_checks():
    z, st = torch.randn(4, 16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ids, w = torch.empty((4, 2), dtype=torch.int32, device="cuda"), torch.empty((4, 2), device="cuda")

    def call(z=z, bias=None, ids=ids, w=w, T=4, k=2, E=16, groups=1, kept=1, top=1, score=0):
        B.moe_route(1, T, k, E, score, [z], bias, groups, kept, top, True, 1.0, [ids], [w], st)

    call()
    for kw in (dict(z=z.cpu()), dict(z=z.t()), dict(z=z.double()), dict(ids=ids.long()), dict(w=w.half()),
               dict(T=5), dict(bias=torch.zeros(8, device="cuda")), dict(z=z.int())):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(k=0), dict(groups=3), dict(groups=4, kept=5), dict(groups=8, kept=1, k=3, T=1), dict(top=3),
               dict(groups=16, kept=16, top=2), dict(score=2), dict(kept=0)):
        with pytest.raises(B.A2avError) as e:
            call(**kw)
        assert e.value.code == B.EARG
