"""Every tile of the microscaled products: the tile that a call takes computed by
the library's rule, with last row tiles of every height, 1 to 11 steps of 256
elements, gated and not, on whole numbers whose sums fp32 holds exactly, so
that every output is known to the bit. Products on the GPU in 64 bits."""
import pytest
import torch

import mx_ref as M
from embeddings_a2av_virtual_amd import _binding as B

pytestmark = pytest.mark.gpu

FORMATS = {"fp8": B.MX_FP8, "fp4": B.MX_FP4}
ROWS, COLS = (256, 128, 64), (256, 128, 128)


def tile_of(rows, experts, cols):
    """The library's choice: the largest tile with enough of them that the mean expert half fills."""
    for i in range(2 if rows <= 64 * experts else 1 if rows <= 128 * experts else 0, 2):
        t = ROWS[i]
        tiles = rows // t + (experts // 2 if rows % (experts * t) else 0)
        if tiles * -(-cols // COLS[i]) >= 200:
            return i
    return 2


def whole(n, K, form, g):
    """Rows of small e2m1 values with scales of 1, and the values."""
    v = M.table(M.FP4).cuda()[torch.randint(0, 8, (n, K), generator=g, device="cuda")]
    v = v * (1 - 2 * torch.randint(0, 2, (n, K), generator=g, device="cuda"))
    code = torch.bucketize(v.abs(), M.table(form).cuda()) + (128 if form == M.FP8 else 8) * (v < 0)
    code = torch.nn.functional.pad(code, (0, M.padded(K) - K))
    if form == M.FP4:
        code = code[:, ::2] + 16 * code[:, 1::2]
    rows = torch.full((n, M.row_bytes(form, K)), 255, dtype=torch.uint8, device="cuda")
    rows[:, :code.shape[1]] = code.to(torch.uint8)
    rows[:, code.shape[1]:M.used_bytes(form, K)] = 127
    return rows, v


def run(per, K, N, form, gated, seed, want):
    g = torch.Generator(device="cuda").manual_seed(seed)
    P, R, NW = len(per), sum(per), 2 * N if gated else N
    assert tile_of(R, P, (N + 15) // 16 * 32 if gated else N) == want
    x, xv = whole(R, K, form, g)
    w, wv = whole(P * NW, K, M.FP4, g)
    if gated:  # silu(64) is 64 in fp32: the gate rows give 64 times the first element of x
        wv = wv.reshape(P, NW, K)
        wv[:, :N] = 0
        code = torch.zeros(P * N, M.padded(K) // 2, dtype=torch.uint8, device="cuda")
        w.reshape(P, NW, -1)[:, :N, :M.padded(K) // 2] = code.reshape(P, N, -1)
    wv = wv.reshape(P, NW, K)
    bias = torch.zeros(P, NW, device="cuda")
    if gated:
        bias[:, :N] = 64
    else:
        bias += torch.randint(-3, 4, (P, NW), generator=g, device="cuda")
    off = torch.tensor([[0] + torch.tensor(per).cumsum(0).tolist()], dtype=torch.int64, device="cuda")
    out = torch.full((R + 1, N), 7.0, dtype=torch.bfloat16, device="cuda")
    act = B.ACT_SWIGLU if gated else B.ACT_NONE
    ws = torch.empty(B.moe_expert_linear_mx_workspace_bytes(1, P, K, N, act, [R]), dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.moe_expert_linear_mx(1, P, K, N, form, act, [x], [R], off, [w], [bias], [out], ws, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and (out[R] == 7).all()
    at = 0
    for e, n in enumerate(per):
        h = xv[at:at + n] @ wv[e].t() + bias[e].double()
        y = h[:, :N] * h[:, N:] if gated else h
        assert (y.abs() < 2 ** 24).all()
        far = out[at:at + n] != y.float().to(torch.bfloat16)
        assert not far.any(), (e, n, far.nonzero()[:4].tolist(), int(far.sum()))
        at += n


@pytest.mark.parametrize("form", FORMATS)
@pytest.mark.parametrize("macros", range(1, 12))
def test_largest_tiles(form, macros):
    # last tiles of 1, 64, 65, 128, 129 and 256 rows, and experts of fewer
    per = [257, 320, 321, 384, 385, 512, 1, 0, 63]
    run(per, macros * 256 - 5, 6008, FORMATS[form], False, macros, 0)


@pytest.mark.parametrize("form", FORMATS)
@pytest.mark.parametrize("macros", [1, 4, 5, 9])
def test_largest_tiles_gated(form, macros):
    run([300, 256, 40, 513, 0, 100], macros * 256, 4000, FORMATS[form], True, macros, 0)


@pytest.mark.parametrize("form", FORMATS)
@pytest.mark.parametrize("macros", [1, 2, 3, 4, 5, 8, 10])
def test_middle_tiles(form, macros):
    run([129, 192, 193, 256, 1, 0, 64], macros * 256 - 7, 3000, FORMATS[form], False, macros, 1)
    run([129, 60, 200], macros * 256 - 7, 3500, FORMATS[form], True, macros, 1)


@pytest.mark.parametrize("form", FORMATS)
@pytest.mark.parametrize("macros", [1, 2, 3, 4, 5, 8, 10])
def test_smallest_tiles(form, macros):
    run([65, 32, 33, 64, 1, 0, 128], macros * 256 - 9, 330, FORMATS[form], False, macros, 2)
    run([70, 60, 3], macros * 256 - 9, 250, FORMATS[form], True, macros, 2)
