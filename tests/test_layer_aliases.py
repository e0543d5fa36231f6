"""Arrays that a call writes while others still read them are refused at the C
ABI, before any HIP call is made (no GPU needed). Every array has a base of its
own but the two in question."""
import ctypes

import pytest

EARG = -1
vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    from embeddings_a2av_virtual_amd import _binding
    return _binding.lib()


def _ptrs(*v):
    return (ctypes.c_void_p * len(v))(*v)


def _rows(*v):
    return (ctypes.c_int64 * len(v))(*v)


def test_gated_gradient_over_d_out(L):
    """SwiGLU's d_pre has rows twice as wide as d_out's: row r lands on rows
    that other workgroups have not read."""
    bases = {n: _ptrs(1 << 20 | i << 12, 1 << 21 | i << 12) for i, n in
             enumerate(("x", "w", "pre", "d_out", "d_pre", "d_x", "d_w", "d_b"))}
    r = _rows(20, 7)
    need = L.moe_expert_linear_backward_workspace_bytes(2, 4, 64, 32, 4, r)

    def call(**kw):
        b = dict(bases, **kw)
        return L.moe_expert_linear_backward(2, 4, 64, 32, 1, 4, b["x"], r, vp(1 << 22), b["w"], b["pre"], b["d_out"],
                                            b["d_pre"], b["d_x"], b["d_w"], b["d_b"], vp(1 << 23), need, vp(1 << 24),
                                            None)

    assert call(d_pre=bases["d_out"]) == EARG
    assert call(d_pre=_ptrs(bases["d_pre"][0], bases["d_out"][1])) == EARG
    assert call(d_pre=bases["x"]) == EARG and call(d_x=bases["d_pre"]) == EARG


def test_combine_gradient_over_d_out(L):
    """d_out's rows are read for all of a token's slots, by waves of their own."""
    names = ("back", "perm", "w", "d_out", "d_back", "d_w")
    b = {n: _ptrs(1 << 20 | i << 12, 1 << 21 | i << 12) for i, n in enumerate(names)}
    need = L.moe_combine_backward_workspace_bytes(2, 10, 2)
    own_need = L.moe_combine_return_backward_workspace_bytes(2, 10, 2, 8)

    def call(**kw):
        a = dict(b, **kw)
        return L.moe_combine_backward(2, 10, 2, 8, *(a[n] for n in names), vp(1 << 23), need, vp(1 << 24), None)

    def call_owners(rows=_rows(20, 20), **kw):
        a = dict(b, **kw)
        return L.moe_combine_return_backward(2, 10, 2, 8, 8, vp(1 << 22), b["perm"], a["perm"], a["back"], rows, a["w"],
                                             a["d_out"], a["d_back"], a["d_w"], 1, vp(1 << 23), own_need, vp(1 << 24),
                                             None)

    g, d = b["d_out"], b["d_back"]
    for over in (g, _ptrs(d[0], g[1]), _ptrs(g[1], d[1]), _ptrs(g[0], d[1])):
        assert call(d_back=over) == EARG
        assert call_owners(d_back=over) == EARG
    assert call_owners(d_back=_ptrs(d[0], g[0]), rows=_rows(0, 20)) == EARG
