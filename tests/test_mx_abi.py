"""Argument errors of the microscaled layer's calls that the C ABI reports
before any HIP call is made, and their sizes (no GPU needed)."""
import ctypes

import pytest

import mx_ref as M

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


def test_row_bytes(L):
    for form in (M.FP8, M.FP4):
        for H in (1, 31, 32, 255, 256, 257, 1000, 2048, 7168, 1 << 20):
            assert L.moe_mx_row_bytes(form, H) == M.row_bytes(form, H)
        assert L.moe_mx_row_bytes(form, 0) == 0 and L.moe_mx_row_bytes(form, (1 << 20) + 1) == 0
    assert L.moe_mx_row_bytes(2, 64) == 0 and L.moe_mx_row_bytes(5, 64) == 0


@pytest.mark.parametrize("name", ["moe_mx_quantize", "moe_mx_dequantize"])
def test_conversions(L, name):
    p, q, n = _ptrs(16, 32), _ptrs(48, 64), _rows(4, 4)
    wide, narrow = (q, p) if name == "moe_mx_quantize" else (p, q)

    def call(W=2, H=64, type=1, form=3, a=p, rows=n, b=q, st=vp(16)):
        return getattr(L, name)(W, H, type, form, a, rows, b, st, None)

    for kw in (dict(W=0), dict(W=65), dict(H=0), dict(H=(1 << 20) + 1), dict(type=3), dict(type=-1), dict(form=2),
               dict(form=5), dict(a=None), dict(b=None), dict(rows=None), dict(st=None), dict(a=_ptrs(16, None)),
               dict(b=_ptrs(None, 64)), dict(rows=_rows(4, -1)), dict(rows=_rows(1 << 31, 0)),
               dict(H=257, rows=_rows(1 << 30, 0)), dict(a=q)):
        assert call(**kw) == EARG, kw
    assert call(**({"b": _ptrs(48, 68)} if name == "moe_mx_quantize" else {"a": _ptrs(16, 36)})) == EARG
    assert call(rows=_rows(0, 0), a=_ptrs(None, None), b=_ptrs(None, None)) == 0


def test_rms_norm(L):
    x, r, s, o, m = (_ptrs(16 * i, 16 * i) for i in range(1, 6))

    def call(W=2, T=4, H=64, type=1, eps=1e-6, x=x, residual=r, weight=vp(16), sum=s, out=o, rows=m, form=3, st=vp(16)):
        return L.moe_rms_norm(W, T, H, type, ctypes.c_double(eps), x, residual, weight, sum, out, rows, form, st, None)

    half = _ptrs(16, None)
    for kw in (dict(W=0), dict(W=65), dict(T=-1), dict(T=(1 << 30) + 1), dict(H=0), dict(H=(1 << 20) + 1), dict(type=3),
               dict(eps=-1e-9), dict(eps=float("nan")), dict(x=None), dict(weight=None), dict(st=None),
               dict(out=None, rows=None), dict(residual=None), dict(form=2), dict(form=5), dict(x=half),
               dict(residual=half), dict(sum=half), dict(out=half), dict(rows=half), dict(rows=_ptrs(80, 84)),
               dict(rows=x), dict(rows=r), dict(rows=s), dict(rows=o), dict(sum=o)):
        assert call(**kw) == EARG, kw
    none = _ptrs(None, None)
    assert call(T=0, x=none, residual=none, sum=none, out=none, rows=none) == 0


def test_rms_norm_backward(L):
    x, g, s, d = (_ptrs(16 * i, 16 * i) for i in range(1, 5))
    need = L.moe_rms_norm_backward_workspace_bytes(2, 10, 64)
    assert need >= 20 * 64 * 4
    for bad in ((0, 10, 64), (65, 10, 64), (2, -1, 64), (2, (1 << 30) + 1, 64), (2, 10, 0), (2, 10, (1 << 20) + 1)):
        assert L.moe_rms_norm_backward_workspace_bytes(*bad) == 0

    def call(W=2, T=10, H=64, type=1, eps=1e-6, x=x, weight=vp(16), d_out=g, d_sum=s, d_x=d, dw=vp(16), ws=vp(256),
             n=need, st=vp(16)):
        return L.moe_rms_norm_backward(W, T, H, type, ctypes.c_double(eps), x, weight, d_out, d_sum, d_x, dw, ws, n, st,
                                       None)

    half = _ptrs(16, None)
    for kw in (dict(W=0), dict(T=-1), dict(H=0), dict(type=3), dict(eps=-1.0), dict(x=None), dict(weight=None),
               dict(d_out=None), dict(d_x=None), dict(ws=None), dict(ws=vp(264)), dict(n=need - 1), dict(st=None),
               dict(x=half), dict(d_out=half), dict(d_sum=half), dict(d_x=half)):
        assert call(**kw) == EARG, kw
    assert call(T=0, dw=None) == 0


def test_expert_linear_mx(L):
    p, q, w, r = _ptrs(16, 16), _ptrs(32, 32), _ptrs(48, 48), _rows(20, 0)
    need = L.moe_expert_linear_mx_workspace_bytes(2, 4, 64, 32, 0, r)
    assert need > 0
    for bad in ((0, 4, 64, 32, 0, r), (2, 0, 64, 32, 0, r), (2, 2049, 64, 32, 0, r), (2, 4, 0, 32, 0, r),
                (2, 4, 64, 0, 0, r), (2, 4, (1 << 20) + 1, 32, 0, r), (2, 4, 64, (1 << 20) + 1, 0, r),
                (2, 4, 64, 32, 5, r), (2, 4, 64, 32, 0, _rows(20, -1)), (2, 4, 64, 32, 0, _rows(20, (1 << 30) + 1)),
                (2, 4, 64, 32, 0, None)):
        assert L.moe_expert_linear_mx_workspace_bytes(*bad) == 0

    def call(form=3, act=0, x=p, rows=r, off=vp(16), w=w, bias=None, out=q, type=1, ws=vp(256), n=need, st=vp(16)):
        return L.moe_expert_linear_mx(2, 4, 64, 32, form, act, x, rows, off, w, bias, out, type, ws, n, st, None)

    half = _ptrs(None, 16)
    for kw in (dict(form=2), dict(form=1), dict(form=5), dict(act=5), dict(act=-1), dict(x=None), dict(rows=None),
               dict(off=None), dict(w=None), dict(out=None), dict(type=0), dict(type=4), dict(ws=None),
               dict(ws=vp(260)), dict(n=need - 1), dict(st=None), dict(x=half), dict(w=_ptrs(16, None)),
               dict(bias=half), dict(out=half), dict(out=p), dict(x=_ptrs(20, 16)), dict(w=_ptrs(48, 52)),
               dict(type=3, out=_ptrs(36, 32))):
        assert call(**kw) == EARG, kw
