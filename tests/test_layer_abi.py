"""Argument errors of the layer's calls that the C ABI reports before any HIP
call is made, and their workspace sizes (no GPU needed)."""
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


def test_route(L):
    p, one = _ptrs(16, 16), ctypes.c_float(1.0)

    def call(W=2, T=4, k=2, E=8, type=0, score=0, z=p, bias=None, groups=1, kept=1, top=1, ids=p, w=p, st=vp(16)):
        return L.moe_route(W, T, k, E, type, score, z, bias, groups, kept, top, 1, one, ids, w, st, None)

    for kw in (dict(W=0), dict(W=65), dict(T=-1), dict(k=0), dict(k=9), dict(E=0), dict(E=4097, k=1), dict(type=3),
               dict(type=-1), dict(score=2), dict(groups=0), dict(groups=3), dict(groups=4, kept=0),
               dict(groups=4, kept=5), dict(groups=4, kept=1, k=3), dict(top=0), dict(top=3),
               dict(groups=8, kept=8, top=2), dict(z=None), dict(ids=None), dict(w=None), dict(st=None),
               dict(z=_ptrs(16, None)), dict(ids=_ptrs(None, 16)), dict(w=_ptrs(16, None)),
               dict(T=1 << 30, k=2), dict(T=1 << 62, k=2), dict(E=4096, k=65),
               dict(E=4096, groups=128, kept=2, k=2)):
        assert call(**kw) == EARG, kw
    assert call(T=0, z=_ptrs(None, None), ids=_ptrs(None, None), w=_ptrs(None, None)) == 0


def test_route_backward(L):
    p, one = _ptrs(16, 16), ctypes.c_float(1.0)

    def call(W=2, T=4, k=2, E=8, type=0, score=0, z=p, ids=p, w=p, dw=p, dz=p, st=vp(16)):
        return L.moe_route_backward(W, T, k, E, type, score, z, ids, w, 1, one, dw, dz, st, None)

    for kw in (dict(W=0), dict(T=-1), dict(k=65, E=4096), dict(E=0), dict(type=3), dict(score=-1), dict(z=None),
               dict(ids=None), dict(w=None), dict(dw=None), dict(dz=None), dict(st=None), dict(dz=_ptrs(16, None)),
               dict(dw=_ptrs(None, 16)), dict(T=1 << 31, k=1)):
        assert call(**kw) == EARG, kw
    assert call(T=0) == 0


def test_combine_backward(L):
    p = _ptrs(16, 16)
    need = L.moe_combine_backward_workspace_bytes(2, 10, 2)
    assert need >= 2 * 10 * 2 * 4
    for bad in ((0, 10, 2), (65, 10, 2), (2, -1, 2), (2, 10, 0), (2, 1 << 30, 2)):
        assert L.moe_combine_backward_workspace_bytes(*bad) == 0

    def call(W=2, T=10, k=2, H=8, a=(p,) * 6, ws=vp(256), n=need, st=vp(16)):
        return L.moe_combine_backward(W, T, k, H, *a, ws, n, st, None)

    for kw in (dict(W=0), dict(T=-1), dict(k=0), dict(H=0), dict(H=1 << 62), dict(n=need - 1), dict(ws=None), dict(st=None)):
        assert call(**kw) == EARG, kw
    for i in range(6):
        for x in (None, _ptrs(16, None)):
            a = [p] * 6
            a[i] = x
            assert call(a=a) == EARG
    assert call(T=0) == 0


def test_combine_return_backward(L):
    p, r = _ptrs(16, 16), _rows(20, 20)
    need = L.moe_combine_return_backward_workspace_bytes(2, 10, 2, 8)
    assert need > L.moe_combine_return_workspace_bytes(2, 10, 2, 8)
    assert L.moe_combine_return_backward_workspace_bytes(3, 10, 2, 8) == 0

    def call(W=2, T=10, k=2, E=8, H=8, counts=vp(16), a=(p, p, p, r, p, p, p, p), layout=1, ws=vp(256), n=need,
             st=vp(16)):
        return L.moe_combine_return_backward(W, T, k, E, H, counts, *a, layout, ws, n, st, None)

    for kw in (dict(W=3), dict(T=-1), dict(k=0), dict(H=0), dict(layout=2), dict(layout=-1), dict(counts=None),
               dict(n=need - 1), dict(ws=None), dict(st=None), dict(H=1 << 62)):
        assert call(**kw) == EARG, kw
    for i in range(8):
        for x in (None, _rows(20, -1) if i == 3 else _ptrs(16, None)):
            a = [p, p, p, r, p, p, p, p]
            a[i] = x
            assert call(a=a) == EARG, i


def test_expert_linear(L):
    p, q, s, r = _ptrs(16, 16), _ptrs(32, 32), _ptrs(48, 48), _rows(20, 0)
    need = L.moe_expert_linear_workspace_bytes(2, 4, 64, 32, 0, r)
    assert need > 0
    for bad in ((0, 4, 64, 32, 0, r), (2, 0, 64, 32, 0, r), (2, 2049, 64, 32, 0, r), (2, 4, 0, 32, 0, r),
                (2, 4, 64, 0, 0, r), (2, 4, (1 << 20) + 1, 32, 0, r), (2, 4, 64, (1 << 20) + 1, 0, r),
                (2, 4, 64, 32, 5, r), (2, 4, 64, 32, -1, r), (2, 4, 64, 32, 0, _rows(20, -1)),
                (2, 4, 64, 32, 0, _rows(20, (1 << 30) + 1)), (2, 4, 64, 32, 0, None)):
        assert L.moe_expert_linear_workspace_bytes(*bad) == 0
        assert L.moe_expert_linear_backward_workspace_bytes(*bad) == 0

    def call(type=1, act=0, x=p, rows=r, off=vp(16), w=p, bias=None, res=None, out=q, pre=None, ws=vp(256), n=need,
             st=vp(16)):
        return L.moe_expert_linear(2, 4, 64, 32, type, act, x, rows, off, w, bias, res, out, pre, ws, n, st, None)

    half = _ptrs(None, 16)
    for kw in (dict(type=0), dict(type=3), dict(act=5), dict(x=None), dict(rows=None), dict(off=None), dict(w=None),
               dict(out=None), dict(ws=None), dict(ws=vp(260)), dict(n=need - 1), dict(st=None), dict(x=half),
               dict(w=_ptrs(16, None)), dict(bias=half), dict(res=half), dict(out=half), dict(pre=half),
               dict(out=p), dict(pre=p), dict(pre=q), dict(pre=s, res=s)):
        assert call(**kw) == EARG, kw


def test_expert_linear_backward(L):
    p, q, s, r = _ptrs(16, 16), _ptrs(32, 32), _ptrs(48, 48), _rows(20, 0)
    need = L.moe_expert_linear_backward_workspace_bytes(2, 4, 64, 32, 3, r)
    assert need > L.moe_expert_linear_workspace_bytes(2, 4, 64, 32, 3, r)

    def call(type=1, act=3, x=p, off=vp(16), w=p, pre=p, g=p, dpre=q, dx=s, dw=p, db=p, ws=vp(256), n=need, st=vp(16)):
        return L.moe_expert_linear_backward(2, 4, 64, 32, type, act, x, r, off, w, pre, g, dpre, dx, dw, db, ws, n,
                                            st, None)

    half = _ptrs(None, 16)
    for kw in (dict(type=0), dict(act=9), dict(x=None), dict(off=None), dict(w=None), dict(pre=None), dict(g=None),
               dict(dpre=None), dict(act=0), dict(act=0, pre=None), dict(act=0, dpre=None), dict(ws=None),
               dict(n=need - 1), dict(st=None), dict(x=half), dict(pre=half), dict(g=half), dict(dpre=half),
               dict(dx=half), dict(dw=half), dict(db=half), dict(dx=p), dict(dx=q), dict(dpre=p),
               dict(act=0, pre=None, dpre=None, g=s)):
        assert call(**kw) == EARG, kw
