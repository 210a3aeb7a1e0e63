"""CPU checks of the entry points on adapters of many requests and of the
gradient clipping: every call here fails validation, or has nothing to do,
before the library touches the HIP runtime."""
import ctypes as C

import pytest
import torch

import orthogonal_fine_tuning_amd as oft
from orthogonal_fine_tuning_amd import _lib

OK = C.c_void_p(0x100000)
FAR = C.c_void_p(0x4000000000)
OUT = C.c_void_p(0x8000000000)
BAD = C.c_void_p(0x100008)


def _rows(T=4, n=3, order=OK, offsets=OK, tiles=OK):
    r = oft.oft_adapter_rows()
    r.T, r.n = T, n
    r.order, r.offsets, r.tiles = (p.value if p is not None else None for p in (order, offsets, tiles))
    return r


# ------------------------------------------------------------------ rows
@pytest.mark.parametrize("T,n,code", [(0, 1, 0), (1, 1024, 0), (1 << 22, 1, 0), (-1, 1, _lib.OFT_EINVAL), (1, 0, _lib.OFT_EINVAL),
                                      (1, 1025, _lib.OFT_EUNSUPPORTED), ((1 << 22) + 1, 1, _lib.OFT_EUNSUPPORTED)])
def test_rows_bytes(T, n, code):
    a, b = C.c_size_t(7), C.c_size_t(7)
    assert _lib.load().oft_adapter_rows_bytes(T, n, C.byref(a), C.byref(b)) == code
    if code == 0:
        assert a.value >= 32 and a.value % 16 == 0 and (b.value == 0) == (T <= 4096)


def test_rows_bytes_rejects_null():
    b = C.c_size_t(0)
    lib = _lib.load()
    assert lib.oft_adapter_rows_bytes(1, 1, None, C.byref(b)) == _lib.OFT_EINVAL
    assert lib.oft_adapter_rows_bytes(1, 1, C.byref(b), None) == _lib.OFT_EINVAL


def test_route_validation():
    f = _lib.load().oft_adapter_route
    call = lambda r, a=OK, ws=OK, n=1 << 40: f(a, C.byref(r) if r is not None else None, ws, n, None)  # noqa: E731
    assert call(None) == _lib.OFT_EINVAL
    for r in (_rows(T=-1), _rows(n=0), _rows(order=None), _rows(offsets=None), _rows(tiles=None), _rows(order=BAD),
              _rows(offsets=BAD), _rows(tiles=BAD)):
        assert call(r) == _lib.OFT_EINVAL
    assert call(_rows(n=1025)) == _lib.OFT_EUNSUPPORTED
    assert call(_rows(), a=None) == _lib.OFT_EINVAL
    assert call(_rows(), a=BAD) == _lib.OFT_EINVAL
    big = _rows(T=5000)
    need = oft.oft_adapter_rows_bytes(5000, 3)[1]
    assert call(big, ws=None) == _lib.OFT_EINVAL
    assert call(big, n=need - 1) == _lib.OFT_EWORKSPACE


# -------------------------------------------------------------- low rank
def _ld(**kw):
    a = dict(T=4, n=3, K=64, segs=(16, 32), r=8, dtype=oft.OFT_DT_BF16)
    a.update(kw)
    return oft.lowrank_desc(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(), 0), (dict(T=0), 0), (dict(dtype=1), 0), (dict(segs=(16,) * 8), 0), (dict(r=128), 0), (dict(n=1024), 0),
    (dict(T=-1), _lib.OFT_EINVAL), (dict(n=0), _lib.OFT_EINVAL), (dict(K=0), _lib.OFT_EINVAL),
    (dict(r=0), _lib.OFT_EINVAL), (dict(segs=()), _lib.OFT_EINVAL),
    (dict(K=96), _lib.OFT_ESHAPE), (dict(segs=(16, 24)), _lib.OFT_ESHAPE), (dict(r=12), _lib.OFT_ESHAPE),
    (dict(segs=(32, -16)), _lib.OFT_ESHAPE), (dict(dtype=2), _lib.OFT_EDTYPE),
    (dict(r=136), _lib.OFT_EUNSUPPORTED), (dict(segs=(16,) * 9), _lib.OFT_EUNSUPPORTED),
    (dict(K=(1 << 20) + 64), _lib.OFT_EUNSUPPORTED), (dict(segs=(1 << 20, 16)), _lib.OFT_EUNSUPPORTED),
    (dict(n=1025), _lib.OFT_EUNSUPPORTED), (dict(T=(1 << 22) + 1), _lib.OFT_EUNSUPPORTED),
    (dict(T=1 << 14, K=1 << 20, segs=(1 << 20,), r=128, n=1024), 0),
    (dict(T=(1 << 14) + 1, K=1 << 20), _lib.OFT_EUNSUPPORTED), (dict(T=(1 << 14) + 1, segs=(1 << 20,)), _lib.OFT_EUNSUPPORTED),
])
def test_lowrank_descriptor(kw, code):
    d, n = _ld(**kw), C.c_size_t(0)
    for which in (oft.OFT_PASS_FWD, oft.OFT_PASS_BWD):
        assert _lib.load().oft_lowrank_workspace_bytes(C.byref(d), which, C.byref(n)) == code
    if code == 0:
        assert (n.value == 0) == (d.T == 0)


def test_workspace_queries_reject():
    lib, n = _lib.load(), C.c_size_t(0)
    d, r = _ld(), oft.rotate_desc(4, 3, 64, 32)
    for f, desc in ((lib.oft_lowrank_workspace_bytes, d), (lib.oft_rotate_workspace_bytes, r)):
        assert f(None, 0, C.byref(n)) == _lib.OFT_EINVAL
        assert f(C.byref(desc), 0, None) == _lib.OFT_EINVAL
        assert f(C.byref(desc), 2, C.byref(n)) == _lib.OFT_EINVAL
    wrong = _ld()
    wrong.N = 64  # not the segments' sum
    assert lib.oft_lowrank_workspace_bytes(C.byref(wrong), 0, C.byref(n)) == _lib.OFT_ESHAPE


def _lfwd(d=None, rows=None, **kw):
    a = dict(x=OK, A=OK, B=OK, scale=OK, y_base=FAR, y=FAR, v=OK, ws=OK, n=1 << 40)
    a.update(kw)
    return _lib.load().oft_lowrank_fwd(C.byref(d or _ld()), C.byref(rows or _rows()), *a.values(), None)


def test_lowrank_fwd_validation():
    assert _lfwd(_ld(T=0), x=None, y=None) == _lib.OFT_OK
    assert _lfwd(rows=_rows(T=5)) == _lib.OFT_ESHAPE
    assert _lfwd(rows=_rows(n=2)) == _lib.OFT_ESHAPE
    assert _lfwd(rows=_rows(tiles=None)) == _lib.OFT_EINVAL
    for name in ("x", "A", "B", "scale", "y_base", "y", "ws"):
        assert _lfwd(**{name: None}) == _lib.OFT_EINVAL, name
        assert _lfwd(**{name: BAD}) == _lib.OFT_EINVAL, name
    assert _lfwd(v=BAD) == _lib.OFT_EINVAL
    need = oft.oft_lowrank_workspace_bytes(_ld(), oft.OFT_PASS_FWD)
    assert _lfwd(n=need - 1) == _lib.OFT_EWORKSPACE
    # y is y_base (4 rows of 48 bf16: 384 bytes) or apart from it, and apart from x (512 bytes)
    assert _lfwd(y=C.c_void_p(FAR.value + 368)) == _lib.OFT_EINVAL
    assert _lfwd(y=C.c_void_p(OK.value + 496), y_base=FAR) == _lib.OFT_EINVAL
    assert _lfwd(y=C.c_void_p(OK.value + 512), n=0) == _lib.OFT_EWORKSPACE


def _lbwd(d=None, rows=None, **kw):
    a = dict(dy=OK, x=OK, v=OK, A=OK, B=OK, scale=OK, dx_base=FAR, dx=FAR, dA=OUT, dB=OUT, ws=OK, n=1 << 40)
    a.update(kw)
    return _lib.load().oft_lowrank_bwd(C.byref(d or _ld()), C.byref(rows or _rows()), *a.values(), None)


def test_lowrank_bwd_validation():
    assert _lbwd(dx=None, dA=None, dB=None, dy=None) == _lib.OFT_OK  # nothing asked for
    assert _lbwd(rows=_rows(n=4)) == _lib.OFT_ESHAPE
    for name in ("dy", "scale", "ws"):
        assert _lbwd(**{name: None}) == _lib.OFT_EINVAL, name
    for name in ("dy", "x", "v", "A", "B", "scale", "dx_base", "dx", "dA", "dB", "ws"):
        assert _lbwd(**{name: BAD}) == _lib.OFT_EINVAL, name
    assert _lbwd(x=None) == _lib.OFT_EINVAL and _lbwd(v=None) == _lib.OFT_EINVAL
    assert _lbwd(A=None) == _lib.OFT_EINVAL and _lbwd(B=None) == _lib.OFT_EINVAL
    # what no gradient asked for reads may be missing
    assert _lbwd(dA=None, dB=None, x=None, v=None, n=0) == _lib.OFT_EWORKSPACE
    assert _lbwd(dx=None, dA=None, x=None, A=None, B=None, n=0) == _lib.OFT_EWORKSPACE
    # dx: dx_base or apart from it (512 bytes), x and dy
    assert _lbwd(dx=C.c_void_p(FAR.value + 496)) == _lib.OFT_EINVAL
    assert _lbwd(dx=OK, dx_base=None, dy=FAR) == _lib.OFT_EINVAL
    assert _lbwd(dx=C.c_void_p(OK.value + 368), dx_base=None, x=FAR) == _lib.OFT_EINVAL
    need = oft.oft_lowrank_workspace_bytes(_ld(), oft.OFT_PASS_BWD)
    assert _lbwd(n=need - 1) == _lib.OFT_EWORKSPACE


# -------------------------------------------------------------- rotations
@pytest.mark.parametrize("kw,code", [
    (dict(), 0), (dict(T=0), 0), (dict(b=16, N=96), 0), (dict(N=1 << 20), 0),
    (dict(T=-1), _lib.OFT_EINVAL), (dict(N=0), _lib.OFT_EINVAL), (dict(N=48), _lib.OFT_ESHAPE),
    (dict(b=8), _lib.OFT_EUNSUPPORTED), (dict(N=(1 << 20) + 32), _lib.OFT_EUNSUPPORTED),
    (dict(T=1 << 22, N=4096), 0), (dict(T=1 << 22, N=4128), _lib.OFT_EUNSUPPORTED), (dict(dtype=3), _lib.OFT_EDTYPE),
])
def test_rotate_descriptor(kw, code):
    a = dict(T=4, n=3, N=64, b=32, dtype=oft.OFT_DT_BF16)
    a.update(kw)
    d, n = oft.rotate_desc(**a), C.c_size_t(0)
    assert _lib.load().oft_rotate_workspace_bytes(C.byref(d), oft.OFT_PASS_FWD, C.byref(n)) == code
    if code == 0:
        assert n.value == 0
        assert _lib.load().oft_rotate_workspace_bytes(C.byref(d), oft.OFT_PASS_BWD, C.byref(n)) == 0
        assert (n.value == 0) == (d.T == 0)


def test_rotate_validation():
    lib = _lib.load()
    d = oft.rotate_desc(4, 3, 64, 32)
    fwd = lambda rows=_rows(), z=OK, R=OK, y=OK, d=d: lib.oft_rotate_fwd(C.byref(d), C.byref(rows), z, R, y, None)  # noqa: E731
    assert fwd(d=oft.rotate_desc(0, 3, 64, 32), z=None) == _lib.OFT_OK
    assert fwd(rows=_rows(T=3)) == _lib.OFT_ESHAPE
    for kw in (dict(z=None), dict(z=BAD), dict(R=None), dict(R=BAD), dict(y=None), dict(y=BAD),
               dict(y=C.c_void_p(OK.value + 496)), dict(rows=_rows(order=None))):
        assert fwd(**kw) == _lib.OFT_EINVAL, kw

    def bwd(rows=_rows(), **kw):
        a = dict(dy=OK, y=FAR, Rf=OK, R=OK, dz=OUT, dq=OUT, ws=OK, n=1 << 40)
        a.update(kw)
        return lib.oft_rotate_bwd(C.byref(d), C.byref(rows), *a.values(), None)

    assert bwd(dz=None, dq=None, dy=None) == _lib.OFT_OK
    assert bwd(rows=_rows(n=1)) == _lib.OFT_ESHAPE
    for kw in (dict(dy=None), dict(y=None), dict(Rf=None), dict(R=None), dict(ws=None), dict(dy=BAD), dict(y=BAD),
               dict(Rf=BAD), dict(R=BAD), dict(dz=BAD), dict(dq=BAD), dict(ws=BAD),
               dict(dz=C.c_void_p(OK.value + 16)), dict(dz=FAR)):
        assert bwd(**kw) == _lib.OFT_EINVAL, kw
    need = oft.oft_rotate_workspace_bytes(d, oft.OFT_PASS_BWD)
    assert bwd(n=need - 1) == _lib.OFT_EWORKSPACE


# -------------------------------------------------------------- gradients
def _ptrs(*a):
    return (C.c_void_p * len(a))(*[p.value if isinstance(p, C.c_void_p) else p for p in a])


def _counts(*a):
    return (C.c_int64 * len(a))(*a)


def test_grad_sizes():
    lib, n = _lib.load(), C.c_size_t(0)
    f = lambda m, c, dt=1: lib.oft_grad_workspace_bytes(m, c, dt, C.byref(n))  # noqa: E731
    assert f(0, None) == 0 and n.value == 0
    assert f(3, _counts(5, 0, 100000)) == 0 and n.value > 0
    assert f(-1, None) == _lib.OFT_EINVAL and f(1, None) == _lib.OFT_EINVAL and f(1, _counts(-1)) == _lib.OFT_EINVAL
    assert f(1, _counts(1), 2) == _lib.OFT_EDTYPE
    assert f(65537, _counts(*([1] * 65537))) == _lib.OFT_EUNSUPPORTED
    assert f(1, _counts((1 << 36) - 1)) == 0
    assert f(1, _counts(1 << 36)) == _lib.OFT_EUNSUPPORTED
    assert f(2, _counts(1 << 35, 1 << 35)) == _lib.OFT_EUNSUPPORTED
    assert lib.oft_grad_workspace_bytes(0, None, 1, None) == _lib.OFT_EINVAL


def test_grad_validation():
    lib = _lib.load()
    sums = lambda g=_ptrs(OK), c=_counts(8), dt=1, s=OK, ws=OK, n=1 << 20: lib.oft_grad_sumsq(1, g, c, dt, s, ws, n, None)  # noqa: E731
    for kw in (dict(g=None), dict(g=_ptrs(None)), dict(g=_ptrs(0x100002)), dict(g=_ptrs(0x100001), dt=0), dict(s=None),
               dict(s=C.c_void_p(0x100004)), dict(ws=None), dict(ws=BAD)):
        assert sums(**kw) == _lib.OFT_EINVAL, kw
    assert sums(n=7) == _lib.OFT_EWORKSPACE

    def clip(g=_ptrs(OK), c=_counts(8), dt=1, s=OK, most=1.0, out=_ptrs(OK), stats=OK):
        return lib.oft_grad_clip(1, g, c, dt, s, most, out, stats, None)

    for kw in (dict(g=_ptrs(None)), dict(s=None), dict(most=-1.0), dict(most=float("nan")), dict(out=None),
               dict(out=_ptrs(None)), dict(out=_ptrs(0x100002)), dict(stats=None), dict(stats=C.c_void_p(0x100004)),
               dict(out=_ptrs(OK.value + 28)), dict(out=_ptrs(OK.value - 28))):
        assert clip(**kw) == _lib.OFT_EINVAL, kw


def test_grad_list_refuses():
    t = torch.zeros(64)
    for grads, out in (([], None), ([t], []), ([t], None)):  # (the last: not on a GPU)
        with pytest.raises(ValueError):
            oft.grad_list(grads, out)
