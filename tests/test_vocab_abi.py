"""CPU checks of the vocabulary losses' and the balance loss's entry points:
every call here fails validation, or has nothing to do, before the library
touches the HIP runtime."""
import ctypes as C

import numpy as np
import pytest
import torch

import orthogonal_fine_tuning_amd as oft
from orthogonal_fine_tuning_amd import _lib

OK = C.c_void_p(0x100000)
OUT = C.c_void_p(0x40000000)
ODD = C.c_void_p(0x100001)
BAD = C.c_void_p(0x100008)


def _d(**kw):
    base = dict(T=4, V=100, dtype=oft.OFT_DT_BF16, k=3, ld=104, ld_grad=100)
    base.update(kw)
    return oft.vocab_desc(**base)


def _query(d):
    n = C.c_size_t(0)
    return _lib.load().oft_vocab_workspace_bytes(C.byref(d), C.byref(n))


@pytest.mark.parametrize("kw,code", [
    (dict(), _lib.OFT_OK),
    (dict(T=0), _lib.OFT_OK),
    (dict(T=-1), _lib.OFT_EINVAL),
    (dict(V=0), _lib.OFT_EINVAL),
    (dict(ld=99), _lib.OFT_EINVAL),
    (dict(ld_grad=99), _lib.OFT_EINVAL),
    (dict(dtype=2), _lib.OFT_EDTYPE),
    (dict(temperature=0.0), _lib.OFT_EINVAL),
    (dict(temperature=-1.0), _lib.OFT_EINVAL),
    (dict(temperature=float("nan")), _lib.OFT_EINVAL),
    (dict(temperature=float("inf")), _lib.OFT_EINVAL),
    (dict(temperature=2.0 ** -20), _lib.OFT_OK),
    (dict(temperature=2.0 ** -21), _lib.OFT_EINVAL),
    (dict(temperature=2.0 ** 20), _lib.OFT_OK),
    (dict(temperature=2.0 ** 21), _lib.OFT_EINVAL),
    (dict(accumulate=2), _lib.OFT_EINVAL),
    (dict(k=-1), _lib.OFT_EUNSUPPORTED),
    (dict(k=257), _lib.OFT_EUNSUPPORTED),
    (dict(T=1 << 22), _lib.OFT_OK),
    (dict(T=(1 << 22) + 1), _lib.OFT_EUNSUPPORTED),
    (dict(V=1 << 24, ld=1 << 24, ld_grad=1 << 24), _lib.OFT_OK),
    (dict(V=(1 << 24) + 1, ld=1 << 25, ld_grad=1 << 25), _lib.OFT_EUNSUPPORTED),
    (dict(T=1 << 20, V=1 << 14, ld=1 << 14, ld_grad=1 << 14), _lib.OFT_OK),
    (dict(T=(1 << 20) + 1, V=1 << 14, ld=1 << 14, ld_grad=1 << 14), _lib.OFT_EUNSUPPORTED),
    (dict(T=2, ld=(1 << 39) - 1), _lib.OFT_OK),
    (dict(T=2, ld=1 << 39), _lib.OFT_EUNSUPPORTED),
    (dict(T=2, ld_grad=1 << 39), _lib.OFT_EUNSUPPORTED),
    (dict(T=1 << 22, ld=1 << 62), _lib.OFT_EUNSUPPORTED),  # the product would pass 64 bits
])
def test_descriptor(kw, code):
    assert _query(_d(**kw)) == code


def test_workspace_query_rejects_null():
    lib = _lib.load()
    n = C.c_size_t(0)
    assert lib.oft_vocab_workspace_bytes(None, C.byref(n)) == _lib.OFT_EINVAL
    assert lib.oft_vocab_workspace_bytes(C.byref(_d()), None) == _lib.OFT_EINVAL
    assert oft.oft_vocab_workspace_bytes(_d(T=0)) == 0


def _fwd(d, **kw):
    a = dict(logits=OK, labels=OK, logp=OK, entropy=OK, top_idx=OK, top_logp=OK, stats=OK, ws=OK, n=1 << 40)
    a.update(kw)
    return _lib.load().oft_token_logprobs(C.byref(d), a["logits"], a["labels"], a["logp"], a["entropy"], a["top_idx"],
                                          a["top_logp"], a["stats"], a["ws"], a["n"], None)


def test_token_logprobs_validation():
    assert _fwd(_d(T=0), logits=None, stats=None) == _lib.OFT_OK
    assert _fwd(_d(k=129), logits=None) == _lib.OFT_EUNSUPPORTED
    assert _fwd(_d(k=101)) == _lib.OFT_ESHAPE  # more alternatives than columns
    for kw in (dict(logits=None), dict(logits=ODD), dict(stats=None), dict(stats=BAD), dict(labels=None),
               dict(logp=None), dict(labels=BAD), dict(logp=BAD), dict(entropy=BAD), dict(top_idx=None),
               dict(top_logp=None), dict(top_logp=BAD)):
        assert _fwd(_d(), **kw) == _lib.OFT_EINVAL, kw
    # fp32 rows need 4-byte alignment, and no more
    assert _fwd(_d(dtype=oft.OFT_DT_F32), logits=C.c_void_p(0x100002)) == _lib.OFT_EINVAL
    assert _fwd(_d(dtype=oft.OFT_DT_F32), logits=C.c_void_p(0x100004), stats=None) == _lib.OFT_EINVAL
    need = oft.oft_vocab_workspace_bytes(_d())
    if need:
        assert _fwd(_d(), ws=None) == _lib.OFT_EINVAL
        assert _fwd(_d(), ws=BAD) == _lib.OFT_EINVAL
        assert _fwd(_d(), n=need - 1) == _lib.OFT_EWORKSPACE


def _bwd(d, **kw):
    a = dict(logits=OK, labels=OK, stats=OK, entropy=OK, g_logp=OK, g_entropy=OK, d_logits=OUT)
    a.update(kw)
    return _lib.load().oft_token_logprobs_bwd(C.byref(d), *a.values(), None)


def test_token_logprobs_bwd_validation():
    assert _bwd(_d(T=0), logits=None) == _lib.OFT_OK
    for kw in (dict(logits=None), dict(d_logits=None), dict(d_logits=ODD), dict(stats=None), dict(stats=BAD),
               dict(labels=None), dict(g_logp=None), dict(labels=None, g_logp=None, g_entropy=None),
               dict(entropy=None), dict(entropy=BAD), dict(g_entropy=BAD), dict(g_logp=BAD), dict(labels=BAD)):
        assert _bwd(_d(), **kw) == _lib.OFT_EINVAL, kw


@pytest.mark.parametrize("kw,off", [
    (dict(), 0),                                # in place with other row distances (104 and 100)
    (dict(ld=100, accumulate=1), 0),            # in place and accumulating
    (dict(ld=100), 2),                          # shifted by one element
    (dict(ld=100), 2 * (3 * 100 + 99)),         # the last element of logits
    (dict(ld=100), -2 * (3 * 100 + 99)),        # the last element of d_logits
])
def test_overlapping_gradient_is_refused(kw, off):
    d = _d(**kw)
    out = C.c_void_p(0x100000 + off)
    assert _bwd(d, d_logits=out) == _lib.OFT_EINVAL
    assert _lib.load().oft_distill_topk_bwd(C.byref(d), OK, OUT, OUT, OUT, OUT, out, None) == _lib.OFT_EINVAL


def test_distill_validation():
    lib = _lib.load()
    f, b = lib.oft_distill_topk, lib.oft_distill_topk_bwd
    assert f(C.byref(_d(T=0)), None, None, None, None, None, None, 0, None) == _lib.OFT_OK
    assert b(C.byref(_d(T=0)), None, None, None, None, None, None, None) == _lib.OFT_OK
    for k in (0, 257):
        assert f(C.byref(_d(k=k)), OK, OK, OK, OK, OK, OK, 1 << 40, None) == _lib.OFT_EUNSUPPORTED
        assert b(C.byref(_d(k=k)), OK, OK, OK, OK, OK, OUT, None) == _lib.OFT_EUNSUPPORTED
    d = _d()
    for i in range(5):
        for p in (None, ODD):
            a = [OK] * 5
            a[i] = p
            assert f(C.byref(d), *a, OK, 1 << 40, None) == _lib.OFT_EINVAL
    for i in range(6):
        for p in (None, ODD):
            a = [OK] * 5 + [OUT]
            a[i] = p
            assert b(C.byref(d), *a, None) == _lib.OFT_EINVAL
    need = oft.oft_vocab_workspace_bytes(d)
    if need:
        assert f(C.byref(d), OK, OK, OK, OK, OK, OK, need - 1, None) == _lib.OFT_EWORKSPACE


def _moe(**kw):
    base = dict(T=128, E=16, k=4, H=256, I=128, g=32, b=32, chunk=4, renorm=0)
    base.update(kw)
    return oft.moe_desc(**base)


def test_balance_validation():
    lib = _lib.load()
    n = C.c_size_t(0)
    q = lib.oft_moe_balance_workspace_bytes
    assert q(C.byref(_moe()), 32, C.byref(n)) == _lib.OFT_OK and n.value > 0
    assert q(C.byref(_moe()), 32, None) == _lib.OFT_EINVAL
    assert q(C.byref(_moe()), 0, C.byref(n)) == _lib.OFT_EINVAL
    assert q(C.byref(_moe()), 33, C.byref(n)) == _lib.OFT_ESHAPE
    assert q(C.byref(_moe(k=17)), 32, C.byref(n)) == _lib.OFT_EUNSUPPORTED
    assert q(None, 32, C.byref(n)) == _lib.OFT_EINVAL
    f, b = lib.oft_moe_balance, lib.oft_moe_balance_bwd
    # logits, topk_idx, mask (optional), counts, tokens, loss, mean_prob (optional), ws
    assert f(C.byref(_moe(T=0)), 32, *[None] * 8, 0, None) == _lib.OFT_OK
    for i in range(8):
        for p in (None, BAD):
            if p is None and i in (2, 6):
                continue
            a = [OK] * 8
            a[i] = p
            assert f(C.byref(_moe()), 32, *a, 1 << 40, None) == _lib.OFT_EINVAL, (i, p)
    assert f(C.byref(_moe()), 32, *[OK] * 8, n.value - 1, None) == _lib.OFT_EWORKSPACE
    assert f(C.byref(_moe()), 33, *[OK] * 8, 1 << 40, None) == _lib.OFT_ESHAPE
    # logits, mask (optional), counts, tokens, g_loss, d_logits
    assert b(C.byref(_moe(T=0)), 32, *[None] * 6, 0, None) == _lib.OFT_OK
    assert b(C.byref(_moe()), 32, *[OK] * 6, 2, None) == _lib.OFT_EINVAL
    for i in range(6):
        for p in (None, BAD):
            if p is None and i == 1:
                continue
            a = [OK] * 6
            a[i] = p
            assert b(C.byref(_moe()), 32, *a, 0, None) == _lib.OFT_EINVAL, (i, p)


def test_binding_refuses_tensors_that_do_not_fit():
    """The binding's own checks come before the library is called: tensors
    on the host, and (on any device) wrong types, shapes and strides."""
    d = _d(ld=100)
    x = torch.zeros((4, 100), dtype=torch.bfloat16)
    f = torch.zeros(4)
    i = torch.zeros(4, dtype=torch.int32)
    s = torch.zeros((4, 2))
    with pytest.raises(ValueError, match="cpu"):
        oft.oft_token_logprobs(d, x, i, f, s, f, torch.zeros((4, 3), dtype=torch.int32), torch.zeros((4, 3)))
    with pytest.raises(ValueError, match="cpu"):
        oft.oft_token_logprobs_bwd(d, x, i, s, f, x)
    with pytest.raises(ValueError, match="cpu"):
        oft.oft_distill_topk(d, x, torch.zeros((4, 3), dtype=torch.int32), torch.zeros((4, 3)), f, s)
    with pytest.raises(ValueError, match="cpu"):
        oft.oft_distill_topk_bwd(d, x, torch.zeros((4, 3), dtype=torch.int32), torch.zeros((4, 3)), s, f, x)
    m = _moe()
    y = torch.zeros((128, 16))
    with pytest.raises(ValueError, match="cpu"):
        oft.oft_moe_balance(m, 32, y, torch.zeros((128, 4), dtype=torch.int32), torch.zeros((4, 16)), f, f)
    with pytest.raises(ValueError, match="cpu"):
        oft.oft_moe_balance_bwd(m, 32, y, torch.zeros((4, 16), dtype=torch.int32), i, f, y)
    with pytest.raises(ValueError, match="divisor"):
        oft.oft_moe_balance(m, 33, y, None, None, None, None)


def test_every_gpu_test_shape_passes_validation():
    """The shapes the GPU tests run are valid descriptors, checked here so
    that a bad test shape never reaches the GPU."""
    from tests import test_gpu_balance as tb
    from tests import test_gpu_vocab as tv

    for c in tv.SHAPES:
        for dtype in (oft.OFT_DT_BF16, oft.OFT_DT_F32):
            assert c["k"] <= min(c["V"], 128)
            assert _query(_d(T=c["T"], V=c["V"], k=c["k"], ld=c["V"] + c["pad"], ld_grad=c["V"] + c["gpad"],
                             dtype=dtype, temperature=c["tau"])) == _lib.OFT_OK
    n = C.c_size_t(0)
    for S, L, E, k in tb.SHAPES:
        d = oft.moe_desc(S * L, E, k, 64, 64, 32, 32, 16)
        assert _lib.load().oft_moe_balance_workspace_bytes(C.byref(d), L, C.byref(n)) == _lib.OFT_OK
