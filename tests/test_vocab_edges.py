"""CPU pins of the vocabulary losses' conventions at their borders, and checks
of their workspaces that fail before the library touches the HIP runtime."""
import ctypes as C

import numpy as np
import pytest

import orthogonal_fine_tuning_amd as oft
from oracle import vocab
from orthogonal_fine_tuning_amd import _lib

OK = C.c_void_p(0x100000)
BAD = C.c_void_p(0x100008)


@pytest.mark.parametrize("tau", [0.6, 1.0, 2.0])
def test_a_teacher_list_of_log_probabilities(tau):
    """Log-probabilities at temperature 1 are the teacher's logits up to a
    shift, those of x / s are it times s; as they stand they are the teacher at
    temperature tau s."""
    rng = np.random.default_rng(3)
    teacher, student = rng.normal(0, 2.5, (2, 5, 400))
    idx = vocab.top(teacher, 16)

    def listed(values):
        return np.take_along_axis(values, idx, axis=1)

    want = vocab.distill(student, idx, listed(teacher), tau)
    q = np.exp(listed(teacher) / tau)
    assert np.allclose(vocab.teacher_probs(idx, listed(teacher), 400, tau)[0], q / q.sum(axis=1, keepdims=True), atol=1e-14)
    assert np.allclose(vocab.distill(student, idx, listed(vocab.log_probs(teacher)[0]), tau), want, atol=1e-12)
    for s in (0.7, 1.5):
        scored = listed(vocab.log_probs(teacher, s)[0])
        assert np.allclose(vocab.distill(student, idx, s * scored, tau), want, atol=1e-12)
        twice = vocab.teacher_probs(idx, scored, 400, tau)[0]
        assert np.allclose(twice, vocab.teacher_probs(idx, listed(teacher), 400, tau * s)[0], atol=1e-12)
        assert np.abs(vocab.distill(student, idx, scored, tau) - want).min() > 1e-3


# -------------------------------------------------------------- workspaces
# Few long rows are read in slices and need one, with alternatives from fewer
# columns on.
@pytest.mark.parametrize("T,V,k", [(4, 151936, 3), (4, 70001, 0), (199, 40009, 20), (1, 300001, 128)])
@pytest.mark.parametrize("dtype", [oft.OFT_DT_BF16, oft.OFT_DT_F32])
def test_scoring_checks_its_workspace(T, V, k, dtype):
    d = oft.vocab_desc(T, V, dtype, k=k)
    need = oft.oft_vocab_workspace_bytes(d)
    assert need > 0

    def call(ws, n):
        return _lib.load().oft_token_logprobs(C.byref(d), OK, OK, OK, OK, OK, OK, OK, ws, n, None)

    assert call(None, need) == _lib.OFT_EINVAL
    assert call(BAD, need) == _lib.OFT_EINVAL
    assert call(OK, need - 1) == _lib.OFT_EWORKSPACE
    assert call(OK, 0) == _lib.OFT_EWORKSPACE


@pytest.mark.parametrize("T,V,k", [(4, 151936, 64), (199, 70001, 1), (4, 300001, 256)])
@pytest.mark.parametrize("dtype", [oft.OFT_DT_BF16, oft.OFT_DT_F32])
def test_distillation_checks_its_workspace(T, V, k, dtype):
    d = oft.vocab_desc(T, V, dtype, k=k)
    need = oft.oft_vocab_workspace_bytes(d)
    assert need > 0

    def call(ws, n):
        return _lib.load().oft_distill_topk(C.byref(d), OK, OK, OK, OK, OK, ws, n, None)

    assert call(None, need) == _lib.OFT_EINVAL
    assert call(BAD, need) == _lib.OFT_EINVAL
    assert call(OK, need - 1) == _lib.OFT_EWORKSPACE
    assert call(OK, 0) == _lib.OFT_EWORKSPACE
