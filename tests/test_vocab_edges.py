"""CPU pins of the vocabulary losses' conventions at their borders."""
import numpy as np
import pytest

from oracle import vocab


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
