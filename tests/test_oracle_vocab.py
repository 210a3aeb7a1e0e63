"""Pins for the oracle's vocabulary losses and router balance loss: closed
forms, explicit probabilities, central differences."""
import math

import numpy as np
import pytest

from oracle import moe, policy, vocab


def _x(seed, T=5, V=23, scale=2.0):
    return np.random.default_rng(seed).normal(0, scale, (T, V))


def _central(f, x, h=1e-5):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        g[i] = (f(a) - f(b)) / (2 * h)
    return g


@pytest.mark.parametrize("tau", [1.0, 0.6, 2.5])
def test_log_probs_are_normalised_and_match_the_policy_oracle(tau):
    x = _x(0)
    lp, m, l = vocab.log_probs(x, tau)
    assert np.allclose(np.exp(lp).sum(axis=1), 1.0, atol=1e-13)
    assert np.array_equal(m, x.max(axis=1))
    lab = np.array([0, 3, 22, 7, 11])
    assert np.allclose(vocab.given(lp, lab), policy.log_softmax_at(x / tau, lab), atol=1e-13)
    assert np.allclose(l, np.log(np.exp((x - m[:, None]) / tau).sum(axis=1)), atol=1e-13)


def test_entropy_closed_forms():
    x = np.zeros((2, 8))
    x[1] = -np.inf
    x[1, 3] = 5.0
    assert np.allclose(vocab.entropy(vocab.log_probs(x)[0]), [math.log(8), 0.0])


def test_rows_without_a_plain_meaning():
    x = np.array([[-np.inf] * 3, [np.nan, 0, 1], [np.inf, 0, 1]])
    lp, m, l = vocab.log_probs(x)
    assert np.all(lp[0] == -np.inf) and l[0] == -np.inf and m[0] == -np.inf
    assert np.all(np.isnan(lp[1:])) and np.all(np.isnan(l[1:]))
    assert vocab.entropy(lp)[0] == 0
    d = vocab.logprobs_grad(x, [0, 0, 0], np.ones(3), np.ones(3))
    assert np.all(d[0] == 0) and np.all(np.isnan(d[1:]))
    assert np.all(vocab.logprobs_grad(x, [0, -1, 0], [1.0, 1.0, 0.0], None)[1:] == 0)
    assert np.array_equal(vocab.given(np.zeros((3, 3)), [-1, 3, -2]), [0.0, np.nan, np.nan], equal_nan=True)


def test_top_breaks_ties_by_column_and_ranks_nan_last():
    x = np.array([[1.0, 3.0, 3.0, np.nan, -np.inf, 2.0], [0.0, -0.0, 0.0, 0.0, -0.0, 0.0]])
    assert vocab.top(x, 6).tolist() == [[1, 2, 5, 0, 3, 4], [0, 1, 2, 3, 4, 5]]


@pytest.mark.parametrize("tau", [1.0, 0.7])
def test_logprob_and_entropy_gradient_by_differences(tau):
    x = _x(1)
    lab = np.array([2, -1, 0, 22, 5])
    rng = np.random.default_rng(9)
    gl, ge = rng.normal(size=5), rng.normal(size=5)

    def f(y):
        lp = vocab.log_probs(y, tau)[0]
        return float((gl * vocab.given(lp, lab)).sum() + (ge * vocab.entropy(lp)).sum())

    assert np.allclose(vocab.logprobs_grad(x, lab, gl, ge, tau), _central(f, x), atol=1e-8)


@pytest.mark.parametrize("tau", [1.0, 2.0])
def test_distillation_gradient_by_differences(tau):
    x = _x(2)
    rng = np.random.default_rng(4)
    idx = rng.integers(0, 23, (5, 6))  # with repeated entries
    idx[1, 2] = idx[1, 0]
    idx[3, 1:] = -1
    val = rng.normal(0, 2, (5, 6))
    g = rng.normal(size=5)
    f = lambda y: float((g * vocab.distill(y, idx, val, tau)).sum())  # noqa: E731
    assert np.allclose(vocab.distill_grad(x, idx, val, g, tau), _central(f, x), atol=1e-8)


def test_distillation_is_the_divergence_of_full_lists():
    """A teacher that lists the whole vocabulary: KL(q || p), 0 when it lists
    the student's own logits in any order and shift."""
    x = _x(3, T=2, V=9)
    order = np.array([np.random.default_rng(i).permutation(9) for i in range(2)])
    own = np.take_along_axis(x, order, axis=1) + np.array([[3.0], [-50.0]])
    assert np.allclose(vocab.distill(x, order, own), 0.0, atol=1e-13)
    y = _x(5, T=2, V=9)
    p = np.exp(x) / np.exp(x).sum(axis=1, keepdims=True)
    q = np.exp(y) / np.exp(y).sum(axis=1, keepdims=True)
    want = (q * (np.log(q) - np.log(p))).sum(axis=1)
    assert np.allclose(vocab.distill(x, np.tile(np.arange(9), (2, 1)), y), want, atol=1e-13)


def test_distillation_of_rows_without_weight_or_with_bad_entries():
    x = _x(6, T=4, V=5)
    idx = np.array([[-1, -1], [0, 1], [0, 5], [2, 3]])
    val = np.array([[1.0, 2.0], [-np.inf, -np.inf], [0.0, 0.0], [np.nan, 0.0]])
    v = vocab.distill(x, idx, val)
    assert v[0] == 0 and v[1] == 0 and np.isnan(v[2]) and np.isnan(v[3])
    d = vocab.distill_grad(x, idx, val, np.ones(4))
    assert np.all(d[:2] == 0) and np.all(np.isnan(d[2:]))
    assert np.all(vocab.distill_grad(x, idx, val, np.zeros(4)) == 0)


def test_planted_mistakes_fail():
    x = _x(7)
    lab = np.array([2, 4, 0, 22, 5])
    gl = np.ones(5)
    right = vocab.logprobs_grad(x, lab, gl, None, 0.7)
    no_tau = vocab.logprobs_grad(x / 0.7, lab, gl, None, 1.0)  # without the 1 / tau of the chain rule
    assert np.abs(right - no_tau).max() > 1e-2
    idx = np.array([[1, 1]] * 5)
    q_once = vocab.distill_grad(x, idx[:, :1], np.zeros((5, 1)), gl)
    twice = vocab.distill_grad(x, idx, np.array([[0.0, 0.0]] * 5), gl)
    assert np.allclose(q_once, twice)  # two halves of the same entry are one entry
    assert np.abs(twice[:, 1] - (np.exp(vocab.log_probs(x)[0][:, 1]) - 0.5)).min() > 0.4


def _router(seed, S=3, L=7, E=11, k=3):
    rng = np.random.default_rng(seed)
    x = rng.normal(0, 1.5, (S * L, E))
    idx = np.argsort(-x, axis=1, kind="stable")[:, :k]
    mask = rng.random(S * L) < 0.7
    return x, idx, mask


@pytest.mark.parametrize("masked", [False, True])
def test_balance_gradient_by_differences(masked):
    x, idx, mask = _router(1)
    mask = mask if masked else None
    g = np.array([0.3, -1.0, 2.0])
    b = moe.balance(x, idx, 7, mask)
    f = lambda y: float((g * moe.balance(y, idx, 7, mask)["loss"]).sum())  # noqa: E731
    d = moe.balance_grad(x, b["counts"], b["tokens"], g, 3, 7, mask)
    assert np.allclose(d, _central(f, x), atol=1e-8)
    if masked:
        assert np.all(d[~mask] == 0)


def test_balance_closed_forms():
    # evenly spread: loss 1 with uniform probabilities; everything on one expert
    x = np.zeros((8, 4))
    even = np.array([[t % 4] for t in range(8)])
    b = moe.balance(x, even, 8)
    assert np.allclose(b["loss"], 1.0) and b["counts"].tolist() == [[2, 2, 2, 2]]
    x[:, 1] = 50.0
    b = moe.balance(x, np.full((8, 1), 1), 8)
    assert np.allclose(b["loss"], 4.0)
    # no tokens; an index out of range; a row of nothing but -inf; NaN as -inf
    z = moe.balance(x, even, 8, np.zeros(8, bool))
    assert z["loss"][0] == 0 and z["tokens"][0] == 0 and np.all(z["mean_prob"] == 0)
    assert moe.balance(x, np.full((8, 1), 9), 8)["counts"].sum() == 0
    x[0], x[1, 0] = -np.inf, np.nan
    b = moe.balance(x, even, 8)
    assert np.all(np.isfinite(b["mean_prob"])) and b["tokens"][0] == 8
