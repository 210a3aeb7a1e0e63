"""Losses on vocabulary logits, in fp64.

Test infrastructure only (see the package header).

[P2] "Five design features of the adapter-first architecture" trains the
adapter by reinforcement learning, whose losses are functions of the
log-probabilities log p_i = z_i - log(sum_j exp z_j), z = (x - max x) / tau,
of a row x of logits.  Written out here: the log-probabilities of given
tokens with the row's entropy and its largest entries, the Kullback-Leibler
divergence from a teacher's renormalised top list, and both gradients.

A logit of -inf has p = 0.  A row of nothing but -inf has log p = -inf,
entropy 0 and gradient 0.
"""
from __future__ import annotations

import numpy as np

NO_LABEL = -1


def _f64(x):
    return np.asarray(x, dtype=np.float64)


def log_probs(x, tau=1.0):
    """(log p [T, V], m [T], l [T]); rows without a maximum give -inf."""
    x = _f64(x)
    with np.errstate(all="ignore"):
        m = np.where(np.isnan(x), -np.inf, x).max(axis=1)
        z = (x - np.where(np.isinf(m) & (m < 0), 0.0, m)[:, None]) / tau
        l = np.log(np.exp(z).sum(axis=1))
        lp = np.where((l == -np.inf)[:, None], -np.inf, z - l[:, None])
    return lp, m, l


def entropy(lp):
    with np.errstate(all="ignore"):
        p = np.exp(lp)
        return -np.where(p == 0, 0.0, p * lp).sum(axis=1)


def top(x, k):
    """Columns of the k largest, ties to the lower column, NaN as -inf."""
    x = _f64(x)
    return np.argsort(-np.where(np.isnan(x), -np.inf, x), axis=1, kind="stable")[:, :k].astype(np.int32)


def given(lp, labels):
    """log p at labels: 0 for NO_LABEL, NaN for another label out of range."""
    labels = np.asarray(labels, dtype=np.int64)
    V = lp.shape[1]
    ok = (labels >= 0) & (labels < V)
    v = lp[np.arange(len(labels)), np.where(ok, labels, 0)]
    return np.where(ok, v, np.where(labels == NO_LABEL, 0.0, np.nan))


def logprobs_grad(x, labels, g_logp, g_entropy, tau=1.0):
    """Gradient of sum g_logp log p_label + g_entropy H with respect to x."""
    lp, _, l = log_probs(x, tau)
    T, V = lp.shape
    H = entropy(lp)
    labels = np.full(T, NO_LABEL) if labels is None else np.asarray(labels, dtype=np.int64)
    gl = np.where(labels == NO_LABEL, 0.0, 0.0 if g_logp is None else _f64(g_logp))
    ge = np.zeros(T) if g_entropy is None else _f64(g_entropy)
    with np.errstate(all="ignore"):
        p = np.exp(lp)
        d = -p * (gl[:, None] + ge[:, None] * (np.where(p == 0, 0.0, lp) + H[:, None]))
    ok = (labels >= 0) & (labels < V)
    d[np.arange(T)[ok], labels[ok]] += gl[ok]
    d /= tau
    d[l == -np.inf] = 0.0
    d[(labels < NO_LABEL) | (labels >= V)] = np.nan
    d[(gl == 0) & (ge == 0)] = 0.0
    return d


def teacher_probs(idx, val, V, tau=1.0):
    """q [T, K] of the listed entries (NaN rows where an entry is invalid,
    0 where there is none) and log q."""
    idx = np.asarray(idx, dtype=np.int64)
    val = np.where(idx == NO_LABEL, -np.inf, _f64(val))
    bad = (((idx < NO_LABEL) | (idx >= V)) | np.isnan(val) | (val == np.inf)).any(axis=1)
    with np.errstate(all="ignore"):
        m = np.where(bad, 0.0, val.max(axis=1))
        none = m == -np.inf
        z = (val - np.where(none, 0.0, m)[:, None]) / tau
        lq = z - np.log(np.exp(z).sum(axis=1))[:, None]
        q = np.where(none[:, None], 0.0, np.exp(lq))
    q[bad] = np.nan
    return q, lq


def distill(x, idx, val, tau=1.0):
    """KL(q || p) of every row, q the teacher's renormalised list."""
    lp, _, _ = log_probs(x, tau)
    q, lq = teacher_probs(idx, val, lp.shape[1], tau)
    idx = np.asarray(idx, dtype=np.int64)
    at = np.take_along_axis(lp, np.clip(idx, 0, lp.shape[1] - 1), axis=1)
    with np.errstate(all="ignore"):
        return np.where(q == 0, 0.0, q * (lq - at)).sum(axis=1)


def distill_grad(x, idx, val, g, tau=1.0):
    lp, _, l = log_probs(x, tau)
    T, V = lp.shape
    q, _ = teacher_probs(idx, val, V, tau)
    g = _f64(g)
    d = np.exp(lp)
    idx = np.asarray(idx, dtype=np.int64)
    for t in range(T):
        for j in range(idx.shape[1]):
            if q[t, j] > 0:
                d[t, idx[t, j]] -= q[t, j]
    d *= g[:, None] / tau
    d[(l == -np.inf) | (q == 0).all(axis=1)] = 0.0
    d[np.isnan(q).any(axis=1)] = np.nan
    d[g == 0] = 0.0
    return d
