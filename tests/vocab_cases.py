"""Rows of logits for the tests of the vocabulary losses, and how far fp32
arithmetic may be from the fp64 oracle on them.

Error bounds.  u = 2^-24 is half a step of fp32 arithmetic (one rounding).
With A = sum p |z| (z = (x - m) / tau):
  * z: the subtraction, the rounded 1 / tau and the product, 3u |z|;
  * e^z as 2^(z log2 e): z's own error, the rounded constant and the product
    (2u |z| more), the hardware exponential (one step, 2u): (5 |z| + 2) u
    relative;
  * s: that, averaged with weights p, and one rounding per addition of a
    chain of at most V / 256 + 16 terms: (5 A + V / 256 + 18) u relative, which
    l = log s takes over absolutely, plus log's own steps 4u |l| + 2u;
  * log p_i: l's error, 3u |z_i| and the subtraction u |z_i - l|;
  * H = l - sum e z / s: both errors, each term of the sum off by
    (5 |z| + 3) u relative;
  * p_i = e^(log p_i): log p_i's error, 2u |log p_i| and the exponential, 2u.
An exponential below 2^-126 may be flushed to 0: 2^-125 absolute.
A result rounded to a type is off by half its step more (eps / 2 relative).
"""
import numpy as np

from oracle import vocab

U = 2.0 ** -24
FLUSH = 2.0 ** -125
NEG = -np.inf


def rows(T, V, dtype, seed, kinds=None):
    """fp32 array [T, V] of values that `dtype` ("bf16", "f32") holds exactly.
    `kinds`: the kind of each row in turn ("plain" if None)."""
    rng = np.random.default_rng(seed)
    x = rng.normal(0, 2.5, (T, V)).astype(np.float32)
    kinds = kinds or ["plain"]
    low = -3.3895314e38 if dtype == "bf16" else -3.4028235e38  # the type's lowest value
    for t in range(T):
        kind = kinds[t % len(kinds)]
        r = x[t]
        if kind == "ties":
            r[:] = np.round(r)
        elif kind == "constant":
            r[:] = 1.5
        elif kind == "zeros":
            r[:] = np.where(rng.random(V) < 0.5, -0.0, 0.0)
        elif kind == "masked":
            r[rng.random(V) < 0.6] = NEG
        elif kind == "lowest":
            r[rng.random(V) < 0.6] = low
        elif kind == "all_lowest":
            r[:] = low
        elif kind == "empty":
            r[:] = NEG
        elif kind == "one":
            r[:] = NEG
            r[rng.integers(V)] = -7.0
        elif kind == "nan":
            r[rng.integers(V)] = np.nan
        elif kind == "all_nan":
            r[:] = np.nan
        elif kind == "inf":
            r[rng.integers(V)] = np.inf
        elif kind == "wide":
            r *= 400.0
        elif kind == "shifted":
            r += 800.0
        elif kind == "up":
            r[:] = np.linspace(-20.0, 20.0, V)
        elif kind == "down":
            r[:] = np.linspace(20.0, -20.0, V)
        elif kind == "peak_last":
            r[-1] = 30.0
        elif kind == "peak_first":
            r[0] = 30.0
        elif kind == "border":
            # c x crosses 2^20 at temperature 1, where the reference of the
            # sums changes its form
            r += 2.0 ** 20 * np.log(2.0)
        elif kind == "narrow":
            r[:] = 3.0 + r * 1e-6
        elif kind != "plain":
            raise ValueError(kind)
    return as_type(x, dtype)


MORE_KINDS = ["border", "narrow", "plain", "masked"]
ALL_KINDS = ["plain", "ties", "constant", "zeros", "masked", "lowest", "all_lowest", "empty", "one", "nan", "all_nan",
             "inf", "wide", "shifted", "up", "down", "peak_last", "peak_first"]


def as_type(x, dtype):
    import torch

    t = torch.from_numpy(np.ascontiguousarray(x))
    return (t.to(torch.bfloat16).float() if dtype == "bf16" else t).numpy()


class Bounds:
    """Absolute error bounds of one row batch's results (arrays)."""

    def __init__(self, x, tau):
        with np.errstate(all="ignore"):
            self.lp, self.m, self.l = vocab.log_probs(x, tau)
            V = x.shape[1]
            self.tau = tau
            self.p = np.where(np.isfinite(self.lp), np.exp(self.lp), 0.0)
            fin = np.isfinite(self.lp)
            l = np.where(np.isfinite(self.l), self.l, 0.0)
            self.z = np.where(fin, self.lp + l[:, None], 0.0)
            az = np.abs(self.z)
            self.chain = V / 256 + 18
            A = (self.p * az).sum(axis=1)
            self.l_tol = (5 * A + self.chain + 4 * np.abs(l) + 4) * U
            self.lp_tol = self.l_tol[:, None] + U * (3 * az + np.where(fin, np.abs(self.lp), 0.0))
            self.H = vocab.entropy(self.lp)
            H = np.where(np.isfinite(self.H), self.H, 0.0)
            self.H_tol = self.l_tol + U * ((self.p * az * (5 * az + 5)).sum(axis=1) + A * (2 * self.chain + 5 * A + 8)
                                           + np.abs(H) * 2)
            alp = np.where(fin, np.abs(self.lp), 0.0)
            self.p_rel = self.lp_tol + U * (2 * alp + 4)
            self.alp = alp
            self.aH = np.abs(H)

    def grad(self, ref, gl, ge, dtype):
        """Bound of logprobs_grad (gl, ge [T]) rounded to dtype."""
        gl, ge = np.abs(gl)[:, None], np.abs(ge)[:, None]
        aH = self.aH[:, None]
        tol = self.p * (gl * (self.p_rel + 4 * U) + ge * ((self.p_rel + 6 * U) * (self.alp + aH) + self.lp_tol
                                                          + self.H_tol[:, None]))
        tol = tol + FLUSH * (gl + ge * (128 + aH))
        return self._rounded(ref, tol / self.tau, dtype)

    def _rounded(self, ref, tol, dtype):
        a = np.where(np.isfinite(ref), np.abs(ref), 0.0)
        tol = tol + 4 * U * a + FLUSH
        return tol + (2.0 ** -8 * (a + tol) if dtype == "bf16" else 0.0)

    def teacher(self, idx, val):
        """Bounds of the loss and of q [T, K]."""
        V = self.lp.shape[1]
        q, lq = vocab.teacher_probs(idx, val, V, self.tau)
        K = q.shape[1]
        live = np.where(np.isfinite(lq) & (q > 0), lq, 0.0)
        q = np.where(q > 0, q, 0.0)
        zt = np.abs(live - live.max(axis=1, keepdims=True))
        lq_tol = ((5 * (q * zt).sum(axis=1) + K / 64 + 18)[:, None] + 3 * zt + np.abs(live) + 8) * U
        q_rel = (5 * zt + 4) * U + ((5 * (q * zt).sum(axis=1) + K / 64 + 18) * U)[:, None]
        at = np.take_along_axis(self.lp, np.clip(np.asarray(idx, np.int64), 0, V - 1), axis=1)
        at_tol = np.take_along_axis(self.lp_tol, np.clip(np.asarray(idx, np.int64), 0, V - 1), axis=1)
        gap = np.abs(live - np.where(np.isfinite(at), at, 0.0))
        loss = (q * ((q_rel + (K / 64 + 14) * U) * gap + lq_tol + at_tol)).sum(axis=1)
        loss = loss + FLUSH * K * 256
        return loss, q * q_rel

    def distill_grad(self, ref, idx, val, g, dtype):
        _, q_tol = self.teacher(idx, val)
        tol = self.p * (self.p_rel + 2 * U) + FLUSH
        idx = np.asarray(idx, np.int64)
        q, _ = vocab.teacher_probs(idx, val, self.lp.shape[1], self.tau)
        q = np.where(q > 0, q, 0.0)
        K = idx.shape[1]
        for j in range(K):
            ok = (idx[:, j] >= 0) & (idx[:, j] < self.lp.shape[1])
            t = np.arange(len(idx))[ok]
            # (an entry listed more than once is a sum of at most K terms)
            tol[t, idx[ok, j]] += q_tol[ok, j] + (K + 2) * U * q[ok, j] + FLUSH
        return self._rounded(ref, tol * (np.abs(g) / self.tau)[:, None], dtype)


def check(got, ref, tol, what):
    """NaN where the oracle has NaN, the same infinities, and within tol."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    other = np.isnan(got) != np.isnan(ref)
    assert not other.any(), f"{what}: NaN at other places: {np.argwhere(other)[:4].tolist()} of {int(other.sum())}"
    inf = np.isinf(ref)
    tol = np.broadcast_to(tol, ref.shape)
    # an exact value beyond fp32's range is its infinity, and one whose bound
    # reaches past the range may be: ref (1 + e) is above the largest number
    # for an e that the bound allows
    big = np.isfinite(ref) & (np.abs(ref) + np.where(np.isfinite(ref), tol, 0.0) > 3.4028235e38)
    assert np.array_equal(got[inf], ref[inf]), f"{what}: infinities"
    fin = np.isfinite(ref) & ~big
    assert np.all(np.isfinite(got[fin])), f"{what}: not finite"
    d = np.abs(got[fin] - ref[fin])
    worst = float((d / np.maximum(tol[fin], 1e-300)).max()) if d.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} of the bound (error {d.max():.3g})"
    return worst
