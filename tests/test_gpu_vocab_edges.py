"""Rows at the borders of the vocabulary losses' definitions, against the
oracle: columns that rank alike, ranges that a division by the temperature
brings back, calls that depend on each other."""
import numpy as np
import pytest

from oracle import vocab
from tests.helpers import host
from tests.test_gpu_vocab import DTYPES, _c, _logprobs
from tests.vocab_cases import NEG, Bounds, as_type, check

pytestmark = pytest.mark.gpu


# ------------------------------------------ NaN and -inf among the alternatives
# Both rank last and alike, by column.  Rows shorter than the candidates' lists
# and longer, whole (from 200 rows on, or short) and in slices, at odd
# addresses, and of more columns than the selection holds maxima of.
RANKED_ALIKE = [_c(12, 6, 5), _c(12, 8, 2), _c(12, 8, 8), _c(24, 128, 20, pad=3, offset=1), _c(24, 257, 128),
                _c(24, 500, 128, pad=1), _c(24, 700, 100), _c(24, 2049, 33, pad=1), _c(24, 9000, 128, offset=5),
                _c(205, 5001, 20), _c(12, 70001, 20, pad=2), _c(12, 151936, 64), _c(6, 300001, 40)]


def _few_numbers(T, V, k, dtype, seed):
    """Rows with fewer than k numbers above -inf where t % 3 < 2 (none at all
    where t % 12 is 0), k and more otherwise; -inf and NaN elsewhere, half of
    each, a NaN in a thousand columns, in the first columns alone, or none."""
    rng = np.random.default_rng(seed)
    x = np.full((T, V), NEG, np.float32)
    low = -3.3895314e38 if dtype == "bf16" else -3.4028235e38  # the type's lowest value
    for t in range(T):
        r = x[t]
        nan = (rng.random(V) < 0.5, rng.random(V) < 1e-3, np.arange(V) < 3, np.zeros(V, bool))[t % 4]
        if t % 4 == 1:
            nan[rng.integers(V)] = True
        r[nan] = np.nan
        n = 0 if t % 12 == 0 else int(rng.integers(1, k)) if t % 3 < 2 and k > 1 else k + int(rng.integers(0, 40))
        at = rng.permutation(V)[:min(n, V - 1)]
        r[at] = rng.normal(0, 3, at.size)
        r[at[::5]] = low
    return as_type(x, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("c", RANKED_ALIKE, ids=["T{T}-V{V}-k{k}-o{offset}".format(**c) for c in RANKED_ALIKE])
def test_nan_ranks_as_minus_infinity_beside_it(c, dtype):
    print(f"[ranked alike] {c} {dtype}", flush=True)
    T, V, k = c["T"], c["V"], c["k"]
    x = _few_numbers(T, V, k, dtype, V + k)
    if V == 6:
        x[0] = [1.0, 3.0, 3.0, np.nan, NEG, 2.0]
    if V == 8:
        x[0] = [np.nan] + [NEG] * 7
    labels = np.arange(T, dtype=np.int32) % V
    _, got = _logprobs(c, dtype, x, labels)
    want = vocab.top(x, k)
    wrong = np.flatnonzero((host(got["top_idx"]) != want).any(axis=1))
    assert wrong.size == 0, f"rows {wrong[:8].tolist()} of {wrong.size}"
    b = Bounds(x, 1.0)
    check(host(got["top_logp"]), np.take_along_axis(b.lp, want, 1), np.take_along_axis(b.lp_tol, want, 1), "top_logp")
    check(host(got["entropy"]), b.H, b.H_tol, "entropy")
