"""Batches of rows with adapters for the tests, and how far the library may be
from the fp64 oracle on them.

u = 2^-24 is half a step of fp32.  A sum of k products in fp32 is off by at
most 2 u (k + c) sum |a b|, c the additions that join partial sums (64 is more
than any call has): a matrix step adds exact products of bf16 numbers, and each
of its additions is off by at most a whole step.  Splitting an fp32 number into three bf16 parts
loses nothing (below 2^-100 parts may be flushed: FLUSH absolute), into two
2^-16 of it.  A result in bf16 is off by half its step more, 2^-8 of it.
"""
import numpy as np

from oracle import adapters as oracle

U = 2.0 ** -24
FLUSH = 2.0 ** -100
HALF = {"bf16": 2.0 ** -8, "f32": U}


def sum_err(k, total):
    """Error of an fp32 sum of k products whose magnitudes add to `total`."""
    return 2 * U * (k + 64) * total + FLUSH


def rounded(e, value, dtype):
    return e + HALF[dtype] * (np.abs(value) + e)


def bf16(a):
    """To the nearest bf16 value, as fp32."""
    u = np.ascontiguousarray(a, dtype=np.float32).view(np.uint32)
    u = (u + 0x7FFF + ((u >> 16) & 1)) & np.uint32(0xFFFF0000)
    return u.view(np.float32)


def as_type(a, dtype):
    return bf16(a) if dtype == "bf16" else np.ascontiguousarray(a, dtype=np.float32)


def adapters(T, n, kind, seed=0):
    """int32 [T] adapter numbers.  kinds: "runs" of consecutive rows, "mixed"
    row by row, "one" adapter for all, "none", "some" (a third without one,
    by several numbers outside the range), "skewed" (nearly all rows the last
    adapter's)."""
    rng = np.random.default_rng([seed, T, n])
    if kind == "runs":
        cuts = np.sort(rng.integers(0, T + 1, max(1, min(T, n) - 1)))
        return rng.permutation(max(n, len(cuts) + 1))[np.searchsorted(cuts, np.arange(T), "right")].astype(np.int32) % n
    a = rng.integers(0, n, T)
    if kind == "one":
        a[:] = n // 2
    elif kind == "none":
        a[:] = -1
    elif kind == "some":
        out = rng.random(T) < 0.34
        a[out] = rng.choice([-1, n, n + 5, -2 ** 31, 2 ** 31 - 1], int(out.sum()))
    elif kind == "skewed":
        a[rng.random(T) < 0.95] = n - 1
    return a.astype(np.int32)


def lowrank(T, n, K, segs, r, dtype, kind, seed=0):
    rng = np.random.default_rng([seed, T, n, K, r])
    N, R = sum(segs), r * len(segs)
    return {"adapter": adapters(T, n, kind, seed),
            "x": as_type(rng.normal(0, 1, (T, K)), dtype), "y_base": as_type(rng.normal(0, 1, (T, N)), dtype),
            "dx_base": as_type(rng.normal(0, 1, (T, K)), dtype), "dy": bf16(rng.normal(0, 1, (T, N))),
            "A": bf16(rng.normal(0, K ** -0.5, (n, R, K))), "B": bf16(rng.normal(0, 0.2, (n, N, r))),
            "scale": rng.uniform(0.5, 2.0, n).astype(np.float32)}


def _f64(c, *names):
    return [np.asarray(c[k], dtype=np.float64) for k in names]


def lowrank_fwd(c, segs, dtype):
    """((y, tolerance), (v, tolerance))."""
    x, A, B, scale, y0 = _f64(c, "x", "A", "B", "scale", "y_base")
    y, v = oracle.lowrank_fwd(x, A, B, scale, y0, c["adapter"], segs)
    zero = np.zeros_like(y0)
    _, vmag = oracle.lowrank_fwd(abs(x), abs(A), abs(B), scale, zero, c["adapter"], segs)
    ev = sum_err(x.shape[1], vmag)
    # y's products, with v off by ev and by what its parts leave out
    n, r = len(A), B.shape[2]
    lost = 2.0 ** -16 if dtype == "bf16" else 0.0
    mag, ey = np.zeros_like(y), np.zeros_like(y)
    for a, rows in oracle._used(c["adapter"], n):
        for cols, js in oracle._pieces(segs, r):
            mag[rows, cols] = scale[a] * (abs(v[rows][:, js]) @ abs(B[a, cols]).T)
            ey[rows, cols] = scale[a] * ((ev[rows][:, js] + lost * abs(v[rows][:, js])) @ abs(B[a, cols]).T)
    ey = ey + sum_err(r, mag) + 2 * U * mag + U * (abs(y0) + mag)  # the scale's product, and the last addition
    return (y, rounded(ey, y, dtype)), (v, ev)


def lowrank_bwd(c, v, segs, dtype, with_base=True):
    """((dx, tol), (dA, tol), (dB, tol)) for the saved v (fp32 values)."""
    dy, x, A, B, scale = _f64(c, "dy", "x", "A", "B", "scale")
    v = np.asarray(v, dtype=np.float64)
    base = np.asarray(c["dx_base"], dtype=np.float64) if with_base else np.zeros_like(x)
    dx, dA, dB = oracle.lowrank_bwd(dy, x, v, A, B, scale, base, c["adapter"], segs)
    n, r = len(A), B.shape[2]
    lost = 2.0 ** -16 if dtype == "bf16" else 0.0
    # fp32 times fp32 leaves the products of parts at 2^-24 of the whole out:
    # three of them
    pairs = 3 * 2.0 ** -23 if dtype == "f32" else 0.0
    edx, edA, edB = U * abs(base), np.zeros_like(dA), np.zeros_like(dB)
    mag = np.zeros_like(dx)
    for a, rows in oracle._used(c["adapter"], n):
        k = len(rows)
        for cols, js in oracle._pieces(segs, r):
            u = abs(dy[rows, cols] @ B[a, cols])
            eu = sum_err(dy[:, cols].shape[1], abs(dy[rows, cols]) @ abs(B[a, cols]))
            mag[rows] += scale[a] * (u @ abs(A[a, js]))
            edx[rows] += scale[a] * ((eu + lost * u) @ abs(A[a, js]))
            m = scale[a] * ((u + eu).T @ abs(x[rows]))
            edA[a, js] = scale[a] * (eu.T @ abs(x[rows])) + sum_err(k, m) + (2 * U + pairs) * m
            m = scale[a] * (abs(dy[rows, cols]).T @ abs(v[rows][:, js]))
            edB[a, cols] = sum_err(k, m) + 2 * U * m
    edx += sum_err(r * len(segs), mag) + 3 * U * mag
    return (dx, rounded(edx, dx, dtype)), (dA, edA), (dB, edB)


def rotations(n, nblk, b, seed=0, size=0.05):
    """(bf16 parameters [n, nblk, b(b-1)/2], the fp64 R of those)."""
    rng = np.random.default_rng([seed, n, nblk, b])
    p = bf16(rng.normal(0, size, (n, nblk, b * (b - 1) // 2)))
    q = np.zeros((n, nblk, b, b))
    i, l = np.triu_indices(b, 1)
    q[..., i, l] = p
    q[..., l, i] = -p
    return p, np.linalg.solve(np.eye(b) - q, np.eye(b) + q)


def rotate_fwd(z, R_op, adapter, dtype):
    y = oracle.rotate_fwd(z, R_op, adapter)
    mag = oracle.rotate_fwd(abs(z), abs(R_op), adapter)
    return y, rounded(sum_err(R_op.shape[2], mag), y, dtype)


def rotate_bwd(dy, y, R_op, R, adapter, dtype):
    """((dz, tol), (dq, tol)), R_op the bf16 operand and R the fp32 one the call is given."""
    dz, dq = oracle.rotate_bwd(dy, y, R_op, R, adapter)
    mag = oracle.rotate_fwd(abs(dy), abs(np.swapaxes(R_op, 2, 3)), adapter)
    n, nblk, b, _ = R.shape
    edq = np.zeros_like(dq)
    i, l = np.triu_indices(b, 1)
    eye = np.eye(b)
    for a, rows in oracle._used(adapter, n):
        d = abs(dy[rows]).reshape(len(rows), nblk, b)
        o = abs(y[rows]).reshape(len(rows), nblk, b)
        for j in range(nblk):
            S = d[:, j].T @ o[:, j]
            Ra = abs(R[a, j])
            # S off by its own sum; two products of b terms each, in order
            g = 0.5 * (Ra.T + eye) @ (sum_err(len(rows), S) + 2 * 2 * U * (b + 64) * S) @ (eye + Ra)
            edq[a, j] = (g + g.T)[i, l]
    return (dz, rounded(sum_err(b, mag), dz, "bf16")), (dq, edq)
