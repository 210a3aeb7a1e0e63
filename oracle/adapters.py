"""fp64 CPU oracle of the operators on adapters of many requests and of the
gradient clipping.  Arrays hold plain values (bf16 and fp32 inputs as the fp64
numbers they stand for); shares no code with the GPU path."""
from __future__ import annotations

import numpy as np


def route(adapter, n):
    """(order, offsets): rows by adapter, stable, rows without one (outside 0 .. n - 1) last."""
    a = np.asarray(adapter, dtype=np.int64)
    lists = [[] for _ in range(n + 1)]
    for t, i in enumerate(a.tolist()):
        lists[i if 0 <= i < n else n].append(t)
    order = np.array([t for rows in lists for t in rows], dtype=np.int32)
    offsets = np.cumsum([0] + [len(rows) for rows in lists[:n]]).astype(np.int32)
    return order, offsets


def _used(adapter, n):
    a = np.asarray(adapter)
    return [(i, np.nonzero(a == i)[0]) for i in range(n) if (a == i).any()]


def _pieces(segs, r):
    at = 0
    for s, width in enumerate(segs):
        yield slice(at, at + width), slice(s * r, (s + 1) * r)
        at += width


def lowrank_fwd(x, A, B, scale, y_base, adapter, segs):
    """(y, v)."""
    n, r = len(A), B.shape[2]
    y, v = np.array(y_base, dtype=np.float64), np.zeros((len(x), len(segs) * r))
    for a, rows in _used(adapter, n):
        v[rows] = x[rows] @ A[a].T
        for cols, js in _pieces(segs, r):
            y[rows, cols] += scale[a] * (v[rows][:, js] @ B[a, cols].T)
    return y, v


def lowrank_bwd(dy, x, v, A, B, scale, dx_base, adapter, segs):
    """(dx, dA, dB)."""
    n, r = len(A), B.shape[2]
    dx = np.array(dx_base, dtype=np.float64)
    dA, dB = np.zeros(A.shape), np.zeros(B.shape)
    for a, rows in _used(adapter, n):
        for cols, js in _pieces(segs, r):
            u = dy[rows, cols] @ B[a, cols]
            dx[rows] += scale[a] * (u @ A[a, js])
            dA[a, js] = scale[a] * (u.T @ x[rows])
            dB[a, cols] = scale[a] * (dy[rows, cols].T @ v[rows][:, js])
    return dx, dA, dB


def rotate_fwd(z, R, adapter):
    """R [n, nblk, b, b]: y_blk = R_j z_blk."""
    n, nblk, b, _ = R.shape
    y = np.array(z, dtype=np.float64)
    for a, rows in _used(adapter, n):
        zb = np.asarray(z, dtype=np.float64)[rows].reshape(len(rows), nblk, b)
        y[rows] = np.einsum("jil,tjl->tji", R[a], zb).reshape(len(rows), nblk * b)
    return y


def rotate_bwd(dy, y, R_op, R, adapter):
    """(dz, dq): dz by the operand R_op, dq by the exact R (as the library takes them)."""
    n, nblk, b, _ = R.shape
    dz = rotate_fwd(dy, np.swapaxes(R_op, 2, 3), adapter)
    dq = np.zeros((n, nblk, b * (b - 1) // 2))
    i, l = np.triu_indices(b, 1)
    eye = np.eye(b)
    for a, rows in _used(adapter, n):
        d = dy[rows].reshape(len(rows), nblk, b)
        o = y[rows].reshape(len(rows), nblk, b)
        for j in range(nblk):
            S = d[:, j].T @ o[:, j]
            g = 0.5 * (R[a, j].T + eye) @ S @ (eye + R[a, j])
            dq[a, j] = (g - g.T)[i, l]
    return dz, dq


def clip(grads, max_norm):
    """(norm, coefficient, clipped gradients)."""
    norm = float(np.sqrt(sum(float(np.sum(np.square(g, dtype=np.float64))) for g in grads)))
    coef = min(1.0, max_norm / (norm + 1e-6))
    return norm, coef, [coef * np.asarray(g, dtype=np.float64) for g in grads]
