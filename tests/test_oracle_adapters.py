"""Pins for the oracle of the operators on adapters of many requests and of the
gradient clipping: closed forms and central differences."""
import math

import numpy as np
import pytest

from oracle import adapters as oracle
from oracle import dense


def _central(f, x, h=1e-5):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        g[i] = (f(a) - f(b)) / (2 * h)
    return g


def test_route_is_stable_and_puts_rows_without_an_adapter_last():
    order, offsets = oracle.route([2, -1, 0, 2, 3, 0, 7], 3)
    assert order.tolist() == [2, 5, 0, 3, 1, 4, 6]
    assert offsets.tolist() == [0, 2, 2, 4]
    order, offsets = oracle.route([], 2)
    assert order.size == 0 and offsets.tolist() == [0, 0, 0]


SEGS = (3, 5)
ADAPTER = np.array([1, 0, -1, 1, 2, 1])


def _lowrank(seed):
    rng = np.random.default_rng(seed)
    n, r, K, N = 4, 2, 6, sum(SEGS)
    return (rng.normal(size=(6, K)), rng.normal(size=(n, r * len(SEGS), K)), rng.normal(size=(n, N, r)),
            rng.uniform(0.5, 2, n), rng.normal(size=(6, N)), rng.normal(size=(6, N)))


def test_lowrank_row_by_row():
    x, A, B, scale, y0, _ = _lowrank(0)
    y, v = oracle.lowrank_fwd(x, A, B, scale, y0, ADAPTER, SEGS)
    assert np.array_equal(y[2], y0[2]) and not v[2].any()
    for t in (0, 1, 3, 4, 5):
        a = ADAPTER[t]
        up = np.concatenate([B[a, :3] @ A[a, :2], B[a, 3:] @ A[a, 2:]])  # the whole update
        assert np.allclose(y[t], y0[t] + scale[a] * (up @ x[t]), atol=1e-13)


def test_lowrank_gradients_by_differences():
    x, A, B, scale, y0, dy = _lowrank(1)
    _, v = oracle.lowrank_fwd(x, A, B, scale, y0, ADAPTER, SEGS)
    base = np.random.default_rng(2).normal(size=x.shape)
    dx, dA, dB = oracle.lowrank_bwd(dy, x, v, A, B, scale, base, ADAPTER, SEGS)
    loss = lambda x, A, B: float((dy * oracle.lowrank_fwd(x, A, B, scale, y0, ADAPTER, SEGS)[0]).sum())  # noqa: E731
    assert np.allclose(dx - base, _central(lambda z: loss(z, A, B), x), atol=1e-8)
    assert np.allclose(dA, _central(lambda z: loss(x, z, B), A), atol=1e-8)
    assert np.allclose(dB, _central(lambda z: loss(x, A, z), B), atol=1e-8)
    assert not dA[3].any() and not dB[3].any()  # no rows


def _cayley(p, b):
    n, nblk, _ = p.shape
    q = np.zeros((n, nblk, b, b))
    i, l = np.triu_indices(b, 1)
    q[..., i, l] = p
    q[..., l, i] = -p
    return np.linalg.solve(np.eye(b) - q, np.eye(b) + q)


def test_rotation_gradients_by_differences():
    rng = np.random.default_rng(3)
    n, nblk, b = 3, 2, 4
    p = rng.normal(0, 0.3, (n, nblk, 6))
    z, dy = rng.normal(size=(6, nblk * b)), rng.normal(size=(6, nblk * b))
    adapter = np.array([1, 0, 5, 1, 1, 0])
    R = _cayley(p, b)
    y = oracle.rotate_fwd(z, R, adapter)
    assert np.array_equal(y[2], z[2])
    assert np.allclose(np.linalg.norm(y, axis=1), np.linalg.norm(z, axis=1))
    dz, dq = oracle.rotate_bwd(dy, y, R, R, adapter)
    assert np.allclose(dz, _central(lambda t: float((dy * oracle.rotate_fwd(t, R, adapter)).sum()), z), atol=1e-8)
    assert np.allclose(dq, _central(lambda t: float((dy * oracle.rotate_fwd(z, _cayley(t, b), adapter)).sum()), p), atol=1e-7)
    assert not dq[2].any()


def test_rotation_of_one_adapter_is_the_dense_layers():
    rng = np.random.default_rng(4)
    b, nblk, T = 16, 2, 5
    p = rng.normal(0, 0.1, (nblk, b * (b - 1) // 2)).astype(np.float32)
    bits = (p.view(np.uint32) >> 16).astype(np.uint16)
    R = dense.cayley(bits, b)
    z = rng.normal(size=(T, nblk * b))
    want = np.concatenate([z[:, j * b:(j + 1) * b] @ R[j].T for j in range(nblk)], axis=1)
    assert np.allclose(oracle.rotate_fwd(z, R[None], np.zeros(T, int)), want, atol=1e-13)


@pytest.mark.parametrize("max_norm,coef", [(10.0, 1.0), (2.5, 2.5 / (5 + 1e-6)), (0.0, 0.0)])
def test_clip(max_norm, coef):
    norm, c, out = oracle.clip([np.array([3.0]), np.zeros(0), np.array([0.0, -4.0])], max_norm)
    assert norm == 5.0 and math.isclose(c, coef, rel_tol=1e-15)
    assert np.allclose(np.concatenate(out), c * np.array([3.0, 0.0, -4.0]))
