"""Edges of the operators on adapters of many requests: what the second product
of a low-rank update holds of the first one, what a NaN reaches, sums over very
many rows, rows and factors that only the streamed kernels see."""
import numpy as np
import pytest

from oracle import adapters as oracle
from tests import adapter_cases as cases
from tests.test_gpu_adapters import _down, _empty, _rows, _up, _ws

pytestmark = pytest.mark.gpu


def _oft():
    import orthogonal_fine_tuning_amd as oft

    return oft


# ------------------------------------- what is held between the two products
def _two_of(rng, n, rows, cols):
    """[n, rows, cols]: two entries of each row +-1, the rest 0."""
    m = np.zeros((n, rows, cols))
    at = np.argsort(rng.random((n, rows, cols)), axis=2)[:, :, :2]
    np.put_along_axis(m, at, rng.choice([-1.0, 1.0], (n, rows, 2)), axis=2)
    return m


HELD = [(5, 8), (600, 24), (600, 40), (2100, 8), (2100, 48), (700, 72)]  # T, r: both tile heights, every length of v


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,r", HELD)
def test_update_that_cancels_its_base(T, r, dtype):
    """x and A are whole numbers, and so are v (22 bits of it), the update and
    every partial sum of them, below 2^24: fp32 holds all of it.  y_base is the
    update's bf16 value, negated, and y what that rounding left: 13 bits, which
    a v of fewer than 32 bits would not have."""
    oft = _oft()
    n, K, segs = 3, 1024, (64, 80)
    rng = np.random.default_rng([T, r])
    N, R = sum(segs), 2 * r
    x, A = rng.integers(0, 128, (T, K)).astype(np.float64), rng.integers(0, 128, (n, R, K)).astype(np.float64)
    B, scale = _two_of(rng, n, N, r), np.array([0.5, 1.0, 2.0])
    a = cases.adapters(T, n, "some", 1)
    zero = np.zeros((T, N))
    update, v = oracle.lowrank_fwd(x, A, B, scale, zero, a, segs)
    mag, _ = oracle.lowrank_fwd(x, A, abs(B), scale, zero, a, segs)
    assert v.max() < 2 ** 24 and mag.max() < 2 ** 25  # (a scale of 2 is a step of 2)
    base = -cases.bf16(update).astype(np.float64)
    base[update == 0] = 1.0
    want = cases.as_type(base + update, dtype)
    d = oft.lowrank_desc(T, n, K, segs, r, oft.OFT_DT_F32 if dtype == "f32" else oft.OFT_DT_BF16)
    rows = _rows(a, n)
    ws, nb = _ws(oft.oft_lowrank_workspace_bytes(d, oft.OFT_PASS_FWD))
    gy, gv = _empty((T, N), dtype), _empty((T, R))
    f32 = lambda t: t.astype(np.float32)  # noqa: E731
    oft.oft_lowrank_fwd(d, rows, _up(f32(x), dtype), _up(f32(A), "bf16"), _up(f32(B), "bf16"), _up(f32(scale)),
                        _up(f32(base), dtype), gy, v=gv, ws=ws, ws_bytes=nb)
    assert np.array_equal(_down(gv), v)
    assert np.array_equal(_down(gy), want.astype(np.float64))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,r", HELD)
def test_gradient_that_cancels_its_base(T, r, dtype):
    """The same of dx, whose u takes the place of v."""
    oft = _oft()
    n, K, segs = 3, 128, (512, 768)
    rng = np.random.default_rng([T, r, 1])
    N, R = sum(segs), 2 * r
    dy, B = rng.integers(0, 128, (T, N)).astype(np.float64), rng.integers(0, 128, (n, N, r)).astype(np.float64)
    A, scale = np.swapaxes(_two_of(rng, n, K, R), 1, 2).copy(), np.array([0.5, 1.0, 2.0])
    a = cases.adapters(T, n, "some", 2)
    zero = np.zeros((T, K))
    v = np.zeros((T, R))
    dx, _, _ = oracle.lowrank_bwd(dy, zero, v, A, B, scale, zero, a, segs)
    mag, _, _ = oracle.lowrank_bwd(dy, zero, v, abs(A), B, scale, zero, a, segs)
    assert mag.max() < 2 ** 25
    base = -cases.bf16(dx).astype(np.float64)
    base[dx == 0] = 1.0
    want = cases.as_type(base + dx, dtype)
    d = oft.lowrank_desc(T, n, K, segs, r, oft.OFT_DT_F32 if dtype == "f32" else oft.OFT_DT_BF16)
    rows = _rows(a, n)
    ws, nb = _ws(oft.oft_lowrank_workspace_bytes(d, oft.OFT_PASS_BWD))
    gx = _empty((T, K), dtype)
    f32 = lambda t: t.astype(np.float32)  # noqa: E731
    oft.oft_lowrank_bwd(d, rows, _up(f32(dy), "bf16"), None, None, _up(f32(A), "bf16"), _up(f32(B), "bf16"),
                        _up(f32(scale)), dx=gx, dx_base=_up(f32(base), dtype), ws=ws, ws_bytes=nb)
    assert np.array_equal(_down(gx), want.astype(np.float64))
