"""The operators on adapters of many requests against the fp64 oracle: rows
sorted by adapter, low-rank updates, block rotations, and their gradients."""
import numpy as np
import pytest

from tests import adapter_cases as cases
from oracle import adapters as oracle

pytestmark = pytest.mark.gpu


def _oft():
    import orthogonal_fine_tuning_amd as oft

    return oft


def _up(a, dtype="f32"):
    import torch

    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t.to(torch.bfloat16) if dtype == "bf16" else t


def _empty(shape, dtype="f32", fill=float("nan")):
    import torch

    return torch.full(shape, fill, dtype=torch.bfloat16 if dtype == "bf16" else torch.float32, device="cuda")


def _down(t):
    return t.float().cpu().numpy().astype(np.float64)


def _within(got, want, tol, what):
    off = np.abs(_down(got) - want)
    bad = ~(off <= tol)
    assert not bad.any(), (what, int(bad.sum()), float(np.nanmax(off)), np.argwhere(bad)[:4].tolist())


def _rows(adapter, n):
    oft = _oft()
    rows = oft.adapter_rows(len(adapter), n)
    oft.oft_adapter_route(rows, _up(adapter))
    return rows


def _ws(nbytes):
    import torch

    return torch.full((max(16, nbytes),), 0xFF, dtype=torch.uint8, device="cuda"), nbytes


# --------------------------------------------------------------------- route
@pytest.mark.parametrize("kind", ["mixed", "runs", "one", "none", "some"])
@pytest.mark.parametrize("T,n", [(1, 1), (3, 2), (64, 64), (256, 128), (256, 129), (257, 128), (65, 1), (1000, 7), (1024, 1024), (1025, 1000), (4097, 33),
                                 (30001, 1024),
                                 (65536, 7), (65537, 300), (524288, 5), (600001, 900)])
def test_route(T, n, kind):
    a = cases.adapters(T, n, kind)
    rows = _rows(a, n)
    order, offsets = oracle.route(a, n)
    assert np.array_equal(rows.offsets.cpu().numpy(), offsets)
    assert np.array_equal(rows.order.cpu().numpy(), order)


@pytest.mark.parametrize("T,n", [(1, 1), (65, 3), (1000, 7), (2048, 40), (2049, 3), (5000, 1024), (20000, 5), (40000, 1000)])
@pytest.mark.parametrize("kind", ["mixed", "some", "none", "skewed"])
def test_route_lists(T, n, kind):
    """Every list covers each row once, in pieces of one adapter and the list's size."""
    a = cases.adapters(T, n, kind)
    rows = _rows(a, n)
    order, offsets = oracle.route(a, n)
    tiles = rows.tiles.cpu().numpy()
    up4 = lambda k: (k + 3) & ~3  # noqa: E731
    at = 8 + 2 * up4(n + 1)
    piece = lambda d: max(64, ((T + d - 1) // d + 63) & ~63)  # noqa: E731
    for i, size in enumerate((16, 64, piece(4), piece(16))):
        cap = 0 if i == 0 and T > 2048 else min(T, T // size + n + 1)
        got = tiles[at:at + 4 * cap].reshape(-1, 4)[:tiles[i]]
        at += 4 * cap
        if i == 0 and T > 2048:
            assert tiles[i] == 0
            continue
        want, slot = [], 0
        bounds = offsets.tolist() + [T]
        for g in range(n + 1):
            lo, hi = bounds[g], bounds[g + 1]
            several = i >= 2 and g < n and hi - lo > size
            for p in range(lo, hi, size):
                want.append((g if g < n else -1, p, min(size, hi - p), slot if several else -1))
                slot += several
        assert got.tolist() == [list(w) for w in want]
        assert slot <= (8 if i == 2 else 32)


# ------------------------------------------------------------------ low rank
SHAPES = [  # T, n, K, segments, r, kind
    (1, 1, 64, (16,), 8, "one"),
    (5, 3, 256, (128, 128, 128), 8, "mixed"),
    (64, 64, 320, (16, 48, 208), 16, "mixed"),
    (33, 4, 128, (32, 1040), 24, "some"),
    (130, 3, 2560, (64, 64), 128, "runs"),
    (1024, 9, 192, (112,), 40, "skewed"),
    (1025, 5, 256, (384,), 72, "mixed"),
    (1500, 3, 128, (80, 176), 32, "some"),
    (2050, 40, 64, (16,) * 8, 16, "runs"),
    (2051, 2, 512, (64,) * 8, 128, "skewed"),
    (40, 5, 128, (64,), 16, "none"),
    (2100, 5, 128, (32,) * 8, 32, "some"),     # 32 rows at a time
    (1300, 3, 128, (80,), 48, "mixed"),
    (1200, 2, 64, (48,), 24, "runs"),
    (2060, 2, 64, (48,), 24, "runs"),
    (2070, 3, 128, (80, 16), 48, "mixed"),
    (513, 2, 64, (48,), 40, "some"),
    (512, 2, 64, (48,), 40, "some"),
    (300, 2, 64, (16384,), 64, "skewed"),      # pieces of a quarter of the rows, by their number
    (2100, 3, 64, (9728,), 128, "skewed"),     # or by the columns
    (40001, 2, 64, (16,), 8, "skewed"),        # pieces of more rows than have their numbers in LDS
]


def _lowrank(shape, dtype):
    T, n, K, segs, r, kind = shape
    oft = _oft()
    c = cases.lowrank(T, n, K, segs, r, dtype, kind)
    t = {k: _up(v, dtype if k in ("x", "y_base", "dx_base") else "bf16" if k in ("A", "B", "dy") else "f32")
         for k, v in c.items()}
    d = oft.lowrank_desc(T, n, K, segs, r, oft.OFT_DT_F32 if dtype == "f32" else oft.OFT_DT_BF16)
    return c, t, d, _rows(c["adapter"], n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_lowrank_fwd(shape, dtype):
    oft = _oft()
    T, n, K, segs, r, _ = shape
    c, t, d, rows = _lowrank(shape, dtype)
    (y, ytol), (v, vtol) = cases.lowrank_fwd(c, segs, dtype)
    gy, gv = _empty((T, sum(segs)), dtype), _empty((T, r * len(segs)))
    ws, nb = _ws(oft.oft_lowrank_workspace_bytes(d, oft.OFT_PASS_FWD))
    oft.oft_lowrank_fwd(d, rows, t["x"], t["A"], t["B"], t["scale"], t["y_base"], gy, v=gv, ws=ws, ws_bytes=nb)
    _within(gy, y, ytol, "y")
    _within(gv, v, vtol, "v")
    # onto y_base itself, without v: the same bits
    oft.oft_lowrank_fwd(d, rows, t["x"], t["A"], t["B"], t["scale"], t["y_base"], t["y_base"], ws=ws, ws_bytes=nb)
    assert (t["y_base"] == gy).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_lowrank_bwd(shape, dtype):
    oft = _oft()
    T, n, K, segs, r, _ = shape
    c, t, d, rows = _lowrank(shape, dtype)
    _, (v, _) = cases.lowrank_fwd(c, segs, dtype)
    v = v.astype(np.float32)
    (dx, xtol), (dA, atol), (dB, btol) = cases.lowrank_bwd(c, v, segs, dtype)
    gx, gA, gB = _empty((T, K), dtype), _empty(dA.shape), _empty(dB.shape)
    ws, nb = _ws(oft.oft_lowrank_workspace_bytes(d, oft.OFT_PASS_BWD))
    args = (d, rows, t["dy"], t["x"], _up(v), t["A"], t["B"], t["scale"])
    oft.oft_lowrank_bwd(*args, dx=gx, dx_base=t["dx_base"], dA=gA, dB=gB, ws=ws, ws_bytes=nb)
    _within(gx, dx, xtol, "dx")
    _within(gA, dA, atol, "dA")
    _within(gB, dB, btol, "dB")
    # each alone, dx without a base and onto its base: the same bits
    one = _empty(dA.shape)
    oft.oft_lowrank_bwd(*args, dA=one, ws=ws, ws_bytes=nb)
    assert (one == gA).all()
    one = _empty(dB.shape)
    oft.oft_lowrank_bwd(*args, dB=one, ws=ws, ws_bytes=nb)
    assert (one == gB).all()
    oft.oft_lowrank_bwd(*args, dx=t["dx_base"], dx_base=t["dx_base"], ws=ws, ws_bytes=nb)
    assert (t["dx_base"] == gx).all()
    (dx, xtol), _, _ = cases.lowrank_bwd(c, v, segs, dtype, with_base=False)
    oft.oft_lowrank_bwd(*args, dx=gx, ws=ws, ws_bytes=nb)
    _within(gx, dx, xtol, "dx alone")


# ------------------------------------------------------------------- rotations
ROT = [  # T, n, N, kind
    (1, 1, 32, "one"),
    (7, 3, 96, "mixed"),
    (64, 64, 384, "mixed"),
    (65, 4, 160, "some"),
    (1024, 6, 128, "runs"),
    (1025, 6, 416, "skewed"),
    (2500, 3, 64, "some"),
    (3001, 70, 32, "mixed"),
    (50, 2, 96, "none"),
    (300, 2, 16416, "skewed"),  # pieces of a quarter of the rows
    (40001, 2, 32, "skewed"),   # pieces of more rows than have their numbers in LDS
]


def _rotate(shape, b, dtype):
    T, n, N, kind = shape
    oft = _oft()
    import torch

    rng = np.random.default_rng([T, n, N, b])
    p, _ = cases.rotations(n, N // b, b)
    Rf = torch.empty((n, N // b, b, b), dtype=torch.float32, device="cuda")
    Rops = torch.empty((n, N // b, 2, b, b), dtype=torch.bfloat16, device="cuda")
    oft.cayley_build(_up(p, "bf16"), n * (N // b), b, Rf, Rops)
    a = cases.adapters(T, n, kind)
    z, dy = cases.as_type(rng.normal(0, 1, (T, N)), dtype), cases.bf16(rng.normal(0, 1, (T, N)))
    d = oft.rotate_desc(T, n, N, b, oft.OFT_DT_F32 if dtype == "f32" else oft.OFT_DT_BF16)
    return a, z, dy, Rf, Rops, d, _rows(a, n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("b", [16, 32])
@pytest.mark.parametrize("shape", ROT, ids=str)
def test_rotate_fwd(shape, b, dtype):
    oft = _oft()
    T, n, N, _ = shape
    a, z, _, Rf, Rops, d, rows = _rotate(shape, b, dtype)
    y, tol = cases.rotate_fwd(z.astype(np.float64), _down(Rops[:, :, 0]), a, dtype)
    tz, gy = _up(z, dtype), _empty((T, N), dtype)
    oft.oft_rotate_fwd(d, rows, tz, Rops, gy)
    _within(gy, y, tol, "y")
    oft.oft_rotate_fwd(d, rows, tz, Rops, tz)
    assert (tz == gy).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("b", [16, 32])
@pytest.mark.parametrize("shape", ROT, ids=str)
def test_rotate_bwd(shape, b, dtype):
    oft = _oft()
    T, n, N, _ = shape
    a, y, dy, Rf, Rops, d, rows = _rotate(shape, b, dtype)
    (dz, ztol), (dq, qtol) = cases.rotate_bwd(dy.astype(np.float64), y.astype(np.float64), _down(Rops[:, :, 0]),
                                              _down(Rf), a, dtype)
    tdy, ty = _up(dy, "bf16"), _up(y, dtype)
    gz, gq = _empty((T, N), "bf16"), _empty(dq.shape)
    ws, nb = _ws(oft.oft_rotate_workspace_bytes(d, oft.OFT_PASS_BWD))
    oft.oft_rotate_bwd(d, rows, tdy, ty, Rf, Rops, dz=gz, dq=gq, ws=ws, ws_bytes=nb)
    _within(gz, dz, ztol, "dz")
    _within(gq, dq, qtol, "dq")
    one = _empty(dq.shape)
    oft.oft_rotate_bwd(d, rows, tdy, ty, Rf, Rops, dq=one, ws=ws, ws_bytes=nb)
    assert (one == gq).all()
    one = _empty((T, N), "bf16")
    oft.oft_rotate_bwd(d, rows, tdy, None, None, Rops, dz=one)
    assert (one == gz).all()
    oft.oft_rotate_bwd(d, rows, tdy, ty, Rf, Rops, dz=tdy, dq=one_dq(dq.shape), ws=ws, ws_bytes=nb)
    assert (tdy == gz).all()


def one_dq(shape):
    return _empty(shape)
