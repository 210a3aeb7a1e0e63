"""Edges of the operators on adapters of many requests: what the second product
of a low-rank update holds of the first one, what a NaN reaches, sums over very
many rows, rows and factors that only the streamed kernels see."""
import numpy as np
import pytest

from oracle import adapters as oracle
from tests import adapter_cases as cases
from tests import test_gpu_adapters as plain
from tests import test_gpu_adapters_use as use
from tests.test_gpu_adapters import _down, _empty, _rows, _up, _within, _ws

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


# ------------------------------------------------ what a NaN or infinity reaches
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("b", [16, 32])
@pytest.mark.parametrize("T", [40, 1500])
def test_blocks_of_a_rotated_row_are_apart(T, b, dtype, bad):
    """A block's y, dz and dq depend on the block alone: one bad channel leaves
    all others as they are, bit for bit."""
    import torch

    oft = _oft()
    n, N = 3, 160
    rng = np.random.default_rng([T, b])
    p, _ = cases.rotations(n, N // b, b)
    Rf = torch.empty((n, N // b, b, b), device="cuda")
    Rops = torch.empty((n, N // b, 2, b, b), dtype=torch.bfloat16, device="cuda")
    oft.cayley_build(_up(p, "bf16"), n * (N // b), b, Rf, Rops)
    a = cases.adapters(T, n, "mixed")
    rows = _rows(a, n)
    d = oft.rotate_desc(T, n, N, b, oft.OFT_DT_F32 if dtype == "f32" else oft.OFT_DT_BF16)
    z, dy = _up(cases.as_type(rng.normal(0, 1, (T, N)), dtype), dtype), _up(cases.bf16(rng.normal(0, 1, (T, N))), "bf16")
    ws, nb = _ws(oft.oft_rotate_workspace_bytes(d, oft.OFT_PASS_BWD))
    saved = z.clone()  # (any rows do for the saved output)

    def run(z, dy, saved):
        y, dz, alone = _empty((T, N), dtype), _empty((T, N), "bf16"), _empty((T, N), "bf16")
        dq = _empty((n, N // b, b * (b - 1) // 2))
        oft.oft_rotate_fwd(d, rows, z, Rops, y)
        oft.oft_rotate_bwd(d, rows, dy, None, None, Rops, dz=alone)
        oft.oft_rotate_bwd(d, rows, dy, saved, Rf, Rops, dz=dz, dq=dq, ws=ws, ws_bytes=nb)
        return y, alone, dz, dq

    clean = run(z, dy, saved)
    for t, ch in ((0, 5), (T // 2, N - 20), (T - 1, 37)):
        blk, ad = ch // b, int(a[t])
        bz, bd, bs = z.clone(), dy.clone(), saved.clone()
        bz[t, ch] = bd[t, ch] = bad
        got = run(bz, bd, bs)
        for g, c in zip(got[:3], clean[:3]):
            hit = torch.zeros((T, N), dtype=torch.bool, device="cuda")
            hit[t, blk * b:(blk + 1) * b] = True
            assert torch.equal(g[~hit], c[~hit]), (t, ch)
            assert not torch.isfinite(g[hit]).all()
        hit = torch.zeros((n, N // b), dtype=torch.bool, device="cuda")
        hit[ad, blk] = True
        assert torch.equal(got[3][~hit], clean[3][~hit]) and not torch.isfinite(got[3][hit]).all(), (t, ch)


# ------------------------------------------------------ sums over very many rows
# A few large products and then small ones, LARGE / 2^30 each: the 32 of a
# matrix step are a quarter of a step of fp32 beside the large ones' sum, and a
# sum of them all in one accumulator loses every one.  Sums of at most 2048
# rows that are then added to each other lose those beside the large ones
# alone: the small sums are whole multiples of the large one's step.
LONG_T, LARGE, SMALL, FIRST, CHAIN = 1 << 20, 2.0 ** 20, 2.0 ** -5, 32, 2048


def _long(n):
    """(adapters of LONG_T rows in n runs, the row's values, sums by adapter, how far they may be off)."""
    a = (np.arange(LONG_T, dtype=np.int64) * n // LONG_T).astype(np.int32)
    counts = np.bincount(a, minlength=n)
    first = np.concatenate([[0], np.cumsum(counts)[:-1]])
    val = np.full(LONG_T, SMALL, dtype=np.float32)
    for f in first:
        val[f:f + FIRST] = LARGE
    want = FIRST * LARGE + (counts - FIRST) * SMALL
    # what a chain beside the large products may lose, and two steps of the
    # whole (4 each) for the last chain, whose sum is no multiple of them
    return a, val, want, CHAIN * SMALL + 8.0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 20])
def test_lowrank_sums_over_many_rows(n, dtype):
    import torch

    oft = _oft()
    K, N, r = 64, 16, 8
    a, val, want, tol = _long(n)
    rows = _rows(a, n)
    col = _up(val)[:, None]
    one = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    x = torch.zeros((LONG_T, K), dtype=torch.float32 if dtype == "f32" else torch.bfloat16, device="cuda")
    x[:, 3:5] = col
    v = torch.zeros((LONG_T, r), device="cuda")
    v[:, 2:4] = col
    dy, A, B = one(LONG_T, N), one(n, r, K), one(n, N, r)
    dy[:, 1] = 1.0
    B[:, 1, 6] = 1.0  # u = 1 in column 6
    d = oft.lowrank_desc(LONG_T, n, K, (N,), r, oft.OFT_DT_F32 if dtype == "f32" else oft.OFT_DT_BF16)
    dA, dB = _empty((n, r, K)), _empty((n, N, r))
    ws, nb = _ws(oft.oft_lowrank_workspace_bytes(d, oft.OFT_PASS_BWD))
    oft.oft_lowrank_bwd(d, rows, dy, x, v, A, B, torch.ones(n, device="cuda"), dA=dA, dB=dB, ws=ws, ws_bytes=nb)
    gA, gB = _down(dA), _down(dB)
    for got in (gA[:, 6, 3], gA[:, 6, 4], gB[:, 1, 2], gB[:, 1, 3]):
        assert (np.abs(got - want) <= tol).all(), (got - want, tol)
    gA[:, 6, 3:5] = 0
    gB[:, 1, 2:4] = 0
    assert not gA.any() and not gB.any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 20])
@pytest.mark.parametrize("b", [16, 32])
def test_rotation_sums_over_many_rows(b, n, dtype):
    """Identity rotations: dq = 2 (S - S^T)."""
    import torch

    oft = _oft()
    N = 32
    a, val, want, tol = _long(n)
    rows = _rows(a, n)
    y = torch.zeros((LONG_T, N), dtype=torch.float32 if dtype == "f32" else torch.bfloat16, device="cuda")
    y[:, 7] = _up(val)
    dy = torch.zeros((LONG_T, N), dtype=torch.bfloat16, device="cuda")
    dy[:, 2] = 1.0
    eye = torch.eye(b, device="cuda").expand(n, N // b, b, b).contiguous()
    ops = torch.stack([eye, eye], 2).bfloat16().contiguous()
    d = oft.rotate_desc(LONG_T, n, N, b, oft.OFT_DT_F32 if dtype == "f32" else oft.OFT_DT_BF16)
    dq, dz = _empty((n, N // b, b * (b - 1) // 2)), _empty((LONG_T, N), "bf16")
    ws, nb = _ws(oft.oft_rotate_workspace_bytes(d, oft.OFT_PASS_BWD))
    oft.oft_rotate_bwd(d, rows, dy, y, eye, ops, dz=dz, dq=dq, ws=ws, ws_bytes=nb)
    assert torch.equal(dz, dy)
    got = _down(dq)
    i, l = np.triu_indices(b, 1)
    at = int(np.flatnonzero((i == 2) & (l == 7))[0])
    assert (np.abs(got[:, 0, at] - 2 * want) <= 2 * tol).all(), (got[:, 0, at] - 2 * want, tol)
    got[:, 0, at] = 0
    assert not got.any()


# ------------------------------------------------------------- rows never sorted
@pytest.mark.parametrize("fill", [-2 ** 31, -1, 0, 5, 2 ** 31 - 1, None])
@pytest.mark.parametrize("T", [70, 3000])
def test_arrays_that_were_never_written_stay_inside(T, fill):
    """Whatever an order, its offsets and lists hold, a call writes to its own
    results and nothing else: guards around every one of them are left alone."""
    import torch

    oft = _oft()
    n, K, segs, r, b = 4, 128, (64, 96), 16, 32
    N, R = sum(segs), 2 * r
    rng = np.random.default_rng([T, 0 if fill is None else fill % 1000])
    rows = oft.adapter_rows(T, n)
    for t in (rows.order, rows.offsets, rows.tiles):
        if fill is None:
            t.copy_(torch.from_numpy(rng.integers(-2 ** 31, 2 ** 31, t.numel()).astype(np.int32)))
        else:
            t.fill_(fill)
    guarded = []

    def out(*shape, dtype=torch.float32):
        count = int(np.prod(shape))
        buf = torch.full((count + 512,), 7.0, dtype=dtype, device="cuda")
        guarded.append((buf, count))
        return buf[256:256 + count].view(*shape)

    bf = dict(dtype=torch.bfloat16)
    ones = lambda *s: torch.ones(s, device="cuda", **bf)  # noqa: E731
    ld, rd = oft.lowrank_desc(T, n, K, segs, r), oft.rotate_desc(T, n, N, b)
    need = [oft.oft_lowrank_workspace_bytes(ld, 0), oft.oft_lowrank_workspace_bytes(ld, 1), oft.oft_rotate_workspace_bytes(rd, 1)]
    ws = [out(nb // 4) for nb in need]
    scale = torch.ones(n, device="cuda")
    Rf = torch.eye(b, device="cuda").expand(n, N // b, b, b).contiguous()
    Rops = torch.stack([Rf, Rf], 2).bfloat16().contiguous()
    oft.oft_lowrank_fwd(ld, rows, ones(T, K), ones(n, R, K), ones(n, N, r), scale, ones(T, N), out(T, N, **bf), v=out(T, R),
                        ws=ws[0], ws_bytes=need[0])
    oft.oft_lowrank_bwd(ld, rows, ones(T, N), ones(T, K), torch.ones((T, R), device="cuda"), ones(n, R, K), ones(n, N, r),
                        scale, dx=out(T, K, **bf), dA=out(n, R, K), dB=out(n, N, r), ws=ws[1], ws_bytes=need[1])
    oft.oft_rotate_fwd(rd, rows, ones(T, N), Rops, out(T, N, **bf))
    oft.oft_rotate_bwd(rd, rows, ones(T, N), ones(T, N), Rf, Rops, dz=out(T, N, **bf), dq=out(n, N // b, b * (b - 1) // 2),
                       ws=ws[2], ws_bytes=need[2])
    torch.cuda.synchronize()
    for buf, count in guarded:
        assert bool((buf[:256] == 7).all()) and bool((buf[256 + count:] == 7).all())


# --------------------------------------------------- fp32 rows times an fp32 u
@pytest.mark.parametrize("T", [3, 70])
def test_products_of_fp32_values_keep_their_bits(T):
    """A row an adapter: dA is one product u x.  Both factors are 1 and then all
    ones from the eighth bit on, so that their parts below the first are as
    large as parts can be.  The product is exact but for the parts' own sums
    (the last is off by a step at most, 2^-23 of it, those before it by 2^-7 of
    that each) and the scale's rounding (half a step)."""
    import torch

    oft = _oft()
    K, N, r = 64, 32, 8
    val = 1.0 + 2.0 ** -7 - 2.0 ** -23
    rows = _rows(np.arange(T, dtype=np.int32), T)
    x = torch.full((T, K), val, device="cuda")
    x[:, 1::2] *= -4.0
    dy, B = torch.zeros((T, N), device="cuda"), torch.zeros((T, N, r), device="cuda")
    dy[:, 2:5] = 1.0
    B[:, 2], B[:, 3], B[:, 4] = 1.0, 2.0 ** -7, -(2.0 ** -23)  # u = val, exactly
    d = oft.lowrank_desc(T, T, K, (N,), r, oft.OFT_DT_F32)
    dA = _empty((T, r, K))
    ws, nb = _ws(oft.oft_lowrank_workspace_bytes(d, oft.OFT_PASS_BWD))
    oft.oft_lowrank_bwd(d, rows, dy.bfloat16(), x, None, None, B.bfloat16(), torch.ones(T, device="cuda"), dA=dA, ws=ws,
                        ws_bytes=nb)
    want = val * _down(x)[:, None, :]
    assert (np.abs(_down(dA) - want) <= 4 * cases.U * np.abs(want)).all()


def test_descriptor_without_blocks_is_refused():
    import torch

    oft = _oft()
    rows = _rows(np.zeros(4, dtype=np.int32), 2)
    bf = lambda *s: torch.ones(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    d = oft.rotate_desc(4, 2, 64, 0)
    with pytest.raises(ValueError):  # (no R_ops has blocks of 0 channels)
        oft.oft_rotate_fwd(d, rows, bf(4, 64), bf(2, 2, 2, 32, 32), bf(4, 64))
    with pytest.raises(oft.OftError):
        oft.oft_rotate_fwd(d, rows, bf(4, 64), bf(2, 0, 2, 0, 0), bf(4, 64))
    with pytest.raises(oft.OftError):
        oft.oft_rotate_bwd(d, rows, bf(4, 64), None, None, bf(2, 0, 2, 0, 0), dz=bf(4, 64))


# ------------------------------------------- rows and ranks of the streamed kernels
def _picked(T):
    return np.concatenate([[0, 1, T - 2, T - 1], np.random.default_rng(1).integers(0, T, 60)])


@pytest.mark.parametrize("r", [16, 48, 72])
def test_streamed_low_rank(r):
    """Rows of more bytes than the caches hold, both directions, every length
    of v that the kernel keeps in another way: rows picked from them, in 64 bits."""
    import torch

    oft = _oft()
    T, n, wide, thin = 36000, 3, 2048, 64
    g = torch.Generator(device="cuda").manual_seed(r)
    bf = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    ad = torch.randint(-1, n, (T,), generator=g, device="cuda").int()
    rows = oft.adapter_rows(T, n)
    oft.oft_adapter_route(rows, ad)
    scale = torch.tensor([0.5, 1.0, 2.0], device="cuda")
    pick = _picked(T)
    base = bf(T, wide)
    for K, N in ((thin, wide), (wide, thin)):
        d = oft.lowrank_desc(T, n, K, (N,), r)
        x, dy, A, B = bf(T, K), bf(T, N), bf(n, r, K) / 8, bf(n, N, r) / 4
        c = {"x": _down(x[pick]), "dy": _down(dy[pick]), "A": _down(A), "B": _down(B), "scale": _down(scale),
             "adapter": ad.cpu().numpy()[pick]}
        got = torch.empty_like(base)
        if N == wide:
            ws, nb = _ws(oft.oft_lowrank_workspace_bytes(d, oft.OFT_PASS_FWD))
            oft.oft_lowrank_fwd(d, rows, x, A, B, scale, base, got, ws=ws, ws_bytes=nb)
            (want, tol), _ = cases.lowrank_fwd({**c, "y_base": _down(base[pick])}, (N,), "bf16")
        else:
            ws, nb = _ws(oft.oft_lowrank_workspace_bytes(d, oft.OFT_PASS_BWD))
            oft.oft_lowrank_bwd(d, rows, dy, None, None, A, B, scale, dx=got, dx_base=base, ws=ws, ws_bytes=nb)
            (want, tol), _, _ = cases.lowrank_bwd({**c, "dx_base": _down(base[pick])}, np.zeros((len(pick), r)), (N,), "bf16")
        _within(got[pick], want, tol, (r, K, N))
        none = ad < 0
        assert torch.equal(got[none], base[none])


@pytest.mark.parametrize("b", [16, 32])
def test_streamed_rotation_gradients_of_fp32_rows(b):
    """dz against calls of 1000 rows, bit for bit; dq of some blocks in 64 bits."""
    import torch

    oft = _oft()
    T, n, N, few = 36000, 3, 2048, 4
    g = torch.Generator(device="cuda").manual_seed(b)
    ad = torch.randint(-1, n, (T,), generator=g, device="cuda").int()
    y, dy = torch.randn((T, N), generator=g, device="cuda"), torch.randn((T, N), generator=g, device="cuda").bfloat16()
    p, _ = cases.rotations(n, N // b, b)
    Rf = torch.empty((n, N // b, b, b), device="cuda")
    Rops = torch.empty((n, N // b, 2, b, b), dtype=torch.bfloat16, device="cuda")
    oft.cayley_build(_up(p, "bf16"), n * (N // b), b, Rf, Rops)
    rows = oft.adapter_rows(T, n)
    oft.oft_adapter_route(rows, ad)
    d = oft.rotate_desc(T, n, N, b, oft.OFT_DT_F32)
    dz, dq = torch.empty_like(dy), _empty((n, N // b, b * (b - 1) // 2))
    ws, nb = _ws(oft.oft_rotate_workspace_bytes(d, oft.OFT_PASS_BWD))
    oft.oft_rotate_bwd(d, rows, dy, y, Rf, Rops, dz=dz, dq=dq, ws=ws, ws_bytes=nb)
    for at in range(0, T, 1000):
        part = oft.adapter_rows(1000, n)
        oft.oft_adapter_route(part, ad[at:at + 1000].clone())
        one = torch.empty((1000, N), dtype=torch.bfloat16, device="cuda")
        oft.oft_rotate_bwd(oft.rotate_desc(1000, n, N, b), part, dy[at:at + 1000].clone(), None, None, Rops, dz=one)
        assert torch.equal(one, dz[at:at + 1000])
    i, l = np.triu_indices(b, 1)
    eye = np.eye(b)
    for k in range(n):
        sel = (ad == k).nonzero()[:, 0]
        o, s = _down(dy[sel, :few * b]).reshape(-1, few, b), _down(y[sel, :few * b]).reshape(-1, few, b)
        for j in range(few):
            R = _down(Rf[k, j])
            gq = 0.5 * (R.T + eye) @ (o[:, j].T @ s[:, j]) @ (eye + R)
            m = abs(o[:, j]).T @ abs(s[:, j])
            e = 0.5 * (abs(R).T + eye) @ (cases.sum_err(len(sel), m) + 4 * cases.U * (b + 64) * m) @ (eye + abs(R))
            assert (np.abs(_down(dq[k, j]) - (gq - gq.T)[i, l]) <= (e + e.T)[i, l]).all(), (k, j)


@pytest.mark.parametrize("kind", ["mixed", "some", "none", "skewed"])
def test_lists_of_rows_sorted_eight_steps_a_wave(kind):
    plain.test_route_lists(600001, 900, kind)


def test_graphs_of_sums_in_several_chains():
    """Pieces of more rows than one accumulator takes, replayed by two graphs
    that share their workspaces: what a replay before left is not added to."""
    use.test_graphs_that_share_workspaces_follow_their_inputs(41000)
