"""Global gradient norm and clipping against the fp64 oracle."""
import numpy as np
import pytest

from oracle import adapters as oracle
from tests.adapter_cases import HALF, U, as_type

pytestmark = pytest.mark.gpu


def _oft():
    import orthogonal_fine_tuning_amd as oft

    return oft


def _tensors(sizes, dtype, seed, size=1.0, odd=False):
    """Views of one buffer (odd: starting at any element), and their values."""
    import torch

    rng = np.random.default_rng(seed)
    gap = [int(rng.integers(0, 9)) if odd else 0 for _ in sizes]
    buf = torch.full((sum(gap) + sum((s + 15) & ~15 if not odd else s for s in sizes) + 16,), 7.0,
                     dtype=torch.bfloat16 if dtype == "bf16" else torch.float32, device="cuda")
    out, vals, at = [], [], 0
    for s, g in zip(sizes, gap):
        at += g
        v = as_type(size * rng.normal(0, 1, s), dtype)
        t = buf[at:at + s]
        t.copy_(torch.from_numpy(v))
        out.append(t)
        vals.append(v)
        at += s if odd else (s + 15) & ~15
    return buf, out, vals


def _clip(grads, out, max_norm):
    import torch

    oft = _oft()
    lst = oft.grad_list(grads, out)
    nb = oft.oft_grad_workspace_bytes(lst)
    ws = torch.full((max(16, nb),), 0xFF, dtype=torch.uint8, device="cuda")
    sumsq = torch.full((1,), float("nan"), dtype=torch.float64, device="cuda")
    stats = torch.full((2,), float("nan"), device="cuda")
    oft.oft_grad_sumsq(lst, sumsq, ws=ws, ws_bytes=nb)
    oft.oft_grad_clip(lst, sumsq, max_norm, stats)
    return float(sumsq), stats.cpu().numpy().astype(np.float64)


SIZES = [[1], [7], [0, 5, 0], [120, 2880, 1], [16384], [16385, 1], [3] * 17, [1000] * 250, [40000, 1, 99999, 12345],
         [3000001, 17]]


@pytest.mark.parametrize("max_norm", [0.5, 1e6])
@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[0]}")
def test_clip(sizes, dtype, odd, max_norm):
    import torch

    buf, grads, vals = _tensors(sizes, dtype, [len(sizes), sizes[0]], odd=odd)
    norm, coef, want = oracle.clip(vals, max_norm)
    _, outs, _ = _tensors(sizes, dtype, 1, odd=odd)
    before = buf.clone()
    sumsq, stats = _clip(grads, outs, max_norm)
    # squares and sums in fp64: an fp32 rounding of the norm, a few of the coefficient
    assert abs(sumsq - norm ** 2) <= 1e-9 * norm ** 2
    assert abs(stats[0] - norm) <= 2 * U * norm
    assert abs(stats[1] - coef) <= 8 * U * coef
    for o, w, v in zip(outs, want, vals):
        tol = 10 * U * np.abs(w) + HALF[dtype] * np.abs(w) * (1 + 10 * U) + 2.0 ** -126
        assert (np.abs(o.float().cpu().numpy() - w) <= tol).all()
    assert torch.equal(buf, before)
    # in place: the same bits, and nothing between the tensors touched
    _clip(grads, None, max_norm)
    for g, o in zip(grads, outs):
        assert torch.equal(g, o)
        g.fill_(7.0)
    assert (buf == 7.0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_outputs_at_another_alignment(dtype):
    import torch

    _, grads, vals = _tensors([5000, 33], dtype, 3)
    buf = torch.full((5200,), 7.0, dtype=grads[0].dtype, device="cuda")
    outs = [buf[1:5001], buf[5101:5134]]
    _clip(grads, outs, 1.0)
    _clip(grads, None, 1.0)
    for g, o in zip(grads, outs):
        assert torch.equal(g, o)
        o.fill_(7.0)
    assert (buf == 7.0).all()


def test_range_and_specials():
    import torch

    big = torch.full((1000,), 3e38, device="cuda")
    sumsq, stats = _clip([big], None, 1.0)  # the square passes fp32, the norm too
    assert abs(sumsq - 1000 * float(np.float32(3e38)) ** 2) <= 1e-9 * sumsq
    assert np.isinf(stats[0]) and stats[1] == 0.0 and (big == 0).all()
    big = torch.full((4,), 1e38, device="cuda")
    _, stats = _clip([big], None, 1.0)
    want = 2 * float(np.float32(1e38))
    assert abs(stats[0] - want) <= 2 * U * want
    assert np.allclose(big.cpu().numpy(), 0.5, rtol=8 * U)
    small = torch.full((10,), 1e-42, device="cuda")
    _, stats = _clip([small], None, 1.0)
    assert stats[1] == 1.0 and abs(stats[0] - 1e-42 * 10 ** 0.5) <= 2e-45
    for bad, c in ((float("inf"), 0.0), (float("nan"), None)):
        g = torch.ones(3000, device="cuda")
        g[1234] = bad
        _, stats = _clip([g], None, 1.0)
        if c is None:
            assert np.isnan(stats).all() and torch.isnan(g).all()
        else:
            assert np.isinf(stats[0]) and stats[1] == 0.0
            assert torch.isnan(g[1234]) and int((g == 0).sum()) == 2999
    zero = torch.zeros(100, device="cuda")
    sumsq, stats = _clip([zero], None, 0.0)
    assert sumsq == 0.0 and stats[0] == 0.0 and stats[1] == 0.0
