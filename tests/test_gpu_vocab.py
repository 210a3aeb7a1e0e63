"""Token log-probabilities with entropy and top alternatives, distillation
from a teacher's top logits, and their gradients, against the oracle."""
import numpy as np
import pytest

from oft_inputs import DenseConfig, make_dense
from oracle import dense as odense
from oracle import vocab
from tests.helpers import dev, err, host
from tests.vocab_cases import ALL_KINDS, MORE_KINDS, Bounds, as_type, check, rows

pytestmark = pytest.mark.gpu


def _c(T, V, k, pad=0, gpad=0, tau=1.0, offset=0):
    """pad / gpad: elements between rows of logits / d_logits; offset:
    elements from the buffer's start to the first row."""
    return dict(T=T, V=V, k=k, pad=pad, gpad=gpad, tau=tau, offset=offset)


# from one token to many, odd and even rows, rows shorter than a wave and
# longer than any slice, rows that start off 16-byte alignment
SHAPES = [_c(1, 1, 1), _c(3, 2, 2, tau=0.5), _c(20, 7, 7, pad=2), _c(19, 63, 20), _c(18, 64, 64, gpad=3),
          _c(36, 65, 65, offset=3), _c(18, 127, 100), _c(18, 257, 128, pad=7, gpad=7, offset=1), _c(40, 1000, 5, tau=2.5),
          _c(18, 2048, 20, offset=5), _c(37, 2049, 33, pad=1, gpad=2), _c(18, 4097, 128, tau=0.7), _c(1100, 700, 3, pad=13),
          _c(18, 8191, 64, gpad=1, tau=1.3), _c(2, 32768, 128), _c(19, 50021, 20, pad=3, gpad=11, offset=7),
          _c(1, 151936, 20, tau=0.7), _c(18, 151936, 64), _c(2, 300001, 128, tau=0.9), _c(1, 1500000, 17)]
IDS = ["T{T}-V{V}-k{k}-p{pad}-g{gpad}-o{offset}".format(**c) for c in SHAPES]
DTYPES = ["bf16", "f32"]


def _tt(dtype):
    import torch

    return torch.bfloat16 if dtype == "bf16" else torch.float32


def _view(a, dtype, ld, offset, fill):
    """The rows of a [T, V] on the GPU, ld elements apart, inside a buffer
    filled with `fill`: (buffer, view)."""
    import torch

    T, V = a.shape
    buf = torch.full((offset + T * ld + 64,), fill, dtype=_tt(dtype), device="cuda")
    view = buf[offset:offset + T * ld].view(T, ld)[:, :V]
    view.copy_(torch.from_numpy(np.ascontiguousarray(a)).to("cuda"))
    return buf, view


def _desc(c, dtype, k=None, accumulate=0):
    import orthogonal_fine_tuning_amd as oft

    return oft.vocab_desc(c["T"], c["V"], oft.OFT_DT_F32 if dtype == "f32" else oft.OFT_DT_BF16,
                          k=c["k"] if k is None else k, ld=c["V"] + c["pad"], ld_grad=c["V"] + c["gpad"],
                          temperature=c["tau"], accumulate=accumulate)


def _ws(d):
    import torch
    import orthogonal_fine_tuning_amd as oft

    n = oft.oft_vocab_workspace_bytes(d)
    return {"ws": torch.full((max(n, 16),), 0xA5, dtype=torch.uint8, device="cuda"), "ws_bytes": n}


def _f32(*shape):
    import torch

    return torch.full(shape, 9.0, device="cuda")


def _logprobs(c, dtype, x, labels):
    import torch
    import orthogonal_fine_tuning_amd as oft

    T, k = c["T"], c["k"]
    d = _desc(c, dtype)
    # between the rows: NaN, which must not get into any result
    _, xv = _view(x, dtype, d.ld, c["offset"], float("nan"))
    o = dict(logp=_f32(T), entropy=_f32(T), stats=_f32(T, 2))
    top = dict(top_idx=torch.full((T, k), -5, dtype=torch.int32, device="cuda"), top_logp=_f32(T, k)) if k else {}
    oft.oft_token_logprobs(d, xv, dev(labels), o["logp"], o["stats"], entropy=o["entropy"], **top, **_ws(d))
    torch.cuda.synchronize()
    return xv, {**o, **top}


def _labels(rng, T, V):
    lab = rng.integers(0, V, T)
    lab[rng.random(T) < 0.15] = -1
    if T > 4:
        lab[2], lab[4] = V, -2
    return lab.astype(np.int32)


def _check_logprobs(c, x, labels, got, b):
    T, k = c["T"], c["k"]
    w = [check(host(got["stats"])[:, 0], b.m, 0.0, "stats m"),
         check(host(got["stats"])[:, 1], b.l, b.l_tol, "stats l"),
         check(host(got["entropy"]), b.H, b.H_tol, "entropy")]
    ok = (labels >= 0) & (labels < c["V"])
    tol = np.where(ok, b.lp_tol[np.arange(T), np.where(ok, labels, 0)], 0.0)
    w.append(check(host(got["logp"]), vocab.given(b.lp, labels), tol, "logp"))
    if k:
        top = vocab.top(x, k)
        assert np.array_equal(host(got["top_idx"]), top), "top_idx"
        w.append(check(host(got["top_logp"]), np.take_along_axis(b.lp, top, 1), np.take_along_axis(b.lp_tol, top, 1),
                       "top_logp"))
    return max(w)


def _sentinel_ok(buf, c, dtype, fill):
    """Everything outside the rows' own elements is as it was."""
    import torch

    mask = torch.ones(buf.numel(), dtype=torch.bool, device="cuda")
    ld = c["V"] + c["gpad"]
    mask[c["offset"]:c["offset"] + c["T"] * ld].view(c["T"], ld)[:, :c["V"]] = False
    return bool((buf[mask].float() == fill).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("c", SHAPES, ids=IDS)
def test_logprobs_and_gradient(c, dtype):
    import torch
    import orthogonal_fine_tuning_amd as oft

    print(f"[logprobs] {c} {dtype}", flush=True)
    T, V = c["T"], c["V"]
    rng = np.random.default_rng(T + 3 * V)
    x = rows(T, V, dtype, T * 7 + V, ALL_KINDS if T >= 18 else ["plain", "masked"])
    labels = _labels(rng, T, V)
    xv, got = _logprobs(c, dtype, x, labels)
    b = Bounds(x, np.float64(np.float32(c["tau"])))
    w = _check_logprobs(c, x, labels, got, b)
    gl, ge = rng.normal(0, 1, T).astype(np.float32), rng.normal(0, 0.3, T).astype(np.float32)
    gl[rng.random(T) < 0.2] = 0
    ge[rng.random(T) < 0.4] = 0
    d = _desc(c, dtype, k=0)
    buf, dv = _view(np.full((T, V), 3.0, np.float32), dtype, d.ld_grad, c["offset"], 77.0)
    oft.oft_token_logprobs_bwd(d, xv, dev(labels), got["stats"], dev(gl), dv, entropy=got["entropy"], g_entropy=dev(ge))
    torch.cuda.synchronize()
    ref = vocab.logprobs_grad(x, labels, gl, ge, b.tau)
    wg = check(host(dv.float()), ref, b.grad(ref, np.where(labels == -1, 0, gl), ge, dtype), "d_logits")
    assert _sentinel_ok(buf, c, dtype, 77.0)
    print(f"[logprobs] {w:.2f} of the bound, gradient {wg:.2f}", flush=True)


def _teacher_case(rng, x, K, special):
    """A list of K entries per row: distinct columns where V allows, some
    repeated, unused, at -inf; `special` adds rows with bad entries."""
    T, V = x.shape
    idx = rng.integers(0, V, (T, K))
    best = vocab.top(x, min(K, V))
    idx[:, :best.shape[1]] = np.where(rng.random(best.shape) < 0.5, best, idx[:, :best.shape[1]])
    val = rng.normal(0, 3, (T, K)).astype(np.float32)
    idx[rng.random((T, K)) < 0.1] = -1
    val[rng.random((T, K)) < 0.1] = -np.inf
    val[idx == -1] = np.nan  # ignored
    if special and T > 8:
        idx[1] = -1
        val[3] = -np.inf
        idx[5, -1] = V
        idx[6, 0] = -3
        idx[7, 0], val[7, 0] = 0, np.nan
        idx[8, K // 2], val[8, K // 2] = 0, np.inf
    return idx.astype(np.int32), val


def _distill(c, dtype, x, idx, val):
    import torch
    import orthogonal_fine_tuning_amd as oft

    d = _desc(c, dtype, k=idx.shape[1])
    _, xv = _view(x, dtype, d.ld, c["offset"], float("nan"))
    loss, stats = _f32(c["T"]), _f32(c["T"], 2)
    oft.oft_distill_topk(d, xv, dev(idx), dev(val), loss, stats, **_ws(d))
    torch.cuda.synchronize()
    return d, xv, loss, stats


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("c", SHAPES, ids=IDS)
def test_distillation_and_gradient(c, dtype):
    import torch
    import orthogonal_fine_tuning_amd as oft

    T, V = c["T"], c["V"]
    K = min(256, 2 * c["k"])
    print(f"[distill] {c} K={K} {dtype}", flush=True)
    rng = np.random.default_rng(5 * T + V)
    x = rows(T, V, dtype, T * 11 + V, ALL_KINDS if T >= 18 else ["plain"])
    idx, val = _teacher_case(rng, x, K, True)
    d, xv, loss, stats = _distill(c, dtype, x, idx, val)
    b = Bounds(x, np.float64(np.float32(c["tau"])))
    ref = vocab.distill(x, idx, val, b.tau)
    w = check(host(loss), ref, b.teacher(idx, val)[0], "loss")
    check(host(stats)[:, 0], b.m, 0.0, "stats m")
    check(host(stats)[:, 1], b.l, b.l_tol, "stats l")
    g = rng.normal(0, 1, T).astype(np.float32)
    g[rng.random(T) < 0.2] = 0
    buf, dv = _view(np.full((T, V), 3.0, np.float32), dtype, d.ld_grad, c["offset"], 77.0)
    oft.oft_distill_topk_bwd(d, xv, dev(idx), dev(val), stats, dev(g), dv)
    torch.cuda.synchronize()
    gref = vocab.distill_grad(x, idx, val, g, b.tau)
    wg = check(host(dv.float()), gref, b.distill_grad(gref, idx, val, g, dtype), "d_logits")
    assert _sentinel_ok(buf, c, dtype, 77.0)
    print(f"[distill] {w:.2f} of the bound, gradient {wg:.2f}", flush=True)


@pytest.mark.parametrize("dtype", DTYPES)
def test_optional_parts_and_zero_alternatives(dtype):
    """No labels, no entropy, no alternatives; each gradient alone."""
    import torch
    import orthogonal_fine_tuning_amd as oft

    c = _c(20, 3001, 0, pad=3, tau=0.8)
    rng = np.random.default_rng(0)
    x = rows(20, 3001, dtype, 3, ALL_KINDS)
    labels = _labels(rng, 20, 3001)
    xv, full = _logprobs(c, dtype, x, labels)
    b = Bounds(x, np.float64(np.float32(0.8)))
    _check_logprobs(c, x, labels, full, b)
    d = _desc(c, dtype)
    stats = _f32(20, 2)
    oft.oft_token_logprobs(d, xv, None, None, stats, **_ws(d))
    torch.cuda.synchronize()
    assert torch.equal(stats.view(torch.int32), full["stats"].view(torch.int32))
    gl, ge = rng.normal(0, 1, 20).astype(np.float32), rng.normal(0, 1, 20).astype(np.float32)
    for use_l, use_e in ((True, False), (False, True)):
        _, dv = _view(np.zeros((20, 3001), np.float32), dtype, d.ld_grad, 0, 0.0)
        oft.oft_token_logprobs_bwd(d, xv, dev(labels) if use_l else None, full["stats"], dev(gl) if use_l else None, dv,
                                   entropy=full["entropy"] if use_e else None, g_entropy=dev(ge) if use_e else None)
        torch.cuda.synchronize()
        ref = vocab.logprobs_grad(x, labels if use_l else None, gl if use_l else None, ge if use_e else None, b.tau)
        check(host(dv.float()), ref, b.grad(ref, gl * use_l, ge * use_e, dtype), "d_logits")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V,pad", [(1000, 0), (4097, 3), (4097, 0), (13001, 2)])
def test_gradient_in_place_and_accumulated(dtype, V, pad):
    """In place: bit for bit the gradient written elsewhere.  Accumulated:
    one rounding of the sum; rows without a gradient stay as they are."""
    import torch
    import orthogonal_fine_tuning_amd as oft

    T, K = 20, 12
    c = _c(T, V, 0, pad=pad, gpad=pad, tau=1.2)
    rng = np.random.default_rng(V)
    x = rows(T, V, dtype, 1, ALL_KINDS)
    labels = _labels(rng, T, V)
    idx, val = _teacher_case(rng, x, K, True)
    g = rng.normal(0, 1, T).astype(np.float32)
    g[3] = 0
    xv, full = _logprobs(c, dtype, x, labels)
    b = Bounds(x, np.float64(np.float32(1.2)))
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    half = {"bf16": torch.int16, "f32": torch.int32}[dtype]

    def grads(which, accumulate, src, dst):
        d = _desc(c, dtype, k=K if which == "distill" else 0, accumulate=accumulate)
        if which == "distill":
            oft.oft_distill_topk_bwd(d, src, dev(idx), dev(val), full["stats"], dev(g), dst)
        else:
            oft.oft_token_logprobs_bwd(d, src, dev(labels), full["stats"], dev(g), dst, entropy=full["entropy"],
                                       g_entropy=dev(0.1 * g))
        torch.cuda.synchronize()

    for which in ("distill", "logprobs"):
        _, plain = _view(np.zeros((T, V), np.float32), dtype, V + pad, 0, 0.0)
        grads(which, 0, xv, plain)
        buf, same = _view(x, dtype, V + pad, 0, 55.0)
        grads(which, 0, same, same)
        assert torch.equal(same.contiguous().view(half), plain.contiguous().view(half)), which
        assert _sentinel_ok(buf, c, dtype, 55.0)
        start = rows(T, V, dtype, 9)
        _, acc = _view(start, dtype, V + pad, 0, 0.0)
        grads(which, 1, xv, acc)
        if which == "distill":
            ref = vocab.distill_grad(x, idx, val, g, b.tau)
            tol = b.distill_grad(ref, idx, val, g, "f32")
        else:
            ref = vocab.logprobs_grad(x, labels, g, np.float32(0.1) * g, b.tau)
            tol = b.grad(ref, np.where(labels == -1, 0, g), 0.1 * g, "f32")
        want = ref + start
        a = np.where(np.isfinite(want), np.abs(want), 0.0)
        # the fp32 sum and the rounding to the type
        check(host(acc.float()), want, tol + 2.0 ** -24 * (a + tol) + u * (a + tol), which + " accumulated")
        assert np.array_equal(host(acc.float())[3], start[3])


def test_zero_gradient_rows_are_not_read():
    """Padded rows (no label, or upstream gradients of 0) get exact zeros
    whatever the logits and the saved statistics hold."""
    import torch
    import orthogonal_fine_tuning_amd as oft

    T, V = 6, 777
    x = torch.full((T, V), float("nan"), dtype=torch.bfloat16, device="cuda")
    stats = torch.full((T, 2), float("nan"), device="cuda")
    out = torch.full((T, V), 5.0, dtype=torch.bfloat16, device="cuda")
    d = oft.vocab_desc(T, V)
    lab = torch.tensor([-1, 3, -1, 0, 776, -7], dtype=torch.int32, device="cuda")
    g = torch.tensor([2.0, 0.0, float("nan"), 0.0, 0.0, 0.0], device="cuda")
    oft.oft_token_logprobs_bwd(d, x, lab, stats, g, out)
    torch.cuda.synchronize()
    assert bool((out == 0).all())
    out.fill_(5.0)
    d = oft.vocab_desc(T, V, k=4)
    idx = torch.zeros((T, 4), dtype=torch.int32, device="cuda")
    idx[:3] = -1
    val = torch.zeros((T, 4), device="cuda")
    g = torch.tensor([2.0, 1.0, -1.0, 0.0, 0.0, 0.0], device="cuda")
    oft.oft_distill_topk_bwd(d, x, idx, val, stats, g, out)
    torch.cuda.synchronize()
    assert bool((out == 0).all())


@pytest.mark.parametrize("which", ["logprobs", "distill"])
def test_gradient_against_differences_of_the_loss(which):
    """fp32: the loss's change along a direction v against <gradient, v>.
    Each loss is off by at most its bound; what a step of this size leaves
    out of the linear term is the oracle's own difference, in fp64."""
    import torch
    import orthogonal_fine_tuning_amd as oft

    T, V, K, h = 8, 5003, 30, 2.0 ** -6
    c = _c(T, V, 0, tau=1.0)
    rng = np.random.default_rng(2)
    x = rows(T, V, "f32", 4)
    v = np.clip(rng.normal(0, 0.5, (T, V)), -1, 1)
    hi, lo = (x + h * v).astype(np.float32), (x - h * v).astype(np.float32)
    step = (hi.astype(np.float64) - lo.astype(np.float64)) / 2  # the step that was taken
    if which == "logprobs":
        labels = rng.integers(0, V, T).astype(np.int32)

        def loss(y):
            o = _logprobs(c, "f32", y, labels)[1]
            return host(o["logp"]).astype(np.float64) + host(o["entropy"])

        def exact(y):
            lp = vocab.log_probs(y)[0]
            return vocab.given(lp, labels) + vocab.entropy(lp)

        slope = vocab.logprobs_grad(x, labels, np.ones(T), np.ones(T))
        xv, full = _logprobs(c, "f32", x, labels)
        dv = torch.empty((T, V), device="cuda")
        one = torch.ones(T, device="cuda")
        oft.oft_token_logprobs_bwd(_desc(c, "f32"), xv, dev(labels), full["stats"], one, dv, entropy=full["entropy"],
                                   g_entropy=one)
    else:
        idx = np.stack([rng.permutation(V)[:K] for _ in range(T)]).astype(np.int32)
        val = rng.normal(0, 2, (T, K)).astype(np.float32)

        def loss(y):
            return host(_distill(c, "f32", y, idx, val)[2]).astype(np.float64)

        def exact(y):
            return vocab.distill(y, idx, val)

        slope = vocab.distill_grad(x, idx, val, np.ones(T))
        d, xv, _, stats = _distill(c, "f32", x, idx, val)
        dv = torch.empty((T, V), device="cuda")
        oft.oft_distill_topk_bwd(d, xv, dev(idx), dev(val), stats, torch.ones(T, device="cuda"), dv)
    torch.cuda.synchronize()
    diff = loss(hi) - loss(lo)
    want = 2 * (host(dv).astype(np.float64) * step).sum(axis=1)
    beyond = np.abs(exact(hi) - exact(lo) - 2 * (slope * step).sum(axis=1))
    b = Bounds(x, 1.0)
    noise = b.teacher(idx, val)[0] if which == "distill" else b.lp_tol[np.arange(T), labels] + b.H_tol
    # both losses' bounds (taken at x: 1.5 for the rows h away from it), the
    # fp32 gradient's own error (p_rel is below 2^-16 at this size), and
    # the part beyond the linear term
    tol = 3 * noise + 2 * (np.abs(host(dv)) * np.abs(step)).sum(axis=1) * 2.0 ** -16 + beyond * 1.01
    assert np.all(np.abs(diff - want) <= tol), (np.abs(diff - want) / tol).max()
    assert np.abs(diff).max() > 5 * tol.max()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,V,k,pad", [(205, 40001, 20, 0), (207, 33333, 128, 2), (19, 9000, 128, 1)])
def test_rows_enough_to_take_whole(T, V, k, pad, dtype):
    """Rows of several steps, one workgroup each, with every kind of row;
    and few rows with nearly as many alternatives as blocks of columns."""
    import torch
    import orthogonal_fine_tuning_amd as oft

    c = _c(T, V, k, pad=pad, gpad=pad, tau=0.8)
    rng = np.random.default_rng(T)
    x = rows(T, V, dtype, T, ALL_KINDS)
    labels = _labels(rng, T, V)
    xv, got = _logprobs(c, dtype, x, labels)
    b = Bounds(x, np.float64(np.float32(0.8)))
    _check_logprobs(c, x, labels, got, b)
    idx, val = _teacher_case(rng, x, min(256, 2 * k), True)
    d, xv, loss, stats = _distill(c, dtype, x, idx, val)
    check(host(loss), vocab.distill(x, idx, val, b.tau), b.teacher(idx, val)[0], "loss")
    assert torch.equal(stats.view(torch.int32), got["stats"].view(torch.int32))
    g = rng.normal(0, 1, T).astype(np.float32)
    _, dv = _view(np.full((T, V), 3.0, np.float32), dtype, d.ld_grad, 0, 77.0)
    oft.oft_distill_topk_bwd(d, xv, dev(idx), dev(val), stats, dev(g), dv)
    torch.cuda.synchronize()
    ref = vocab.distill_grad(x, idx, val, g, b.tau)
    check(host(dv.float()), ref, b.distill_grad(ref, idx, val, g, dtype), "d_logits")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,V,k", [(6, 151936, 128), (7, 151935, 20), (204, 40001, 128), (12, 20000, 128)])
def test_alternatives_in_clusters(T, V, k, dtype):
    """The best columns next to each other or in the share of one wave, a few
    or some hundred, apart or equal: the lists of candidates run over in one
    wave, in all, or hold nearly all of them."""
    rng = np.random.default_rng(V + k)
    x = rng.normal(0, 2, (T, V)).astype(np.float32)
    for t in range(T):
        kind, n = t % 6, (400, 140, 60)[t // 6 % 3]
        at = np.arange(n) + int(rng.integers(0, V - n))  # a run
        if kind >= 3:
            # 128 columns of every 2048, from a common offset: one wave's vectors
            at = (np.arange(4)[:, None] * 2048 + np.arange(n // 4) + 512 * (kind - 3)).reshape(-1)
        x[t, at] = 12.0 if kind % 3 == 1 else rng.uniform(9.0, 20.0, at.size)
        if kind % 3 == 2:
            x[t, at[::2]] = 12.0
    x = as_type(x, dtype)
    c = _c(T, V, k)
    labels = _labels(rng, T, V)
    _, got = _logprobs(c, dtype, x, labels)
    assert np.array_equal(host(got["top_idx"]), vocab.top(x, k))
    b = Bounds(x[:6], 1.0)
    top = host(got["top_idx"])[:6]
    check(host(got["top_logp"])[:6], np.take_along_axis(b.lp, top, 1), np.take_along_axis(b.lp_tol, top, 1), "top_logp")


@pytest.mark.parametrize("T,V", [(8, 10007), (210, 10007), (8, 70001)])
@pytest.mark.parametrize("tau", [1.0, 2.0 ** -20, 2.0 ** 20, 0.01, 300.0])
def test_temperatures_and_far_references(T, V, tau):
    """The smallest and largest temperature, and rows whose scaled maximum
    crosses the border between the two forms of a sum's reference."""
    import torch
    import orthogonal_fine_tuning_amd as oft

    c = _c(T, V, 9, tau=tau)
    x = rows(T, V, "f32", 5, MORE_KINDS)
    rng = np.random.default_rng(1)
    labels = vocab.top(x, 3)[np.arange(T), rng.integers(0, 3, T)].astype(np.int32)
    xv, got = _logprobs(c, "f32", x, labels)
    b = Bounds(x, tau)
    _check_logprobs(c, x, labels, got, b)
    gl, ge = rng.normal(0, 1, T).astype(np.float32), rng.normal(0, 1, T).astype(np.float32)
    dv = torch.empty((T, V), device="cuda")
    oft.oft_token_logprobs_bwd(_desc(c, "f32"), xv, dev(labels), got["stats"], dev(gl), dv, entropy=got["entropy"],
                               g_entropy=dev(ge))
    torch.cuda.synchronize()
    ref = vocab.logprobs_grad(x, labels, gl, ge, tau)
    check(host(dv), ref, b.grad(ref, gl, ge, "f32"), "d_logits")


def test_streamed_rows_equal_kept_ones():
    """A call large enough to pass the caches by, bit for bit its rows in
    smaller calls that do not, forward and backward."""
    import torch
    import orthogonal_fine_tuning_amd as oft

    T, V, k, part = 690, 120011, 20, 230  # 166 MB of bf16 against 55 MB
    g = torch.Generator(device="cuda").manual_seed(3)
    x = (2.5 * torch.randn((T, V), generator=g, device="cuda")).to(torch.bfloat16)
    lab = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    up = torch.randn(T, generator=g, device="cuda")

    def run(a, b):
        n = b - a
        d = oft.vocab_desc(n, V, k=k, temperature=0.9)
        o = dict(logp=_f32(n), stats=_f32(n, 2), entropy=_f32(n),
                 top_idx=torch.zeros((n, k), dtype=torch.int32, device="cuda"), top_logp=_f32(n, k))
        oft.oft_token_logprobs(d, x[a:b], lab[a:b].clone(), **o, **_ws(d))
        gr = torch.empty((n, V), dtype=torch.bfloat16, device="cuda")
        dg = torch.empty_like(gr)
        oft.oft_token_logprobs_bwd(d, x[a:b], lab[a:b].clone(), o["stats"], up[a:b].clone(), gr, entropy=o["entropy"],
                                   g_entropy=up[a:b].clone())
        loss, st = _f32(n), _f32(n, 2)
        oft.oft_distill_topk(d, x[a:b], o["top_idx"], o["top_logp"], loss, st, **_ws(d))
        oft.oft_distill_topk_bwd(d, x[a:b], o["top_idx"], o["top_logp"], st, up[a:b].clone(), dg)
        torch.cuda.synchronize()
        return {**o, "grad": gr, "loss": loss, "dgrad": dg}

    whole = run(0, T)
    for a in range(0, T, part):
        small = run(a, a + part)
        for name in small:
            assert torch.equal(whole[name][a:a + part], small[name]), (name, a)


def test_deterministic_and_independent_of_other_rows():
    import torch

    T, V = 37, 30011
    c = _c(T, V, 50, tau=0.9)
    x = rows(T, V, "bf16", 3, ["plain", "ties", "masked"])
    labels = np.arange(T, dtype=np.int32)
    a, b = (_logprobs(c, "bf16", x, labels)[1] for _ in range(2))
    for n in a:
        assert torch.equal(a[n], b[n]), n


def test_rows_beyond_32_bit_offsets():
    """Rows more than 2^31 elements apart (and d_logits likewise)."""
    import torch
    import orthogonal_fine_tuning_amd as oft

    T, V, ld = 3, 1501, (1 << 31) + 24
    x = rows(T, V, "bf16", 2)
    labels = np.array([5, 1500, 0], np.int32)
    buf = torch.empty(2 * ld + V, dtype=torch.bfloat16, device="cuda")
    xv = buf.as_strided((T, V), (ld, 1))
    xv.copy_(torch.from_numpy(x).to("cuda"))
    d = oft.vocab_desc(T, V, k=4, ld=ld, ld_grad=ld)
    o = dict(logp=_f32(T), entropy=_f32(T), stats=_f32(T, 2), top_idx=torch.zeros((T, 4), dtype=torch.int32, device="cuda"),
             top_logp=_f32(T, 4))
    oft.oft_token_logprobs(d, xv, dev(labels), o["logp"], o["stats"], o["entropy"], o["top_idx"], o["top_logp"], **_ws(d))
    torch.cuda.synchronize()
    b = Bounds(x, 1.0)
    _check_logprobs(_c(T, V, 4), x, labels, o, b)
    g = np.array([1.0, -2.0, 0.5], np.float32)
    oft.oft_token_logprobs_bwd(d, xv, dev(labels), o["stats"], dev(g), xv)
    torch.cuda.synchronize()
    ref = vocab.logprobs_grad(x, labels, g, None)
    check(host(xv.float()), ref, b.grad(ref, g, 0 * g, "bf16"), "d_logits")


def test_graph_replay_with_a_shared_workspace():
    """Scoring and distillation captured into two graphs that share one
    workspace, replayed in turn with new logits and with eager calls between
    them; everything bit for bit as eager."""
    import torch
    import orthogonal_fine_tuning_amd as oft

    T, V, k = 6, 40009, 20
    d = oft.vocab_desc(T, V, k=k, temperature=0.7)
    n = oft.oft_vocab_workspace_bytes(d)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    ws2 = torch.empty_like(ws)
    x = torch.empty((T, V), dtype=torch.bfloat16, device="cuda")
    lab = torch.arange(T, dtype=torch.int32, device="cuda")
    g = torch.ones(T, device="cuda")

    def outs():
        return dict(logp=_f32(T), entropy=_f32(T), stats=_f32(T, 2), top_logp=_f32(T, k), loss=_f32(T), stats2=_f32(T, 2),
                    top_idx=torch.zeros((T, k), dtype=torch.int32, device="cuda"), d1=torch.empty_like(x),
                    d2=torch.empty_like(x))

    def score(o, w):
        oft.oft_token_logprobs(d, x, lab, o["logp"], o["stats"], o["entropy"], o["top_idx"], o["top_logp"], ws=w,
                               ws_bytes=n)
        oft.oft_token_logprobs_bwd(d, x, lab, o["stats"], g, o["d1"], entropy=o["entropy"], g_entropy=g)

    def distill(o, w):
        oft.oft_distill_topk(d, x, o["top_idx"], o["top_logp"], o["loss"], o["stats2"], ws=w, ws_bytes=n)
        oft.oft_distill_topk_bwd(d, x, o["top_idx"], o["top_logp"], o["stats2"], g, o["d2"])

    a, e = outs(), outs()
    x.copy_(torch.from_numpy(rows(T, V, "bf16", 0)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        score(a, ws)
        distill(a, ws)
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        score(a, ws)
    with torch.cuda.graph(g2):
        distill(a, ws)
    for r in range(4):
        x.copy_(torch.from_numpy(rows(T, V, "bf16", r + 1, ["plain", "masked", "ties"])))
        score(e, ws2)
        distill(e, ws2)
        torch.cuda.synchronize()
        g1.replay()
        g2.replay()
        torch.cuda.synchronize()
        for name in a:
            assert torch.equal(a[name], e[name]), (r, name)


def test_two_streams_at_once():
    """Two calls on two streams, each with its own workspace and outputs."""
    import torch
    import orthogonal_fine_tuning_amd as oft

    T, V, k = 5, 60013, 20
    d = oft.vocab_desc(T, V, k=k)
    xs = [torch.from_numpy(rows(T, V, "bf16", s)).to("cuda").to(torch.bfloat16) for s in (1, 2)]
    lab = torch.zeros(T, dtype=torch.int32, device="cuda")

    def call(x, w, stream=None):
        o = dict(logp=_f32(T), entropy=_f32(T), stats=_f32(T, 2),
                 top_idx=torch.zeros((T, k), dtype=torch.int32, device="cuda"), top_logp=_f32(T, k))
        return o, lambda: oft.oft_token_logprobs(d, x, lab, o["logp"], o["stats"], o["entropy"], o["top_idx"],
                                                 o["top_logp"], **w, stream=stream)

    want = []
    for x in xs:
        o, f = call(x, _ws(d))
        f()
        want.append(o)
    streams = [torch.cuda.Stream() for _ in xs]
    calls = [call(x, _ws(d), s.cuda_stream) for x, s in zip(xs, streams)]
    torch.cuda.synchronize()
    for _ in range(5):
        for _, f in calls:
            f()
    torch.cuda.synchronize()
    for w, (o, _) in zip(want, calls):
        for n in w:
            assert torch.equal(w[n], o[n]), n


def test_binding_refuses_wrong_tensors():
    import torch
    import orthogonal_fine_tuning_amd as oft

    T, V = 4, 100
    d = oft.vocab_desc(T, V, k=3)
    x = torch.zeros((T, V), dtype=torch.bfloat16, device="cuda")
    i = torch.zeros(T, dtype=torch.int32, device="cuda")
    f, s = _f32(T), _f32(T, 2)
    ti, tl = torch.zeros((T, 3), dtype=torch.int32, device="cuda"), _f32(T, 3)
    good = dict(logits=x, labels=i, logp=f, stats=s, entropy=f, top_idx=ti, top_logp=tl, **_ws(d))
    for kw in (dict(logits=x.float()), dict(logits=x.t()), dict(logits=x[:, :99]), dict(labels=i.long()),
               dict(labels=i.cpu()), dict(logp=f.double()), dict(stats=_f32(T, 3)), dict(top_idx=ti[:, :2]),
               dict(top_logp=_f32(3, T).t()), dict(ws=torch.zeros(8, device="cpu", dtype=torch.uint8), ws_bytes=8),
               dict(ws=torch.zeros(8, device="cuda", dtype=torch.uint8), ws_bytes=16)):
        with pytest.raises(ValueError):
            oft.oft_token_logprobs(d, **{**good, **kw})
    oft.oft_token_logprobs(d, **good)
    torch.cuda.synchronize()


def test_adapter_step_distilled_from_the_frozen_base():
    """As an adapter's training step uses them together: a dense layer's
    outputs as logits; the frozen base scores the tokens and lists its top 16
    (oft_linear_fwd_base, oft_token_logprobs), the adapted layer is scored and
    distilled from that list, both gradients meet in one d_logits
    (accumulate), and oft_linear_bwd turns it into dX and dQ."""
    import torch
    import orthogonal_fine_tuning_amd as oft

    cfg = DenseConfig("distil", M=96, K=512, segs=(512, 256), b=32, x_dtype="bf16", w_fmt="int4", g=64, q_std=0.1)
    inp = make_dense(cfg, seed=4)
    ld = oft.linear_desc(cfg.M, cfg.K, cfg.segs, cfg.b, oft.OFT_DT_BF16, oft.OFT_W_INT4, cfg.g)
    x, wc, ws, = dev(inp["x"]), dev(inp["w_codes"]), dev(inp["w_scales"])
    Rf = torch.empty((cfg.nblk, cfg.b, cfg.b), device="cuda")
    Rops = torch.empty((cfg.nblk, 2, cfg.b, cfg.b), dtype=torch.int16, device="cuda")
    oft.cayley_build(dev(inp["p"]), cfg.nblk, cfg.b, Rf, Rops)
    yb = torch.empty((cfg.M, cfg.N), dtype=torch.int16, device="cuda")
    y = torch.empty_like(yb)
    oft.oft_linear_fwd_base(ld, x, wc, ws, yb)
    oft.oft_linear_fwd(ld, x, wc, ws, Rops, y)
    M, V, k, tau = cfg.M, cfg.N, 16, 1.5
    vd = oft.vocab_desc(M, V, k=k, temperature=tau)
    add = oft.vocab_desc(M, V, k=k, temperature=tau, accumulate=1)
    rng = np.random.default_rng(1)
    lab = rng.integers(0, V, M).astype(np.int32)
    g = rng.normal(0, 1, M).astype(np.float32)
    t_logp, t_stats, t_idx, t_top = _f32(M), _f32(M, 2), torch.zeros((M, k), dtype=torch.int32, device="cuda"), _f32(M, k)
    oft.oft_token_logprobs(vd, yb, dev(lab), t_logp, t_stats, top_idx=t_idx, top_logp=t_top, **_ws(vd))
    logp, H, stats, loss, stats2 = _f32(M), _f32(M), _f32(M, 2), _f32(M), _f32(M, 2)
    tops = dict(top_idx=torch.zeros_like(t_idx), top_logp=_f32(M, k))
    oft.oft_token_logprobs(vd, y, dev(lab), logp, stats, entropy=H, **tops, **_ws(vd))
    oft.oft_distill_topk(vd, y, t_idx, t_top, loss, stats2, **_ws(vd))
    dy = torch.empty_like(y)
    oft.oft_token_logprobs_bwd(vd, y, dev(lab), stats, dev(g), dy)
    oft.oft_distill_topk_bwd(add, y, t_idx, t_top, stats2, torch.ones(M, device="cuda"), dy)
    dx = torch.empty((M, cfg.K), dtype=torch.int16, device="cuda")
    dq = torch.empty((cfg.nblk, cfg.npair), device="cuda")
    nb = oft.oft_linear_workspace_bytes(ld, oft.OFT_PASS_BWD)
    oft.oft_linear_bwd(ld, dy, y, wc, ws, Rf, Rops, dx, dq, torch.empty(max(nb, 16), dtype=torch.uint8, device="cuda"), nb)
    torch.cuda.synchronize()
    # the losses on the logits that the layers gave, against the oracle
    yh, bh = (t.view(torch.bfloat16).double().cpu().numpy() for t in (y, yb))
    b, bb = Bounds(yh, tau), Bounds(bh, tau)
    assert torch.equal(stats, stats2)
    assert np.array_equal(host(t_idx), vocab.top(bh, k))
    check(host(logp), vocab.given(b.lp, lab), b.lp_tol[np.arange(M), lab], "logp")
    check(host(t_logp), vocab.given(bb.lp, lab), bb.lp_tol[np.arange(M), lab], "teacher logp")
    top = host(t_top).astype(np.float64)
    check(host(loss), vocab.distill(yh, host(t_idx), top, tau), b.teacher(host(t_idx), top)[0], "loss")
    want = vocab.logprobs_grad(yh, lab, g, None, tau) + vocab.distill_grad(yh, host(t_idx), top, np.ones(M), tau)
    got = dy.view(torch.bfloat16).double().cpu().numpy()
    # two roundings to bf16, the first of the policy gradient alone
    first = np.abs(vocab.logprobs_grad(yh, lab, g, None, tau))
    e = np.abs(got - want).max() / np.abs(want).max()
    assert np.all(np.abs(got - want) <= 2.0 ** -8 * (first + np.abs(want)) * 1.02 + 1e-6), e
    # and through the layer: the layer's own parity bound
    W = odense.dequant(inp)
    xo = odense.x_f64(inp)
    dX, dp = odense.backward(xo, W, odense.cayley(inp["p"], cfg.b), got)
    e_dx, e_dq = err(dx.view(torch.bfloat16).float().cpu().numpy(), dX), err(host(dq), dp)
    print(f"[adapter step] d_logits err {e:.2e}, dx {e_dx:.2e}, dq {e_dq:.2e}", flush=True)
    assert e_dx <= 2e-2 and e_dq <= 2e-2
