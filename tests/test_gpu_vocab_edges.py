"""Rows at the borders of the vocabulary losses' definitions, against the
oracle: columns that rank alike, ranges that a division by the temperature
brings back, calls that depend on each other."""
import numpy as np
import pytest

from oracle import vocab
from tests.helpers import dev, host
from tests.test_gpu_vocab import DTYPES, _c, _distill, _f32, _logprobs, _ws
from tests.vocab_cases import NEG, U, Bounds, as_type, check, rows

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


# ------------------------------------------------ the temperature of a teacher
@pytest.mark.parametrize("scored_at", [1.0, 0.7])
@pytest.mark.parametrize("tau", [0.6, 1.5])
def test_teacher_scored_and_distilled_at_other_temperatures(tau, scored_at):
    """The list that the teacher's scoring wrote at temperature 1 (times the
    temperature, if another one) against the teacher's own logits, divided by
    tau once."""
    import torch
    import orthogonal_fine_tuning_amd as oft

    print(f"[teacher] tau={tau} scored at {scored_at}", flush=True)
    T, V, k = 40, 5003, 16
    rng = np.random.default_rng(8)
    teacher = as_type(rng.normal(0, 2.5, (T, V)).astype(np.float32), "bf16")
    x = as_type((teacher + rng.normal(0, 0.7, (T, V))).astype(np.float32), "bf16")
    _, got = _logprobs(_c(T, V, k, tau=scored_at), "bf16", teacher, np.zeros(T, np.int32))
    idx = vocab.top(teacher, k)
    assert np.array_equal(host(got["top_idx"]), idx)
    values = got["top_logp"] * scored_at if scored_at != 1.0 else got["top_logp"]
    d = oft.vocab_desc(T, V, k=k, temperature=tau)
    xt = torch.from_numpy(x).to("cuda").to(torch.bfloat16)
    loss, stats, dx = _f32(T), _f32(T, 2), torch.empty_like(xt)
    g = rng.normal(0, 1, T).astype(np.float32)
    oft.oft_distill_topk(d, xt, got["top_idx"], values, loss, stats, **_ws(d))
    oft.oft_distill_topk_bwd(d, xt, got["top_idx"], values, stats, dev(g), dx)
    torch.cuda.synchronize()
    t32, s32 = np.float64(np.float32(tau)), np.float64(np.float32(scored_at))
    b, bt = Bounds(x, t32), Bounds(teacher, s32)
    raw = np.take_along_axis(teacher.astype(np.float64), idx, 1)
    # what the list itself is off by: its log-probabilities' bound, and one
    # rounding (and the factor's own) of the product
    at = np.take_along_axis(bt.lp, idx, 1)
    off = np.take_along_axis(bt.lp_tol, idx, 1) * s32 + (0.0 if scored_at == 1.0 else 2 * U * np.abs(at) * s32)
    off = off.max(axis=1, keepdims=True) / t32
    # d loss / d value = q (log q - log p - loss) / tau, d log q at most twice
    # the values' own; 1 % for what the linear terms leave out (off is below 1e-5)
    ref = vocab.distill(x, idx, raw, t32)
    q, lq = vocab.teacher_probs(idx, raw, V, t32)
    gap = np.abs(lq - np.take_along_axis(b.lp, idx, 1) - ref[:, None])
    assert off.max() < 1e-5
    tol = b.teacher(idx, raw)[0] + 1.01 * (q * gap * off).sum(axis=1)
    check(host(loss), ref, tol, "loss")
    # the same list as it stands is another teacher, by its weights (its loss
    # may meet the right one's by chance: it does not grow or fall with tau)
    if scored_at != 1.0:
        assert (np.abs(vocab.teacher_probs(idx, at, V, t32)[0] - q).max(axis=1) > 1e3 * off[:, 0]).all()
    gref = vocab.distill_grad(x, idx, raw, g, t32)
    more = np.zeros((T, V))
    np.put_along_axis(more, idx.astype(np.int64), q * 2.02 * off, 1)
    more *= (np.abs(g) / t32)[:, None]
    check(host(dx.float()), gref, b.distill_grad(gref, idx, raw, g, "bf16") + more * (1 + 2.0 ** -8), "d_logits")


# ----------------------------------------------------- far ends of log p
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tau", [1.0, 4.0, 2.0 ** 20])
@pytest.mark.parametrize("T,V", [(6, 90), (6, 70001), (203, 2100)])
def test_distances_to_the_maximum_beyond_fp32(T, V, tau, dtype):
    """Finite logits of both signs near the type's range: x - m passes fp32's,
    (x - m) / tau does not (from a temperature of 2 on)."""
    print(f"[far] T={T} V={V} tau={tau} {dtype}", flush=True)
    import torch
    import orthogonal_fine_tuning_amd as oft

    rng = np.random.default_rng(V)
    x = rng.normal(0, 2.5, (T, V)).astype(np.float32)
    x[:, ::7] = -3e38
    x[::2, 3] = 3e38
    x[1::2, 5:40] = rng.uniform(1e38, 3.3e38, (len(x[1::2]), 35))
    x[1, 20:30] = NEG
    x = as_type(x, dtype)
    k = 60
    labels = np.where(np.arange(T) % 3 == 0, 7, np.arange(T) % V).astype(np.int32)
    xv, got = _logprobs(_c(T, V, k, tau=tau), dtype, x, labels)
    b = Bounds(x, tau)
    top = vocab.top(x, k)
    assert np.array_equal(host(got["top_idx"]), top)
    check(host(got["logp"]), vocab.given(b.lp, labels), b.lp_tol[np.arange(T), labels], "logp")
    check(host(got["top_logp"]), np.take_along_axis(b.lp, top, 1), np.take_along_axis(b.lp_tol, top, 1), "top_logp")
    check(host(got["entropy"]), b.H, b.H_tol, "entropy")
    idx = np.concatenate([top[:, :5], np.tile(np.array([7, 14, 8], np.int32), (T, 1))], axis=1)
    val = (rng.normal(0, 1, idx.shape) * tau).astype(np.float32)
    d = oft.vocab_desc(T, V, oft.OFT_DT_F32 if dtype == "f32" else oft.OFT_DT_BF16, k=idx.shape[1], temperature=tau)
    loss, stats, dx = _f32(T), _f32(T, 2), torch.empty_like(xv)
    oft.oft_distill_topk(d, xv, dev(idx), dev(val), loss, stats, **_ws(d))
    oft.oft_distill_topk_bwd(d, xv, dev(idx), dev(val), stats, torch.ones(T, device="cuda"), dx)
    torch.cuda.synchronize()
    check(host(loss), vocab.distill(x, idx, val, tau), b.teacher(idx, val)[0], "loss")
    ref = vocab.distill_grad(x, idx, val, np.ones(T), tau)
    check(host(dx.float()), ref, b.distill_grad(ref, idx, val, np.ones(T), dtype), "d_logits")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,V", [(3, 300), (3, 70001), (201, 300)])
def test_a_listed_column_of_little_weight_that_the_student_masks(T, V, dtype):
    """255 equal entries and one just inside the smallest weight (its
    exponential is 2^-125.5, its share of the sum 2^-133.5, and that over the
    largest temperature 0 in fp32): masked by the student, the loss is infinite;
    in a row with a NaN it is NaN, and with the entry unlisted finite."""
    print(f"[little weight] T={T} V={V} {dtype}", flush=True)
    tau, K = 2.0 ** 20, 256
    rng = np.random.default_rng(1)
    x = as_type(rng.normal(0, 2.5, (T, V)).astype(np.float32), dtype)
    x[:, 299] = NEG
    x[1, 298] = np.nan
    idx = np.tile(np.append(np.arange(K - 1), 299).astype(np.int32), (T, 1))
    val = np.zeros((T, K), np.float32)
    val[:, -1] = -125.5 * np.log(2.0) * tau
    idx[2, -1] = -1
    q = vocab.teacher_probs(idx, val, V, tau)[0]
    assert np.all(q[:2, -1] > 2.0 ** -134) and np.all(q[:2, -1] * 2.0 ** -20 < 2.0 ** -151)
    _, _, loss, _ = _distill(_c(T, V, 1, tau=tau), dtype, x, idx, val)
    b = Bounds(x, tau)
    want = vocab.distill(x, idx, val, tau)
    assert want[0] == np.inf and np.isnan(want[1]) and np.isfinite(want[2])
    check(host(loss), want, b.teacher(idx, val)[0], "loss")


# ------------------------------------------------------- rows and their calls
def _everything(x, labels, idx, val, g, k, tau):
    """Scoring, distillation and both gradients of some rows."""
    import torch
    import orthogonal_fine_tuning_amd as oft

    T, V = x.shape
    d = oft.vocab_desc(T, V, oft.OFT_DT_F32 if x.dtype == torch.float32 else oft.OFT_DT_BF16, k=k, temperature=tau)
    o = dict(logp=_f32(T), entropy=_f32(T), stats=_f32(T, 2),
             top_idx=torch.full((T, k), -5, dtype=torch.int32, device="cuda"), top_logp=_f32(T, k))
    oft.oft_token_logprobs(d, x, labels, **o, **_ws(d))
    d1, d2, loss, stats2 = torch.empty_like(x), torch.empty_like(x), _f32(T), _f32(T, 2)
    oft.oft_token_logprobs_bwd(d, x, labels, o["stats"], g, d1, entropy=o["entropy"], g_entropy=g)
    oft.oft_distill_topk(d, x, idx, val, loss, stats2, **_ws(d))
    oft.oft_distill_topk_bwd(d, x, idx, val, stats2, g, d2)
    torch.cuda.synchronize()
    return {**o, "d_logits": d1, "loss": loss, "stats2": stats2, "distilled": d2}


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,V", [(37, 30012), (37, 151936), (9, 300004)])
def test_a_row_alone_and_in_any_order(T, V, dtype):
    """Bit for bit the same results for a row among others, in another order
    and by itself: whole rows, and rows in slices (as many for one row as for
    all of these; rows of an even length start alike)."""
    import torch

    print(f"[any order] T={T} V={V} {dtype}", flush=True)
    k, tau = 50, 0.9
    rng = np.random.default_rng(V)
    kinds = ["plain", "ties", "masked", "nan", "constant", "wide"]
    x = torch.from_numpy(rows(T, V, dtype, 3, kinds)).to("cuda").to(torch.float32 if dtype == "f32" else torch.bfloat16)
    labels, g = dev(rng.integers(0, V, T).astype(np.int32)), dev(rng.normal(0, 1, T).astype(np.float32))
    idx = dev(rng.integers(0, V, (T, k)).astype(np.int32))
    val = dev(rng.normal(0, 2, (T, k)).astype(np.float32))

    def some(at):
        return _everything(*(a[at].contiguous() for a in (x, labels, idx, val, g)), k, tau)

    def same(name, a, b):
        bits = {4: torch.int32, 2: torch.int16}[a.element_size()]
        return torch.equal(a.contiguous().view(bits), b.contiguous().view(bits))

    every = some(torch.arange(T, device="cuda"))
    order = torch.from_numpy(rng.permutation(T)).to("cuda")
    mixed = some(order)
    for name in every:
        assert same(name, mixed[name], every[name][order]), name
    for t in range(0, T, 1 if V < 100000 else 4):
        alone = some(torch.tensor([t], device="cuda"))
        for name in every:
            assert same(name, alone[name], every[name][t:t + 1]), (t, name)


@pytest.mark.parametrize("dtype", DTYPES)
def test_graphs_of_sliced_rows_with_a_shared_workspace(dtype):
    """Scoring and distillation of rows in slices, captured into two graphs
    that share the one workspace both of them write, replayed in turn and one
    of them twice, with new logits and eager calls in between."""
    import torch
    import orthogonal_fine_tuning_amd as oft

    T, V, k = 6, 70001, 20
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    d = oft.vocab_desc(T, V, oft.OFT_DT_F32 if dtype == "f32" else oft.OFT_DT_BF16, k=k)
    n = oft.oft_vocab_workspace_bytes(d)
    assert n > 0
    ws, ws2 = (torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda") for _ in range(2))
    x = torch.empty((T, V), dtype=dt, device="cuda")
    lab, g = torch.arange(T, dtype=torch.int32, device="cuda"), torch.ones(T, device="cuda")

    def outs():
        return dict(logp=_f32(T), entropy=_f32(T), stats=_f32(T, 2), top_logp=_f32(T, k), loss=_f32(T), stats2=_f32(T, 2),
                    top_idx=torch.zeros((T, k), dtype=torch.int32, device="cuda"), d1=torch.empty_like(x),
                    d2=torch.empty_like(x))

    def score(o, w):
        oft.oft_token_logprobs(d, x, lab, o["logp"], o["stats"], o["entropy"], o["top_idx"], o["top_logp"], ws=w, ws_bytes=n)
        oft.oft_token_logprobs_bwd(d, x, lab, o["stats"], g, o["d1"], entropy=o["entropy"], g_entropy=g)

    def distill(o, w):
        oft.oft_distill_topk(d, x, o["top_idx"], o["top_logp"], o["loss"], o["stats2"], ws=w, ws_bytes=n)
        oft.oft_distill_topk_bwd(d, x, o["top_idx"], o["top_logp"], o["stats2"], g, o["d2"])

    a, e = outs(), outs()
    x.copy_(torch.from_numpy(rows(T, V, dtype, 0)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        score(a, ws)
        torch.cuda.synchronize()
        ws.fill_(0xA5)
        distill(a, ws)
    torch.cuda.synchronize()
    assert bool((ws != 0xA5).any())  # the distillation's triples go through it too
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        score(a, ws)
    with torch.cuda.graph(g2):
        distill(a, ws)
    for r in range(4):
        x.copy_(torch.from_numpy(rows(T, V, dtype, r + 1, ["plain", "masked", "ties"])))
        score(e, ws2)
        distill(e, ws2)
        torch.cuda.synchronize()
        for graph in ((g1, g2), (g1, g2, g2), (g1, g1, g2), (g1, g2))[r]:
            graph.replay()
        torch.cuda.synchronize()
        for name in a:
            assert torch.equal(a[name], e[name]), (r, name)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tau", [0.5, 1.0, 2.0])
@pytest.mark.parametrize("T,V", [(4, 31), (4, 70001), (201, 3000)])
def test_masked_columns_below_a_row_of_lowest_values(T, V, tau, dtype):
    """Columns at -inf where the maximum is the type's lowest value (and its
    quotient by a small temperature passes fp32's range): log p is -inf."""
    x = np.full((T, V), NEG, np.float32)
    x[:, 5::9] = -3.3895314e38 if dtype == "bf16" else -3.4028235e38
    labels = np.where(np.arange(T) % 2 == 0, 3, 5).astype(np.int32)
    k = 20
    _, got = _logprobs(_c(T, V, k, tau=tau), dtype, x, labels)
    b, top = Bounds(x, tau), vocab.top(x, k)
    assert np.array_equal(host(got["top_idx"]), top)
    check(host(got["logp"]), vocab.given(b.lp, labels), b.lp_tol[np.arange(T), labels], "logp")
    check(host(got["top_logp"]), np.take_along_axis(b.lp, top, 1), np.take_along_axis(b.lp_tol, top, 1), "top_logp")
    check(host(got["entropy"]), b.H, b.H_tol, "entropy")
    idx = np.tile(np.array([5, 14, 3], np.int32), (T, 1))
    idx[::3, 2] = -1
    val = np.zeros((T, 3), np.float32)
    loss = _distill(_c(T, V, 1, tau=tau), dtype, x, idx, val)[2]
    check(host(loss), vocab.distill(x, idx, val, tau), b.teacher(idx, val)[0], "loss")
