"""The router's balance loss and its gradient against the oracle."""
import numpy as np
import pytest

from oracle import moe as omoe
from tests.helpers import dev, host
from tests.vocab_cases import U, check

pytestmark = pytest.mark.gpu

# sequences, tokens of each, experts, experts per token
SHAPES = [(1, 1, 1, 1), (1, 3, 5, 2), (4, 16, 8, 8), (3, 65, 64, 4), (2, 64, 65, 16), (1, 200, 128, 6), (5, 129, 200, 8),
          (70000, 1, 4, 1), (1, 1500, 384, 8), (2, 257, 500, 16), (1, 90, 1000, 16), (1, 33, 1024, 3), (2, 5000, 16, 2)]


def _case(S, L, E, k, seed, masked):
    rng = np.random.default_rng(seed)
    T = S * L
    x = (rng.normal(0, 1.5, (T, E)) + rng.normal(0, 0.5, E)).astype(np.float32)
    idx = np.argsort(-x, axis=1, kind="stable")[:, :k].astype(np.int32)
    mask = None
    if masked:
        mask = (rng.random(T) < 0.7).astype(np.uint8)
        mask[:L] = 0  # a sequence of padding alone
        x[mask == 0] = np.nan  # what padded rows hold is not read
        idx[mask == 0] = 1 << 30
    return x, idx, mask, rng.normal(0, 1, S).astype(np.float32)


def _run(S, L, E, k, x, idx, mask, g, accumulate=None, mean=True):
    import torch
    import orthogonal_fine_tuning_amd as oft

    d = oft.moe_desc(S * L, E, k, 64, 64, 32, 32, 16)
    n = oft.oft_moe_balance_workspace_bytes(d, L)
    ws = torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")
    o = {"counts": torch.full((S, E), -7, dtype=torch.int32, device="cuda"),
         "tokens": torch.full((S,), -7, dtype=torch.int32, device="cuda"),
         "loss": torch.full((S,), 9.0, device="cuda"), "mean_prob": torch.full((S, E), 9.0, device="cuda")}
    mt = None if mask is None else dev(mask)
    xt = dev(x)
    oft.oft_moe_balance(d, L, xt, dev(idx), o["counts"], o["tokens"], o["loss"],
                        mean_prob=o["mean_prob"] if mean else None, mask=mt, ws=ws, ws_bytes=n)
    dl = torch.full((S * L, E), 3.0, device="cuda") if accumulate is None else dev(accumulate)
    oft.oft_moe_balance_bwd(d, L, xt, o["counts"], o["tokens"], dev(g), dl, mask=mt,
                            accumulate=0 if accumulate is None else 1)
    torch.cuda.synchronize()
    return {**{n: host(v) for n, v in o.items()}, "d_logits": host(dl)}


def _check(S, L, E, k, x, idx, mask, g, got, base=None):
    ref = omoe.balance(x, idx, L, mask)
    assert np.array_equal(got["counts"], ref["counts"]) and np.array_equal(got["tokens"], ref["tokens"])
    use = np.ones(S * L, bool) if mask is None else mask.astype(bool)
    fin = np.where(np.isfinite(x), x, 0.0)
    z = np.abs(np.where(use[:, None], fin - fin.max(axis=1, keepdims=True), 0.0)).max()
    # p: the exponential (5 |z| + 2 as in the vocabulary losses) in the term
    # and in the sum, the sum's chain of at most E / 16 + 8 additions, the
    # reciprocal and the product
    p_rel = (10 * z + E / 16 + 16) * U
    # sums over at most L tokens in any order
    tol_P = ref["mean_prob"] * (p_rel + (L + 8) * U) + 2.0 ** -125
    w = check(got["mean_prob"], ref["mean_prob"], tol_P, "mean_prob")
    n = np.maximum(ref["tokens"], 1)[:, None]
    f = ref["counts"] / (n * k)
    tol_l = E * (f * tol_P).sum(axis=1) + ref["loss"] * (E / 64 + 24) * U
    w2 = check(got["loss"], ref["loss"], tol_l, "loss")
    d = omoe.balance_grad(x, ref["counts"], ref["tokens"], g, k, L, mask)
    s = np.arange(S * L) // L
    p = omoe._router_softmax(np.where(use[:, None], x, 0.0))
    dot = (f[s] * p).sum(axis=1, keepdims=True)
    scale = (np.abs(g)[s] * E / n[s, 0])[:, None]
    tol_d = scale * p * (f[s] + dot) * (2 * p_rel + (E / 16 + 24) * U) + 2.0 ** -120
    if base is not None:
        d = d + base
        tol_d = tol_d + np.abs(d) * U + U * tol_d
    w3 = check(got["d_logits"], d, tol_d, "d_logits")
    print(f"[balance] S={S} L={L} E={E} k={k}: of the bound mean_prob {w:.2f} loss {w2:.2f} d_logits {w3:.2f}", flush=True)


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("S,L,E,k", SHAPES)
def test_balance_against_oracle(S, L, E, k, masked):
    print(f"[balance] S={S} L={L} E={E} k={k} masked={masked}", flush=True)
    x, idx, mask, g = _case(S, L, E, k, S + 7 * L + E + k, masked)
    got = _run(S, L, E, k, x, idx, mask, g)
    _check(S, L, E, k, x, idx, mask, g, got)
    if mask is not None:
        assert np.all(got["d_logits"][mask == 0] == 0)


def test_accumulates_onto_the_router_gradient_and_leaves_padding_alone():
    S, L, E, k = 3, 50, 100, 4
    x, idx, mask, g = _case(S, L, E, k, 5, True)
    base = np.random.default_rng(1).normal(0, 1e-3, (S * L, E)).astype(np.float32)
    base[mask == 0] = np.nan
    got = _run(S, L, E, k, x, idx, mask, g, accumulate=base, mean=False)
    assert np.array_equal(got["d_logits"][mask == 0], base[mask == 0], equal_nan=True)
    assert np.all(got["mean_prob"] == 9.0)  # not asked for: untouched
    base0 = np.where((mask == 0)[:, None], 0.0, base)
    got["d_logits"][mask == 0] = 0.0
    ref = omoe.balance(x, idx, L, mask)
    got["mean_prob"] = ref["mean_prob"]
    _check(S, L, E, k, x, idx, mask, g, got, base0)


def test_rows_without_a_maximum_nan_logits_and_bad_indices():
    S, L, E, k = 2, 40, 96, 3
    x, idx, _, g = _case(S, L, E, k, 8, False)
    x[3] = -np.inf
    x[5] = np.nan
    x[7, :90] = -np.inf
    x[9, 4] = np.nan
    idx[11] = [-1, E, 2]
    idx[12] = [5, 5, 5]  # an expert listed more than once counts each time
    got = _run(S, L, E, k, x, idx, None, g)
    ref = omoe.balance(x, idx, L)
    assert np.array_equal(got["counts"], ref["counts"])
    _check(S, L, E, k, x, idx, None, g, got)
    assert np.all(got["d_logits"][[3, 5]] == 0)


def test_deterministic():
    S, L, E, k = 2, 700, 256, 8
    x, idx, mask, g = _case(S, L, E, k, 2, True)
    a, b = (_run(S, L, E, k, x, idx, mask, g) for _ in range(2))
    for n in a:
        assert np.array_equal(a[n], b[n]), n


def test_router_step_with_balance_loss():
    """oft_moe_route, the balance loss on its selection, oft_moe_router_bwd,
    and the balance gradient added: the sum of both oracle gradients."""
    import torch
    import orthogonal_fine_tuning_amd as oft

    S, L, E, k = 4, 64, 128, 8
    T = S * L
    rng = np.random.default_rng(3)
    x = (rng.normal(0, 1, (T, E)) + rng.normal(0, 0.5, E)).astype(np.float32)
    dw = rng.normal(0, 1e-2, (T, k)).astype(np.float32)
    g = (0.01 * rng.random(S)).astype(np.float32)
    d = oft.moe_desc(T, E, k, 64, 64, 32, 32, 16)
    i32 = dict(dtype=torch.int32, device="cuda")
    tb = dict(topk_idx=torch.empty((T, k), **i32), topk_w=torch.empty((T, k), device="cuda"),
              counts=torch.empty(E, **i32), offsets=torch.empty(E + 1, **i32), perm=torch.empty(T * k, **i32),
              inv_perm=torch.empty(T * k, **i32), active=torch.empty(E, **i32), n_active=torch.empty(1, **i32),
              chunk_of_expert=torch.empty(E, **i32))
    xt = dev(x)
    n = oft.oft_moe_workspace_bytes(d, oft.OFT_PASS_FWD)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    oft.oft_moe_route(d, xt, oft.moe_routing(**tb), ws, n)
    nb = oft.oft_moe_balance_workspace_bytes(d, L)
    wb = torch.empty(nb, dtype=torch.uint8, device="cuda")
    counts, tokens, loss = torch.empty((S, E), **i32), torch.empty(S, **i32), torch.empty(S, device="cuda")
    oft.oft_moe_balance(d, L, xt, tb["topk_idx"], counts, tokens, loss, ws=wb, ws_bytes=nb)
    dl = torch.empty((T, E), device="cuda")
    oft.oft_moe_router_bwd(d, xt, tb["topk_idx"], dev(dw), dl)
    oft.oft_moe_balance_bwd(d, L, xt, counts, tokens, dev(g), dl, accumulate=1)
    torch.cuda.synchronize()
    idx = host(tb["topk_idx"])
    assert np.array_equal(host(counts).sum(axis=0), host(tb["counts"]))  # the router's own histogram
    ref = omoe.balance(x, idx, L)
    want = omoe.router_backward(x, idx, dw, renorm=False) + omoe.balance_grad(x, ref["counts"], ref["tokens"], g, k, L)
    err = np.abs(host(dl) - want).max() / np.abs(want).max()
    print(f"[router + balance] err {err:.2e}", flush=True)
    # |terms| / max |sum| is of order 1; both gradients are fp32 sums of E = 128 terms
    assert err <= 2e-5


def test_graph_replay_and_side_stream():
    """Forward and backward captured once and replayed with new inputs, with
    eager calls between the replays; the same on a stream of its own."""
    import torch
    import orthogonal_fine_tuning_amd as oft

    S, L, E, k = 2, 300, 160, 4
    d = oft.moe_desc(S * L, E, k, 64, 64, 32, 32, 16)
    n = oft.oft_moe_balance_workspace_bytes(d, L)

    def buffers():
        return dict(counts=torch.empty((S, E), dtype=torch.int32, device="cuda"),
                    tokens=torch.empty(S, dtype=torch.int32, device="cuda"), loss=torch.empty(S, device="cuda"),
                    mean_prob=torch.empty((S, E), device="cuda"), d_logits=torch.empty((S * L, E), device="cuda"),
                    ws=torch.empty(n, dtype=torch.uint8, device="cuda"))

    def step(x, idx, g, b):
        oft.oft_moe_balance(d, L, x, idx, b["counts"], b["tokens"], b["loss"], mean_prob=b["mean_prob"], ws=b["ws"],
                            ws_bytes=n)
        oft.oft_moe_balance_bwd(d, L, x, b["counts"], b["tokens"], g, b["d_logits"])

    x, idx, _, g = _case(S, L, E, k, 0, False)
    xs, ids, gs = dev(x), dev(idx), dev(g)
    a, e = buffers(), buffers()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(xs, ids, gs, a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(xs, ids, gs, a)
    for r in range(4):
        x, idx, _, g = _case(S, L, E, k, r + 1, False)
        xs.copy_(dev(x))
        ids.copy_(dev(idx))
        gs.copy_(dev(g))
        step(xs, ids, gs, e)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for name in ("counts", "tokens", "loss", "mean_prob", "d_logits"):
            assert torch.equal(a[name], e[name]), (r, name)


def test_more_sequences_and_experts_than_one_grid_dimension():
    """A million sequences of one token: their finishing workgroups, 17 to a
    sequence, are more threads than one dimension of a grid holds.  With one
    pair to a token the loss is E p of its expert."""
    import torch
    import orthogonal_fine_tuning_amd as oft

    S, E = 1_000_000, 544
    d = oft.moe_desc(S, E, 1, 64, 64, 32, 32, 16)
    n = oft.oft_moe_balance_workspace_bytes(d, 1)
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((S, E), generator=g, device="cuda")
    idx = torch.randint(0, E, (S, 1), generator=g, device="cuda", dtype=torch.int32)
    counts = torch.full((S, E), -7, dtype=torch.int32, device="cuda")
    tokens, loss = torch.full((S,), -7, dtype=torch.int32, device="cuda"), torch.full((S,), -7.0, device="cuda")
    oft.oft_moe_balance(d, 1, x, idx, counts, tokens, loss, ws=torch.empty(n, dtype=torch.uint8, device="cuda"),
                        ws_bytes=n)
    torch.cuda.synchronize()
    assert bool((tokens == 1).all()) and bool((counts.sum(1) == 1).all())
    assert torch.equal(counts.argmax(1), idx[:, 0].long())
    for a in range(0, S, 100_000):
        at = slice(a, a + 100_000)
        want = E * torch.softmax(x[at].double(), 1).gather(1, idx[at].long())[:, 0]
        # as in _check: |z| <= 16 (the maximum less the minimum of E normal values)
        tol = want * (10 * 16 + E / 16 + 16 + E / 64 + 24) * U
        assert bool(((loss[at].double() - want).abs() <= tol).all()), a
