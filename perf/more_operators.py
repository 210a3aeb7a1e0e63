"""The operators on adapters of many requests as measured: their cases, plain forms and 64-bit results.

Adapters over one frozen projection, served and trained together:

  route                  rows sorted by the adapter that they use (stable), once
                         for all the projections of a step;
  lowrank / lowrank_grad low-rank updates beside the shared projection, each row
                         with its own adapter, every fused segment with factors
                         of its own; and the gradients of rows and factors;
  rotate / rotate_grad   the block rotations of each row's own orthogonal adapter
                         after the shared projection; and the gradients of rows
                         and adapter parameters;
  clip                   the global norm of an adapter's gradients, many tensors,
                         and their clipping.

`run` computes them in elementary torch operations in 32 bits, or, where `own`
is set, through orthogonal_fine_tuning_amd.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6  # beside the norm in the clipping coefficient


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _named(name, case):
    return {"name": name, **case} if name else case


def _route(name, T, S, n, free):
    """T rows of S requests, n adapters; free: share of requests that use none."""
    return _named(name, {"kind": "route", "T": T, "S": S, "n": n, "free": free})


def _lowrank(name, kind, T, S, n, K, segs, r, dtype, free=0.0):
    return _named(name, {"kind": kind, "T": T, "S": S, "n": n, "K": K, "segs": segs, "r": r, "dtype": dtype, "free": free})


def _rotate(name, kind, T, S, n, N, b, dtype, free=0.0):
    return _named(name, {"kind": kind, "T": T, "S": S, "n": n, "N": N, "b": b, "dtype": dtype, "free": free})


def _clip(name, layers, blocks, pairs, dtype, max_norm=1.0):
    """layers times tensors of blocks[i] * pairs elements."""
    return _named(name, {"kind": "clip", "layers": layers, "blocks": blocks, "pairs": pairs, "dtype": dtype,
                         "max_norm": max_norm})


QKV, GATE_UP, TINY = "4096,1024,1024", "9728,9728", "128,128,128"


def listed():
    return [
        # a decode batch: one row a request, most with an adapter of their own
        _route("route_decode", 64, 64, 64, 0.1),
        # prompts and decoded tokens of many requests in one batch
        _route("route_batch", 20011, 700, 300, 0.1),
        # a decode batch beside the fused QKV projection
        _lowrank("lowrank_decode", "lowrank", 64, 64, 64, 2560, QKV, 16, "bf16"),
        # prompts of a few requests beside the gate/up projection
        _lowrank("lowrank_prefill", "lowrank", 8192, 24, 16, 2560, GATE_UP, 32, "bf16"),
        # a training batch of four adapters, QKV projection
        _lowrank("lowrank_grad_train", "lowrank_grad", 4096, 16, 4, 2560, QKV, 16, "bf16"),
        # fp32 rows in odd numbers, an odd rank, some rows of the base model
        _lowrank("lowrank_grad_f32_odd", "lowrank_grad", 777, 9, 5, 2560, QKV, 24, "f32", free=0.2),
        # a decode batch whose requests each rotate the fused QKV output their own way
        _rotate("rotate_decode", "rotate", 64, 64, 64, 6144, 32, "bf16"),
        # prompts through the gate/up projection
        _rotate("rotate_prefill", "rotate", 8192, 24, 8, 19456, 32, "bf16"),
        # a training batch of four adapters, gate/up projection
        _rotate("rotate_grad_train", "rotate_grad", 4096, 16, 4, 19456, 32, "bf16"),
        # fp32 rows in odd numbers, small blocks, some rows of the base model
        _rotate("rotate_grad_f32_b16", "rotate_grad", 1501, 11, 6, 6144, 16, "f32", free=0.2),
        # the gradient of one small layer
        _clip("clip_layer", 1, "8,8,8", 120, "f32", max_norm=0.25),
        # the gradients of 48 MoE layers of 128 experts
        _clip("clip_moe", 48, "6144", 496, "f32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["route", "lowrank", "lowrank_grad", "rotate", "rotate_grad", "clip"])
    free = rng.choice([0.0, 0.0, 0.2])
    if kind == "route":
        T = _log_int(rng, 1, 20000)
        return _route(None, T, _log_int(rng, 1, min(T, 1000)), _log_int(rng, 1, 1000), free)
    if kind == "clip":
        blocks = ",".join(str(_log_int(rng, 1, 600)) for _ in range(rng.randint(1, 7)))
        return _clip(None, rng.randint(1, 48), blocks, rng.choice([120, 496]), rng.choice(["f32", "f32", "bf16"]),
                     rng.choice([1.0, 1.0, 1e6]))
    T = _log_int(rng, 1, 8192 if kind in ("lowrank", "rotate") else 4096)
    grad = kind.endswith("_grad")
    S = _log_int(rng, 1, min(T, 16 if grad else 64))
    n = _log_int(rng, 1, 8 if grad else 64)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if dtype == "f32":
        T = min(T, 2048)
        S = min(S, T)
    if kind.startswith("lowrank"):
        K, segs = rng.choice([(256, TINY), (2560, QKV), (2560, QKV), (2560, GATE_UP)])
        return _lowrank(None, kind, T, S, n, K, segs, 8 * rng.randint(1, 4 if grad else 8), dtype, free)
    return _rotate(None, kind, T, S, n, rng.choice([384, 6144, 19456]), rng.choice([16, 32, 32]), dtype, free)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(0xADA + int(seed))


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _requests(case, seed):
    """Row counts [S] (1 or more each, T in all) and adapters [S] (-1: none) of the batch's requests."""
    rng = np.random.default_rng([0xADA, seed])
    T, S, n = case["T"], case["S"], case["n"]
    cuts = np.sort(rng.choice(T - 1, S - 1, replace=False)) + 1 if S > 1 else np.empty(0, np.int64)
    lengths = np.diff(np.concatenate([[0], cuts, [T]]))
    adapter = rng.permutation(n)[np.arange(S) % n] if S <= n else rng.integers(0, n, S)
    return lengths, np.where(rng.random(S) < case["free"], -1, adapter)


def _prepare_rows(case, seed):
    lengths, adapter = _requests(case, seed)
    T, S = case["T"], case["S"]
    first = np.concatenate([[0], np.cumsum(lengths)[:-1]])
    at = np.arange(lengths.max())
    padded = np.where(at < lengths[:, None], first[:, None] + at, T)  # [S, L], T where a request has ended
    dev = dict(device="cuda")
    return {"case": case,
            "adapter": torch.from_numpy(np.repeat(adapter, lengths).astype(np.int32)).to(**dev),
            "request_adapter": torch.from_numpy(adapter.astype(np.int64)).to(**dev),
            "padded": torch.from_numpy(padded.astype(np.int64)).to(**dev)}


def _segs(case):
    return [int(s) for s in case["segs"].split(",")]


def _prepare_lowrank(case, seed):
    s, g = _prepare_rows(case, seed), _gen(seed)
    T, n, K, r, segs = case["T"], case["n"], case["K"], case["r"], _segs(case)
    N, R = sum(segs), case["r"] * len(segs)
    rand = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    s["x"] = rand(T, K).to(_dtype(case))
    s["A"] = (rand(n, R, K) / math.sqrt(K)).bfloat16()
    s["B"] = (0.2 * rand(n, N, r)).bfloat16()
    s["scale"] = 1.0 + torch.rand(n, generator=g, device="cuda")
    f32 = dict(dtype=torch.float32, device="cuda")
    if case["kind"] == "lowrank":
        s["y_base"] = rand(T, N).to(_dtype(case))
        s["y"] = torch.empty_like(s["y_base"])
    else:
        s["dy"] = rand(T, N).bfloat16()
        s["v"] = _lowrank_v(s)
        s["dx_base"] = rand(T, K).to(_dtype(case))
        s["dx"] = torch.empty_like(s["dx_base"])
        s["dA"] = torch.empty((n, R, K), **f32)
        s["dB"] = torch.empty((n, N, r), **f32)
    return s


def _rotations(n, nblk, b, g):
    """R = (I + Q) (I - Q)^-1 of Q skew-symmetric from N(0, 0.02): [n, nblk, b, b]."""
    p = 0.02 * torch.randn((n * nblk, b, b), generator=g, device="cuda")
    q = p.triu(1)
    q = q - q.transpose(1, 2)
    one = torch.eye(b, device="cuda")
    power, inv = q, one + q
    for _ in range(5):  # (I - Q)^-1 = (I + Q) (I + Q^2) (I + Q^4) ...
        power = torch.bmm(power, power)
        inv = inv + torch.bmm(inv, power)
    return torch.bmm(one + q, inv).view(n, nblk, b, b)


def _prepare_rotate(case, seed):
    s, g = _prepare_rows(case, seed), _gen(seed)
    T, n, N, b = case["T"], case["n"], case["N"], case["b"]
    R = _rotations(n, N // b, b, g)
    s["R_f32"] = R.contiguous()
    s["R_ops"] = torch.stack([R, R.transpose(2, 3)], 2).bfloat16().contiguous()  # [n, nblk, 2, b, b]
    z = torch.randn((T, N), generator=g, device="cuda").to(_dtype(case))
    if case["kind"] == "rotate":
        s["z"] = z
        s["y"] = torch.empty_like(z)
    else:
        s["z"] = z
        s["y_saved"] = _rotated(s, z, 0).to(z.dtype)
        del s["z"]
        s["dy"] = torch.randn((T, N), generator=g, device="cuda").bfloat16()
        s["dz"] = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
        s["dq"] = torch.empty((n, N // b, b * (b - 1) // 2), dtype=torch.float32, device="cuda")
    return s


def _prepare_clip(case, seed):
    g = _gen(seed)
    sizes = [int(k) * case["pairs"] for k in case["blocks"].split(",")] * case["layers"]
    grads = [(0.01 * torch.randn(k, generator=g, device="cuda")).to(_dtype(case)) for k in sizes]
    return {"case": case, "grads": grads, "out": [torch.empty_like(t) for t in grads],
            "sumsq": torch.empty(1, dtype=torch.float64, device="cuda"),
            "stats": torch.empty(2, dtype=torch.float32, device="cuda")}


def _prepare(case, seed):
    kind = case["kind"].replace("_grad", "")
    return {"route": _prepare_rows, "lowrank": _prepare_lowrank, "rotate": _prepare_rotate,
            "clip": _prepare_clip}[kind](case, seed)


def prepare(case, seed):
    s = _prepare(case, seed)
    if own:
        import orthogonal_fine_tuning_amd as oft

        # descriptors and workspaces, which a program keeps between calls, and
        # the rows' order, which it keeps for all the projections of a step
        kind, dt = case["kind"], oft.OFT_DT_BF16 if case.get("dtype") == "bf16" else oft.OFT_DT_F32
        which = oft.OFT_PASS_BWD if kind.endswith("_grad") else oft.OFT_PASS_FWD
        need = 0
        if kind == "clip":
            s["list"] = oft.grad_list(s["grads"], s["out"])
            need = oft.oft_grad_workspace_bytes(s["list"])
        else:
            s["rows"] = oft.adapter_rows(case["T"], case["n"], "cuda")
            if kind != "route":
                oft.oft_adapter_route(s["rows"], s["adapter"])
        if kind.startswith("lowrank"):
            s["desc"] = oft.lowrank_desc(case["T"], case["n"], case["K"], _segs(case), case["r"], dt)
            need = oft.oft_lowrank_workspace_bytes(s["desc"], which)
        elif kind.startswith("rotate"):
            s["desc"] = oft.rotate_desc(case["T"], case["n"], case["N"], case["b"], dt)
            need = oft.oft_rotate_workspace_bytes(s["desc"], which)
        s["ws"], s["ws_bytes"] = torch.empty(max(16, need), dtype=torch.uint8, device="cuda"), need
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def _run_own(s):
    import orthogonal_fine_tuning_amd as oft

    kind = s["case"]["kind"]
    if kind == "route":
        oft.oft_adapter_route(s["rows"], s["adapter"])
        return {"order": s["rows"].order, "offsets": s["rows"].offsets}
    if kind == "lowrank":
        oft.oft_lowrank_fwd(s["desc"], s["rows"], s["x"], s["A"], s["B"], s["scale"], s["y_base"], s["y"], ws=s["ws"],
                            ws_bytes=s["ws_bytes"])
        return {"y": s["y"]}
    if kind == "lowrank_grad":
        oft.oft_lowrank_bwd(s["desc"], s["rows"], s["dy"], s["x"], s["v"], s["A"], s["B"], s["scale"], dx=s["dx"],
                            dx_base=s["dx_base"], dA=s["dA"], dB=s["dB"], ws=s["ws"], ws_bytes=s["ws_bytes"])
        return {"dx": s["dx"], "dA": s["dA"], "dB": s["dB"]}
    if kind == "rotate":
        oft.oft_rotate_fwd(s["desc"], s["rows"], s["z"], s["R_ops"], s["y"])
        return {"y": s["y"]}
    if kind == "rotate_grad":
        oft.oft_rotate_bwd(s["desc"], s["rows"], s["dy"], s["y_saved"], s["R_f32"], s["R_ops"], dz=s["dz"], dq=s["dq"],
                           ws=s["ws"], ws_bytes=s["ws_bytes"])
        return {"dz": s["dz"], "dq": s["dq"]}
    oft.oft_grad_sumsq(s["list"], s["sumsq"], ws=s["ws"], ws_bytes=s["ws_bytes"])
    oft.oft_grad_clip(s["list"], s["sumsq"], s["case"]["max_norm"], s["stats"])
    return {"stats": s["stats"], "out": s["out"]}


def _run_route(s):
    n, a = s["case"]["n"], s["adapter"]
    key = torch.where((a >= 0) & (a < n), a, n)
    key, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(key, torch.arange(n + 1, dtype=key.dtype, device=key.device))
    return {"order": order.int(), "offsets": offsets.int()}


def _by_request(s, t):
    """[T, C] -> fp32 [S, L, C], zeros behind a request's end."""
    t = torch.cat([t, t.new_zeros((1, t.shape[1]))])
    return t[s["padded"]].float()


def _by_row(s, t):
    """[S, L, C] -> [T, C]."""
    T = s["case"]["T"]
    out = t.new_empty((T + 1, t.shape[2]))
    out[s["padded"].reshape(-1)] = t.reshape(-1, t.shape[2])
    return out[:T]


def _of_requests(s, name):
    """An adapter tensor for each request in fp32 (any one's where it uses none)."""
    return s[name][s["request_adapter"].clamp(min=0)].float()


def _request_scale(s):
    return torch.where(s["request_adapter"] >= 0, _of_requests(s, "scale"), 0.0)[:, None, None]


def _pieces(case):
    """(first row of B, its end, first row of A, its end) of each segment."""
    ends = np.cumsum([0] + _segs(case)).tolist()
    r = case["r"]
    return [(ends[i], ends[i + 1], i * r, (i + 1) * r) for i in range(len(ends) - 1)]


def _lowrank_v(s):
    v = torch.bmm(_by_request(s, s["x"]), _of_requests(s, "A").transpose(1, 2).contiguous())
    return _by_row(s, v * (s["request_adapter"] >= 0)[:, None, None]).contiguous()


def _run_lowrank(s):
    v, B = _by_request(s, _lowrank_v(s)) * _request_scale(s), _of_requests(s, "B")
    d = torch.cat([torch.bmm(v[:, :, a:b], B[:, p:q].transpose(1, 2).contiguous()) for p, q, a, b in _pieces(s["case"])], 2)
    return {"y": (s["y_base"].float() + _by_row(s, d)).to(s["y_base"].dtype)}


def _run_lowrank_grad(s):
    case, scale = s["case"], _request_scale(s)
    dy, x, v = _by_request(s, s["dy"]), _by_request(s, s["x"]), _by_request(s, s["v"])
    A, B = _of_requests(s, "A"), _of_requests(s, "B")
    u = torch.cat([torch.bmm(dy[:, :, p:q], B[:, p:q].contiguous()) for p, q, a, b in _pieces(case)], 2) * scale
    dx = s["dx_base"].float() + _by_row(s, torch.bmm(u, A))
    dA = torch.bmm(u.transpose(1, 2).contiguous(), x)
    dB = torch.cat([torch.bmm(dy[:, :, p:q].transpose(1, 2).contiguous(), v[:, :, a:b].contiguous())
                    for p, q, a, b in _pieces(case)], 1) * scale
    at = s["request_adapter"].clamp(min=0)
    return {"dx": dx.to(s["x"].dtype), "dA": torch.zeros_like(s["A"], dtype=torch.float32).index_add_(0, at, dA),
            "dB": torch.zeros_like(s["B"], dtype=torch.float32).index_add_(0, at, dB)}


def _blocks(s, t):
    """[T, N] -> fp32 [S, nblk, L, b]."""
    t = _by_request(s, t)
    return t.view(t.shape[0], t.shape[1], -1, s["case"]["b"]).transpose(1, 2).contiguous()


def _rotated(s, t, which):
    """Rows times the transpose of R_ops[which] of their adapter, fp32 (unchanged where they use none)."""
    R = s["R_ops"][s["request_adapter"].clamp(min=0), :, which].float()  # [S, nblk, b, b]
    z = _blocks(s, t)
    S, nblk, L, b = z.shape
    y = torch.bmm(z.view(S * nblk, L, b), R.transpose(2, 3).reshape(S * nblk, b, b)).view(S, nblk, L, b)
    y = torch.where((s["request_adapter"] >= 0)[:, None, None, None], y, z)
    return _by_row(s, y.transpose(1, 2).reshape(S, L, nblk * b))


def _run_rotate_grad(s):
    case, b = s["case"], s["case"]["b"]
    dz = _rotated(s, s["dy"], 1).to(torch.bfloat16)
    dy, y = _blocks(s, s["dy"]), _blocks(s, s["y_saved"])
    S, nblk, L, _ = dy.shape
    cross = torch.bmm(dy.transpose(2, 3).reshape(S * nblk, b, L), y.view(S * nblk, L, b)).view(S, nblk, b, b)
    cross = cross * (s["request_adapter"] >= 0)[:, None, None, None]
    sums = torch.zeros_like(s["R_f32"]).index_add_(0, s["request_adapter"].clamp(min=0), cross).view(-1, b, b)
    R, one = s["R_f32"].view(-1, b, b), torch.eye(b, device="cuda")
    gq = 0.5 * torch.bmm(torch.bmm(R.transpose(1, 2).contiguous() + one, sums), one + R)
    gq = gq - gq.transpose(1, 2)
    i, j = torch.triu_indices(b, b, 1, device="cuda")
    return {"dz": dz, "dq": gq[:, i, j].view(case["n"], nblk, -1)}


def _run_clip(s):
    norm = torch.stack([t.float().square().sum() for t in s["grads"]]).sum().sqrt()
    coef = (s["case"]["max_norm"] / (norm + EPS)).clamp(max=1.0)
    return {"stats": torch.stack([norm, coef]), "out": [(t.float() * coef).to(t.dtype) for t in s["grads"]]}


def run(state):
    if own:
        return _run_own(state)
    kind = state["case"]["kind"]
    if kind == "rotate":
        return {"y": _rotated(state, state["z"], 0).to(state["z"].dtype)}
    return {"route": _run_route, "lowrank": _run_lowrank, "lowrank_grad": _run_lowrank_grad,
            "rotate_grad": _run_rotate_grad, "clip": _run_clip}[kind](state)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    kind = case["kind"]
    if kind == "clip":
        size = 2 if case["dtype"] == "bf16" else 4
        count = sum(int(k) for k in case["blocks"].split(",")) * case["pairs"] * case["layers"]
        # the norm is known only after the last gradient, so each is read again; what
        # a chip's caches could hold of the first read is not counted out
        return {"bytes": 3 * count * size + 16, "flops": 3 * count}
    T, n = case["T"], case["n"]
    if kind == "route":
        return {"bytes": 8 * T + 4 * (n + 1), "flops": T}
    size, rows = 2 if case["dtype"] == "bf16" else 4, T * (1.0 - case["free"])
    used = min(n, case["S"])  # adapters that the batch's requests use, at most
    if kind.startswith("lowrank"):
        segs = _segs(case)
        K, N, r = case["K"], sum(segs), case["r"]
        R = r * len(segs)
        factors = R * K + N * r
        if kind == "lowrank":
            return {"bytes": int(rows * K * size + 2 * T * N * size + 2 * used * factors), "flops": int(2 * rows * factors)}
        return {"bytes": int(rows * (2 * N + size * K + 4 * R) + 2 * T * K * size + 2 * used * factors + 4 * n * factors),
                "flops": int(4 * rows * factors)}
    N, b = case["N"], case["b"]
    if kind == "rotate":
        return {"bytes": int(2 * T * N * size + 2 * used * N * b), "flops": int(2 * rows * N * b)}
    return {"bytes": int(4 * T * N + rows * N * size + 2 * used * N * b + 4 * used * N * b + 2 * n * N * (b - 1)),
            "flops": int(4 * rows * N * b)}


# --------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------
def _exact_route(s):
    n, a = s["case"]["n"], s["adapter"].cpu().numpy()
    key = np.where((a >= 0) & (a < n), a, n)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=n + 1)[:n])])
    return {"order": torch.from_numpy(np.argsort(key, kind="stable").astype(np.int32)),
            "offsets": torch.from_numpy(offsets.astype(np.int32))}


def _rows_of(s):
    """(adapter, its rows) of the batch, adapters in use alone."""
    a = s["adapter"].long()
    return [(i, (a == i).nonzero()[:, 0]) for i in a.unique().tolist() if i >= 0]


def _exact_lowrank(s):
    case = s["case"]
    segs, r = _segs(case), case["r"]
    if case["kind"] == "lowrank":
        y = s["y_base"].double()
        for i, rows in _rows_of(s):
            x = s["x"][rows].double()
            for k, part in enumerate(torch.split(torch.arange(sum(segs), device=x.device), segs)):
                up = s["B"][i, part].double() @ s["A"][i, k * r:(k + 1) * r].double()  # [seg, K], the update itself
                y[rows[:, None], part] += s["scale"][i].double() * (x @ up.T)
        return {"y": y}
    dx = s["dx_base"].double()
    dA, dB = torch.zeros_like(s["A"], dtype=torch.float64), torch.zeros_like(s["B"], dtype=torch.float64)
    for i, rows in _rows_of(s):
        x, dy, v, c = s["x"][rows].double(), s["dy"][rows].double(), s["v"][rows].double(), s["scale"][i].double()
        for k, part in enumerate(torch.split(torch.arange(sum(segs), device=x.device), segs)):
            a, b = s["A"][i, k * r:(k + 1) * r].double(), s["B"][i, part].double()
            dx[rows] += c * (dy[:, part] @ (b @ a))
            dA[i, k * r:(k + 1) * r] = c * (b.T @ (dy[:, part].T @ x))
            dB[i, part] = c * (dy[:, part].T @ v[:, k * r:(k + 1) * r])
    return {"dx": dx, "dA": dA, "dB": dB}


def _exact_rotate(s):
    case = s["case"]
    b, N = case["b"], case["N"]
    grad = case["kind"] == "rotate_grad"
    src = s["dy"] if grad else s["z"]
    out = src.double()
    dq = torch.zeros((case["n"], N // b, b * (b - 1) // 2), dtype=torch.float64, device=src.device)
    i, j = torch.triu_indices(b, b, 1, device=src.device)
    one = torch.eye(b, dtype=torch.float64, device=src.device)
    for a, rows in _rows_of(s):
        for k in range(N // b):
            at = slice(k * b, (k + 1) * b)
            t = src[rows, at].double()
            R = s["R_ops"][a, k, 0].double()
            # y = R z a row, so that dz = R^T dy
            out[rows, at] = t @ (R if grad else R.T)
            if grad:
                R = s["R_f32"][a, k].double()
                G = t.T @ (s["y_saved"][rows, at].double() @ R)  # the gradient of R, z = R^T y
                gq = 0.5 * (R.T + one) @ G @ (R.T + one)
                dq[a, k] = (gq - gq.T)[i, j]
    return {"dz": out, "dq": dq} if grad else {"y": out}


def _exact_clip(s):
    total = sum(float(t.double().square().sum()) for t in s["grads"])
    coef = min(1.0, s["case"]["max_norm"] / (math.sqrt(total) + EPS))
    return {"stats": torch.tensor([math.sqrt(total), coef], dtype=torch.float64),
            "out": [t.double() * coef for t in s["grads"]]}


def exact(case, seed):
    s = _prepare(case, seed)
    kind = case["kind"].replace("_grad", "")
    return {"route": _exact_route, "lowrank": _exact_lowrank, "rotate": _exact_rotate, "clip": _exact_clip}[kind](s)
