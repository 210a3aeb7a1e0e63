"""The policy and router loss operators as measured: their cases, plain forms and 64-bit results.

Three operators that an adapter's training step and a rollout server compute
from logits:

  logprobs / logprobs_grad   log-probabilities of given tokens with the entropy
                             and the top alternatives of each row, and the
                             gradient of the first two with respect to the logits;
  distill / distill_grad     distillation from a teacher's top logits: the
                             cross entropy against the teacher's renormalised
                             list (minus the list's own entropy), and its gradient;
  balance                    the router's balance loss with per-expert counts,
                             forward and then backward, as a training step runs it.

`run` computes them in elementary torch operations in 32 bits, or, where `own`
is set, through orthogonal_fine_tuning_amd.
"""
import math

import torch

own = False

IGNORE = -1  # label of a row without a given token


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _vocab(name, kind, T, V, dtype, k=0, pad=0, temperature=1.0, masked=0):
    """pad: unused elements behind each row; masked: columns at -inf at the end."""
    c = {"kind": kind, "T": T, "V": V, "dtype": dtype, "k": k, "pad": pad, "temperature": temperature, "masked": masked}
    return {"name": name, **c} if name else c


def _balance(name, S, L, E, k, padded):
    c = {"kind": "balance", "S": S, "L": L, "E": E, "k": k, "padded": padded}
    return {"name": name, **c} if name else c


def listed():
    return [
        # one decoded token: its log-probability and the alternatives a server returns
        _vocab("logprobs_one_token", "logprobs", 1, 151936, "bf16", k=20, temperature=0.7, masked=267),
        # a decode batch of the same vocabulary
        _vocab("logprobs_decode_batch", "logprobs", 64, 151936, "bf16", k=5, masked=267),
        # scoring rollouts: a training batch's rows, with alternatives
        _vocab("logprobs_rollout", "logprobs", 4096, 151936, "bf16", k=20, temperature=0.7, masked=267),
        # a teacher's list of 128 from fp32 logits, an odd vocabulary (rows start off alignment)
        _vocab("logprobs_teacher_list_f32", "logprobs", 333, 50021, "f32", k=128),
        # the policy loss's gradient with an entropy bonus, a training batch
        _vocab("logprobs_grad_train", "logprobs_grad", 4096, 151936, "bf16", temperature=0.7, masked=267),
        # the same on fp32 rows that are a slice of wider ones
        _vocab("logprobs_grad_f32_sliced", "logprobs_grad", 129, 32003, "f32", pad=61),
        # distillation from 64 teacher entries, a training batch
        _vocab("distill_train", "distill", 4096, 151936, "bf16", k=64, temperature=2.0),
        # a few odd fp32 rows, 100 entries
        _vocab("distill_f32_odd", "distill", 57, 50021, "f32", k=100),
        # its gradient, a training batch
        _vocab("distill_grad_train", "distill_grad", 2048, 151936, "bf16", k=64, temperature=2.0),
        # and on odd bf16 rows
        _vocab("distill_grad_odd", "distill_grad", 200, 50021, "bf16", k=256, temperature=1.5),
        # a router's balance loss: one sequence, and batches of padded sequences
        _balance("balance_one_sequence", 1, 512, 64, 4, False),
        _balance("balance_batch", 8, 4096, 384, 8, True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["logprobs", "logprobs_grad", "distill", "distill_grad", "balance"])
    if kind == "balance":
        k = rng.randint(1, 8)
        L = _log_int(rng, 32, 4096)
        return _balance(None, _log_int(rng, 1, 8), L, _log_int(rng, max(8, k), 512), k, rng.random() < 0.5)
    V = _log_int(rng, 1000, 151936)
    T = _log_int(rng, 1, 4096)
    k = {"logprobs": rng.choice([0, _log_int(rng, 1, 128)]), "logprobs_grad": 0}.get(kind, _log_int(rng, 1, 256))
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if dtype == "f32":
        T = min(T, 2048)
    return _vocab(None, kind, T, V, dtype, k=k, pad=rng.choice([0, 0, rng.randint(1, 200)]),
                  temperature=rng.choice([1.0, 1.0, round(rng.uniform(0.5, 2.5), 2)]),
                  masked=rng.choice([0, rng.randint(1, 300)]))


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(0x5EED + int(seed))


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _logits(case, g):
    """Rows as a vocabulary projection gives them: a broad bulk and a few
    likely tokens above it; [T, V] inside rows of V + pad elements.  Returns
    the rows and the columns of their likely tokens."""
    T, V, n = case["T"], case["V"], min(300, case["V"] // 2)
    x = torch.randn((T, V + case["pad"]), generator=g, device="cuda").mul_(2.2)
    live = V - case["masked"]
    # distinct columns: one in each of n equal stretches of the live ones
    width = live // n
    likely = torch.arange(n, device="cuda") * width + torch.randint(0, width, (T, n), generator=g, device="cuda")
    x.scatter_add_(1, likely, 10.0 * torch.rand((T, n), generator=g, device="cuda") ** 2)
    x = x.to(_dtype(case))
    if case["masked"]:
        x[:, live:V] = -math.inf
    return x[:, :V], likely


def _rows_without_token(T):
    """Every sixteenth row of a training batch is prompt or padding."""
    return torch.arange(T, device="cuda") % 16 == 15


def _prepare_vocab(case, seed):
    g = _gen(seed)
    T, V, kind, tau = case["T"], case["V"], case["kind"], case["temperature"]
    x, likely = _logits(case, g)
    s = {"case": case, "logits": x}
    f32 = dict(dtype=torch.float32, device="cuda")
    if kind in ("logprobs", "logprobs_grad"):
        pick = torch.randint(0, likely.shape[1], (T, 1), generator=g, device="cuda")
        s["labels"] = torch.where(_rows_without_token(T), IGNORE, likely.gather(1, pick)[:, 0]).int()
    else:
        # the teacher's list: likely tokens first, then other columns, best first
        K, n = case["k"], likely.shape[1]
        order = torch.rand((T, n), generator=g, device="cuda").argsort(1)
        cols = likely.gather(1, order)[:, :K]
        s["teacher_idx"] = cols.int().contiguous()
        s["teacher_logits"] = (8.0 * torch.rand((T, K), generator=g, device="cuda")).sort(1, descending=True)[0]
    if kind.endswith("_grad"):
        # what the forward left: the rows' maximum, log sum and entropy
        y = x.float()
        m = y.amax(1)
        z = (y - m[:, None]) / tau
        e = z.exp()
        S = e.sum(1)
        l = S.log()
        s["stats"] = torch.stack([m, l], 1).contiguous()
        s["entropy"] = l - torch.where(e > 0, e * z, 0.0).sum(1) / S
        s["d_logits"] = torch.empty((T, V + case["pad"]), dtype=x.dtype, device="cuda")[:, :V]
        gr = torch.randn(T, generator=g, **f32)
        if kind == "logprobs_grad":
            off = _rows_without_token(T)
            s["g_logp"] = gr
            s["g_entropy"] = torch.where(off, 0.0, 0.1 * torch.rand(T, generator=g, **f32))
        else:
            s["g_loss"] = gr.abs()
    elif kind == "logprobs":
        s["logp"] = torch.empty(T, **f32)
        s["entropy"] = torch.empty(T, **f32)
        s["stats"] = torch.empty((T, 2), **f32)
        if case["k"]:
            s["top_idx"] = torch.empty((T, case["k"]), dtype=torch.int32, device="cuda")
            s["top_logp"] = torch.empty((T, case["k"]), **f32)
    else:
        s["loss"] = torch.empty(T, **f32)
        s["stats"] = torch.empty((T, 2), **f32)
    return s


def _prepare_balance(case, seed):
    g = _gen(seed)
    S, L, E, k = case["S"], case["L"], case["E"], case["k"]
    T = S * L
    # experts differ in how often they are chosen, as a router's do
    logits = torch.randn((T, E), generator=g, device="cuda") + 0.5 * torch.randn(E, generator=g, device="cuda")
    s = {"case": case, "logits": logits, "topk_idx": logits.topk(k, 1)[1].int().contiguous(), "mask": None}
    if case["padded"]:
        length = torch.randint(max(1, L // 2), L + 1, (S, 1), generator=g, device="cuda")
        s["mask"] = (torch.arange(L, device="cuda") < length).to(torch.uint8).reshape(T)
    f32 = dict(dtype=torch.float32, device="cuda")
    s["g_loss"] = 0.01 * (1.0 + torch.rand(S, generator=g, **f32))
    s["counts"] = torch.empty((S, E), dtype=torch.int32, device="cuda")
    s["tokens"] = torch.empty(S, dtype=torch.int32, device="cuda")
    s["loss"] = torch.empty(S, **f32)
    s["mean_prob"] = torch.empty((S, E), **f32)
    s["d_logits"] = torch.empty((T, E), **f32)
    return s


def prepare(case, seed):
    s = (_prepare_balance if case["kind"] == "balance" else _prepare_vocab)(case, seed)
    if own:
        import orthogonal_fine_tuning_amd as oft

        # the descriptor and the workspace, which a program keeps between calls
        if case["kind"] == "balance":
            # the layer around the router plays no part in its loss
            s["desc"] = oft.moe_desc(case["S"] * case["L"], case["E"], case["k"], 64, 64, 32, 32, 16)
            s["ws_bytes"] = oft.oft_moe_balance_workspace_bytes(s["desc"], case["L"])
        else:
            ld = case["V"] + case["pad"]
            s["desc"] = oft.vocab_desc(case["T"], case["V"], oft.OFT_DT_BF16 if case["dtype"] == "bf16" else oft.OFT_DT_F32,
                                       k=case["k"], ld=ld, ld_grad=ld, temperature=case["temperature"])
            s["ws_bytes"] = oft.oft_vocab_workspace_bytes(s["desc"])
        s["ws"] = torch.empty(max(16, s["ws_bytes"]), dtype=torch.uint8, device="cuda")
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def _run_own(s):
    import orthogonal_fine_tuning_amd as oft

    kind = s["case"]["kind"]
    if kind == "logprobs":
        top = {"top_idx": s["top_idx"], "top_logp": s["top_logp"]} if s["case"]["k"] else {}
        oft.oft_token_logprobs(s["desc"], s["logits"], s["labels"], s["logp"], s["stats"], entropy=s["entropy"],
                               ws=s["ws"], ws_bytes=s["ws_bytes"], **top)
        return {"logp": s["logp"], "stats": s["stats"], "entropy": s["entropy"], **top}
    if kind == "logprobs_grad":
        oft.oft_token_logprobs_bwd(s["desc"], s["logits"], s["labels"], s["stats"], s["g_logp"], s["d_logits"],
                                   entropy=s["entropy"], g_entropy=s["g_entropy"])
        return {"d_logits": s["d_logits"]}
    if kind == "distill":
        oft.oft_distill_topk(s["desc"], s["logits"], s["teacher_idx"], s["teacher_logits"], s["loss"], s["stats"],
                             ws=s["ws"], ws_bytes=s["ws_bytes"])
        return {"loss": s["loss"], "stats": s["stats"]}
    if kind == "distill_grad":
        oft.oft_distill_topk_bwd(s["desc"], s["logits"], s["teacher_idx"], s["teacher_logits"], s["stats"],
                                 s["g_loss"], s["d_logits"])
        return {"d_logits": s["d_logits"]}
    L = s["case"]["L"]
    oft.oft_moe_balance(s["desc"], L, s["logits"], s["topk_idx"], s["counts"], s["tokens"], s["loss"],
                        mean_prob=s["mean_prob"], mask=s["mask"], ws=s["ws"], ws_bytes=s["ws_bytes"])
    oft.oft_moe_balance_bwd(s["desc"], L, s["logits"], s["counts"], s["tokens"], s["g_loss"], s["d_logits"],
                            mask=s["mask"])
    return {k: s[k] for k in ("counts", "tokens", "loss", "mean_prob", "d_logits")}


def _top(x, k):
    """Columns of the k largest of each row, ties to the lower column: one
    integer key of value (its bits in order) and column, so that no two are equal."""
    bits = (x + 0.0).view(torch.int32)
    order = bits ^ ((bits >> 31) & 0x7FFFFFFF)
    key = order.long() * (1 << 32) + ((1 << 32) - 1 - torch.arange(x.shape[1], device=x.device))
    return key.topk(k, 1)[1]


def _run_vocab(s):
    case, tau = s["case"], s["case"]["temperature"]
    x = s["logits"].float()
    rows = torch.arange(x.shape[0], device=x.device)
    if not case["kind"].endswith("_grad"):
        m = x.amax(1, keepdim=True)
        z = (x - m) / tau
        e = z.exp()
        S = e.sum(1)
        l = S.log()
        stats = torch.stack([m[:, 0], l], 1)
        if case["kind"] == "distill":
            u = s["teacher_logits"] / tau
            u = u - u.amax(1, keepdim=True)
            logq = u - u.exp().sum(1, keepdim=True).log()
            logp = z.gather(1, s["teacher_idx"].long()) - l[:, None]
            return {"loss": (logq.exp() * (logq - logp)).sum(1), "stats": stats}
        given = s["labels"].long()
        logp = torch.where(given >= 0, z[rows, given.clamp(min=0)] - l, 0.0)
        entropy = l - torch.where(e > 0, e * z, 0.0).sum(1) / S
        out = {"logp": logp, "stats": stats, "entropy": entropy}
        if case["k"]:
            top = _top(x, case["k"])
            out["top_idx"] = top.int()
            out["top_logp"] = z.gather(1, top) - l[:, None]
        return out
    lp = (x - s["stats"][:, :1]) / tau - s["stats"][:, 1:]  # log p
    p = lp.exp()
    if case["kind"] == "distill_grad":
        u = s["teacher_logits"] / tau
        q = (u - u.amax(1, keepdim=True)).exp()
        d = p.scatter_add(1, s["teacher_idx"].long(), -q / q.sum(1, keepdim=True)) * (s["g_loss"] / tau)[:, None]
        return {"d_logits": d.to(s["logits"].dtype)}
    given = s["labels"].long()
    gl = torch.where(given >= 0, s["g_logp"], 0.0)
    d = -p * (gl[:, None] + s["g_entropy"][:, None] * (torch.where(p > 0, lp, 0.0) + s["entropy"][:, None]))
    d[rows, given.clamp(min=0)] += gl
    return {"d_logits": (d / tau).to(s["logits"].dtype)}


def _run_balance(s):
    S, L, E, k = (s["case"][n] for n in ("S", "L", "E", "k"))
    x = s["logits"]
    use = torch.ones(S * L, device=x.device) if s["mask"] is None else s["mask"].float()
    p = (x - x.amax(1, keepdim=True)).exp()
    p = p / p.sum(1, keepdim=True) * use[:, None]
    hot = torch.zeros_like(x).scatter_(1, s["topk_idx"].long(), 1.0) * use[:, None]
    counts = hot.view(S, L, E).sum(1)
    n = use.view(S, L).sum(1)
    f = counts / (n * k)[:, None]
    P = p.view(S, L, E).sum(1) / n[:, None]
    loss = E * (f * P).sum(1)
    ft = f.repeat_interleave(L, 0)
    scale = (s["g_loss"] * E / n).repeat_interleave(L)
    d = scale[:, None] * p * (ft - (ft * p).sum(1, keepdim=True))
    return {"counts": counts.int(), "tokens": n.int(), "loss": loss, "mean_prob": P, "d_logits": d}


def run(state):
    if own:
        return _run_own(state)
    return _run_balance(state) if state["case"]["kind"] == "balance" else _run_vocab(state)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    if case["kind"] == "balance":
        T, E, S = case["S"] * case["L"], case["E"], case["S"]
        return {"bytes": 4 * T * E + 4 * T * case["k"] + 4 * T * E + 8 * S * E + (T if case["padded"] else 0),
                "flops": 12 * T * E}
    T, V, size = case["T"], case["V"], 2 if case["dtype"] == "bf16" else 4
    row = size * V
    if case["kind"] == "logprobs":
        return {"bytes": T * (row + 20 + 8 * case["k"]), "flops": 6 * T * V}
    if case["kind"] == "distill":
        return {"bytes": T * (row + 12 + 8 * case["k"]), "flops": 4 * T * V}
    if case["kind"] == "logprobs_grad":
        # the rows without a token have no gradient to compute
        return {"bytes": (T - T // 16) * row + T * (row + 24), "flops": 8 * (T - T // 16) * V}
    return {"bytes": T * (2 * row + 12 + 8 * case["k"]), "flops": 4 * T * V}


# --------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------
def _exact_rows(s, a, b):
    """Rows a .. b of a vocabulary case."""
    case, kind = s["case"], s["case"]["kind"]
    x = s["logits"][a:b].double()
    lp = torch.log_softmax(x / case["temperature"], 1)
    out = {}
    if "teacher_idx" in s:
        idx = s["teacher_idx"][a:b].long()
        lq = torch.log_softmax(s["teacher_logits"][a:b].double() / case["temperature"], 1)
        if kind == "distill":
            out["loss"] = (lq.exp() * (lq - lp.gather(1, idx))).sum(1)
        else:
            d = lp.exp()
            d.scatter_add_(1, idx, -lq.exp())
            out["d_logits"] = d * s["g_loss"][a:b, None].double() / case["temperature"]
    else:
        lab = s["labels"][a:b].long()
        has = lab >= 0
        p = lp.exp()
        h = -torch.special.xlogy(p, p).sum(1)
        if kind == "logprobs":
            out["logp"] = torch.where(has, lp.gather(1, lab.clamp(min=0)[:, None])[:, 0], 0.0)
            out["entropy"] = h
            if case["k"]:
                val, col = x.sort(stable=True, dim=1, descending=True)
                out["top_idx"] = col[:, :case["k"]].int()
                out["top_logp"] = lp.gather(1, col[:, :case["k"]])
        else:
            gl = torch.where(has, s["g_logp"][a:b].double(), 0.0)[:, None]
            ge = s["g_entropy"][a:b].double()[:, None]
            d = torch.zeros_like(p).scatter_(1, lab.clamp(min=0)[:, None], gl) - gl * p
            d -= ge * (torch.special.xlogy(p, p) + h[:, None] * p)
            out["d_logits"] = d / case["temperature"]
    if not kind.endswith("_grad"):
        m = x.max(1)[0]
        out["stats"] = torch.stack([m, torch.logsumexp(x / case["temperature"], 1) - m / case["temperature"]], 1)
    return out


def _exact_balance(s):
    S, L, E, k = (s["case"][n] for n in ("S", "L", "E", "k"))
    out = {n: [] for n in ("counts", "tokens", "loss", "mean_prob", "d_logits")}
    for i in range(S):
        at = slice(i * L, (i + 1) * L)
        x = s["logits"][at].double().requires_grad_(True)
        use = torch.ones(L, dtype=torch.bool, device=x.device) if s["mask"] is None else s["mask"][at].bool()
        n = int(use.sum())
        counts = torch.bincount(s["topk_idx"][at][use].long().reshape(-1), minlength=E)
        P = torch.softmax(x, 1)[use].mean(0)
        loss = E * (counts.double() / (n * k) * P).sum()
        (d,) = torch.autograd.grad(loss, x, s["g_loss"][i].double())
        for name, v in (("counts", counts.int()), ("tokens", torch.tensor(n, dtype=torch.int32, device=x.device)),
                        ("loss", loss.detach()), ("mean_prob", P.detach()), ("d_logits", d)):
            out[name].append(v)
    return {n: torch.cat(v) if n == "d_logits" else torch.stack(v) for n, v in out.items()}


def exact(case, seed):
    s = (_prepare_balance if case["kind"] == "balance" else _prepare_vocab)(case, seed)
    if case["kind"] == "balance":
        return _exact_balance(s)
    step = max(1, (1 << 27) // case["V"])
    parts = [_exact_rows(s, a, min(case["T"], a + step)) for a in range(0, case["T"], step)]
    return {name: torch.cat([p[name] for p in parts]) for name in parts[0]}
