"""The operators on adapters of many requests as programs use them: together
with the layers, captured and replayed, on other streams, and on batches that
their documentation allows and no plain case holds."""
import numpy as np
import pytest

from oft_inputs import DenseConfig, make_dense
from oracle import adapters as oracle
from oracle import dense as odense
from tests import adapter_cases as cases
from tests.helpers import dev, err, host
from tests.test_gpu_adapters import _down, _empty, _rows, _up, _within, _ws

pytestmark = pytest.mark.gpu


def _oft():
    import orthogonal_fine_tuning_amd as oft

    return oft


class Batch:
    """Inputs, outputs and workspaces of one call of each operator."""

    def __init__(self, T, n, K, segs, r, b, kind, seed):
        import torch

        oft = _oft()
        self.T, self.n, self.segs, self.N, self.r, self.b = T, n, segs, sum(segs), r, b
        c = cases.lowrank(T, n, K, segs, r, "bf16", kind, seed)
        self.adapter = _up(c["adapter"])
        self.t = {k: _up(v, "f32" if k == "scale" else "bf16") for k, v in c.items() if k != "adapter"}
        p, _ = cases.rotations(n, self.N // b, b, seed)
        self.Rf = torch.empty((n, self.N // b, b, b), device="cuda")
        self.Rops = torch.empty((n, self.N // b, 2, b, b), dtype=torch.bfloat16, device="cuda")
        oft.cayley_build(_up(p, "bf16"), n * (self.N // b), b, self.Rf, self.Rops)
        self.ld = oft.lowrank_desc(T, n, K, segs, r)
        self.rd = oft.rotate_desc(T, n, self.N, b)
        self.rows = oft.adapter_rows(T, n)
        self.ws = [_ws(oft.oft_lowrank_workspace_bytes(self.ld, p)) for p in (0, 1)] + [
            _ws(oft.oft_rotate_workspace_bytes(self.rd, 1))]
        self.out = dict(z=_empty((T, self.N), "bf16"), y=_empty((T, self.N), "bf16"), v=_empty((T, r * len(segs))),
                        dx=_empty((T, K), "bf16"), dA=_empty((n, r * len(segs), K)), dB=_empty((n, self.N, r)),
                        dz=_empty((T, self.N), "bf16"), dq=_empty((n, self.N // b, b * (b - 1) // 2)))
        self.stats = _empty((2,))
        self.sumsq = torch.zeros(1, dtype=torch.float64, device="cuda")
        self.clipped = {k: _empty(self.out[k].shape) for k in ("dA", "dB", "dq")}
        self.grads = oft.grad_list([self.out[k] for k in self.clipped], list(self.clipped.values()))
        self.gws = _ws(oft.oft_grad_workspace_bytes(self.grads))

    def run(self, ws=None, stream=None):
        oft = _oft()
        t, o, w = self.t, self.out, ws or self.ws
        oft.oft_adapter_route(self.rows, self.adapter, stream=stream)
        oft.oft_rotate_fwd(self.rd, self.rows, t["y_base"], self.Rops, o["z"], stream=stream)
        oft.oft_lowrank_fwd(self.ld, self.rows, t["x"], t["A"], t["B"], t["scale"], o["z"], o["y"], v=o["v"], ws=w[0][0],
                            ws_bytes=w[0][1], stream=stream)
        oft.oft_rotate_bwd(self.rd, self.rows, t["dy"], o["z"], self.Rf, self.Rops, dz=o["dz"], dq=o["dq"], ws=w[2][0],
                           ws_bytes=w[2][1], stream=stream)
        oft.oft_lowrank_bwd(self.ld, self.rows, t["dy"], t["x"], o["v"], t["A"], t["B"], t["scale"], dx=o["dx"],
                            dx_base=t["dx_base"], dA=o["dA"], dB=o["dB"], ws=w[1][0], ws_bytes=w[1][1], stream=stream)
        oft.oft_grad_sumsq(self.grads, self.sumsq, ws=self.gws[0], ws_bytes=self.gws[1], stream=stream)
        oft.oft_grad_clip(self.grads, self.sumsq, 0.5, self.stats, stream=stream)

    def results(self):
        return {**self.out, **{"clipped " + k: v for k, v in self.clipped.items()}, "stats": self.stats,
                "order": self.rows.order, "offsets": self.rows.offsets}


def _same(a, b, what):
    import torch

    for k in a:
        assert torch.equal(a[k], b[k]), (what, k)


@pytest.mark.parametrize("T", [70, 1500, 5000])
def test_graphs_that_share_workspaces_follow_their_inputs(T):
    """One batch captured twice into two graphs that share every workspace;
    each replay has another batch (other rows, another mix of adapters) and is
    compared with an eager run in its own memory, bit for bit."""
    import torch

    a, e = (Batch(T, 5, 128, (64, 96), 16, 32, "some", 1) for _ in range(2))
    b = Batch(T, 5, 128, (64, 96), 16, 32, "mixed", 2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a.run()
        b.run(a.ws)
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        a.run()
    with torch.cuda.graph(g2):
        b.run(a.ws)
    for i, kind in enumerate(["runs", "one", "none", "skewed", "some"]):
        ad = _up(cases.adapters(T, 5, kind, i))
        x = _up(cases.bf16(np.random.default_rng(i).normal(0, 1, (T, 128))), "bf16")
        want = []
        for s in (a, b):
            s.adapter.copy_(ad)
            s.t["x"].copy_(x)
            e.adapter.copy_(ad)
            for k in s.t:
                e.t[k].copy_(s.t[k])
            e.Rf.copy_(s.Rf)
            e.Rops.copy_(s.Rops)
            e.run()
            torch.cuda.synchronize()
            want.append({k: v.clone() for k, v in e.results().items()})
        g1.replay()
        g2.replay()
        torch.cuda.synchronize()
        _same(want[0], a.results(), (i, kind))
        _same(want[1], b.results(), (i, kind))


def test_two_streams_at_once_share_the_rows():
    """Two streams, each with its own outputs and workspaces, and calls on one
    batch's order from both."""
    import torch

    want = Batch(1300, 4, 128, (96, 32), 8, 16, "mixed", 3)
    want.run()
    both = [Batch(1300, 4, 128, (96, 32), 8, 16, "mixed", 3) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in both]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, b in zip(streams, both):
            b.run(stream=s.cuda_stream)
    torch.cuda.synchronize()
    for b in both:
        _same(want.results(), b.results(), "streams")
    # the same order, read from two streams at once
    oft = _oft()
    outs = [_empty((1300, 128), "bf16") for _ in both]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, o in zip(streams, outs):
            oft.oft_rotate_fwd(want.rd, want.rows, want.t["y_base"], want.Rops, o, stream=s.cuda_stream)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want.out["z"])


def test_current_stream_is_taken():
    import torch

    want, b = (Batch(200, 3, 64, (32,), 8, 32, "mixed", 4) for _ in range(2))
    want.run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        b.run()
    s.synchronize()
    _same(want.results(), b.results(), "current stream")


@pytest.mark.parametrize("T", [300, 1500])
def test_order_of_the_rows_does_not_show(T):
    """Rows in another order: each row's results move with it, bit for bit, and
    twice the same call gives the same bits."""
    import torch

    a = Batch(T, 4, 128, (64, 64), 16, 32, "some", 5)
    a.run()
    first = {k: v.clone() for k, v in a.results().items()}
    a.run()
    _same(first, a.results(), "again")
    perm = torch.randperm(T, generator=torch.Generator().manual_seed(1)).cuda()
    for k in ("x", "y_base", "dy", "dx_base"):
        a.t[k].copy_(a.t[k][perm])
    a.adapter.copy_(a.adapter[perm])
    a.run()
    for k in ("z", "y", "v", "dx", "dz"):
        assert torch.equal(a.out[k], first[k][perm]), k


@pytest.mark.parametrize("T", [100, 1500])
def test_infinities_and_nan_stay_with_their_rows(T):
    """A row of NaN or infinities reaches its own results and its adapter's
    gradients; an adapter without rows may hold anything."""
    import torch

    n, bad = 4, 2
    a, clean = (Batch(T, n, 128, (64, 64), 16, 32, "mixed", 6) for _ in range(2))
    ad = cases.adapters(T, n - 1, "mixed", 6)  # (adapter 3 has no rows)
    for s in (a, clean):
        s.adapter.copy_(_up(ad))
    rows = np.flatnonzero(ad == bad)[:3]
    for k, what in (("x", float("nan")), ("y_base", float("inf")), ("dy", float("-inf"))):
        a.t[k][torch.from_numpy(rows).cuda()] = what
    a.t["A"][3] = float("nan")
    a.t["B"][3] = float("inf")
    a.t["scale"][3] = float("nan")
    a.Rops[3] = float("nan")
    a.Rf[3] = float("inf")
    a.run()
    clean.run()
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[torch.from_numpy(rows).cuda()] = False
    for k in ("z", "y", "v", "dx", "dz"):
        assert torch.equal(a.out[k][keep], clean.out[k][keep]), k
        assert not torch.isfinite(a.out[k][~keep]).all(), k
    for k in ("dA", "dB", "dq"):
        for i in (0, 1, 3):
            assert torch.equal(a.out[k][i], clean.out[k][i]), (k, i)
        assert (a.out[k][3] == 0).all() and not torch.isfinite(a.out[k][bad]).all()


def test_no_rows_at_all():
    import torch

    oft = _oft()
    rows = oft.adapter_rows(0, 3)
    oft.oft_adapter_route(rows, torch.empty(0, dtype=torch.int32, device="cuda"))
    assert rows.offsets.tolist() == [0, 0, 0, 0]
    bf = lambda *s: torch.ones(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    d = oft.lowrank_desc(0, 3, 64, (32,), 8)
    dA, dB = _empty((3, 8, 64)), _empty((3, 32, 8))
    oft.oft_lowrank_fwd(d, rows, bf(0, 64), bf(3, 8, 64), bf(3, 32, 8), torch.ones(3, device="cuda"), bf(0, 32), bf(0, 32))
    oft.oft_lowrank_bwd(d, rows, bf(0, 32), bf(0, 64), _empty((0, 8)), bf(3, 8, 64), bf(3, 32, 8),
                        torch.ones(3, device="cuda"), dx=bf(0, 64), dA=dA, dB=dB)
    rd = oft.rotate_desc(0, 3, 32, 16)
    dq = _empty((3, 2, 120))
    oft.oft_rotate_fwd(rd, rows, bf(0, 32), bf(3, 2, 2, 16, 16), bf(0, 32))
    oft.oft_rotate_bwd(rd, rows, bf(0, 32), bf(0, 32), _empty((3, 2, 16, 16)), bf(3, 2, 2, 16, 16), dz=bf(0, 32), dq=dq)
    for t in (dA, dB, dq):
        assert (t == 0).all()


def test_streamed_rows():
    """Rows of more bytes than the caches hold take other loads and stores:
    rows picked from them against 64 bits, the rest against calls of 1000 rows."""
    import torch

    oft = _oft()
    T, n, N, K, r, b = 36000, 3, 2048, 64, 16, 32
    g = torch.Generator(device="cuda").manual_seed(3)
    bf = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    ad = torch.randint(-1, n, (T,), generator=g, device="cuda").int()
    z, dy, x, A, B = bf(T, N), bf(T, N), bf(T, K), bf(n, r, K) / 8, bf(n, N, r)
    scale = torch.tensor([0.5, 1.0, 2.0], device="cuda")
    p, _ = cases.rotations(n, N // b, b)
    Rf = torch.empty((n, N // b, b, b), device="cuda")
    Rops = torch.empty((n, N // b, 2, b, b), dtype=torch.bfloat16, device="cuda")
    oft.cayley_build(_up(p, "bf16"), n * (N // b), b, Rf, Rops)
    rows = oft.adapter_rows(T, n)
    oft.oft_adapter_route(rows, ad)
    rd, ld = oft.rotate_desc(T, n, N, b), oft.lowrank_desc(T, n, K, (N,), r)
    y, dz, low = torch.empty_like(z), torch.empty_like(z), torch.empty_like(z)
    dq = _empty((n, N // b, b * (b - 1) // 2))
    ws, nb = _ws(oft.oft_rotate_workspace_bytes(rd, 1))
    oft.oft_rotate_fwd(rd, rows, z, Rops, y)
    oft.oft_rotate_bwd(rd, rows, dy, y, Rf, Rops, dz=dz, dq=dq, ws=ws, ws_bytes=nb)
    ws, nb = _ws(oft.oft_lowrank_workspace_bytes(ld, 0))
    oft.oft_lowrank_fwd(ld, rows, x, A, B, scale, z, low, ws=ws, ws_bytes=nb)
    for at in range(0, T, 1000):  # (rows on their own rotate to the same bits)
        part = oft.adapter_rows(1000, n)
        oft.oft_adapter_route(part, ad[at:at + 1000].clone())
        one = torch.empty((1000, N), dtype=torch.bfloat16, device="cuda")
        d1 = oft.rotate_desc(1000, n, N, b)
        oft.oft_rotate_fwd(d1, part, z[at:at + 1000].clone(), Rops, one)
        assert torch.equal(one, y[at:at + 1000])
        oft.oft_rotate_bwd(d1, part, dy[at:at + 1000].clone(), None, None, Rops, dz=one)
        assert torch.equal(one, dz[at:at + 1000])
    pick = np.concatenate([[0, 1, T - 2, T - 1], np.random.default_rng(1).integers(0, T, 60)])
    a = ad.cpu().numpy()[pick]
    c = {"x": _down(x[pick]), "A": _down(A), "B": _down(B), "scale": _down(scale), "y_base": _down(z[pick]), "adapter": a}
    (want, tol), _ = cases.lowrank_fwd(c, (N,), "bf16")
    _within(low[pick], want, tol, "low rank")
    # dq: the sums of all rows, in 64 bits on the GPU
    i, l = np.triu_indices(b, 1)
    eye = np.eye(b)
    for k in range(n):
        sel = (ad == k).nonzero()[:, 0]
        S = torch.einsum("tjr,tjc->jrc", dy[sel].view(-1, N // b, b)[:, :4].double(), y[sel].view(-1, N // b, b)[:, :4].double())
        M = torch.einsum("tjr,tjc->jrc", dy[sel].view(-1, N // b, b)[:, :4].double().abs(),
                         y[sel].view(-1, N // b, b)[:, :4].double().abs())
        for j in range(4):
            R = _down(Rf[k, j])
            gq = 0.5 * (R.T + eye) @ S[j].cpu().numpy() @ (eye + R)
            m = M[j].cpu().numpy()
            e = 0.5 * (abs(R).T + eye) @ (cases.sum_err(len(sel), m) + 4 * cases.U * (b + 64) * m) @ (eye + abs(R))
            assert (np.abs(_down(dq[k, j]) - (gq - gq.T)[i, l]) <= (e + e.T)[i, l]).all(), (k, j)


def test_offsets_beyond_32_bits():
    """Rows whose bytes, and factors whose elements, pass 2^32 and 2^31."""
    import torch

    oft = _oft()
    T, N, b = 66000, 34816, 32
    z = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    tail = torch.randn((70, N), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    z[-70:] = tail
    p, _ = cases.rotations(1, N // b, b)
    Rf = torch.empty((1, N // b, b, b), device="cuda")
    Rops = torch.empty((1, N // b, 2, b, b), dtype=torch.bfloat16, device="cuda")
    oft.cayley_build(_up(p, "bf16"), N // b, b, Rf, Rops)
    ad = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    ad[-70:] = 0
    rows = oft.adapter_rows(T, 1)
    oft.oft_adapter_route(rows, ad)
    oft.oft_rotate_fwd(oft.rotate_desc(T, 1, N, b), rows, z, Rops, z)  # (the others: left as they are)
    few = oft.adapter_rows(70, 1)
    oft.oft_adapter_route(few, torch.zeros(70, dtype=torch.int32, device="cuda"))
    want = torch.empty_like(tail)
    oft.oft_rotate_fwd(oft.rotate_desc(70, 1, N, b), few, tail, Rops, want)
    assert torch.equal(z[-70:], want)
    del z
    n, N, r, K, T = 600, 32768, 128, 64, 20
    B = torch.empty((n, N, r), dtype=torch.bfloat16, device="cuda")
    B[-1] = torch.randn((N, r), generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").bfloat16() / 8
    c = cases.lowrank(T, 1, K, (N,), r, "bf16", "one")
    c["B"][0] = _down(B[-1])
    A = torch.zeros((n, r, K), dtype=torch.bfloat16, device="cuda")
    A[-1] = _up(c["A"][0], "bf16")
    scale = torch.full((n,), float(c["scale"][0]), device="cuda")
    d = oft.lowrank_desc(T, n, K, (N,), r)
    rows = oft.adapter_rows(T, n)
    oft.oft_adapter_route(rows, torch.full((T,), n - 1, dtype=torch.int32, device="cuda"))
    y = _empty((T, N), "bf16")
    ws, nb = _ws(oft.oft_lowrank_workspace_bytes(d, 0))
    oft.oft_lowrank_fwd(d, rows, _up(c["x"], "bf16"), A, B, scale, _up(c["y_base"], "bf16"), y, ws=ws, ws_bytes=nb)
    (want, tol), _ = cases.lowrank_fwd(c, (N,), "bf16")
    _within(y, want, tol, "y")


def test_binding_refuses_wrong_tensors():
    import torch

    oft = _oft()
    b = Batch(8, 2, 64, (32,), 8, 32, "mixed", 7)
    t, o = b.t, b.out
    with pytest.raises(ValueError):
        oft.oft_adapter_route(b.rows, b.adapter[:7])
    with pytest.raises(ValueError):
        oft.oft_adapter_route(b.rows, b.adapter.long())
    with pytest.raises(ValueError):
        oft.AdapterRows(8, 2, b.rows.order, b.rows.offsets[:2], b.rows.tiles, None)
    with pytest.raises(ValueError):
        oft.AdapterRows(8, 2, b.rows.order, b.rows.offsets, b.rows.tiles[:8], None)
    low = dict(x=t["x"], A=t["A"], B=t["B"], scale=t["scale"], y_base=t["y_base"], y=o["y"], ws=b.ws[0][0],
               ws_bytes=b.ws[0][1])
    for kw in (dict(x=t["x"].float()), dict(x=t["x"][:7]), dict(A=t["A"][0]), dict(B=t["B"].transpose(1, 2)),
               dict(scale=t["scale"].double()), dict(y=o["y"].cpu()), dict(y_base=t["y_base"].t()), dict(v=o["v"][:, :4]),
               dict(ws_bytes=b.ws[0][1] + 999)):
        with pytest.raises(ValueError):
            oft.oft_lowrank_fwd(b.ld, b.rows, **{**low, **kw})
    with pytest.raises(ValueError):
        oft.oft_lowrank_fwd(oft.lowrank_desc(8, 3, 64, (32,), 8), b.rows, **low)
    rot = dict(z=t["y_base"], R_ops=b.Rops, y=o["z"])
    for kw in (dict(z=t["y_base"].float()), dict(R_ops=b.Rops[:1]), dict(y=o["z"][:4])):
        with pytest.raises(ValueError):
            oft.oft_rotate_fwd(b.rd, b.rows, **{**rot, **kw})
    with pytest.raises(ValueError):
        oft.oft_rotate_bwd(b.rd, b.rows, t["dy"].float(), o["z"], b.Rf, b.Rops, dz=o["dz"])
    with pytest.raises(oft.OftError):  # dq without a workspace
        oft.oft_rotate_bwd(b.rd, b.rows, t["dy"], o["z"], b.Rf, b.Rops, dq=o["dq"])
    f = torch.ones(100, device="cuda")
    for grads, out in (([f, f], None), ([f], [f[:50]]), ([f[:60], f[60:]], [f[:60], f[40:80]]), ([f[:50], f[50:]], [f[50:], f[:50]]),
                       ([f, f.bfloat16()], None), ([f.view(10, 10).t()], None), ([f.double()], None)):
        with pytest.raises(ValueError):
            oft.grad_list(grads, out)
    oft.grad_list([f, f], [torch.empty_like(f), torch.empty_like(f)])  # read twice, written apart
    b.run()
    torch.cuda.synchronize()


def test_training_step_of_several_adapters_over_one_frozen_layer():
    """A step as an adapter trainer runs it: the frozen INT4 layer once for all
    rows, each row's rotation, a low-rank update beside it; back through both,
    dX through the frozen layer, and all gradients clipped by their norm."""
    import torch

    oft = _oft()
    cfg = DenseConfig("shared", M=90, K=512, segs=(512, 128, 128), b=32, x_dtype="bf16", w_fmt="int4", g=64, q_std=0.1)
    inp = make_dense(cfg, seed=5)
    M, K, N, b, n, r = cfg.M, cfg.K, cfg.N, cfg.b, 3, 16
    lin = oft.linear_desc(M, K, cfg.segs, b, oft.OFT_DT_BF16, oft.OFT_W_INT4, cfg.g)
    x, wc, wsc = (dev(inp[k]) for k in ("x", "w_codes", "w_scales"))
    c = cases.lowrank(M, n, K, cfg.segs, r, "bf16", "some", 8)
    p, _ = cases.rotations(n, N // b, b, 8, size=0.1)
    Rf = torch.empty((n, N // b, b, b), device="cuda")
    Rops = torch.empty((n, N // b, 2, b, b), dtype=torch.int16, device="cuda")
    oft.cayley_build(_up(p, "bf16"), n * (N // b), b, Rf, Rops)
    rows = _rows(c["adapter"], n)
    rd, ld = oft.rotate_desc(M, n, N, b), oft.lowrank_desc(M, n, K, cfg.segs, r)
    i16 = lambda *s: torch.empty(s, dtype=torch.int16, device="cuda")  # noqa: E731
    z, y, out, v = i16(M, N), i16(M, N), i16(M, N), _empty((M, 3 * r))
    A, B, scale, dy = _up(c["A"], "bf16"), _up(c["B"], "bf16"), _up(c["scale"]), _up(c["dy"], "bf16")
    oft.oft_linear_fwd_base(lin, x, wc, wsc, z)
    oft.oft_rotate_fwd(rd, rows, z, Rops, y)
    ws, nb = _ws(oft.oft_lowrank_workspace_bytes(ld, 0))
    oft.oft_lowrank_fwd(ld, rows, x, A, B, scale, y, out, v=v, ws=ws, ws_bytes=nb)
    # back: rotation, the frozen layer (R = I), the low-rank update onto its dX
    dz, dq, dx = i16(M, N), _empty((n, N // b, 496)), i16(M, K)
    ws, nb = _ws(oft.oft_rotate_workspace_bytes(rd, 1))
    oft.oft_rotate_bwd(rd, rows, dy, y, Rf, Rops, dz=dz, dq=dq, ws=ws, ws_bytes=nb)
    one_f, one_o = torch.empty((N // b, b, b), device="cuda"), i16(N // b, 2, b, b)
    oft.cayley_build(torch.zeros((N // b, 496), dtype=torch.int16, device="cuda"), N // b, b, one_f, one_o)
    nb = oft.oft_linear_workspace_bytes(lin, oft.OFT_PASS_BWD)
    oft.oft_linear_bwd(lin, dz, z, wc, wsc, one_f, one_o, dx, None, torch.empty(max(nb, 16), dtype=torch.uint8, device="cuda"), nb)
    dA, dB = _empty((n, 3 * r, K)), _empty((n, N, r))
    ws, nb = _ws(oft.oft_lowrank_workspace_bytes(ld, 1))
    oft.oft_lowrank_bwd(ld, rows, dy, x, v, A, B, scale, dx=dx, dx_base=dx, dA=dA, dB=dB, ws=ws, ws_bytes=nb)
    raw = [t.clone() for t in (dq, dA, dB)]
    lst = oft.grad_list([dq, dA, dB])
    ws, nb = _ws(oft.oft_grad_workspace_bytes(lst))
    sumsq, stats = torch.zeros(1, dtype=torch.float64, device="cuda"), _empty((2,))
    oft.oft_grad_sumsq(lst, sumsq, ws=ws, ws_bytes=nb)
    oft.oft_grad_clip(lst, sumsq, 1.0, stats)
    torch.cuda.synchronize()
    # the whole step in 64 bits, by the layer's own parity bound
    W, x64 = odense.dequant(inp), odense.x_f64(inp)
    R = _down(Rf)
    z64 = x64 @ W.T
    y64 = oracle.rotate_fwd(z64, R, c["adapter"])
    f64 = {k: np.asarray(c[k], dtype=np.float64) for k in ("A", "B", "scale", "dy")}
    out64, v64 = oracle.lowrank_fwd(x64, f64["A"], f64["B"], f64["scale"], y64, c["adapter"], cfg.segs)
    dz64, dq64 = oracle.rotate_bwd(f64["dy"], y64, R, R, c["adapter"])
    dx64, dA64, dB64 = oracle.lowrank_bwd(f64["dy"], x64, v64, f64["A"], f64["B"], f64["scale"], dz64 @ W, c["adapter"],
                                          cfg.segs)
    bf = lambda t: t.view(torch.bfloat16).float().cpu().numpy()  # noqa: E731
    e = {"out": err(bf(out), out64), "dx": err(bf(dx), dx64), "dq": err(host(raw[0]), dq64), "dA": err(host(raw[1]), dA64),
         "dB": err(host(raw[2]), dB64)}
    print(f"[training step] {e}", flush=True)
    assert all(k <= 2e-2 for k in e.values()), e
    norm, coef, want = oracle.clip([_down(t) for t in raw], 1.0)
    got = _down(stats)
    assert abs(got[0] - norm) <= 2 * cases.U * norm and abs(got[1] - coef) <= 8 * cases.U * coef
    for t, w in zip((dq, dA, dB), want):
        assert (np.abs(_down(t) - w) <= 12 * cases.U * np.abs(w)).all()
    # a row's adapter alone, as the layer with that adapter computes it
    for a in range(n):
        alone = i16(M, N)
        oft.oft_linear_fwd(lin, x, wc, wsc, Rops[a].contiguous(), alone)
        sel = np.flatnonzero(c["adapter"] == a)
        assert err(bf(y)[sel], bf(alone)[sel]) <= 2e-2
