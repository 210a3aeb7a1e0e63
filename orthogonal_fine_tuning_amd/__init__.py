"""OFT dequant-GEMM for AMD Instinct MI355X (gfx950): Python binding.

Every function here marshals torch tensors (device memory) into the C ABI of
liboft.so (include/oft.h) and calls it on the current torch stream.  All
arithmetic runs in the library's HIP kernels; there is no fallback path.
"""
from __future__ import annotations

import ctypes as C

from . import _lib
from ._lib import (OFT_DT_BF16, OFT_DT_F32, OFT_PASS_BWD, OFT_PASS_FWD, OFT_W_BF16,
                   OFT_W_FP4_E2M1, OFT_W_FP8_E4M3, OFT_W_INT4, OFT_W_INT4_TILED, OFT_MAX_TEACHER, OFT_MAX_TOP,
                   OFT_MAX_ADAPTERS, OFT_MAX_GRADS, OFT_MAX_RANK, OFT_NO_LABEL, OftError, oft_adapter_rows,
                   oft_linear_desc, oft_lowrank_desc, oft_moe_desc, oft_moe_routing, oft_rotate_desc, oft_vocab_desc)

__all__ = [
    "OftError", "linear_desc", "moe_desc", "moe_routing", "cayley_build", "oft_dequant", "oft_pack_int4_tiled",
    "oft_linear_workspace_bytes", "oft_linear_fwd", "oft_linear_fwd_base", "oft_linear_bwd", "oft_linear_bwd_noalloc", "oft_logprob_diff",
    "oft_slots_switch", "oft_linear_fwd_slots",
    "oft_moe_workspace_bytes", "oft_moe_route", "oft_moe_router_bwd", "oft_moe_grouped_fwd", "oft_moe_grouped_fwd_base", "oft_moe_grouped_bwd", "abi_version",
    "vocab_desc", "oft_vocab_workspace_bytes", "oft_token_logprobs", "oft_token_logprobs_bwd", "oft_distill_topk",
    "oft_distill_topk_bwd", "oft_moe_balance_workspace_bytes", "oft_moe_balance", "oft_moe_balance_bwd",
    "AdapterRows", "adapter_rows", "oft_adapter_rows_bytes", "oft_adapter_route", "lowrank_desc",
    "oft_lowrank_workspace_bytes", "oft_lowrank_fwd", "oft_lowrank_bwd", "rotate_desc", "oft_rotate_workspace_bytes",
    "oft_rotate_fwd", "oft_rotate_bwd", "GradList", "grad_list", "oft_grad_workspace_bytes", "oft_grad_sumsq",
    "oft_grad_clip",
    "prof_enable", "prof_records",
    "OFT_DT_BF16", "OFT_DT_F32", "OFT_W_INT4", "OFT_W_FP8_E4M3", "OFT_W_BF16", "OFT_W_FP4_E2M1", "OFT_W_INT4_TILED",
    "OFT_PASS_FWD",
    "OFT_PASS_BWD", "OFT_MAX_TOP", "OFT_MAX_TEACHER", "OFT_NO_LABEL", "OFT_MAX_ADAPTERS", "OFT_MAX_RANK",
    "OFT_MAX_GRADS",
]


def _ptr(t):
    if t is None:
        return None
    return C.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is not None:
        return C.c_void_p(int(stream))
    import torch

    return C.c_void_p(torch.cuda.current_stream().cuda_stream)


def abi_version() -> int:
    return _lib.load().oft_abi_version()


def prof_enable(on: bool) -> None:
    """Start (clearing the list) or stop the library's per-step kernel timing."""
    _lib.check(_lib.load().oft_prof_enable(1 if on else 0), "oft_prof_enable")


def prof_records():
    """[(name, milliseconds)] of the recorded steps, in launch order (waits
    for each record's events)."""
    lib = _lib.load()
    out = []
    buf = C.create_string_buffer(64)
    ms = C.c_float(0.0)
    for i in range(lib.oft_prof_count()):
        _lib.check(lib.oft_prof_read(i, buf, 64, C.byref(ms)), "oft_prof_read")
        out.append((buf.value.decode(), float(ms.value)))
    return out


def linear_desc(M, K, segs, b, x_dtype=OFT_DT_BF16, w_fmt=OFT_W_INT4, g=0) -> oft_linear_desc:
    d = oft_linear_desc()
    d.M, d.K, d.N = int(M), int(K), int(sum(segs))
    d.x_dtype, d.w_fmt, d.g, d.b = int(x_dtype), int(w_fmt), int(g), int(b)
    d.n_seg = len(segs)
    for i, s in enumerate(segs):
        d.seg[i] = int(s)
    return d


def moe_desc(T, E, k, H, I, g, b, chunk, renorm=0, w_fmt=OFT_W_INT4) -> oft_moe_desc:
    d = oft_moe_desc()
    d.T, d.E, d.k, d.H, d.I, d.g, d.b, d.chunk, d.renorm, d.w_fmt = (
        int(v) for v in (T, E, k, H, I, g, b, chunk, renorm, w_fmt))
    return d


def moe_routing(topk_idx, topk_w, counts, offsets, perm, inv_perm, active, n_active,
                chunk_of_expert) -> oft_moe_routing:
    rt = oft_moe_routing()
    for name, t in (("topk_idx", topk_idx), ("topk_w", topk_w), ("counts", counts),
                    ("offsets", offsets), ("perm", perm), ("inv_perm", inv_perm),
                    ("active", active), ("n_active", n_active),
                    ("chunk_of_expert", chunk_of_expert)):
        setattr(rt, name, t.data_ptr())
    return rt


def cayley_build(q, nblk, b, R_f32, R_ops=None, stream=None):
    _lib.check(_lib.load().cayley_build(_ptr(q), nblk, b, _ptr(R_f32), _ptr(R_ops),
                                        _stream(stream)), "cayley_build")


def oft_dequant(w_fmt, rows, cols, g, codes, scales, out, stream=None):
    _lib.check(_lib.load().oft_dequant(w_fmt, rows, cols, g, _ptr(codes), _ptr(scales), _ptr(out),
                                       _stream(stream)), "oft_dequant")


def oft_pack_int4_tiled(count, rows, cols, g, codes, scales, codes_tiled, scales_tiled, stream=None):
    _lib.check(_lib.load().oft_pack_int4_tiled(count, rows, cols, g, _ptr(codes), _ptr(scales), _ptr(codes_tiled),
                                               _ptr(scales_tiled), _stream(stream)), "oft_pack_int4_tiled")


def oft_linear_workspace_bytes(desc, pass_) -> int:
    n = C.c_size_t(0)
    _lib.check(_lib.load().oft_linear_workspace_bytes(C.byref(desc), pass_, C.byref(n)),
               "oft_linear_workspace_bytes")
    return n.value


def oft_linear_fwd(desc, x, w_codes, w_scales, R_ops, y, ws=None, ws_bytes=0, stream=None):
    _lib.check(_lib.load().oft_linear_fwd(C.byref(desc), _ptr(x), _ptr(w_codes), _ptr(w_scales),
                                          _ptr(R_ops), _ptr(y), _ptr(ws), ws_bytes,
                                          _stream(stream)), "oft_linear_fwd")


def oft_linear_fwd_base(desc, x, w_codes, w_scales, y, ws=None, ws_bytes=0, stream=None):
    _lib.check(_lib.load().oft_linear_fwd_base(C.byref(desc), _ptr(x), _ptr(w_codes), _ptr(w_scales),
                                               _ptr(y), _ptr(ws), ws_bytes, _stream(stream)),
               "oft_linear_fwd_base")


def oft_slots_switch(state, slot, version, stream=None):
    _lib.check(_lib.load().oft_slots_switch(_ptr(state), int(slot), int(version), _stream(stream)),
               "oft_slots_switch")


def oft_linear_fwd_slots(desc, x, w_codes, w_scales, R_ops0, R_ops1, state, latch, y, ws=None, ws_bytes=0,
                         stream=None):
    _lib.check(_lib.load().oft_linear_fwd_slots(C.byref(desc), _ptr(x), _ptr(w_codes), _ptr(w_scales),
                                                _ptr(R_ops0), _ptr(R_ops1), _ptr(state), _ptr(latch), _ptr(y),
                                                _ptr(ws), ws_bytes, _stream(stream)),
               "oft_linear_fwd_slots")


def oft_linear_bwd(desc, dy, y_saved, w_codes, w_scales, R_f32, R_ops, dx=None, dq=None, ws=None,
                   ws_bytes=0, stream=None):
    _lib.check(_lib.load().oft_linear_bwd(C.byref(desc), _ptr(dy), _ptr(y_saved), _ptr(w_codes),
                                          _ptr(w_scales), _ptr(R_f32), _ptr(R_ops), _ptr(dx),
                                          _ptr(dq), _ptr(ws), ws_bytes, _stream(stream)),
               "oft_linear_bwd")


def oft_linear_bwd_noalloc(desc, dy, y_saved, w_codes, w_scales, R_f32, R_ops, dx=None, dq=None, stream=None):
    _lib.check(_lib.load().oft_linear_bwd_noalloc(C.byref(desc), _ptr(dy), _ptr(y_saved), _ptr(w_codes),
                                                  _ptr(w_scales), _ptr(R_f32), _ptr(R_ops), _ptr(dx), _ptr(dq),
                                                  _stream(stream)),
               "oft_linear_bwd_noalloc")


def oft_logprob_diff(logits_actor, logits_ref, labels, out, stream=None):
    T, V = logits_actor.shape
    _lib.check(_lib.load().oft_logprob_diff(int(T), int(V), _ptr(logits_actor), _ptr(logits_ref), _ptr(labels),
                                            _ptr(out), _stream(stream)), "oft_logprob_diff")


# ---- losses on vocabulary logits and the router's balance loss -------------
# These calls check their tensors against the descriptor (device, type, shape,
# strides) and launch on the logits' device, on its current stream unless one
# is given.
def vocab_desc(T, V, dtype=OFT_DT_BF16, k=0, ld=None, ld_grad=None, temperature=1.0, accumulate=0) -> oft_vocab_desc:
    """ld, ld_grad: elements from one row of logits / d_logits to the next
    (ld defaults to V, ld_grad to ld)."""
    d = oft_vocab_desc()
    ld = V if ld is None else ld
    d.T, d.V, d.dtype, d.k = int(T), int(V), int(dtype), int(k)
    d.ld, d.ld_grad = int(ld), int(ld if ld_grad is None else ld_grad)
    d.temperature, d.accumulate = float(temperature), int(accumulate)
    return d


_TYPES = {}


def _types(names):
    """The torch types of a kind of tensor ("int32", "bfloat16 int16 uint16"), looked up once."""
    if names not in _TYPES:
        import torch

        _TYPES[names] = tuple(getattr(torch, n) for n in names.split())
    return _TYPES[names]


def _tensor(what, t, names, shape, dev, ld=None):
    """The address of t: a tensor on GPU `dev` of one of the named types and
    the given shape, contiguous or with rows `ld` apart."""
    if t.get_device() != dev or dev < 0:
        raise ValueError(f"{what}: on {t.device}, want the logits' GPU")
    if t.dtype not in _types(names):
        raise ValueError(f"{what}: {t.dtype}, want one of {names}")
    if t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(t.shape)}, want {shape}")
    if ld is None:
        if not t.is_contiguous():
            raise ValueError(f"{what}: not contiguous")
    elif (shape[1] > 1 and t.stride(1) != 1) or (shape[0] > 1 and t.stride(0) != ld):
        raise ValueError(f"{what}: strides {t.stride()}, want ({ld}, 1)")
    return t.data_ptr()


def _maybe(what, t, names, shape, dev):
    return None if t is None else _tensor(what, t, names, shape, dev)


def _rows(what, t, d, ld, dev):
    return _tensor(what, t, "float32" if d.dtype == OFT_DT_F32 else "bfloat16 int16 uint16", (d.T, d.V), dev, ld)


def _workspace(ws, ws_bytes, dev):
    if ws is None:
        return None
    if ws.get_device() != dev or not ws.is_contiguous() or ws.numel() * ws.element_size() < ws_bytes:
        raise ValueError("ws: want a contiguous tensor of at least ws_bytes on the logits' GPU")
    return ws.data_ptr()


_ASK = []


def _asked():
    """(the current stream of a GPU, the current GPU): below torch.cuda's objects
    where torch has that (0.2 us; 1.3 through them, of the 7.3 us that a call of
    one short kernel takes), else through them."""
    if not _ASK:
        import torch

        _ASK[:] = (getattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: torch.cuda.current_stream(dev).cuda_stream),
                   getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device))
    return _ASK


def _launch(name, dev, stream, *args):
    """Call `name` with the logits' GPU current, on its current stream unless one is given."""
    f = getattr(_lib.load(), name)
    current_stream, current_device = _asked()
    if stream is None:
        stream = current_stream(dev)
    if current_device() == dev:
        status = f(*args, int(stream))
    else:
        import torch

        with torch.cuda.device(dev):
            status = f(*args, int(stream))
    _lib.check(status, name)


def oft_vocab_workspace_bytes(desc) -> int:
    n = C.c_size_t(0)
    _lib.check(_lib.load().oft_vocab_workspace_bytes(C.byref(desc), C.byref(n)), "oft_vocab_workspace_bytes")
    return n.value


def oft_token_logprobs(desc, logits, labels, logp, stats, entropy=None, top_idx=None, top_logp=None, ws=None,
                       ws_bytes=0, stream=None):
    """Log-probabilities of the given tokens, entropy and top alternatives of
    each row of logits; labels and logp may both be None."""
    d, dev, row = desc, logits.get_device(), (desc.T,)
    x = _rows("logits", logits, d, d.ld, dev)
    lab = _maybe("labels", labels, "int32", row, dev)
    lp = _maybe("logp", logp, "float32", row, dev)
    ent = _maybe("entropy", entropy, "float32", row, dev)
    st = _tensor("stats", stats, "float32", (d.T, 2), dev)
    ti = tl = None
    if d.k > 0:
        ti = _maybe("top_idx", top_idx, "int32", (d.T, d.k), dev)
        tl = _maybe("top_logp", top_logp, "float32", (d.T, d.k), dev)
    _launch("oft_token_logprobs", dev, stream, C.byref(d), x, lab, lp, ent, ti, tl, st, _workspace(ws, ws_bytes, dev),
            ws_bytes)


def oft_token_logprobs_bwd(desc, logits, labels, stats, g_logp, d_logits, entropy=None, g_entropy=None, stream=None):
    """d_logits of g_logp . logp + g_entropy . entropy; labels and g_logp may
    both be None, and g_entropy may be None."""
    d, dev, row = desc, logits.get_device(), (desc.T,)
    x = _rows("logits", logits, d, d.ld, dev)
    dx = _rows("d_logits", d_logits, d, d.ld_grad, dev)
    lab = _maybe("labels", labels, "int32", row, dev)
    st = _tensor("stats", stats, "float32", (d.T, 2), dev)
    gl = _maybe("g_logp", g_logp, "float32", row, dev)
    ent = _maybe("entropy", entropy, "float32", row, dev)
    ge = _maybe("g_entropy", g_entropy, "float32", row, dev)
    _launch("oft_token_logprobs_bwd", dev, stream, C.byref(d), x, lab, st, ent, gl, ge, dx)


def oft_distill_topk(desc, logits, teacher_idx, teacher_logits, loss, stats, ws=None, ws_bytes=0, stream=None):
    """Per-row loss against the teacher's renormalised top list.  The list is
    divided by desc.temperature here: logits, or log-probabilities at
    temperature 1 (top_logp of another temperature times that temperature)."""
    d, dev, listed = desc, logits.get_device(), (desc.T, desc.k)
    x = _rows("logits", logits, d, d.ld, dev)
    ti = _tensor("teacher_idx", teacher_idx, "int32", listed, dev)
    tl = _tensor("teacher_logits", teacher_logits, "float32", listed, dev)
    out = _tensor("loss", loss, "float32", (d.T,), dev)
    st = _tensor("stats", stats, "float32", (d.T, 2), dev)
    _launch("oft_distill_topk", dev, stream, C.byref(d), x, ti, tl, out, st, _workspace(ws, ws_bytes, dev), ws_bytes)


def oft_distill_topk_bwd(desc, logits, teacher_idx, teacher_logits, stats, g_loss, d_logits, stream=None):
    """d_logits of g_loss . loss."""
    d, dev, listed = desc, logits.get_device(), (desc.T, desc.k)
    x = _rows("logits", logits, d, d.ld, dev)
    dx = _rows("d_logits", d_logits, d, d.ld_grad, dev)
    ti = _tensor("teacher_idx", teacher_idx, "int32", listed, dev)
    tl = _tensor("teacher_logits", teacher_logits, "float32", listed, dev)
    st = _tensor("stats", stats, "float32", (d.T, 2), dev)
    g = _tensor("g_loss", g_loss, "float32", (d.T,), dev)
    _launch("oft_distill_topk_bwd", dev, stream, C.byref(d), x, ti, tl, st, g, dx)


def oft_moe_balance_workspace_bytes(desc, seq_len) -> int:
    n = C.c_size_t(0)
    _lib.check(_lib.load().oft_moe_balance_workspace_bytes(C.byref(desc), int(seq_len), C.byref(n)),
               "oft_moe_balance_workspace_bytes")
    return n.value


def _sequences(desc, seq_len):
    if seq_len < 1 or desc.T % seq_len:
        raise ValueError(f"seq_len {seq_len}: want a divisor of the {desc.T} tokens")
    return desc.T // seq_len


def oft_moe_balance(desc, seq_len, logits, topk_idx, counts, tokens, loss, mean_prob=None, mask=None, ws=None,
                    ws_bytes=0, stream=None):
    """Balance loss, per-expert counts and mean probabilities of each
    sequence of seq_len tokens; mask: uint8 or bool, false for padding."""
    d, dev, S = desc, logits.get_device(), _sequences(desc, seq_len)
    x = _tensor("logits", logits, "float32", (d.T, d.E), dev)
    ti = _tensor("topk_idx", topk_idx, "int32", (d.T, d.k), dev)
    mk = _maybe("mask", mask, "uint8 bool", (d.T,), dev)
    cn = _tensor("counts", counts, "int32", (S, d.E), dev)
    tk = _tensor("tokens", tokens, "int32", (S,), dev)
    out = _tensor("loss", loss, "float32", (S,), dev)
    mp = _maybe("mean_prob", mean_prob, "float32", (S, d.E), dev)
    _launch("oft_moe_balance", dev, stream, C.byref(d), int(seq_len), x, ti, mk, cn, tk, out, mp,
            _workspace(ws, ws_bytes, dev), ws_bytes)


def oft_moe_balance_bwd(desc, seq_len, logits, counts, tokens, g_loss, d_logits, mask=None, accumulate=0,
                        stream=None):
    """d_logits of g_loss . loss, written or (accumulate=1) added."""
    d, dev, S = desc, logits.get_device(), _sequences(desc, seq_len)
    x = _tensor("logits", logits, "float32", (d.T, d.E), dev)
    mk = _maybe("mask", mask, "uint8 bool", (d.T,), dev)
    cn = _tensor("counts", counts, "int32", (S, d.E), dev)
    tk = _tensor("tokens", tokens, "int32", (S,), dev)
    g = _tensor("g_loss", g_loss, "float32", (S,), dev)
    dx = _tensor("d_logits", d_logits, "float32", (d.T, d.E), dev)
    _launch("oft_moe_balance_bwd", dev, stream, C.byref(d), int(seq_len), x, mk, cn, tk, g, dx, int(accumulate))


# ---- adapters of many requests ---------------------------------------------
# These calls check their tensors as those above do, against the descriptor
# and on the GPU of the rows' order.
class AdapterRows:
    """A batch's rows sorted by adapter: order int32 [T], offsets int32 [n + 1]
    and the work lists of the calls that run over them, with the workspace of
    oft_adapter_route.  Calls that overlap on different streams may share one
    that none of them writes."""

    def __init__(self, T, n, order, offsets, tiles, ws):
        self.T, self.n, self.order, self.offsets, self.tiles, self.ws = int(T), int(n), order, offsets, tiles, ws
        dev = self.dev = offsets.get_device()
        tiles_bytes, ws_bytes = oft_adapter_rows_bytes(T, n)
        self.c = oft_adapter_rows()
        self.c.T, self.c.n = self.T, self.n
        self.c.order = _tensor("order", order, "int32", (self.T,), dev) or None
        self.c.offsets = _tensor("offsets", offsets, "int32", (self.n + 1,), dev)
        self.c.tiles = _buffer("tiles", tiles, tiles_bytes, dev)
        self.ws_bytes = ws_bytes
        self._ws = _buffer("ws", ws, ws_bytes, dev) if ws_bytes else None


def _buffer(what, t, nbytes, dev):
    if t.get_device() != dev or not t.is_contiguous() or t.numel() * t.element_size() < nbytes:
        raise ValueError(f"{what}: want a contiguous tensor of at least {nbytes} bytes on the rows' GPU")
    return t.data_ptr()


def oft_adapter_rows_bytes(T, n):
    """(bytes of the work lists, bytes of oft_adapter_route's workspace)."""
    a, b = C.c_size_t(0), C.c_size_t(0)
    _lib.check(_lib.load().oft_adapter_rows_bytes(int(T), int(n), C.byref(a), C.byref(b)), "oft_adapter_rows_bytes")
    return a.value, b.value


def adapter_rows(T, n, device="cuda") -> AdapterRows:
    """AdapterRows with tensors of its own on `device`, for oft_adapter_route to fill."""
    import torch

    tiles, ws = oft_adapter_rows_bytes(T, n)
    new = lambda k: torch.empty(k, dtype=torch.int32, device=device)  # noqa: E731
    return AdapterRows(T, n, new(T), new(n + 1), new(tiles // 4), new((ws + 3) // 4))


def oft_adapter_route(rows, adapter, stream=None):
    """Sort the batch's rows by adapter int32 [T] (outside 0 .. n - 1: none)."""
    a = _tensor("adapter", adapter, "int32", (rows.T,), rows.dev)
    _launch("oft_adapter_route", rows.dev, stream, a or None, C.byref(rows.c), rows._ws, rows.ws_bytes)


def lowrank_desc(T, n, K, segs, r, dtype=OFT_DT_BF16) -> oft_lowrank_desc:
    d = oft_lowrank_desc()
    d.T, d.n, d.K, d.N, d.r, d.dtype = int(T), int(n), int(K), int(sum(segs)), int(r), int(dtype)
    d.n_seg = len(segs)
    for i, s in enumerate(segs[:len(d.seg)]):
        d.seg[i] = int(s)
    return d


def oft_lowrank_workspace_bytes(desc, pass_) -> int:
    n = C.c_size_t(0)
    _lib.check(_lib.load().oft_lowrank_workspace_bytes(C.byref(desc), pass_, C.byref(n)),
               "oft_lowrank_workspace_bytes")
    return n.value


_BF16 = "bfloat16 int16 uint16"


def _row_type(desc):
    return "float32" if desc.dtype == OFT_DT_F32 else _BF16


def _same_batch(desc, rows):
    if desc.T != rows.T or desc.n != rows.n:
        raise ValueError(f"rows: of {rows.T} rows and {rows.n} adapters, want {desc.T} and {desc.n}")


def oft_lowrank_fwd(desc, rows, x, A, B, scale, y_base, y, v=None, ws=None, ws_bytes=0, stream=None):
    """y = y_base + scale v B^T, v = x A^T, with each row's own factors; y may be y_base."""
    d, dev, t = desc, rows.dev, _row_type(desc)
    _same_batch(d, rows)
    R = d.n_seg * d.r
    _launch("oft_lowrank_fwd", dev, stream, C.byref(d), C.byref(rows.c), _tensor("x", x, t, (d.T, d.K), dev),
            _tensor("A", A, _BF16, (d.n, R, d.K), dev), _tensor("B", B, _BF16, (d.n, d.N, d.r), dev),
            _tensor("scale", scale, "float32", (d.n,), dev), _tensor("y_base", y_base, t, (d.T, d.N), dev),
            _tensor("y", y, t, (d.T, d.N), dev), _maybe("v", v, "float32", (d.T, R), dev),
            _workspace(ws, ws_bytes, dev), ws_bytes)


def oft_lowrank_bwd(desc, rows, dy, x, v, A, B, scale, dx=None, dx_base=None, dA=None, dB=None, ws=None, ws_bytes=0,
                    stream=None):
    """dx (added to dx_base, which may be dx), dA and dB of <dy, y>."""
    d, dev, t = desc, rows.dev, _row_type(desc)
    _same_batch(d, rows)
    R = d.n_seg * d.r
    _launch("oft_lowrank_bwd", dev, stream, C.byref(d), C.byref(rows.c),
            _tensor("dy", dy, _BF16, (d.T, d.N), dev), _maybe("x", x, t, (d.T, d.K), dev),
            _maybe("v", v, "float32", (d.T, R), dev), _maybe("A", A, _BF16, (d.n, R, d.K), dev),
            _maybe("B", B, _BF16, (d.n, d.N, d.r), dev), _tensor("scale", scale, "float32", (d.n,), dev),
            _maybe("dx_base", dx_base, t, (d.T, d.K), dev), _maybe("dx", dx, t, (d.T, d.K), dev),
            _maybe("dA", dA, "float32", (d.n, R, d.K), dev), _maybe("dB", dB, "float32", (d.n, d.N, d.r), dev),
            _workspace(ws, ws_bytes, dev), ws_bytes)


def rotate_desc(T, n, N, b, dtype=OFT_DT_BF16) -> oft_rotate_desc:
    d = oft_rotate_desc()
    d.T, d.n, d.N, d.b, d.dtype = int(T), int(n), int(N), int(b), int(dtype)
    return d


def oft_rotate_workspace_bytes(desc, pass_) -> int:
    n = C.c_size_t(0)
    _lib.check(_lib.load().oft_rotate_workspace_bytes(C.byref(desc), pass_, C.byref(n)), "oft_rotate_workspace_bytes")
    return n.value


def _blocks(desc):
    return desc.N // desc.b if desc.b > 0 else 0  # (the library refuses other blocks)


def oft_rotate_fwd(desc, rows, z, R_ops, y, stream=None):
    """y = R z in every block of channels, with each row's own R; y may be z."""
    d, dev, t = desc, rows.dev, _row_type(desc)
    _same_batch(d, rows)
    _launch("oft_rotate_fwd", dev, stream, C.byref(d), C.byref(rows.c), _tensor("z", z, t, (d.T, d.N), dev),
            _tensor("R_ops", R_ops, _BF16, (d.n, _blocks(d), 2, d.b, d.b), dev), _tensor("y", y, t, (d.T, d.N), dev))


def oft_rotate_bwd(desc, rows, dy, y_saved, R_f32, R_ops, dz=None, dq=None, ws=None, ws_bytes=0, stream=None):
    """dz (may be dy) and dq of <dy, y>."""
    d, dev = desc, rows.dev
    _same_batch(d, rows)
    nblk = _blocks(d)
    _launch("oft_rotate_bwd", dev, stream, C.byref(d), C.byref(rows.c), _tensor("dy", dy, _BF16, (d.T, d.N), dev),
            _maybe("y_saved", y_saved, _row_type(d), (d.T, d.N), dev),
            _maybe("R_f32", R_f32, "float32", (d.n, nblk, d.b, d.b), dev),
            _maybe("R_ops", R_ops, _BF16, (d.n, nblk, 2, d.b, d.b), dev), _maybe("dz", dz, _BF16, (d.T, d.N), dev),
            _maybe("dq", dq, "float32", (d.n, nblk, d.b * (d.b - 1) // 2), dev), _workspace(ws, ws_bytes, dev), ws_bytes)


# ---- global gradient norm and clipping --------------------------------------
class GradList:
    """Gradients and where their clipped values go, checked once: a program
    whose gradients keep their addresses makes one and uses it every step.  The
    list means the memory that they have when it is made, and keeps it: after
    t.data = other or t.set_(other) make another list; no tensor of a list may
    be resized."""

    def __init__(self, grads, out=None):
        import torch

        self.grads = list(grads)
        self.out = self.grads if out is None else list(out)
        # (a tensor that is given other memory does not free what the list names)
        self._memory = [t.untyped_storage() for t in self.grads + self.out]
        self.m = len(self.grads)
        if len(self.out) != self.m or self.m == 0:
            raise ValueError(f"grad_list: {self.m} gradients, {len(self.out)} outputs: want as many, and one at least")
        first = self.grads[0]
        self.dev = first.get_device()
        self.dtype = OFT_DT_F32 if first.dtype == torch.float32 else OFT_DT_BF16
        kind = "float32" if self.dtype == OFT_DT_F32 else "bfloat16"
        for g, o in zip(self.grads, self.out):
            _tensor("grads", g, kind, g.shape, self.dev)
            _tensor("out", o, kind, g.shape, self.dev)
        at = lambda t: (t.data_ptr(), t.data_ptr() + t.numel() * t.element_size())  # noqa: E731
        written = sorted(at(o) for o in self.out if o.numel())
        for a, b in zip(written, written[1:]):
            if b[0] < a[1]:
                raise ValueError("grad_list: two outputs overlap")
        apart = sorted([(at(g), 0) for g, o in zip(self.grads, self.out) if g.numel() and g.data_ptr() != o.data_ptr()] +
                       [(w, 1) for w in written])
        end = [0, 0]
        for (lo, hi), kind_ in apart:
            if lo < end[1 - kind_]:
                raise ValueError("grad_list: an output overlaps a gradient that is not its own")
            end[kind_] = max(end[kind_], hi)
        self._grads = (C.c_void_p * self.m)(*[t.data_ptr() for t in self.grads])
        self._out = (C.c_void_p * self.m)(*[t.data_ptr() for t in self.out])
        self._numel = (C.c_int64 * self.m)(*[t.numel() for t in self.grads])


def grad_list(grads, out=None) -> GradList:
    """out: where the clipped gradients go (the gradients themselves if None)."""
    return GradList(grads, out)


def oft_grad_workspace_bytes(grads) -> int:
    n = C.c_size_t(0)
    _lib.check(_lib.load().oft_grad_workspace_bytes(grads.m, grads._numel, grads.dtype, C.byref(n)),
               "oft_grad_workspace_bytes")
    return n.value


def oft_grad_sumsq(grads, sumsq, ws=None, ws_bytes=0, stream=None):
    """sumsq fp64 [1]: the sum of the squares of all gradients of a GradList."""
    _launch("oft_grad_sumsq", grads.dev, stream, grads.m, grads._grads, grads._numel, grads.dtype,
            _tensor("sumsq", sumsq, "float64", (1,), grads.dev), _workspace(ws, ws_bytes, grads.dev), ws_bytes)


def oft_grad_clip(grads, sumsq, max_norm, stats, stream=None):
    """Scale the gradients so that their norm is at most max_norm; stats fp32
    [2]: the norm before, and the coefficient."""
    _launch("oft_grad_clip", grads.dev, stream, grads.m, grads._grads, grads._numel, grads.dtype,
            _tensor("sumsq", sumsq, "float64", (1,), grads.dev), float(max_norm), grads._out,
            _tensor("stats", stats, "float32", (2,), grads.dev))


def oft_moe_workspace_bytes(desc, pass_) -> int:
    n = C.c_size_t(0)
    _lib.check(_lib.load().oft_moe_workspace_bytes(C.byref(desc), pass_, C.byref(n)),
               "oft_moe_workspace_bytes")
    return n.value


def oft_moe_route(desc, logits, rt, ws, ws_bytes, stream=None):
    _lib.check(_lib.load().oft_moe_route(C.byref(desc), _ptr(logits), C.byref(rt), _ptr(ws),
                                         ws_bytes, _stream(stream)), "oft_moe_route")


def oft_moe_router_bwd(desc, logits, topk_idx, dw, d_logits, stream=None):
    _lib.check(_lib.load().oft_moe_router_bwd(C.byref(desc), _ptr(logits), _ptr(topk_idx), _ptr(dw),
                                              _ptr(d_logits), _stream(stream)), "oft_moe_router_bwd")


def oft_moe_grouped_fwd(desc, x, logits, wgu_codes, wgu_scales, wd_codes, wd_scales, R_ops, rt,
                        h_saved, y, ws, ws_bytes, stream=None):
    _lib.check(_lib.load().oft_moe_grouped_fwd(
        C.byref(desc), _ptr(x), _ptr(logits), _ptr(wgu_codes), _ptr(wgu_scales), _ptr(wd_codes),
        _ptr(wd_scales), _ptr(R_ops), C.byref(rt), _ptr(h_saved), _ptr(y), _ptr(ws), ws_bytes,
        _stream(stream)), "oft_moe_grouped_fwd")


def oft_moe_grouped_fwd_base(desc, x, logits, wgu_codes, wgu_scales, wd_codes, wd_scales, rt, h=None, y=None,
                             ws=None, ws_bytes=0, stream=None):
    _lib.check(_lib.load().oft_moe_grouped_fwd_base(
        C.byref(desc), _ptr(x), _ptr(logits), _ptr(wgu_codes), _ptr(wgu_scales), _ptr(wd_codes), _ptr(wd_scales),
        C.byref(rt), _ptr(h), _ptr(y), _ptr(ws), ws_bytes, _stream(stream)), "oft_moe_grouped_fwd_base")


def oft_moe_grouped_bwd(desc, dy, rt, h_saved, wgu_codes, wgu_scales, wd_codes, wd_scales, R_f32,
                        R_ops, dx=None, dq=None, dw=None, ws=None, ws_bytes=0, stream=None):
    _lib.check(_lib.load().oft_moe_grouped_bwd(
        C.byref(desc), _ptr(dy), C.byref(rt), _ptr(h_saved), _ptr(wgu_codes), _ptr(wgu_scales),
        _ptr(wd_codes), _ptr(wd_scales), _ptr(R_f32), _ptr(R_ops), _ptr(dx), _ptr(dq), _ptr(dw),
        _ptr(ws), ws_bytes, _stream(stream)), "oft_moe_grouped_bwd")
