"""The serving operators of libmk (include/mk.h, "Serving operators") on torch tensors: page tables and slot maps,
per-head norms with rotation and cache append, attention over a paged cache, and logit controls. Argument checks
and marshalling only; every result is computed by the library's kernels.

Tensors live on one CUDA device and outputs are preallocated, as in ``Megakernel``; each call enqueues and returns.
``stream`` is a raw CUDA stream (an int, 0 = the legacy default stream); None takes torch's current stream of the
tensors' device, so a call inside ``torch.cuda.stream`` or a graph capture lands there. On any other stream than that the
caller orders the call with the work that makes and frees its tensors, as for every use of torch on two streams. Tensors that do not fit
together raise ValueError; what the library refuses raises MKError. ``status``, where given, is an int32 tensor of one
element that collects the OP_* flags of what only the device can see.
"""
from __future__ import annotations

import ctypes as C
import struct

import torch

from .binding import (MK_OK, LogitControlsArgs, MKError, PagedAttentionArgs, PageTablesArgs, QkNormRopeArgs, load)

OP_BAD_PAGE, OP_BAD_LENGTH, OP_NO_PAGES, OP_NO_ROOM, OP_TIMEOUT = 1, 2, 4, 8, 16

_DTYPE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2, torch.float8_e4m3fn: 3}
_I32, _I64, _F32, _F64 = torch.int32, torch.int64, torch.float32, torch.float64


def _packer(cls):
    """A struct.Struct with the C layout of a ctypes structure (filling one is several times faster)."""
    code = {C.c_void_p: "P", C.c_int64: "q", C.c_int32: "i", C.c_float: "f"}
    fmt = "@"
    for _, t in cls._fields_:
        fmt += code[t._type_] * t._length_ if hasattr(t, "_length_") else code[t]
    s = struct.Struct(fmt + "0q")
    assert s.size == C.sizeof(cls), cls
    return s.pack


_pack_tables = _packer(PageTablesArgs)
_pack_qk = _packer(QkNormRopeArgs)
_pack_attention = _packer(PagedAttentionArgs)
_pack_logits = _packer(LogitControlsArgs)
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _vector(t, dtype, n, dev, what):
    """The address of an optional contiguous tensor of n elements (n None: any number); 0 for None."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous() or (n is not None and t.numel() != n):
        raise ValueError(f"{what}: a contiguous {dtype} tensor of {n} elements on device {dev} is needed, got "
                         f"{tuple(t.shape)} {t.dtype} on {t.device}")
    return t.data_ptr()


def _rows(t, dtype, n, dev, what):
    """(address, row stride, row length) of an optional [n, length] tensor with contiguous rows."""
    if t is None:
        return 0, 0, 0
    if t.dim() != 2 or t.dtype is not dtype or t.get_device() != dev or t.shape[0] != n:
        raise ValueError(f"{what}: a {dtype} tensor [{n}, ...] on device {dev} is needed, got {tuple(t.shape)} "
                         f"{t.dtype} on {t.device}")
    length = t.shape[1]
    row, one = t.stride()
    if length > 1 and one != 1:
        raise ValueError(f"{what}: rows have to be contiguous")
    return t.data_ptr(), row if n > 1 else length, length


def _heads(t, shape, dtype, dev, what):
    """(address, strides without the last) of a tensor of `shape` whose last dimension is contiguous."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev:
        raise ValueError(f"{what}: {dtype} {tuple(shape)} on device {dev} is needed, got {tuple(t.shape)} {t.dtype} "
                         f"on {t.device}")
    s = t.stride()
    if s[-1] != 1:
        raise ValueError(f"{what}: the last dimension has to be contiguous")
    return t.data_ptr(), s[:-1]


def _call(fn, packed, dev, stream, what):
    rc = fn(packed, dev, _raw_stream(dev) if stream is None else stream)
    if rc != MK_OK:
        raise MKError(rc, f"{what} (details on stderr)")


def page_tables(table, held, start, count, ring, ring_state, page_size: int, n_pages: int, *, slots, positions=None,
                owners=None, starts=None, lens=None, ring_state_out=None, status=None, stream=None) -> None:
    """mk_page_tables: the page table rows and the slot map of a step, on the device.

    table: int32 [B, max_pages], rows contiguous, updated in place. held / start / count: int32 [B], the tokens whose
    pages a row holds, the position of its first new token (<= held; less drops tokens) and how many are new.
    ring: int32 [ring size >= n_pages] of free pages with ring_state int32 [2] = (head, number free).
    slots: int64 [places of the slot map]. Optional: positions, owners (int32, as many places), starts (int32 [B + 1]),
    lens (int32 [B], may be held), ring_state_out (int32 [2]; None updates ring_state itself)."""
    dev = table.get_device()
    _need(dev >= 0, "page_tables needs CUDA tensors")
    n = held.numel()
    tp, ts, max_pages = _rows(table, _I32, n, dev, "table")
    places = slots.numel()
    _need(places < 2 ** 31 and ring.numel() < 2 ** 31, "slots and ring have less than 2^31 entries")
    packed = _pack_tables(
        tp, ts, _vector(held, _I32, n, dev, "held"), _vector(start, _I32, n, dev, "start"),
        _vector(count, _I32, n, dev, "count"), _vector(ring, _I32, None, dev, "ring"),
        _vector(ring_state, _I32, 2, dev, "ring_state"),
        _vector(ring_state if ring_state_out is None else ring_state_out, _I32, 2, dev, "ring_state_out"),
        _vector(slots, _I64, places, dev, "slots"), _vector(positions, _I32, places, dev, "positions"),
        _vector(owners, _I32, places, dev, "owners"), _vector(starts, _I32, n + 1, dev, "starts"),
        _vector(lens, _I32, n, dev, "lens"), _vector(status, _I32, 1, dev, "status"), n, max_pages, page_size, n_pages,
        ring.numel(), places)
    _call(load().mk_page_tables, packed, dev, stream, "page_tables")


_NO2, _NO3 = (0, 0), (0, 0, 0)


def qk_norm_rope(q, k, positions, inv_freq, q_out, *, k_out=None, q_gain=None, k_gain=None, eps: float = 1e-6, v=None,
                 k_pages=None, v_pages=None, slots=None, k_scale=None, v_scale=None, status=None, stream=None) -> None:
    """mk_qk_norm_rope: per-head RMSNorm (with q_gain / k_gain) and rotate-half RoPE of queries and keys in one
    pass, with the append of keys and values to a paged cache.

    q: [N, Hq, D], k, v: [N, Hkv, D] bf16 or fp16 by any strides with D contiguous (slices of a fused projection).
    positions: int32 [N]; inv_freq: float64 [rope_dim / 2], radians per position (None: no rotation). q_out [N, Hq, D]
    may be q; k_out [N, Hkv, D] may be k. Cache: k_pages, v_pages [n_pages, Hkv, page size, D] of q's type or
    float8_e4m3fn (with k_scale, v_scale float32 [Hkv]), slots int64 [N] (negative: not stored)."""
    dev = q.get_device()
    _need(dev >= 0 and q.dim() == 3, "qk_norm_rope needs q [tokens, heads, head_dim] on a CUDA device")
    n, hq, d = q.shape
    dt = q.dtype
    _need(dt in _DTYPE and k.dim() == 3, "q and k are bf16 or fp16 [tokens, heads, head_dim]")
    hkv = k.shape[1]
    kv = (n, hkv, d)
    qp, qs = _heads(q, (n, hq, d), dt, dev, "q")
    kp, ks = _heads(k, kv, dt, dev, "k")
    op, os_ = _heads(q_out, (n, hq, d), dt, dev, "q_out")
    kop, kos = (0, _NO2) if k_out is None else _heads(k_out, kv, dt, dev, "k_out")
    half = 0 if inv_freq is None else inv_freq.numel()
    vp, vs, n_pages, page, cdt = 0, _NO2, 0, 0, _DTYPE[dt]
    kpp, kps, vpp, vps, ksp, vsp, sp = 0, _NO3, 0, _NO3, 0, 0, 0
    if k_pages is not None or v_pages is not None:
        _need(k_pages is not None and v_pages is not None and v is not None and slots is not None,
              "a cache needs k_pages, v_pages, v and slots")
        _need(k_pages.dim() == 4 and k_pages.dtype in _DTYPE, "k_pages is [n_pages, kv heads, page size, head_dim]")
        n_pages, _, page, _ = k_pages.shape
        cache = (n_pages, hkv, page, d)
        vp, vs = _heads(v, kv, dt, dev, "v")
        kpp, kps = _heads(k_pages, cache, k_pages.dtype, dev, "k_pages")
        vpp, vps = _heads(v_pages, cache, k_pages.dtype, dev, "v_pages")
        cdt = _DTYPE[k_pages.dtype]
        sp = _vector(slots, _I64, n, dev, "slots")
        if cdt == 3:
            ksp, vsp = _vector(k_scale, _F32, hkv, dev, "k_scale"), _vector(v_scale, _F32, hkv, dev, "v_scale")
    packed = _pack_qk(
        qp, kp, vp, op, kop, _vector(q_gain, dt, d, dev, "q_gain"), _vector(k_gain, dt, d, dev, "k_gain"),
        _vector(inv_freq, _F64, half, dev, "inv_freq"), _vector(positions, _I32, n, dev, "positions"), sp, kpp, vpp,
        ksp, vsp, _vector(status, _I32, 1, dev, "status"), *qs, *ks, *vs, *os_, *kos, *kps, *vps, n, hq, hkv, d,
        2 * half, n_pages, page, _DTYPE[dt], cdt, eps)
    _call(load().mk_qk_norm_rope, packed, dev, stream, "qk_norm_rope")


def _pack_attention_args(q, k_pages, v_pages, table, lens, out, scale, lse, k_scale, v_scale, dev):
    """The argument struct's fields before the workspace's address and those after its size."""
    shape, cache = q.shape, k_pages.shape
    if len(shape) != 4 or len(cache) != 4:
        raise ValueError("q is [batch, rows, heads, head_dim] and k_pages [n_pages, kv heads, page size, head_dim]")
    b, rows, hq, d = shape
    n_pages, hkv, page, width = cache
    dt, ct = q.dtype, k_pages.dtype
    if dt not in _DTYPE or ct not in _DTYPE or width != d:
        raise ValueError(f"types {dt}, {ct}, widths {d}, {width}")
    qp, qs = _heads(q, shape, dt, dev, "q")
    op, os_ = _heads(out, shape, dt, dev, "out")
    kp, ks = _heads(k_pages, cache, ct, dev, "k_pages")
    vp, vs = _heads(v_pages, cache, ct, dev, "v_pages")
    tp, ts, max_pages = _rows(table, _I32, b, dev, "table")
    ksp = vsp = 0
    if ct is torch.float8_e4m3fn:
        ksp, vsp = _vector(k_scale, _F32, hkv, dev, "k_scale"), _vector(v_scale, _F32, hkv, dev, "v_scale")
    return ((qp, kp, vp, tp, _vector(lens, _I32, b, dev, "lens"), ksp, vsp, op, _vector(lse, _F32, b * rows * hq, dev, "lse")),
            (ts, *qs, *os_, *ks, *vs, b, rows, hq, hkv, d, n_pages, page, max_pages, _DTYPE[dt], _DTYPE[ct],
             d ** -0.5 if scale is None else scale))


def _workspace_size(fn, packed, dev, what) -> int:
    size = C.c_uint64(0)
    rc = fn(packed, dev, C.byref(size))
    if rc != MK_OK:
        raise MKError(rc, f"{what} (details on stderr)")
    return size.value


def _workspace(size, device, dev, stream):
    """Scratch for one call, from torch's allocator (inside a graph capture: from the graph's pool)."""
    if stream is None or stream == _raw_stream(dev):
        return torch.empty(size, dtype=torch.uint8, device=device)
    # The memory has to be the other stream's: what torch has free for its current stream may be in use there until the work
    # enqueued on it so far has run, and nothing orders the two.
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)):
        return torch.empty(size, dtype=torch.uint8, device=device)


def paged_attention_workspace(q, k_pages, table) -> int:
    """Bytes of device scratch paged_attention needs for q, k_pages and table of these shapes and types (0 for small
    calls; else the heads, rows and types alone decide)."""
    dev = q.get_device()
    _need(dev >= 0, "paged_attention needs CUDA tensors")
    lens = torch.empty(q.shape[0], dtype=_I32, device=q.device)
    scale = torch.empty(k_pages.shape[1], dtype=_F32, device=q.device)
    head, tail = _pack_attention_args(q, k_pages, k_pages, table, lens, q, None, None, scale, scale, dev)
    return _workspace_size(load().mk_paged_attention_workspace, _pack_attention(*head, 0, 0, 0, *tail), dev,
                           "paged_attention_workspace")


def paged_attention(q, k_pages, v_pages, table, lens, out, *, scale: float | None = None, lse=None, k_scale=None,
                    v_scale=None, workspace=None, status=None, stream=None) -> None:
    """mk_paged_attention: attention of each request's newest R tokens over its paged cache.

    q, out: [B, R, Hq, D] bf16 or fp16; k_pages, v_pages: [n_pages, Hkv, page size, D] of q's type or float8_e4m3fn
    (with k_scale, v_scale float32 [Hkv]); any strides with D contiguous. table: int32 [B, max_pages]; lens: int32 [B],
    positions in the cache with the R new ones (row r sees lens - (R - 1 - r)). scale: 1 / sqrt(D) by default.
    lse: float32 [B, R, Hq] or None. workspace: a uint8 tensor of paged_attention_workspace bytes that no overlapping
    call uses; None allocates what the call needs from torch's allocator (inside a graph capture: from the graph's
    pool, so that graphs do not share it)."""
    dev = q.get_device()
    if dev < 0:
        raise ValueError("paged_attention needs CUDA tensors")
    head, tail = _pack_attention_args(q, k_pages, v_pages, table, lens, out, scale, lse, k_scale, v_scale, dev)
    st = _vector(status, _I32, 1, dev, "status")
    if workspace is None:
        packed = _pack_attention(*head, 0, st, 0, *tail)
        size = _workspace_size(load().mk_paged_attention_workspace, packed, dev, "paged_attention")
        if size:
            workspace = _workspace(size, q.device, dev, stream)
    if workspace is not None:
        packed = _pack_attention(*head, _vector(workspace, torch.uint8, None, dev, "workspace"), st, workspace.numel(), *tail)
    _call(load().mk_paged_attention, packed, dev, stream, "paged_attention")


def logit_controls(logits, out, *, history=None, prompt_len=None, total_len=None, repetition=None, presence=None,
                   frequency=None, bias_ids=None, bias_vals=None, allowed=None, token=None, workspace=None,
                   stream=None) -> None:
    """mk_logit_controls: penalties, biases and masks on logits, and the greedy token of what is left.

    logits: [rows, vocab] fp32, bf16 or fp16, rows contiguous; out: fp32 [rows, vocab] (may be logits). history: int32
    [rows, n] of token ids with prompt_len / total_len int32 [rows]; repetition, presence, frequency: fp32 [rows];
    bias_ids int32 / bias_vals fp32 [rows, m] (pad ids with -1; the last entry of a token counts); allowed: int32
    [rows, ceil(vocab / 32)] bit mask; token: int32 [rows], -1 where nothing is allowed. workspace: a uint8 tensor of
    what mk_logit_controls_workspace says; None allocates what the call needs from torch's allocator."""
    call, workspace = prepare_logit_controls(logits, out, history, prompt_len, total_len, repetition, presence, frequency,
                                             bias_ids, bias_vals, allowed, token, workspace, stream)
    _call(*call)


def prepare_logit_controls(logits, out, history=None, prompt_len=None, total_len=None, repetition=None, presence=None,
                           frequency=None, bias_ids=None, bias_vals=None, allowed=None, token=None, workspace=None,
                           stream=None):
    """logit_controls' marshalling without its launch: (_call's arguments, the workspace, to be kept until the call)."""
    dev = logits.get_device()
    _need(dev >= 0 and logits.dim() == 2, "logit_controls needs logits [rows, vocab] on a CUDA device")
    n, vocab = logits.shape
    dt = logits.dtype
    _need(dt in _DTYPE, f"logits of {dt}")
    lp, ls, _ = _rows(logits, dt, n, dev, "logits")
    op, os_, width = _rows(out, _F32, n, dev, "out")
    _need(width == vocab, "out has another vocabulary")
    hp, hs, hist = _rows(history, _I32, n, dev, "history")
    bp, bs, nb = _rows(bias_ids, _I32, n, dev, "bias_ids")
    bvp, bvs, nbv = _rows(bias_vals, _F32, n, dev, "bias_vals")
    _need(nb == nbv and bs == bvs, "bias_ids and bias_vals have one layout")
    _need(history is not None or (repetition is None and presence is None and frequency is None), "penalties need a history")
    ap, as_, words = _rows(allowed, _I32, n, dev, "allowed")
    _need(allowed is None or words >= (vocab + 31) // 32, "allowed holds a bit for each token")
    head = (lp, op, _vector(token, _I32, n, dev, "token"), hp, _vector(prompt_len, _I32, n, dev, "prompt_len"),
            _vector(total_len, _I32, n, dev, "total_len"), _vector(repetition, _F32, n, dev, "repetition"),
            _vector(presence, _F32, n, dev, "presence"), _vector(frequency, _F32, n, dev, "frequency"), bp, bvp, ap)
    tail = (ls, os_, hs, bs, as_, n, vocab, hist, nb, _DTYPE[dt])
    if workspace is None:
        packed = _pack_logits(*head, 0, 0, *tail)
        size = _workspace_size(load().mk_logit_controls_workspace, packed, dev, "logit_controls")
        if size:
            workspace = _workspace(size, logits.device, dev, stream)
    if workspace is not None:
        packed = _pack_logits(*head, _vector(workspace, torch.uint8, None, dev, "workspace"), workspace.numel(), *tail)
    return (load().mk_logit_controls, packed, dev, stream, "logit_controls"), workspace


def check_logit_controls(call) -> None:
    """Raises what the library would refuse of a prepared call, without enqueueing it."""
    _, packed, dev, _, what = call
    rc = load().mk_logit_controls_check(packed, dev)
    if rc != MK_OK:
        raise MKError(rc, f"{what} (details on stderr)")
