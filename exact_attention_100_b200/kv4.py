"""Serving over a paged key/value cache held in 4 bits: Python binding of ``include/attn_kv.h``.

One serving step, in order (every tensor on the current CUDA device):

    slots, pos, cu, lens, cursor, table = ea.attn_kv_tables(lens, new_lens, table, free, cursor, page, total)
    q, k = ea.attn_rope_axes(q, k, cos, sin, pos, [d // 2])     # or [t, h, w] sections, pos [3, total]
    ea.attn_kv4_append(k, v, cache, slots, signs=signs)
    o, lse = ea.attn_fwd_kv4(q, cache, table, lens, cu_seqlens_q=cu, max_seqlen_q=longest, signs=signs)

``q`` [total, Hq, d], ``k`` and ``v`` [total, Hk, d] are bf16 with any row and head strides (views of
one fused projection); the cache is a uint8 tensor [num_blocks, Hk, page / 16, 18 d] from
:func:`attn_kv4_cache`.  All of it can be captured into a CUDA graph (after one call outside a
capture has set the library up).  What only the device can see (lengths, offsets, slots, positions and
block ids out of range) is reported by the next ``attn_device_status()``.

With ``stream`` the call runs on that stream, and the tensors it makes belong to that stream.
"""

from __future__ import annotations

import contextlib
import ctypes
import math

from . import (ATTN_BF16, ATTN_FP32, _check, _out, _ptr, _signs, _stream_ptr, _workspace, lib)


def declare(L) -> None:
    vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    L.attn_kv_tables.argtypes = [vp] * 10 + [i] * 5 + [vp]
    L.attn_kv_tables.restype = i
    L.attn_rope_axes.argtypes = [vp] * 7 + [i] * 6 + [vp, i, vp, i, i, i, vp]
    L.attn_rope_axes.restype = i
    L.attn_kv4_tile_bytes.argtypes = [i]
    L.attn_kv4_tile_bytes.restype = ctypes.c_ulonglong
    L.attn_kv4_append.argtypes = [vp] * 5 + [i] * 5 + [vp, vp]
    L.attn_kv4_append.restype = i
    L.attn_kv4_read.argtypes = [vp] * 4 + [i] * 6 + [vp]
    L.attn_kv4_read.restype = i
    L.attn_fwd_kv4_workspace_bytes.argtypes = [i, i]
    L.attn_fwd_kv4_workspace_bytes.restype = ctypes.c_ulonglong
    L.attn_fwd_kv4.argtypes = [vp] * 9 + [i] * 9 + [vp, f, i, vp]
    L.attn_fwd_kv4.restype = i


def _on(stream):
    """The stream that a call's own tensors are made on (and whose device is then the current one)."""
    import torch
    return torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext()


def _ints(t, shape, what):
    import torch
    return _out(t, shape, (torch.int32,), what)


def _strides(*values):
    a = (ctypes.c_longlong * len(values))(*[int(v) for v in values])
    return ctypes.cast(a, ctypes.c_void_p)


def attn_kv_tables(lens, new_lens, block_table, free_blocks, cursor, page_size, total, slots=None, positions=None,
                   cu_seqlens=None, lens_out=None, cursor_out=None, stream=None):
    """Block tables and slot maps of one serving step, on the GPU.

    ``lens``, ``new_lens`` [B] int32: tokens each request holds, and adds now; ``block_table``
    [B, width] int32 (new entries written in place); ``free_blocks`` [n] int32 ids and ``cursor`` [1] int32,
    how many of them are taken; ``total``: the host's bound on the sum of ``new_lens``.  Returns ``(slots
    [total], positions [total], cu_seqlens [B + 1], lens_out [B], cursor_out [1], block_table)``, int32.
    ``lens_out=lens`` and ``cursor_out=cursor`` update in place.  A request for which the free blocks do
    not suffice is not served: its slots are -1 and its length stays.
    """
    import torch
    B = int(lens.shape[0]) if lens.dim() == 1 else 0
    if B == 0 or block_table.dim() != 2 or free_blocks.dim() != 1:
        raise ValueError("expected lens [B], block_table [B, width], free_blocks [n]")
    width, total = int(block_table.shape[1]), int(total)
    _ints(lens, (B,), "lens")
    _ints(new_lens, (B,), "new_lens")
    _ints(block_table, (B, width), "block_table")
    _ints(free_blocks, tuple(free_blocks.shape), "free_blocks")
    _ints(cursor, (1,), "cursor")
    if total < 0:
        raise ValueError("total must not be negative")
    with _on(stream):
        new = lambda t, n: t if t is not None else torch.empty(n, dtype=torch.int32, device=lens.device)
        slots, positions = new(slots, total), new(positions, total)
        cu_seqlens, lens_out, cursor_out = new(cu_seqlens, B + 1), new(lens_out, B), new(cursor_out, 1)
        for t, n, what in ((slots, total, "slots"), (positions, total, "positions"), (cu_seqlens, B + 1, "cu_seqlens"),
                           (lens_out, B, "lens_out"), (cursor_out, 1, "cursor_out")):
            _ints(t, (n,), what)
        _check(lib().attn_kv_tables(_ptr(lens), _ptr(new_lens), _ptr(block_table), _ptr(free_blocks), _ptr(cursor),
                                    _ptr(slots), _ptr(positions), _ptr(cu_seqlens), _ptr(lens_out), _ptr(cursor_out), B,
                                    width, int(page_size), int(free_blocks.shape[0]), total, _stream_ptr(stream)),
               "attn_kv_tables")
    return slots, positions, cu_seqlens, lens_out, cursor_out, block_table


def _rope(q, k, cos, sin, positions, sections, q_out, k_out, out_dtype, inverse, stream, name):
    import torch
    sections = [int(s) for s in sections]
    half = sum(sections)
    if q.dim() not in (3, 4) or (k is not None and k.dim() != q.dim()):
        raise ValueError("q and k must be [tokens, heads, d] or [B, heads, N, d]")
    packed = q.dim() == 3
    dims = lambda t: (1, int(t.shape[1]), int(t.shape[0]), int(t.shape[2])) if packed else tuple(int(x) for x in t.shape)
    st = lambda t: (8, t.stride(1), t.stride(0)) if packed else t.stride()[:3]
    B, Hq, N, d = dims(q)
    if k is not None and (dims(k)[0], dims(k)[2], dims(k)[3]) != (B, N, d):
        raise ValueError("k must have q's tokens and d")
    if k is not None and k.dtype != q.dtype:
        raise ValueError("q and k must have one dtype")
    types = (torch.bfloat16, torch.float32)
    for t, what in ((q, "q"), (k, "k")):
        if t is not None:
            _out(t, tuple(t.shape), types, what, strided=True)
    for t, what in ((cos, "cos"), (sin, "sin")):
        if t.dim() != 2 or t.shape[0] == 0:
            raise ValueError("cos and sin must be float32 [n_pos, sum of the sections]")
        _out(t, (int(cos.shape[0]), half), (torch.float32,), what)
    if positions.dim() == 1 and packed and len(sections) == 1:
        positions = positions[None]
    _ints(positions, (len(sections), N) if packed else (len(sections), B, N), "positions")
    with _on(stream):
        outs = []
        for x, y, what in ((q, q_out, "q_out"), (k, k_out, "k_out")):
            if x is None:
                if y is not None:
                    raise ValueError("k_out without k")
                outs.append(None)
                continue
            if y is None:
                y = torch.empty_like(x, dtype=out_dtype or x.dtype)
            outs.append(_out(y, tuple(x.shape), types, what, strided=True))
        q_out, k_out = outs
        if k_out is not None and k_out.dtype != q_out.dtype:
            raise ValueError("q_out and k_out must have one dtype")
        if B * N == 0 or Hq == 0:
            return q_out, k_out
        one = (8, 8, 8)
        strides = _strides(*st(q), *(st(k) if k is not None else one), *st(q_out), *(st(k_out) if k is not None else one))
        sec = (ctypes.c_int * len(sections))(*sections)
        code = lambda t: ATTN_FP32 if t.dtype == torch.float32 else ATTN_BF16
        _check(lib().attn_rope_axes(_ptr(q), _ptr(k), _ptr(q_out), _ptr(k_out), _ptr(cos), _ptr(sin), _ptr(positions), B,
                                    Hq, dims(k)[1] if k is not None else 0, N, d, len(sections),
                                    ctypes.cast(sec, ctypes.c_void_p), int(cos.shape[0]), strides, inverse, code(q),
                                    code(q_out), _stream_ptr(stream)), name)
    return q_out, k_out


def attn_rope_axes(q, k, cos, sin, positions, sections, q_out=None, k_out=None, out_dtype=None, stream=None):
    """Rotary embedding of ``q`` and ``k`` (``k`` may be None) with one to four position axes.

    ``q``, ``k``: [tokens, heads, d] or [B, heads, N, d], bf16 or float32, last dimension contiguous;
    ``cos``, ``sin`` float32 [n_pos, half] (position-major, row p: the angles of position p);
    ``positions`` int32 [axes, tokens] or [axes, B, N]; ``sections``: how many of the ``half`` pairs turn
    with each axis, in order.  Coordinates i and i + half form pair i; dimensions past 2 * half are
    copied.  ``q_out=q``, ``k_out=k`` rotate in place.  Returns ``(q_out, k_out)``."""
    return _rope(q, k, cos, sin, positions, sections, q_out, k_out, out_dtype, 0, stream, "attn_rope_axes")


def attn_rope_axes_bwd(dq, dk, cos, sin, positions, sections, dq_out=None, dk_out=None, out_dtype=None, stream=None):
    """The backward of :func:`attn_rope_axes`: gradients of its outputs to gradients of its inputs
    (bf16 or float32 each), with the same tables, positions and sections."""
    return _rope(dq, dk, cos, sin, positions, sections, dq_out, dk_out, out_dtype, 1, stream, "attn_rope_axes_bwd")


def attn_kv4_cache(num_blocks, Hk, page_size, d, device=None):
    """An empty cache: uint8 zeros [num_blocks, Hk, page_size / 16, 18 d] (every value it holds is 0)."""
    import torch
    tile = int(lib().attn_kv4_tile_bytes(int(d)))
    if tile == 0 or page_size < 16 or page_size > 4096 or page_size % 16:
        raise ValueError("d must be 64, 128 or 256 and page_size a multiple of 16 up to 4096")
    return torch.zeros((int(num_blocks), int(Hk), int(page_size) // 16, tile), dtype=torch.uint8,
                       device=device if device is not None else torch.device("cuda", torch.cuda.current_device()))


def _cache_dims(cache):
    """(num_blocks, Hk, page_size, d) of a cache."""
    import torch
    if cache.dim() != 4 or cache.dtype != torch.uint8 or not cache.is_contiguous() or cache.shape[3] % 18:
        raise ValueError("cache must be contiguous uint8 [num_blocks, Hk, page / 16, 18 d]")
    nb, hk, tiles, tile = (int(x) for x in cache.shape)
    return nb, hk, 16 * tiles, tile // 18


def attn_kv4_append(k, v, cache, slots, signs=None, stream=None):
    """Quantises ``k``, ``v`` [T, Hk, d] bf16 (row and head strides free) to 4 bits and writes them to
    ``slots`` [T] int32 of ``cache``, in place (slot -1: skipped).  ``signs`` (d int8 entries +-1) puts
    K through the random-sign Hadamard transform first; give the same to :func:`attn_fwd_kv4`.
    Returns ``cache``."""
    import torch
    nb, Hk, page, d = _cache_dims(cache)
    T = int(slots.shape[0]) if slots.dim() == 1 else -1
    _ints(slots, (T,), "slots")
    for t, what in ((k, "k"), (v, "v")):
        _out(t, (T, Hk, d), (torch.bfloat16,), what, strided=True)
    if T == 0:
        return cache
    with _on(stream):
        _check(lib().attn_kv4_append(_ptr(k), _ptr(v), _ptr(cache), _ptr(slots), _ptr(_signs(signs, d)), T, Hk, d, page,
                                     nb, _strides(*k.stride()[:2], *v.stride()[:2]), _stream_ptr(stream)),
               "attn_kv4_append")
    return cache


def attn_kv4_read(cache, slots, k=None, v=None, dtype=None, stream=None):
    """The values held at ``slots`` [T] int32 of ``cache``: ``(k, v)`` [T, Hk, d] in ``dtype``
    (torch.bfloat16, the default, or torch.float32); slot -1 gives zeros.  A K that was transformed comes
    back transformed."""
    import torch
    nb, Hk, page, d = _cache_dims(cache)
    T = int(slots.shape[0]) if slots.dim() == 1 else -1
    _ints(slots, (T,), "slots")
    with _on(stream):
        dt = dtype or (k.dtype if k is not None else v.dtype if v is not None else torch.bfloat16)
        k = k if k is not None else torch.empty((T, Hk, d), dtype=dt, device=cache.device)
        v = v if v is not None else torch.empty((T, Hk, d), dtype=dt, device=cache.device)
        for t, what in ((k, "k"), (v, "v")):
            _out(t, (T, Hk, d), (torch.bfloat16, torch.float32), what)
        if k.dtype != v.dtype:
            raise ValueError("k and v must have one dtype")
        if T == 0:
            return k, v
        _check(lib().attn_kv4_read(_ptr(cache), _ptr(slots), _ptr(k), _ptr(v), T, Hk, d, page, nb,
                                   ATTN_FP32 if k.dtype == torch.float32 else ATTN_BF16, _stream_ptr(stream)),
               "attn_kv4_read")
    return k, v


def attn_fwd_kv4_workspace_bytes(d, num_sms=0) -> int:
    """Bytes of the workspace :func:`attn_fwd_kv4` needs on the current device (or on one of
    ``num_sms`` processors)."""
    return int(lib().attn_fwd_kv4_workspace_bytes(int(d), int(num_sms)))


def attn_fwd_kv4(q, cache, block_table, seq_lens, cu_seqlens_q=None, max_seqlen_q=1, o=None, lse=None, workspace=None,
                 signs=None, scale=None, causal=True, stream=None, want_lse=True):
    """Attention of ``q`` [total_q, Hq, d] bf16 (row and head strides free) over the 4-bit ``cache``,
    query head h reading key/value head ``h // (Hq // Hk)``.

    ``block_table`` [B, width] int32, ``seq_lens`` [B] int32 (keys of each request, its new tokens
    among them).  Without ``cu_seqlens_q`` each request has one query (total_q = B); with it (int32
    [B + 1]) request b owns query rows ``cu_seqlens_q[b]:cu_seqlens_q[b + 1]``, at most ``max_seqlen_q`` of
    them, and with ``causal`` they are its last tokens.  ``signs`` as given to :func:`attn_kv4_append`.
    Rows that see no key get O = 0, LSE = -inf.  Returns ``(o [total_q, Hq, d] bf16, lse [Hq, total_q]
    float32)``; rows behind the last request are left as they were.
    """
    import torch
    nb, Hk, page, d = _cache_dims(cache)
    if q.dim() != 3 or int(q.shape[2]) != d or int(q.shape[1]) % Hk:
        raise ValueError("q must be [total_q, Hq, d] with the cache's d and a multiple of its heads")
    total_q, Hq = int(q.shape[0]), int(q.shape[1])
    _out(q, (total_q, Hq, d), (torch.bfloat16,), "q", strided=True)
    if block_table.dim() != 2 or int(block_table.shape[0]) == 0:
        raise ValueError("block_table must be [B, width]")
    B, width = (int(x) for x in block_table.shape)
    _ints(block_table, (B, width), "block_table")
    _ints(seq_lens, (B,), "seq_lens")
    if cu_seqlens_q is not None:
        _ints(cu_seqlens_q, (B + 1,), "cu_seqlens_q")
    elif total_q != B or int(max_seqlen_q) != 1:
        raise ValueError("without cu_seqlens_q there is one query per request")
    with _on(stream):
        if o is None:
            o = torch.empty((total_q, Hq, d), dtype=torch.bfloat16, device=q.device)
        _out(o, (total_q, Hq, d), (torch.bfloat16,), "o", strided=True)
        if lse is None and want_lse:
            lse = torch.empty((Hq, total_q), dtype=torch.float32, device=q.device)
        if lse is not None:
            _out(lse, (Hq, total_q), (torch.float32,), "lse")
        if total_q == 0:
            return o, lse
        args = [_ptr(q), _ptr(cache), _ptr(block_table), _ptr(seq_lens), _ptr(cu_seqlens_q), _ptr(o), _ptr(lse)]
        nbytes = attn_fwd_kv4_workspace_bytes(d)
        workspace = _workspace(workspace, nbytes, q.device, "attn_fwd_kv4")
        s = float(scale) if scale is not None else 1.0 / math.sqrt(d)
        _check(lib().attn_fwd_kv4(*args, _ptr(workspace), _ptr(_signs(signs, d)), B, Hq, Hk, total_q, int(max_seqlen_q),
                                  d, page, nb, width, _strides(*q.stride()[:2], *o.stride()[:2]), s,
                                  int(bool(causal)), _stream_ptr(stream)), "attn_fwd_kv4")
    return o, lse
