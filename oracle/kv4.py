"""Plain float64 forms of the serving operators: block tables, rotary embedding over several axes,
the 4-bit cache and attention over it.  One element, token or request at a time where that is the
definition; shares no code with the CUDA path.

The 4-bit format (``include/attn_kv.h``): per token, head and group of 64 values z = the largest bf16
<= min, s = the smallest bf16 >= (max - z) / 15, u = rint((x - z) / s) in 0 .. 15, in float32
arithmetic; the value is u s + z.  K may go through the random-sign Hadamard transform first
("FlashAttention-3", section "FP8 路径与低精度误差").
"""

from __future__ import annotations

import math

import numpy as np

from .fp8 import fwht_f32


def bf16_down(x: np.ndarray) -> np.ndarray:
    """The largest bf16 value not above each float32 of ``x``."""
    x = np.asarray(x, dtype=np.float32)
    u = x.view(np.uint32)
    cut = u & np.uint32(0xFFFF0000)
    neg = (x < 0) & (cut != u)
    return np.where(neg, cut + np.uint32(0x10000), cut).astype(np.uint32).view(np.float32)


def quantise(x: np.ndarray):
    """(codes uint8 [..., d], s, z float32 [..., d / 64]) of float32 ``x`` [..., d]."""
    x = np.asarray(x, dtype=np.float32)
    g = x.reshape(x.shape[:-1] + (x.shape[-1] // 64, 64))
    with np.errstate(all="ignore"):
        z = bf16_down(g.min(-1))
        rng = (g.max(-1) - z).astype(np.float32)
        s = -bf16_down(-(rng / np.float32(15)).astype(np.float32))
        safe = np.where(s > 0, s, np.float32(1)).astype(np.float32)
        u = np.rint(((g - z[..., None]).astype(np.float32) / safe[..., None]).astype(np.float32))
        u = np.where(s[..., None] > 0, np.clip(u, 0, 15), 0)
        bad = ~(np.isfinite(g).all(-1) & np.isfinite(rng))
    s = np.where(bad, np.float32(np.nan), s)
    z = np.where(bad, np.float32(np.nan), z)
    u = np.where(bad[..., None], 0, u).astype(np.uint8)
    return u.reshape(x.shape), s, z


def values(u, s, z) -> np.ndarray:
    """u s + z in float64."""
    r = lambda a: np.repeat(np.asarray(a, dtype=np.float64), 64, axis=-1)
    return u.astype(np.float64) * r(s) + r(z)


def transformed(x: np.ndarray, signs) -> np.ndarray:
    """What is quantised for K: float32 (1/sqrt d) H_d (D x), stage by stage, or x itself."""
    x = np.asarray(x, dtype=np.float32)
    if signs is None:
        return x
    d = x.shape[-1]
    return (fwht_f32(x * np.asarray(signs, dtype=np.float32)) * np.float32(1 / math.sqrt(d))).astype(np.float32)


def hadamard_f64(x: np.ndarray, signs) -> np.ndarray:
    """(1/sqrt d) H_d (D x) in float64 by the matrix."""
    d = x.shape[-1]
    h = np.ones((1, 1))
    while h.shape[0] < d:
        h = np.block([[h, h], [h, -h]])
    return (np.asarray(x, dtype=np.float64) * np.asarray(signs, dtype=np.float64)) @ h.T / math.sqrt(d)


def code_place(d: int, dim: int, is_v: bool):
    """(byte offset of a dimension's code from the start of its tensor's codes, for row 0; bytes from
    one row to the next; nibble) in a tile."""
    w = min(d, 128)
    n = w // 64
    plane, x = divmod(dim, w)
    g, r = divmod(x, 64)
    if is_v:
        byte = 4 * n * (r // 8) + 4 * g + (r % 8) // 2
    else:
        byte = 8 * n * (r // 16) + 8 * g + (r % 16) // 2
    return plane * 16 * (w // 2) + byte, w // 2, r & 1


def write_token(cache: np.ndarray, page: int, slot: int, head: int, ku, ks, kz, vu, vs, vz) -> None:
    """Writes one token of one head into ``cache`` uint8 [blocks, Hk, page / 16, 18 d]."""
    d = ku.shape[-1]
    block, off = divmod(slot, page)
    tile = cache[block, head, off // 16]
    row = off % 16
    for base, u, is_v in ((0, ku, False), (8 * d, vu, True)):
        for x in range(d):
            at, step, odd = code_place(d, x, is_v)
            at += base + row * step
            tile[at] = (tile[at] & 0x0F) | (int(u[x]) << 4) if odd else (tile[at] & 0xF0) | int(u[x])
    for base, s, z in ((16 * d, ks, kz), (17 * d, vs, vz)):
        pair = np.stack([s, z], -1).astype(np.float32).reshape(-1)
        raw = (pair.view(np.uint32) >> 16).astype(np.uint16).view(np.uint8)
        tile[base + row * (d // 16): base + (row + 1) * (d // 16)] = raw


def read_token(cache: np.ndarray, page: int, slot: int, head: int):
    """(k, v) float64 [d] held at a slot."""
    d = cache.shape[-1] // 18
    block, off = divmod(slot, page)
    tile = cache[block, head, off // 16]
    row = off % 16
    out = []
    for base, pairs, is_v in ((0, 16 * d, False), (8 * d, 17 * d, True)):
        u = np.empty(d, dtype=np.uint8)
        for x in range(d):
            at, step, odd = code_place(d, x, is_v)
            u[x] = (tile[base + row * step + at] >> (4 if odd else 0)) & 15
        raw = tile[pairs + row * (d // 16): pairs + (row + 1) * (d // 16)].copy().view(np.uint16).astype(np.uint32)
        p = (raw << 16).view(np.float32).reshape(-1, 2)
        out.append(values(u, p[:, 0], p[:, 1]))
    return tuple(out)


def attention_kv4_ref(q, k, v, cu_q, lens, scale, causal, signs=None):
    """(O [total_q, Hq, d], LSE [Hq, total_q]) in float64.  ``q`` [total_q, Hq, d]; ``k``, ``v``: per
    request the values held, [ctx, Hk, d]; rows of no request stay NaN; rows that see no key are (0, -inf)."""
    q = np.asarray(q, dtype=np.float64)
    if signs is not None:
        q = hadamard_f64(q, signs)
    total, Hq, d = q.shape
    o = np.full(q.shape, np.nan)
    lse = np.full((Hq, total), np.nan)
    for b, n in enumerate(lens):
        lo, hi = int(cu_q[b]), int(cu_q[b + 1])
        for h in range(Hq):
            kh = h // (Hq // k[b].shape[1])
            for i in range(lo, hi):
                seen = max(0, n - (hi - lo) + (i - lo) + 1) if causal else n
                if seen == 0:
                    o[i, h], lse[h, i] = 0.0, -np.inf
                    continue
                s = scale * (k[b][:seen, kh] @ q[i, h])
                m = s.max()
                p = np.exp(s - m)
                o[i, h] = p @ v[b][:seen, kh] / p.sum()
                lse[h, i] = m + math.log(p.sum())
    return o, lse


def rope_axes_ref(x, cos, sin, positions, sections, inverse=False):
    """``x`` [tokens, heads, d] rotated in float64; ``cos``, ``sin`` [n_pos, half]; ``positions``
    [axes, tokens]."""
    y = np.array(x, dtype=np.float64)
    half = sum(sections)
    i = 0
    for a, n in enumerate(sections):
        c = np.asarray(cos, dtype=np.float64)[positions[a], i:i + n][:, None]
        s = np.asarray(sin, dtype=np.float64)[positions[a], i:i + n][:, None]
        if inverse:
            s = -s
        u, w = np.array(x[..., i:i + n], dtype=np.float64), np.array(x[..., half + i:half + i + n], dtype=np.float64)
        y[..., i:i + n] = u * c - w * s
        y[..., half + i:half + i + n] = w * c + u * s
        i += n
    return y


def tables_ref(lens, new_lens, table, free, cursor, page, total):
    """What attn_kv_tables writes: (slots, positions, cu, lens_out, cursor_out, table); requests one
    after another.  Lengths in range."""
    table = np.array(table)
    slots, positions = np.full(total, -1, np.int64), np.zeros(total, np.int64)
    cu, lens_out, wanted, taken = [0], [], cursor, cursor
    for b, (n0, n) in enumerate(zip(lens, new_lens)):
        held, want = -(-int(n0) // page), -(-(int(n0) + int(n)) // page)
        wanted += want - held
        served = want == held or wanted <= len(free)
        if served:
            if want > held:
                table[b, held:want] = free[taken:wanted]
                taken = wanted
        for i in range(int(n)):
            t = cu[-1] + i
            positions[t] = n0 + i
            if served:
                slots[t] = table[b, (n0 + i) // page] * page + (n0 + i) % page
        cu.append(cu[-1] + int(n))
        lens_out.append(int(n0) + int(n) if served else int(n0))
    return slots, positions, np.array(cu), np.array(lens_out), taken, table
