"""Helpers of the serving tests: caches filled through the library or by random bytes, the values they
hold in float64, and the bound on attention over them."""

from __future__ import annotations

import math

import numpy as np
import torch

import exact_attention_100_b200 as ea
from oracle import attention_kv4_ref
from oracle.kv4 import hadamard_f64


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def random_table(rng, ctx, page, extra_cols=1, spare=3):
    """(block_table int32 [B, width] with -1 where a request has no block, number of blocks)."""
    per = [-(-c // page) for c in ctx]
    nb = sum(per) + spare
    order = rng.permutation(nb)
    table = np.full((len(ctx), max(per + [0]) + extra_cols), -1, dtype=np.int64)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
    return table, nb


def slots_of(table, b, n, page):
    t = np.arange(n)
    return table[b, t // page] * page + t % page


def filled_cache(rng, ctx, table, nb, Hk, d, page, signs=None, k_std=1.0, v_std=1.0, junk=True):
    """A cache whose pages hold normal K and V of each request (through attn_kv4_append); everywhere else
    random bytes (``junk``), among them scales that are NaN or infinite."""
    cache = ea.attn_kv4_cache(nb, Hk, page, d)
    if junk:
        cache.copy_(torch.from_numpy(rng.integers(0, 256, tuple(cache.shape), dtype=np.uint8)).cuda())
        cache[..., 16 * d:] = 0xFF  # (s, z) = NaN
    for b, n in enumerate(ctx):
        if n:
            k, v = (torch.from_numpy((rng.standard_normal((n, Hk, d)) * s).astype(np.float32)).cuda().to(torch.bfloat16)
                    for s in (k_std, v_std))
            ea.attn_kv4_append(k, v, cache, i32(slots_of(table, b, n, page)), signs=signs)
    return cache


def held(cache, ctx, table, page):
    """Per request (k, v) float64 [n, Hk, d] as attn_kv4_read gives them (checked on its own against the
    oracle): float32 values, exact to 2^-24."""
    ks, vs = [], []
    for b, n in enumerate(ctx):
        k, v = ea.attn_kv4_read(cache, i32(slots_of(table, b, n, page)), dtype=torch.float32)
        ks.append(k.cpu().numpy().astype(np.float64))
        vs.append(v.cpu().numpy().astype(np.float64))
    return ks, vs


def reference(q, ks, vs, cu, ctx, scale, causal, signs=None):
    return attention_kv4_ref(q.float().cpu().numpy(), ks, vs, cu, ctx, scale, causal,
                             None if signs is None else signs.cpu().numpy())


# Requests with more rows (queries times heads per key/value head) than this, and 128 keys if Q is transformed, go to
# the kernel that brings K and V to float16
FEW_ROWS = {64: 64, 128: 48, 256: 32}


def bounds(q, ks, vs, cu, ctx, scale, causal, signs, o_ref, lse_ref):
    """Elementwise bounds on |O - ref| and |LSE - ref|, from first-order error propagation.

    A score s_j = scale q . k_j is off by at most d_j = scale e sum_i |q_i| |k_ji| + x |s_j| + x, with e the relative
    roundings of q's and k's entries and of the sums, x those of the scale factors and the exponential.
    LSE is then off by at most sum_j p_j d_j, O by sum_j p_j d_j |v_j - O|.
    Few rows: q is kept in 22 bits and the codes are exact: e = 2^-21 + 2^-18 (float32 sums of up to 256 products
    whose codes carry an offset, at most 16 times the value's own size, cut off at 2^-23 each), x = 2^-20; p_j times
    V's step is rounded by 2^-11, which moves O by 2^-11 sum_j p_j (|v_j| + 15 s_j) <= 2^-11 3 sum_j p_j max|v_j| (a code
    times its step is at most the range, twice the largest value).
    Many rows: q (transformed) and k are rounded to float16, 2^-11 each: e = 2^-10 + 2^-18, x as above, and the row's
    factor is corrected by sum q_i dq_i / sum q_i^2 <= 2^-11: 2^-11 |s_j| more; V is rounded by 2^-11, p too, twice
    where the maximum moved: 3 2^-11 sum_j p_j |v_j|.
    O is rounded to bf16, 2^-8.  Second order: the whole times 1.1."""
    q = q.float().cpu().numpy().astype(np.float64)
    if signs is not None:
        q = hadamard_f64(q, signs.cpu().numpy())
    ob, lb = np.full(o_ref.shape, np.inf), np.full(lse_ref.shape, np.inf)
    group = q.shape[1] // ks[0].shape[1]
    few = FEW_ROWS[q.shape[2]]
    most = max((int(cu[b + 1]) - int(cu[b])) * group for b in range(len(ctx)))
    for b, n in enumerate(ctx):
        lo, hi = int(cu[b]), int(cu[b + 1])
        short = signs is not None and n < 128
        many = most > few and ((hi - lo) * group > few and not short or len(ctx) == 1 and (signs is None or hi - lo >= 128))
        e, x = (2.0 ** -10 if many else 2.0 ** -21) + 2.0 ** -18, 2.0 ** -20
        for h in range(q.shape[1]):
            kh = h // group
            for i in range(lo, hi):
                seen = max(0, n - (hi - lo) + (i - lo) + 1) if causal else n
                if seen == 0:
                    ob[i, h], lb[h, i] = 0, 0
                    continue
                k, v = ks[b][:seen, kh], vs[b][:seen, kh]
                s = scale * (k @ q[i, h])
                p = np.exp(s - lse_ref[h, i])
                dj = scale * e * (np.abs(k) @ np.abs(q[i, h])) + x * np.abs(s) + x
                if many:
                    dj += 2.0 ** -11 * np.abs(s)
                vmax = np.abs(v).max(-1, keepdims=True)
                round_p = 3 * 2.0 ** -11 * (p @ np.abs(v)) if many else 2.0 ** -11 * 3 * (p @ vmax)
                ob[i, h] = 1.1 * ((p * dj) @ np.abs(v - o_ref[i, h]) + round_p) + 2.0 ** -8 * np.abs(o_ref[i, h])
                lb[h, i] = 1.1 * (p @ dj) + 2.0 ** -22 * (abs(lse_ref[h, i]) + 8)
    return ob, lb


def check(o, lse, q, ks, vs, cu, ctx, scale, causal, signs=None):
    o_ref, lse_ref = reference(q, ks, vs, cu, ctx, scale, causal, signs)
    ob, lb = bounds(q, ks, vs, cu, ctx, scale, causal, signs, o_ref, lse_ref)
    rows = int(cu[-1])
    o, lse = o.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    worst = np.max(np.abs(o[:rows] - o_ref[:rows]) / (ob[:rows] + 1e-300))
    assert np.isfinite(o[:rows]).all() and worst <= 1, worst
    ninf = np.isneginf(lse_ref[:, :rows])
    assert np.array_equal(ninf, np.isneginf(lse[:, :rows]))
    with np.errstate(invalid="ignore"):
        off = np.where(ninf, 0, np.abs(lse[:, :rows] - lse_ref[:, :rows])) / (lb[:, :rows] + 1e-300)
    assert off.max() <= 1, off.max()
    return o_ref, lse_ref


def default_scale(d):
    return 1.0 / math.sqrt(d)
