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


def bounds(q, ks, vs, cu, ctx, scale, causal, signs, o_ref, lse_ref, q_step=0.0, k_step=0.0, p_step=2.0 ** -11,
           v_step=0.0):
    """Elementwise bounds on |O - ref| and |LSE - ref|, from first-order error propagation:

    a score s_j = scale q . k_j is off by at most d_j = scale (q_step + k_step + 2^-18) sum_i |q_i| |k_ji|
    (relative roundings of q's and k's entries, and of float32 sums of up to 256 products whose codes
    carry an offset, at most 16 times the value's own size, 2^-24 each) + 2^-20 |s_j| (scale factors, exp2);
    LSE is then off by at most sum_j p_j d_j, O by sum_j p_j d_j |v_j - O|; p_j times V's step is rounded
    by p_step, which moves O by p_step sum_j p_j (|v_j| + 15 s_j) <= p_step 3 sum_j p_j max|v_j| (a code times
    its step is at most the range, twice the largest value); V's own rounding adds v_step sum_j p_j |v_j|;
    O is rounded to bf16, 2^-8.  Second order: the whole times 1.1."""
    q = q.float().cpu().numpy().astype(np.float64)
    if signs is not None:
        q = hadamard_f64(q, signs.cpu().numpy())
    ob, lb = np.full(o_ref.shape, np.inf), np.full(lse_ref.shape, np.inf)
    for b, n in enumerate(ctx):
        lo, hi = int(cu[b]), int(cu[b + 1])
        for h in range(q.shape[1]):
            kh = h // (q.shape[1] // ks[b].shape[1])
            for i in range(lo, hi):
                seen = max(0, n - (hi - lo) + (i - lo) + 1) if causal else n
                if seen == 0:
                    ob[i, h], lb[h, i] = 0, 0
                    continue
                k, v = ks[b][:seen, kh], vs[b][:seen, kh]
                s = scale * (k @ q[i, h])
                p = np.exp(s - lse_ref[h, i])
                dj = scale * (q_step + k_step + 2.0 ** -18) * (np.abs(k) @ np.abs(q[i, h])) + 2.0 ** -20 * np.abs(s)
                vmax = np.abs(v).max(-1, keepdims=True)
                ob[i, h] = 1.1 * ((p * dj) @ np.abs(v - o_ref[i, h]) + (p_step * 3 * (p @ vmax))
                                  + v_step * (p @ np.abs(v))) + 2.0 ** -8 * np.abs(o_ref[i, h])
                lb[h, i] = 1.1 * (p @ dj) + 2.0 ** -22 * (abs(lse_ref[h, i]) + 8)
    return ob, lb


def check(o, lse, q, ks, vs, cu, ctx, scale, causal, signs=None, **steps):
    o_ref, lse_ref = reference(q, ks, vs, cu, ctx, scale, causal, signs)
    if signs is not None:
        steps.setdefault("q_step", 2.0 ** -11)  # the transformed q in float16
    ob, lb = bounds(q, ks, vs, cu, ctx, scale, causal, signs, o_ref, lse_ref, **steps)
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
