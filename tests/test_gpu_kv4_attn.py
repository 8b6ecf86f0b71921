"""attn_fwd_kv4 against the float64 form on the values the cache holds; the bounds are derived in
kv_util.bounds."""

import numpy as np
import pytest
import torch

import exact_attention_100_b200 as ea
from exact_attention_100_b200 import build as ea_build
from exact_attention_100_b200.inputs import hadamard_signs
from kv_util import check, default_scale, filled_cache, held, i32, random_table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ea_build.build()


def _q(rng, rows, Hq, d, std=1.0):
    return torch.from_numpy((rng.standard_normal((rows, Hq, d)) * std).astype(np.float32)).cuda().to(torch.bfloat16)


def _run(ctx, nq, Hq, Hk, d, page, causal=True, transform=False, seed=0, q_std=1.0, k_std=1.0, v_std=1.0, scale=None):
    rng = np.random.default_rng(seed)
    table, nb = random_table(rng, ctx, page)
    signs = torch.from_numpy(hadamard_signs(d)).cuda() if transform else None
    cache = filled_cache(rng, ctx, table, nb, Hk, d, page, signs, k_std, v_std)
    cu = np.concatenate([[0], np.cumsum(nq)])
    q = _q(rng, int(cu[-1]), Hq, d, q_std)
    scale = scale or default_scale(d)
    o, lse = ea.attn_fwd_kv4(q, cache, i32(table), i32(ctx), cu_seqlens_q=i32(cu), max_seqlen_q=max(max(nq), 1), signs=signs,
                             scale=scale, causal=causal)
    assert ea.attn_device_status() == ea.ATTN_OK
    ks, vs = held(cache, ctx, table, page)
    check(o, lse, q, ks, vs, cu, ctx, scale, causal, signs)
    return q, cache, table, cu, signs, o, lse


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("transform", [False, True])
@pytest.mark.parametrize("ctx,nq,Hq,Hk,page", [
    ([1], [1], 1, 1, 16), ([16], [1], 4, 1, 16), ([17, 15, 33], [1, 1, 1], 8, 2, 16), ([129, 1, 700], [1, 1, 1], 6, 2, 48),
    ([2000], [1], 7, 1, 64), ([300, 40, 5, 64], [3, 5, 5, 1], 4, 2, 32), ([90, 257], [9, 20], 6, 3, 128),
    ([5000, 3], [2, 2], 16, 1, 64)])
def test_matches_the_oracle(d, transform, ctx, nq, Hq, Hk, page):
    _run(ctx, nq, Hq, Hk, d, page, True, transform, seed=sum(ctx) + d)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_without_the_causal_mask(d):
    _run([33, 0, 170], [4, 2, 1], 6, 3, d, 16, causal=False, seed=d)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_rows_that_see_no_key(d):
    """Requests without keys, with fewer keys than queries, and without queries."""
    _, _, _, _, _, o, lse = _run([0, 3, 20, 2], [1, 6, 0, 2], 4, 2, d, 16, seed=d)
    assert (o[0] == 0).all() and torch.isneginf(lse[:, 0]).all() and (o[1:4] == 0).all() and (o[4] != 0).any()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_std,k_std,v_std,scale", [(1e-3, 1e3, 1e-6, None), (30.0, 1.0, 1e5, None), (1.0, 1.0, 1e-30, None),
                                                     (1e-20, 1e20, 1.0, None), (4.0, 4.0, 1.0, 1.0)])
def test_values_of_any_size(d, q_std, k_std, v_std, scale):
    _run([700, 31], [1, 2], 4, 2, d, 16, True, True, 7, q_std, k_std, v_std, scale)


def test_steps_of_v_that_grow_along_the_keys():
    """The reference of V's steps has to move: later keys' values are 2^20 times the first ones'."""
    rng = np.random.default_rng(0)
    d, page, ctx = 128, 16, [640]
    table, nb = random_table(rng, ctx, page)
    cache = ea.attn_kv4_cache(nb, 1, page, d)
    k = _q(rng, 640, 1, d)
    v = (_q(rng, 640, 1, d).float() * torch.exp2(torch.arange(640, device="cuda") / 32)[:, None, None]).to(torch.bfloat16)
    t = np.arange(640)
    ea.attn_kv4_append(k, v, cache, i32(table[0, t // page] * page + t % page))
    q = _q(rng, 1, 4, d)
    o, lse = ea.attn_fwd_kv4(q, cache, i32(table), i32(ctx))
    ks, vs = held(cache, ctx, table, page)
    check(o, lse, q, ks, vs, [0, 1], ctx, default_scale(d), True)


def test_strides_other_streams_and_rows_behind_the_last_request():
    rng = np.random.default_rng(3)
    d, page, Hq, Hk, ctx, nq = 128, 32, 6, 2, [77, 200], [2, 1]
    table, nb = random_table(rng, ctx, page)
    cache = filled_cache(rng, ctx, table, nb, Hk, d, page)
    cu = np.array([0, 2, 3])
    wide = _q(rng, 5, Hq + 4, d)
    q = wide[:, 2:2 + Hq]
    room = torch.full((5, Hq, d + 8), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((Hq, 5), 3.0, device="cuda")
    ea.attn_fwd_kv4(q, cache, i32(table), i32(ctx), i32(cu), 2, o=room[..., :d], lse=lse)
    ks, vs = held(cache, ctx, table, page)
    check(room[:, :, :d], lse, q, ks, vs, cu, ctx, default_scale(d), True)
    assert (room[3:] == 3).all() and (room[..., d:] == 3).all() and (lse[:, 3:] == 3).all()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    o2, lse2 = ea.attn_fwd_kv4(q, cache, i32(table), i32(ctx), i32(cu), 2, stream=s)
    torch.cuda.synchronize()
    s.synchronize()
    assert torch.equal(o2[:3], room[:3, :, :d]) and torch.equal(lse2[:, :3], lse[:, :3])
    none, _ = ea.attn_fwd_kv4(q[:0], cache, i32(table), i32(ctx), i32([0, 0, 0]), 1)
    assert none.shape == (0, Hq, d)


def test_a_token_that_is_not_finite_spoils_only_the_rows_that_see_it():
    rng = np.random.default_rng(4)
    d, page, ctx = 128, 16, [40]
    table, nb = random_table(rng, ctx, page)
    for which in (0, 1):
        kv = [_q(rng, 40, 1, d), _q(rng, 40, 1, d)]
        kv[which][39, 0, 3] = float("nan")
        cache = ea.attn_kv4_cache(nb, 1, page, d)
        t = np.arange(40)
        ea.attn_kv4_append(*kv, cache, i32(table[0, t // page] * page + t % page))
        q = _q(rng, 3, 2, d)
        o, _ = ea.attn_fwd_kv4(q, cache, i32(table), i32(ctx), i32([0, 3]), 3)
        assert torch.isfinite(o[:2]).all()
        assert torch.isnan(o[2]).all() if which == 0 else torch.isnan(o[2, :, :64]).all()


def test_tables_and_lengths_out_of_range_are_reported():
    rng = np.random.default_rng(5)
    d, page, Hq, Hk, ctx = 64, 16, 4, 2, [50, 60, 20]
    table, nb = random_table(rng, ctx, page)
    cache = filled_cache(rng, ctx, table, nb, Hk, d, page)
    q = _q(rng, 3, Hq, d)
    good, _ = ea.attn_fwd_kv4(q, cache, i32(table), i32(ctx))
    for entry in (-1, nb, 2 ** 31 - 1):
        t = table.copy()
        t[1, 3] = entry  # keys 48 .. 59 of request 1 are left out
        o, _ = ea.attn_fwd_kv4(q, cache, i32(t), i32(ctx))
        assert ea.attn_device_status() == ea.ATTN_ERR_INVALID_ARG
        assert torch.equal(o[0], good[0]) and torch.equal(o[2], good[2])
        short, _ = ea.attn_fwd_kv4(q, cache, i32(table), i32([50, 48, 20]))
        assert torch.allclose(o[1].float(), short[1].float(), atol=0.02, rtol=0.02)
    for lens, cu in (([50, -1, 20], [0, 1, 2, 3]), ([50, 10 ** 6, 20], [0, 1, 2, 3]), (ctx, [0, 1, 0, 3]), (ctx, [0, 1, 9, 3])):
        o = torch.full((3, Hq, d), 9.0, dtype=torch.bfloat16, device="cuda")
        ea.attn_fwd_kv4(q, cache, i32(table), i32(lens), i32(cu), 1, o=o)
        assert ea.attn_device_status() == ea.ATTN_ERR_INVALID_ARG
        # the batch's keys are split elsewhere: two results within the same bounds
        assert torch.allclose(o[0].float(), good[0].float(), atol=0.02, rtol=0.02) and (o[1] == 9).all()
    assert ea.attn_device_status() == ea.ATTN_OK


def test_results_repeat():
    q, cache, table, cu, signs, o, lse = _run([3000, 100, 900], [1, 1, 1], 8, 2, 128, 64, True, True, 11)
    again = ea.attn_fwd_kv4(q, cache, i32(table), i32([3000, 100, 900]), i32(cu), 1, signs=signs)
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)


@pytest.mark.parametrize("seed", range(12))
def test_random_shapes(seed):
    rng = np.random.default_rng(100 + seed)
    B, Hk, G = int(rng.integers(1, 6)), int(rng.choice([1, 2, 3])), int(rng.choice([1, 2, 3, 5, 8, 11]))
    nq = rng.integers(0, int(rng.choice([2, 4, 40])) + 1, B)
    nq[0] = max(nq[0], 1)
    ctx = [int(x) for x in rng.integers(0, int(rng.choice([20, 300, 1500])), B)]
    _run(ctx, nq, Hk * G, Hk, int(rng.choice([64, 128, 256])), int(rng.choice([16, 48, 64, 128])), bool(rng.integers(2)),
         bool(rng.integers(2)), seed)


@pytest.mark.parametrize("d,Hq,Hk,B", [(64, 3, 1, 1100), (128, 4, 2, 900), (128, 9, 1, 500), (256, 2, 1, 700)])
def test_more_requests_than_threads(d, Hq, Hk, B):
    """Several requests per thread of the pass that cuts the work into spans, many of them without keys or queries."""
    rng = np.random.default_rng(d)
    ctx = [int(x) for x in rng.integers(0, 50, B) * rng.integers(0, 2, B)]
    _run(ctx, rng.integers(0, 3, B), Hq, Hk, d, 16, True, d == 128, seed=d)


@pytest.mark.parametrize("d,G", [(64, 1), (64, 12), (128, 4), (128, 12), (256, 3)])
def test_one_request_over_every_span(d, G):
    """A chunk of rows whose parts are more than the join looks over at once, with a short request on either side."""
    _run([3, 90000, 40], [1, 1, 1], G, 1, d, 64, True, True, seed=d + G)


@pytest.mark.parametrize("bound", [1, 200])
def test_a_batch_without_queries(bound):
    rng = np.random.default_rng(0)
    table, nb = random_table(rng, [40, 20], 16)
    cache = filled_cache(rng, [40, 20], table, nb, 1, 128, 16)
    o, lse = torch.full((3, 2, 128), 5.0, dtype=torch.bfloat16, device="cuda"), torch.full((2, 3), 5.0, device="cuda")
    ea.attn_fwd_kv4(_q(rng, 3, 2, 128), cache, i32(table), i32([40, 20]), i32([0, 0, 0]), bound, o=o, lse=lse)
    assert ea.attn_device_status() == ea.ATTN_OK and (o == 5).all() and (lse == 5).all()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("nq", [[1, 2, 1], [100, 1, 70]])
def test_blocks_of_many_tokens(d, nq):
    _run([5000, 3, 4097], nq, 4, 2, d, 4096, True, True, seed=d)


def test_binding_refuses_shapes_of_no_sense():
    q, table, lens = torch.zeros(1, 2, 64, device="cuda", dtype=torch.bfloat16), i32([[0]]), i32([1])
    good = ea.attn_kv4_cache(1, 1, 16, 64)
    before = ea.attn_num_kernel_launches()
    for cache in (good[:, :0], good[:0], good[..., :17], good[0], good.float(), good.cpu()):
        with pytest.raises((ValueError, ea.AttnError)):
            ea.attn_fwd_kv4(q, cache, table, lens)
        with pytest.raises((ValueError, ea.AttnError)):
            ea.attn_kv4_append(q[:, :1], q[:, :1], cache, i32([0]))
        with pytest.raises((ValueError, ea.AttnError)):
            ea.attn_kv4_read(cache, i32([0]))
    for bad in (q[0], q[0, 0, 0], q[:, :0], q.float(), q[..., :32], q[..., ::2]):
        with pytest.raises((ValueError, ea.AttnError)):
            ea.attn_fwd_kv4(bad, good, table, lens)
        with pytest.raises((ValueError, ea.AttnError)):
            ea.attn_kv4_append(bad, bad, good, i32([0]))
    assert ea.attn_num_kernel_launches() == before
