"""attn_fwd_kv4 on requests of many rows (the tensor-memory kernel) and on batches that mix them with
requests of few rows; bounds as derived in kv_util.bounds."""

import numpy as np
import pytest
import torch

import exact_attention_100_b200 as ea
from exact_attention_100_b200 import build as ea_build
from exact_attention_100_b200.inputs import hadamard_signs
from kv_util import check, default_scale, filled_cache, held, i32, random_table
from test_gpu_kv4_attn import _q, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ea_build.build()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("transform", [False, True])
@pytest.mark.parametrize("ctx,nq,Hq,Hk,page", [
    ([40], [40], 1, 1, 16), ([128], [128], 2, 2, 16), ([300], [100], 4, 1, 48), ([129, 640], [33, 129], 3, 3, 64),
    ([257], [257], 2, 1, 16), ([700, 5, 90, 1], [70, 1, 40, 1], 8, 2, 32), ([1500, 600], [40, 300], 6, 2, 128)])
def test_matches_the_oracle(d, transform, ctx, nq, Hq, Hk, page):
    _run(ctx, nq, Hq, Hk, d, page, True, transform, seed=sum(ctx) + d)


@pytest.mark.parametrize("d,rows", [(64, 64), (64, 66), (128, 48), (128, 50), (256, 32), (256, 34)])
def test_requests_on_both_sides_of_the_choice_of_kernel(d, rows):
    _run([rows, 210, 77], [rows // 2, rows // 2, 1], 4, 2, d, 16, True, True, seed=rows)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_without_the_causal_mask(d):
    _run([333, 1], [150, 40], 4, 2, d, 16, causal=False, transform=True, seed=d)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_rows_that_see_no_key(d):
    _, _, _, _, _, o, lse = _run([0, 30, 200], [50, 170, 60], 4, 2, d, 16, seed=d)
    assert (o[:50] == 0).all() and torch.isneginf(lse[:, :50]).all()
    assert (o[50:190] == 0).all() and (o[190] != 0).any()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_std,k_std,v_std,scale", [(1e-3, 1e3, 1e-6, None), (30.0, 1.0, 1e5, None), (1.0, 1.0, 1e-25, None),
                                                     (1e-20, 1e20, 1.0, None), (4.0, 4.0, 1.0, 1.0)])
def test_values_of_any_size(d, q_std, k_std, v_std, scale):
    _run([500], [60], 4, 2, d, 16, True, True, 7, q_std, k_std, v_std, scale)


@pytest.mark.parametrize("down", [False, True])
def test_sizes_of_v_and_k_that_change_along_the_keys(down):
    rng = np.random.default_rng(0)
    d, page, n, nq = 128, 16, 640, 40
    table, nb = random_table(rng, [n], page)
    cache = ea.attn_kv4_cache(nb, 1, page, d)
    t = np.arange(n)
    size = torch.exp2((torch.arange(n, device="cuda") // 64 - 5.0) * (-3 if down else 3))[:, None, None]
    k = (_q(rng, n, 1, d).float() * size.pow(0.1)).to(torch.bfloat16)
    v = (_q(rng, n, 1, d).float() * size).to(torch.bfloat16)
    ea.attn_kv4_append(k, v, cache, i32(table[0, t // page] * page + t % page))
    q = _q(rng, nq, 4, d)
    o, lse = ea.attn_fwd_kv4(q, cache, i32(table), i32([n]), i32([0, nq]), nq)
    ks, vs = held(cache, [n], table, page)
    check(o, lse, q, ks, vs, [0, nq], [n], default_scale(d), True)


def test_a_token_that_is_not_finite_spoils_only_the_rows_that_see_it():
    rng = np.random.default_rng(4)
    d, page, n, nq = 128, 16, 140, 40
    table, nb = random_table(rng, [n], page)
    t = np.arange(n)
    for which in (0, 1):
        kv = [_q(rng, n, 1, d), _q(rng, n, 1, d)]
        kv[which][n - 10, 0, 3] = float("inf")
        cache = ea.attn_kv4_cache(nb, 1, page, d)
        ea.attn_kv4_append(*kv, cache, i32(table[0, t // page] * page + t % page))
        o, _ = ea.attn_fwd_kv4(_q(rng, nq, 2, d), cache, i32(table), i32([n]), i32([0, nq]), nq)
        assert torch.isfinite(o[:nq - 10]).all() and torch.isnan(o[nq - 10:, :, :64]).all()


def test_strides_and_rows_behind_the_last_request():
    rng = np.random.default_rng(3)
    d, page, Hq, Hk, ctx, nq = 128, 32, 6, 2, [77, 200, 30], [50, 13, 1]
    table, nb = random_table(rng, ctx, page)
    cache = filled_cache(rng, ctx, table, nb, Hk, d, page)
    cu = np.concatenate([[0], np.cumsum(nq)])
    rows = int(cu[-1])
    wide = _q(rng, rows + 3, Hq + 4, d)
    room = torch.full((rows + 3, Hq, d + 8), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((Hq, rows + 3), 3.0, device="cuda")
    ea.attn_fwd_kv4(wide[:, 2:2 + Hq], cache, i32(table), i32(ctx), i32(cu), 50, o=room[..., :d], lse=lse)
    ks, vs = held(cache, ctx, table, page)
    check(room[:, :, :d], lse, wide[:, 2:2 + Hq], ks, vs, cu, ctx, default_scale(d), True)
    assert (room[rows:] == 3).all() and (room[..., d:] == 3).all() and (lse[:, rows:] == 3).all()


def test_a_bound_on_the_queries_that_is_too_large_changes_nothing():
    """max_seqlen_q only bounds: one request, or several, of few rows under a large bound."""
    rng = np.random.default_rng(6)
    for ctx, nq in (([90], [2]), ([90, 33], [2, 1])):
        table, nb = random_table(rng, ctx, 16)
        cache = filled_cache(rng, ctx, table, nb, 2, 64, 16)
        cu = np.concatenate([[0], np.cumsum(nq)])
        q = _q(rng, int(cu[-1]), 4, 64)
        ks, vs = held(cache, ctx, table, 16)
        for bound in (2, 3, 1000):
            o, lse = ea.attn_fwd_kv4(q, cache, i32(table), i32(ctx), i32(cu), bound)
            assert ea.attn_device_status() == ea.ATTN_OK
            if bound < 1000 or len(ctx) > 1:
                check(o, lse, q, ks, vs, cu, ctx, 0.125, True)
            assert torch.isfinite(o).all()


def test_tables_and_lengths_out_of_range_are_reported():
    rng = np.random.default_rng(5)
    d, page, Hq, Hk, ctx, nq = 64, 16, 4, 2, [300, 260, 200], [40, 50, 60]
    table, nb = random_table(rng, ctx, page)
    cache = filled_cache(rng, ctx, table, nb, Hk, d, page)
    cu = np.concatenate([[0], np.cumsum(nq)])
    q = _q(rng, 150, Hq, d)
    good, _ = ea.attn_fwd_kv4(q, cache, i32(table), i32(ctx), i32(cu), 60)
    near = lambda a, b: torch.allclose(a.float(), b.float(), atol=0.02, rtol=0.02)
    for entry in (-1, nb, 2 ** 31 - 1):
        t = table.copy()
        t[1, 3] = entry  # keys 48 .. 63 of request 1 are left out
        o, lse = ea.attn_fwd_kv4(q, cache, i32(t), i32(ctx), i32(cu), 60)
        assert ea.attn_device_status() == ea.ATTN_ERR_INVALID_ARG
        assert near(o[:40], good[:40]) and near(o[90:], good[90:])
        ks, vs = held(cache, ctx, table, page)
        keep = np.r_[0:48, 64:260]
        check(o[40:90], lse[:, 40:90], q[40:90], [ks[1][keep]], [vs[1][keep]], [0, 50], [244], default_scale(d), True)
    for lens, cu2 in (([300, -1, 200], cu), ([300, 10 ** 6, 200], cu), (ctx, [0, 40, 1000, 150]), (ctx, [0, 40, 101, 150])):
        o = torch.full((150, Hq, d), 9.0, dtype=torch.bfloat16, device="cuda")
        ea.attn_fwd_kv4(q, cache, i32(table), i32(lens), i32(cu2), 60, o=o)
        assert ea.attn_device_status() == ea.ATTN_ERR_INVALID_ARG
        assert near(o[:40], good[:40]) and (o[40:90] == 9).all()
    assert ea.attn_device_status() == ea.ATTN_OK


def test_results_repeat_and_replay():
    q, cache, table, cu, signs, o, lse = _run([900, 100, 400], [300, 1, 50], 8, 2, 128, 64, True, True, 11)
    args = (q, cache, i32(table), i32([900, 100, 400]), i32(cu), 300)
    again = ea.attn_fwd_kv4(*args, signs=signs)
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c, _ = ea.attn_fwd_kv4(*args, signs=signs)
    graph.replay()
    assert torch.equal(c, o)


@pytest.mark.parametrize("seed", range(8))
def test_random_shapes(seed):
    rng = np.random.default_rng(200 + seed)
    B, Hk, G = int(rng.integers(1, 5)), int(rng.choice([1, 2, 3])), int(rng.choice([1, 2, 3, 5, 8]))
    nq = rng.integers(0, int(rng.choice([40, 150, 300])) + 1, B)
    nq[0] = max(nq[0], 1)
    ctx = [int(x) for x in rng.integers(0, int(rng.choice([60, 300, 900])), B)]
    _run(ctx, nq, Hk * G, Hk, int(rng.choice([64, 128])), int(rng.choice([16, 48, 64, 128])), bool(rng.integers(2)),
         bool(rng.integers(2)), seed)
