"""attn_kv_tables against the request-by-request form (whole numbers: equal)."""

import numpy as np
import pytest
import torch

import exact_attention_100_b200 as ea
from exact_attention_100_b200 import build as ea_build
from kv_util import i32
from oracle import tables_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ea_build.build()


def _inputs(seed, B, len_hi, new_hi, page, cursor=2, short=0):
    rng = np.random.default_rng(seed)
    lens, new = rng.integers(0, len_hi + 1, B), rng.integers(0, new_hi + 1, B)
    held, want = -(-lens // page), -(-(lens + new) // page)
    width = int(want.max()) + 2
    order = rng.permutation(int(want.sum()) + cursor + 3)
    table = np.full((B, width), -1)
    at = 0
    for b in range(B):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    free = order[at:]
    free = free[:len(free) - short] if short else free
    return lens, new, table, free, cursor


def _same(got, want):
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1))


@pytest.mark.parametrize("B,len_hi,new_hi,page", [(1, 0, 1, 16), (1, 100, 5000, 16), (3, 40, 0, 64), (37, 500, 1, 16),
                                                  (255, 1000, 60, 48), (512, 300, 700, 128), (513, 9, 33, 16),
                                                  (8192, 20, 3, 32)])
def test_matches_the_plain_form(B, len_hi, new_hi, page):
    lens, new, table, free, cursor = _inputs(B + page, B, len_hi, new_hi, page)
    for extra in (0, 5):
        total = int(new.sum()) + extra
        want = tables_ref(lens, new, table, free, cursor, page, total)
        got = ea.attn_kv_tables(i32(lens), i32(new), i32(table), i32(free), i32([cursor]), page, total)
        _same(got, want)
    assert ea.attn_device_status() == ea.ATTN_OK


@pytest.mark.parametrize("B,new_hi", [(5, 3), (200, 40), (64, 900)])
def test_in_place_over_several_steps(B, new_hi):
    page = 16
    lens, new, table, free, cursor = _inputs(B, B, 100, new_hi, page)
    free = np.concatenate([free, 100000 + np.arange(3 * (int(new.sum()) // page + B))])
    dl, dt, df, dc = i32(lens), i32(np.pad(table, ((0, 0), (0, 3 * (new_hi // page + 1))), constant_values=-1)), i32(free), i32([cursor])
    table = dt.cpu().numpy()
    for _ in range(3):
        want = tables_ref(lens, new, table, free, cursor, page, int(new.sum()))
        got = ea.attn_kv_tables(dl, i32(new), dt, df, dc, page, int(new.sum()), lens_out=dl, cursor_out=dc)
        _same(got, want)
        assert got[3].data_ptr() == dl.data_ptr() and got[5].data_ptr() == dt.data_ptr()
        lens, cursor, table = want[3], want[4], want[5]
    assert ea.attn_device_status() == ea.ATTN_OK


def test_requests_without_blocks_are_not_served():
    page = 16
    for short in (5, 12, 10 ** 6):  # three blocks more than needed are there
        lens, new, table, free, cursor = _inputs(3, 60, 90, 50, page, cursor=0, short=min(short, 60))
        if short == 10 ** 6:
            free = free[:0]
        want = tables_ref(lens, new, table, free, 0, page, int(new.sum()))
        got = ea.attn_kv_tables(i32(lens), i32(new), i32(table), i32(free), i32([0]), page, int(new.sum()))
        _same(got, want)
        assert (want[3] != lens + new).any()
    assert ea.attn_device_status() == ea.ATTN_OK


def test_lengths_out_of_range_are_reported_and_not_served():
    page, table = 16, np.arange(12).reshape(3, 4)
    free = i32(np.arange(100, 120))
    for lens, new, total, cu, out in [([5, -1, 7], [3, 2, 1], 10, [0, 3, 3, 4], [8, -1, 8]),
                                      ([5, 6, 7], [3, -2, 1], 10, [0, 3, 3, 4], [8, 6, 8]),
                                      ([5, 60, 7], [3, 5, 1], 10, [0, 3, 3, 4], [8, 60, 8]),
                                      ([5, 6, 7], [3, 2 ** 31 - 1, 1], 10, [0, 3, 3, 4], [8, 6, 8]),
                                      ([5, 6, 7], [3, 9, 1], 10, [0, 3, 10, 10], [8, 6, 7])]:
        slots, pos, c, lo, cur, _ = ea.attn_kv_tables(i32(lens), i32(new), i32(table), free, i32([4]), page, total)
        assert ea.attn_device_status() == ea.ATTN_ERR_INVALID_ARG
        assert c.tolist() == cu and lo.tolist() == out and cur.item() == 4
        assert slots[:3].tolist() == [5, 6, 7]
    for cursor in (-1, 21):
        slots, _, _, lo, cur, _ = ea.attn_kv_tables(i32([16, 3]), i32([1, 1]), i32([[1, -1], [2, -1]]), free, i32([cursor]), page, 2)
        assert ea.attn_device_status() == ea.ATTN_ERR_INVALID_ARG
        assert slots.tolist() == [-1, 35] and lo.tolist() == [16, 4] and cur.item() == cursor
    # a request whose own table misses a block
    slots = ea.attn_kv_tables(i32([3]), i32([1]), i32([[-1]]), free, i32([0]), page, 1)[0]
    assert slots.tolist() == [-1] and ea.attn_device_status() == ea.ATTN_ERR_INVALID_ARG
    assert ea.attn_device_status() == ea.ATTN_OK


def test_no_new_tokens_and_no_free_blocks():
    got = ea.attn_kv_tables(i32([3, 0]), i32([0, 0]), i32([[4], [-1]]), i32(np.zeros(0)), i32([0]), 16, 0)
    assert [t.tolist() for t in got] == [[], [], [0, 0, 0], [3, 0], [0], [[4], [-1]]]
    assert ea.attn_device_status() == ea.ATTN_OK
