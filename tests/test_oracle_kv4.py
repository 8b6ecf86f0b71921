"""Pins of the float64 forms in ``oracle.kv4``: hand-worked values, invariants, and other ways to the
same result."""

import math

import numpy as np
import pytest

from exact_attention_100_b200.inputs import hadamard_signs, round_to_bf16, rope_tables
from oracle import attention_kv4_ref, attention_ref, rope_axes_ref, rope_ref, tables_ref
from oracle.kv4 import bf16_down, code_place, hadamard_f64, quantise, read_token, transformed, values, write_token


def test_bf16_down_by_hand_and_by_rounding():
    x = np.array([1.0, 1.001, -1.001, 0.0, -0.0, 3.0e-40, -3.0e-40], dtype=np.float32)
    assert bf16_down(x)[:2].tolist() == [1.0, 1.0]
    assert bf16_down(x)[2] == np.float32(-1.0078125)
    r = np.random.default_rng(0).standard_normal(4096).astype(np.float32)
    y = bf16_down(r)
    assert np.array_equal(y, round_to_bf16(y)) and (y <= r).all() and (r - y <= np.abs(r) * 2.0 ** -7).all()


def test_quantise_by_hand():
    x = np.zeros((1, 64), dtype=np.float32)
    x[0, :16] = np.arange(16) - 4
    u, s, z = quantise(x)
    assert s[0, 0] == 1.0 and z[0, 0] == -4.0
    assert u[0, :16].tolist() == list(range(16)) and (u[0, 16:] == 4).all()
    u, s, z = quantise(np.full((1, 64), 2.5, dtype=np.float32))
    assert s[0, 0] == 0 and z[0, 0] == 2.5 and (u == 0).all()


@pytest.mark.parametrize("scale", [1e-38, 1e-3, 1.0, 1e30])
def test_values_lie_within_half_a_step(scale):
    x = round_to_bf16((np.random.default_rng(3).standard_normal((50, 128)) * scale).astype(np.float32))
    u, s, z = quantise(x)
    err = np.abs(values(u, s, z) - x)
    # half a step, and the float32 roundings of (x - z) / s: three of 2^-24 of at most 15 steps
    assert (err <= np.repeat(s, 64, -1) * (0.5 + 15 * 3 * 2.0 ** -24)).all()


def test_values_not_finite_spoil_their_group_only():
    x = np.ones((1, 128), dtype=np.float32)
    x[0, 3] = np.inf
    v = values(*quantise(x))
    assert np.isnan(v[0, :64]).all() and (v[0, 64:] == 1).all()
    x = np.full((1, 64), 3e38, dtype=np.float32)
    x[0, 0] = -3e38  # the range is not finite
    assert np.isnan(values(*quantise(x))).all()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("is_v", [False, True])
def test_code_places_fill_the_codes_once(d, is_v):
    seen = {(at + row * step, odd) for x in range(d) for row in range(16) for at, step, odd in [code_place(d, x, is_v)]}
    assert seen == {(b, n) for b in range(8 * d) for n in (0, 1)}


@pytest.mark.parametrize("d", [64, 128, 256])
def test_cache_round_trip(d):
    rng = np.random.default_rng(d)
    page, Hk = 32, 2
    cache = np.full((3, Hk, 2, 18 * d), 0xAB, dtype=np.uint8)
    held = {}
    for slot in (0, 15, 16, 33, 95):
        for h in range(Hk):
            kq, vq = quantise(rng.standard_normal(d)), quantise(rng.standard_normal(d))
            write_token(cache, page, slot, h, *kq, *vq)
            held[slot, h] = values(*kq), values(*vq)
    for (slot, h), (k, v) in held.items():
        a, b = read_token(cache, page, slot, h)
        assert np.array_equal(a, k) and np.array_equal(b, v)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_transform_is_orthogonal_and_float32_form_is_near(d):
    signs = hadamard_signs(d)
    x = round_to_bf16(np.random.default_rng(1).standard_normal((20, d)).astype(np.float32))
    y = hadamard_f64(x, signs)
    assert np.allclose((y * y).sum(-1), (x.astype(np.float64) ** 2).sum(-1), rtol=1e-12)
    # log2 d + 1 roundings of at most 2^-24 of the running sums, whose size is at most sum |x| / sqrt d
    bound = (math.log2(d) + 1) * 2.0 ** -24 * np.abs(x).sum(-1, keepdims=True) / math.sqrt(d) * 2
    assert (np.abs(transformed(x, signs) - y) <= bound).all()


def test_attention_agrees_with_the_dense_definition():
    rng = np.random.default_rng(5)
    Hq, Hk, d, nq, n = 6, 2, 64, 5, 40
    q, k, v = rng.standard_normal((nq, Hq, d)), rng.standard_normal((n, Hk, d)), rng.standard_normal((n, Hk, d))
    o, lse = attention_kv4_ref(q, [k], [v], [0, nq], [n], 0.2, True)
    for h in range(Hq):
        for i in range(nq):
            seen = n - nq + i + 1
            o2, l2 = attention_ref(q[None, None, i:i + 1, h], k[None, None, :seen, h // 3], v[None, None, :seen, h // 3], 0.2,
                                   False)
            assert np.allclose(o[i, h], o2[0, 0, 0], atol=1e-12) and abs(lse[h, i] - l2[0, 0, 0]) < 1e-12


def test_attention_rows_without_keys_and_rows_of_nobody():
    q = np.ones((4, 1, 64))
    o, lse = attention_kv4_ref(q, [np.ones((1, 1, 64))], [np.ones((1, 1, 64))], [0, 3], [1], 1.0, True)
    assert (o[:2] == 0).all() and np.isneginf(lse[0, :2]).all() and (o[2] == 1).all() and np.isnan(o[3]).all()


def test_rope_axes_with_one_axis_is_rope_and_its_inverse_undoes_it():
    cos, sin = rope_tables(50, 64)
    x = round_to_bf16(np.random.default_rng(2).standard_normal((50, 3, 64)).astype(np.float32))
    y = rope_axes_ref(x, cos, sin, np.arange(50)[None], [32])
    one = rope_ref(x.transpose(1, 0, 2)[None], cos, sin)[0].transpose(1, 0, 2)
    assert np.abs(y - one).max() <= 3 * 2.0 ** -24 * np.abs(x).max() * 2
    back = rope_axes_ref(y, cos, sin, np.arange(50)[None], [32], inverse=True)
    assert np.abs(back - x).max() < 1e-6  # the tables are float32: cos^2 + sin^2 is 1 to 2^-23


def test_rope_axes_gradient_by_differences():
    rng = np.random.default_rng(4)
    cos, sin = rope_tables(9, 32)
    pos, sections = rng.integers(0, 9, (3, 5)), [4, 8, 4]
    x, w = rng.standard_normal((5, 2, 40)), rng.standard_normal((5, 2, 40))
    grad = rope_axes_ref(w, cos, sin, pos, sections, inverse=True)
    f = lambda a: (rope_axes_ref(a, cos, sin, pos, sections) * w).sum()
    for at in [(0, 0, 0), (1, 1, 5), (2, 0, 17), (3, 1, 31), (4, 0, 39)]:
        e = np.zeros_like(x)
        e[at] = 1e-4
        assert abs((f(x + e) - f(x - e)) / 2e-4 - grad[at]) < 1e-9


def test_tables_by_hand():
    table = np.array([[7, -1, -1], [-1, -1, -1], [3, 4, -1]])
    slots, pos, cu, lens, cursor, out = tables_ref([10, 0, 32], [10, 3, 1], table, [9, 8, 5], 0, 16, 16)
    assert out.tolist() == [[7, 9, -1], [8, -1, -1], [3, 4, 5]] and cursor == 3
    assert cu.tolist() == [0, 10, 13, 14] and lens.tolist() == [20, 3, 33]
    assert slots.tolist() == [122, 123, 124, 125, 126, 127, 144, 145, 146, 147, 128, 129, 130, 80, -1, -1]
    assert pos.tolist() == [*range(10, 20), 0, 1, 2, 32, 0, 0]


def test_tables_out_of_blocks():
    table = np.full((3, 2), -1)
    slots, _, _, lens, cursor, out = tables_ref([0, 0, 0], [1, 20, 1], table, [5, 6], 0, 16, 22)
    assert cursor == 1 and lens.tolist() == [1, 0, 0]
    assert slots.tolist() == [80] + [-1] * 21 and out.tolist() == [[5, -1], [-1, -1], [-1, -1]]
