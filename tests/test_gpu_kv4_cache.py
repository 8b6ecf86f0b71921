"""attn_kv4_append and attn_kv4_read against the float32 definition (equal) and byte by byte."""

import numpy as np
import pytest
import torch

import exact_attention_100_b200 as ea
from exact_attention_100_b200 import build as ea_build
from exact_attention_100_b200.inputs import hadamard_signs
from kv_util import i32
from oracle.kv4 import quantise, read_token, transformed, values, write_token

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ea_build.build()


def _kv(seed, T, Hk, d, std=1.0):
    rng = np.random.default_rng(seed)
    return [torch.from_numpy((rng.standard_normal((T, Hk, d)) * std).astype(np.float32)).cuda().to(torch.bfloat16)
            for _ in range(2)]


@pytest.mark.parametrize("T,Hk,d,page,transform,std", [
    (1, 1, 64, 16, False, 1.0), (1, 1, 128, 16, True, 1.0), (1, 1, 256, 16, True, 1.0), (17, 3, 64, 48, True, 1.0),
    (33, 2, 128, 64, False, 1e-3), (40, 5, 256, 32, False, 1.0), (70, 4, 128, 4096, True, 30.0),
    (9, 2, 128, 16, True, 1e-38), (9, 2, 128, 16, True, 1e36), (300, 8, 128, 16, True, 1.0)])
def test_codes_scales_and_places(T, Hk, d, page, transform, std):
    k, v = _kv(T + d, T, Hk, d, std)
    signs = hadamard_signs(d)
    nb = -(-T // page) + 2
    slots = np.random.default_rng(1).permutation(nb * page)[:T]
    cache = ea.attn_kv4_cache(nb, Hk, page, d)
    cache.fill_(0x5A)
    want = cache.cpu().numpy()
    ea.attn_kv4_append(k, v, cache, i32(slots), signs=torch.from_numpy(signs).cuda() if transform else None)
    kq = quantise(transformed(k.float().cpu().numpy(), signs if transform else None))
    vq = quantise(v.float().cpu().numpy())
    some = range(T) if T <= 40 else range(0, T, 7)
    got = cache.cpu().numpy()
    for t in some:
        for h in range(Hk):
            write_token(want, page, int(slots[t]), h, *(a[t, h] for a in kq), *(a[t, h] for a in vq))
    if T <= 40:
        assert np.array_equal(got, want)  # every byte, the untouched ones too
    rk, rv = ea.attn_kv4_read(cache, i32(slots), dtype=torch.float32)
    for r, q, i in ((rk, kq, 0), (rv, vq, 1)):
        # u s + z in float64, rounded once
        assert np.array_equal(r.cpu().numpy(), values(*q).astype(np.float32))
        for t in list(some)[:5]:
            assert np.array_equal(read_token(got, page, int(slots[t]), 0)[i], values(*(a[t, 0] for a in q)))
    bk, bv = ea.attn_kv4_read(cache, i32(slots))
    assert torch.equal(bk, rk.to(torch.bfloat16)) and torch.equal(bv, rv.to(torch.bfloat16))
    assert ea.attn_device_status() == ea.ATTN_OK


def test_strided_views_of_a_fused_projection():
    T, Hq, Hk, d, page = 50, 6, 2, 128, 16
    g = torch.Generator(device="cuda").manual_seed(0)
    qkv = torch.randn(T, Hq + 2 * Hk, d, device="cuda", generator=g).to(torch.bfloat16)
    slots = i32(np.arange(T))
    a, b = ea.attn_kv4_cache(5, Hk, page, d), ea.attn_kv4_cache(5, Hk, page, d)
    ea.attn_kv4_append(qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:], a, slots)
    ea.attn_kv4_append(qkv[:, Hq:Hq + Hk].contiguous(), qkv[:, Hq + Hk:].contiguous(), b, slots)
    assert torch.equal(a, b)
    one = ea.attn_kv4_cache(5, 1, page, d)  # one head: its head stride is not used
    ea.attn_kv4_append(qkv[:, Hq:Hq + 1], qkv[:, -1:], one, slots)
    assert torch.equal(ea.attn_kv4_read(one, slots)[0][:, 0], ea.attn_kv4_read(a, slots)[0][:, 0])


@pytest.mark.parametrize("d", [64, 128, 256])
def test_many_tokens_at_once(d):
    """As many rows as make a thread take several of them, the last ones ragged: the same as in small calls."""
    T, Hk, page = 20011, 4, 64
    wide = _kv(d, T, Hk + 1, d, 3.0)
    k, v = wide[0][:, 1:], wide[1][:, :Hk]
    signs = torch.from_numpy(hadamard_signs(d)).cuda()
    slots = np.random.default_rng(d).permutation((T // page + 3) * page)[:T]
    slots[::17] = -1
    a, b = ea.attn_kv4_cache(T // page + 3, Hk, page, d), ea.attn_kv4_cache(T // page + 3, Hk, page, d)
    ea.attn_kv4_append(k, v, a, i32(slots), signs=signs)
    for i in range(0, T, 1000):
        ea.attn_kv4_append(k[i:i + 1000], v[i:i + 1000], b, i32(slots[i:i + 1000]), signs=signs)
    assert torch.equal(a, b) and a.any()
    big = ea.attn_kv4_read(a, i32(slots), dtype=torch.float32)
    for i in range(0, T, 5000):
        small = ea.attn_kv4_read(a, i32(slots[i:i + 5000]), dtype=torch.float32)
        assert all(torch.equal(x[i:i + 5000], y) for x, y in zip(big, small))
    assert (big[0][::17] == 0).all() and ea.attn_device_status() == ea.ATTN_OK


def test_slots_of_nobody_and_slots_out_of_range():
    Hk, d, page, nb = 2, 64, 16, 2
    k, v = _kv(5, 6, Hk, d)
    cache = ea.attn_kv4_cache(nb, Hk, page, d)
    ea.attn_kv4_append(k, v, cache, i32([-1, 3, -1, 31, -1, -1]))
    assert ea.attn_device_status() == ea.ATTN_OK
    rk, rv = ea.attn_kv4_read(cache, i32([3, -1, 31, 3, 0]), dtype=torch.float32)
    assert torch.equal(rk[0], rk[3]) and (rk[1] == 0).all() and (rv[4] == 0).all() and (rk[2] != 0).any()
    assert ea.attn_device_status() == ea.ATTN_OK
    for bad in (32, -2, 2 ** 31 - 1, -2 ** 31):
        before = cache.clone()
        ea.attn_kv4_append(k[:1], v[:1], cache, i32([bad]))
        assert ea.attn_device_status() == ea.ATTN_ERR_INVALID_ARG and torch.equal(cache, before)
        assert (ea.attn_kv4_read(cache, i32([bad]))[0] == 0).all()
        assert ea.attn_device_status() == ea.ATTN_ERR_INVALID_ARG
    ea.attn_kv4_append(k[:0], v[:0], cache, i32(np.zeros(0)))
    assert ea.attn_kv4_read(cache, i32(np.zeros(0)))[0].shape == (0, Hk, d)


def test_constant_zero_and_not_finite_groups():
    k, v = (torch.zeros(4, 1, 128, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    k[1] = 2.5
    v[2, 0, 5], v[3, 0, 70] = float("inf"), float("nan")
    cache = ea.attn_kv4_cache(1, 1, 16, 128)
    ea.attn_kv4_append(k, v, cache, i32(np.arange(4)))
    rk, rv = ea.attn_kv4_read(cache, i32(np.arange(4)), dtype=torch.float32)
    assert torch.equal(rk, k.float())
    nan = torch.isnan(rv[:, 0])
    assert nan[2, :64].all() and not nan[2, 64:].any() and nan[3, 64:].all() and not nan[3, :64].any()
    assert ea.attn_device_status() == ea.ATTN_OK


def test_offsets_past_32_bits():
    """A cache of 5 GB: its last block lies past 2^32 bytes."""
    Hk, d, page = 8, 128, 64
    nb = (5 << 30) // (Hk * page // 16 * 18 * d)
    cache = torch.empty(nb, Hk, page // 16, 18 * d, dtype=torch.uint8, device="cuda")
    k, v = _kv(8, 3, Hk, d)
    slots = i32([0, nb * page // 2, nb * page - 1])
    ea.attn_kv4_append(k, v, cache, slots)
    rk, rv = ea.attn_kv4_read(cache, slots, dtype=torch.float32)
    assert np.array_equal(rk.cpu().numpy(), values(*quantise(k.float().cpu().numpy())).astype(np.float32))
    q = torch.randn(1, Hk, d, device="cuda").to(torch.bfloat16)
    table = i32([[nb - 1]])
    cache[nb - 1] = 0
    ea.attn_kv4_append(k[:1], v[:1], cache, i32([(nb - 1) * page]))
    o, _ = ea.attn_fwd_kv4(q, cache, table, i32([1]))  # one key: O is its V
    want = ea.attn_kv4_read(cache, i32([(nb - 1) * page]), dtype=torch.float32)[1]
    # p = 1; p s in float16 (2^-11 of 15 steps, under the range), then bf16
    tol = 2.0 ** -11 * 2 * want.abs().max() + 2.0 ** -8 * want.abs()
    assert ((o.float() - want).abs() <= tol).all()
    assert ea.attn_device_status() == ea.ATTN_OK
