"""attn_rope_axes and its backward against the float64 form.

Tolerance: each product is rounded (2^-24 relative) and their sum (2^-24): at most 3 * 2^-24 (|a| + |b|)
with |cos|, |sin| <= 1; then half a step of the output type."""

import numpy as np
import pytest
import torch

import exact_attention_100_b200 as ea
from exact_attention_100_b200 import build as ea_build
from exact_attention_100_b200.inputs import rope_tables
from kv_util import i32
from oracle import rope_axes_ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ea_build.build()


def _tables(n_pos, half):
    cos, sin = rope_tables(n_pos, 2 * half)
    return torch.from_numpy(cos).cuda(), torch.from_numpy(sin).cuda()


def _check(x, y, cos, sin, pos, sections, inverse):
    half = sum(sections)
    xn = x.float().cpu().numpy()
    ref = rope_axes_ref(xn, cos.cpu().numpy(), sin.cpu().numpy(), pos.cpu().numpy(), sections, inverse)
    size = np.abs(xn).astype(np.float64)
    tol = np.zeros_like(size)
    tol[..., :half] = tol[..., half:2 * half] = 3 * 2.0 ** -24 * (size[..., :half] + size[..., half:2 * half])
    step = torch.finfo(y.dtype).eps / 2
    err = np.abs(y.float().cpu().numpy() - ref)
    assert (err <= tol + step * (np.abs(ref) + tol)).all(), (err - tol).max()


CASES = [  # tokens, Hq, Hk, d, sections, n_pos
    (1, 1, 1, 64, [32], 5), (7, 5, 2, 128, [16, 24, 24], 40), (130, 32, 8, 128, [64], 130), (33, 3, 3, 80, [20, 20], 9),
    (65, 4, 1, 72, [12, 12, 12], 70), (50, 2, 2, 256, [32, 48, 48], 100), (29, 4, 4, 96, [7, 11, 13, 5], 30),
    (12, 2, 1, 128, [8, 8], 12), (9, 6, 2, 64, [3, 1], 3), (300, 9, 3, 40, [4], 300), (5, 1, 1, 1024, [512], 6),
]


@pytest.mark.parametrize("T,Hq,Hk,d,sections,n_pos", CASES)
@pytest.mark.parametrize("ti,to", [(BF, BF), (F32, F32), (F32, BF), (BF, F32)])
def test_forward_and_backward(T, Hq, Hk, d, sections, n_pos, ti, to):
    g = torch.Generator(device="cuda").manual_seed(T + d)
    q, k = (torch.randn(T, h, d, device="cuda", generator=g).to(ti) for h in (Hq, Hk))
    cos, sin = _tables(n_pos, sum(sections))
    pos = torch.randint(0, n_pos, (len(sections), T), device="cuda", generator=g, dtype=torch.int32)
    for inverse, f in ((False, ea.attn_rope_axes), (True, ea.attn_rope_axes_bwd)):
        a, b = f(q, k, cos, sin, pos, sections, out_dtype=to)
        _check(q, a, cos, sin, pos, sections, inverse)
        _check(k, b, cos, sin, pos, sections, inverse)
        c, none = f(q, None, cos, sin, pos, sections, out_dtype=to)
        assert none is None and torch.equal(c, a)
    assert ea.attn_device_status() == ea.ATTN_OK


def test_gradient_by_differences():
    """Along any direction e, (f(x + e) - f(x - e)) / 2 . w = e . grad: f is linear, so only the float32
    roundings remain (sums over 2^13 products of unit size: 1e-3 is far above them)."""
    g = torch.Generator(device="cuda").manual_seed(0)
    cos, sin = _tables(50, 32)
    pos = torch.randint(0, 50, (3, 16), device="cuda", generator=g, dtype=torch.int32)
    x, w, e = (torch.randn(16, 8, 64, device="cuda", generator=g) for _ in range(3))
    run = lambda t: ea.attn_rope_axes(t, None, cos, sin, pos, [8, 12, 12])[0]
    grad = ea.attn_rope_axes_bwd(w, None, cos, sin, pos, [8, 12, 12])[0]
    diff = ((run(x + e) - run(x - e)).double() / 2 * w.double()).sum()
    assert abs(diff.item() - (e.double() * grad.double()).sum().item()) < 1e-3


@pytest.mark.parametrize("dt", [BF, F32])
def test_strides_orders_and_in_place(dt):
    B, H, N, d, sections = 2, 6, 37, 128, [16, 24, 24]
    g = torch.Generator(device="cuda").manual_seed(1)
    cos, sin = _tables(64, 64)
    qkv = torch.randn(B, N, 3, H, d, device="cuda", generator=g).to(dt)
    pos = torch.randint(0, 64, (3, B, N), device="cuda", generator=g, dtype=torch.int32)
    q, k = qkv[:, :, 0].transpose(1, 2), qkv[:, :, 1].transpose(1, 2)  # [B, H, N, d] views
    a, b = ea.attn_rope_axes(q, k, cos, sin, pos, sections)
    for bi in range(B):
        _check(q[bi].transpose(0, 1), a[bi].transpose(0, 1), cos, sin, pos[:, bi], sections, False)
    # packed views of one batch entry, written through the strides of another buffer
    room = torch.full((N, 2 * H, d + 8), 7.0, device="cuda", dtype=dt)
    c, e = ea.attn_rope_axes(qkv[0, :, 0], qkv[0, :, 1], cos, sin, pos[:, 0].contiguous(), sections,
                             q_out=room[:, ::2, :d], k_out=room[:, 1::2, :d])
    assert torch.equal(c, a[0].transpose(0, 1)) and torch.equal(e, b[0].transpose(0, 1))
    assert (room[..., d:] == 7).all()
    before = qkv.clone()
    ea.attn_rope_axes(q, k, cos, sin, pos, sections, q_out=q, k_out=k)
    assert torch.equal(q, a) and torch.equal(k, b) and torch.equal(qkv[:, :, 2], before[:, :, 2])
    assert ea.attn_device_status() == ea.ATTN_OK


def test_positions_out_of_range_are_reported():
    cos, sin = _tables(10, 32)
    q = torch.randn(4, 2, 64, device="cuda")
    pos = i32([[0, 9, 10, -1], [1, 2, 3, 4]])
    out = torch.full_like(q, 5.0)
    ea.attn_rope_axes(q, None, cos, sin, pos, [16, 16], q_out=out)
    assert ea.attn_device_status() == ea.ATTN_ERR_INVALID_ARG
    ok = ea.attn_rope_axes(q, None, cos, sin, i32([[0, 9, 0, 0], [1, 2, 3, 4]]), [16, 16])[0]
    assert torch.equal(out[:2], ok[:2]) and torch.equal(out[2:, :, 16:32], ok[2:, :, 16:32])
    assert (out[2:, :, :16] == 5).all() and (out[2:, :, 32:48] == 5).all()
    assert ea.attn_device_status() == ea.ATTN_OK


def test_no_tokens():
    cos, sin = _tables(10, 32)
    q = torch.zeros(0, 2, 64, device="cuda")
    assert ea.attn_rope_axes(q, q, cos, sin, i32(np.zeros((1, 0))), [32])[0].shape == (0, 2, 64)


@pytest.mark.parametrize("bad", [dict(sections=[30]), dict(sections=[16, 16]), dict(n=3), dict(out=F32)])
def test_binding_refuses(bad):
    cos, sin = _tables(10, 32)
    q = torch.zeros(4, 2, 64, device="cuda", dtype=BF)
    pos = i32(np.zeros((1, bad.get("n", 4))))
    before = ea.attn_num_kernel_launches()
    with pytest.raises((ValueError, ea.AttnError)):
        ea.attn_rope_axes(q, None, cos, sin, pos, bad.get("sections", [32]),
                          q_out=q.view(4, 2, 64)[:3] if "out" in bad else None)
    assert ea.attn_num_kernel_launches() == before


def test_binding_refuses_other_types_and_rows_that_overlap():
    cos, sin = _tables(10, 32)
    q, pos = torch.zeros(4, 2, 64, device="cuda", dtype=BF), i32(np.zeros((1, 4)))
    before = ea.attn_num_kernel_launches()
    for bad in (dict(out_dtype=torch.float16), dict(q_out=q.half()), dict(k=q[:, :1].expand(4, 2, 64)), dict(q=q[:1].expand(4, 2, 64))):
        with pytest.raises((ValueError, ea.AttnError)):
            ea.attn_rope_axes(bad.get("q", q), bad.get("k"), cos, sin, pos, [32], q_out=bad.get("q_out"), out_dtype=bad.get("out_dtype"))
    assert ea.attn_num_kernel_launches() == before
