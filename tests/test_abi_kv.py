"""The serving entry points without a GPU: the library exports what ``include/attn_kv.h`` declares, and
bad arguments are refused before any CUDA call."""

import ctypes
import os
import re

import pytest

import exact_attention_100_b200 as ea
from exact_attention_100_b200 import build as ea_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BAD, UNSUP = ea.ATTN_ERR_INVALID_ARG, ea.ATTN_ERR_UNSUPPORTED
# never dereferenced: the calls fail their checks first
P, P2, MIS, ODD, NULL = (ctypes.c_void_p(x) for x in (0x10000, 0x20000, 0x10008, 0x10002, 0))


@pytest.fixture(scope="module")
def L():
    ea_build.build()
    return ea.lib()


def _arr(ct, *v):
    return ctypes.cast((ct * len(v))(*v), ctypes.c_void_p)


def _each(f, ok, changes, want):
    for idx, val in changes:
        a = list(ok)
        a[idx] = val
        assert f(*a) == want, (idx, val)


def test_library_exports_what_the_header_declares(L):
    with open(os.path.join(ROOT, "include", "attn_kv.h")) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    names = re.findall(r"^\s*(?:int|unsigned long long)\s+(attn_\w+)\s*\(", text, re.M)
    assert sorted(names) == sorted(["attn_kv_tables", "attn_rope_axes", "attn_kv4_tile_bytes", "attn_kv4_append",
                                    "attn_kv4_read", "attn_fwd_kv4_workspace_bytes", "attn_fwd_kv4"])
    for n in names:
        assert hasattr(L, n)
    for n in ["attn_kv_tables", "attn_rope_axes", "attn_rope_axes_bwd", "attn_kv4_cache", "attn_kv4_append",
              "attn_kv4_read", "attn_fwd_kv4", "attn_fwd_kv4_workspace_bytes"]:
        assert callable(getattr(ea, n))


def test_kv_tables_refusals(L):
    ok = [P] * 10 + [4, 8, 64, 10, 100, NULL]
    _each(L.attn_kv_tables, ok, [(i, NULL) for i in range(10)] + [(i, ODD) for i in range(10)] +
          [(10, 0), (10, 8193), (11, 0), (12, 0), (12, 24), (12, 8192), (13, -1), (14, -1), (11, 1 << 26), (11, 1 << 30)], BAD)


def test_rope_axes_refusals(L):
    sec, st = _arr(ctypes.c_int, 16, 24, 24), _arr(ctypes.c_longlong, *[1024, 128, 4096] * 4)
    ok = [P, P, P2, P2, P, P, P, 1, 8, 2, 100, 128, 3, sec, 50, st, 0, ea.ATTN_BF16, ea.ATTN_BF16, NULL]
    _each(L.attn_rope_axes, ok, [(0, NULL), (2, NULL), (1, NULL), (3, NULL), (4, NULL), (5, NULL), (6, NULL), (13, NULL),
                                 (15, NULL), (0, MIS), (3, MIS), (4, MIS), (6, ODD), (7, 0), (8, 0), (9, 0), (10, 0), (12, 0),
                                 (12, 5), (14, 0), (16, 2), (17, 7), (11, 120), (8, 1 << 21),
                                 (13, _arr(ctypes.c_int, 16, 0, 24)), (13, _arr(ctypes.c_int, 16, 24, 32)),
                                 (15, _arr(ctypes.c_longlong, *[1024, 130, 4096] * 4)),
                                 (15, _arr(ctypes.c_longlong, *[1024, 128, -8] * 4))], BAD)
    _each(L.attn_rope_axes, ok, [(11, 132), (11, 2048), (13, _arr(ctypes.c_int, 16, 24, 22)), (17, ea.ATTN_E4M3)], UNSUP)
    # in place with other strides, or another type
    other = _arr(ctypes.c_longlong, *[1024, 128, 4096] * 2, *[1024, 128, 8192] * 2)
    _each(L.attn_rope_axes, [P, P, P, P] + ok[4:], [(15, other), (18, ea.ATTN_FP32)], BAD)


def test_kv4_append_and_read_refusals(L):
    st = _arr(ctypes.c_longlong, 1024, 128, 1024, 128)
    ok = [P, P, P2, P, P, 10, 8, 128, 64, 100, st, NULL]
    _each(L.attn_kv4_append, ok, [(0, NULL), (1, NULL), (2, NULL), (3, NULL), (10, NULL), (0, MIS), (1, MIS), (2, MIS),
                                  (3, ODD), (4, MIS), (5, 0), (6, 0), (8, 0), (8, 24), (8, 8192), (9, 0), (9, 1 << 26),
                                  (10, _arr(ctypes.c_longlong, 1024, 120 + 4, 1024, 128))], BAD)
    _each(L.attn_kv4_append, ok, [(7, 96), (7, 512)], UNSUP)
    ok = [P2, P, P, P, 10, 8, 128, 64, 100, ea.ATTN_FP32, NULL]
    _each(L.attn_kv4_read, ok, [(0, NULL), (1, NULL), (2, NULL), (3, NULL), (2, MIS), (3, MIS), (4, 0), (5, 0), (7, 40),
                                (8, 0), (9, 9)], BAD)
    _each(L.attn_kv4_read, ok, [(6, 32), (9, ea.ATTN_E4M3)], UNSUP)
    assert [L.attn_kv4_tile_bytes(d) for d in (64, 128, 256, 96, 0)] == [1152, 2304, 4608, 0, 0]


def test_fwd_kv4_refusals(L):
    st = _arr(ctypes.c_longlong, 4096, 128, 4096, 128)
    ok = [P, P2, P, P, P, P2, P, P, P, 4, 32, 8, 40, 16, 128, 64, 100, 20, st, 0.1, 1, NULL]
    inf, nan = float("inf"), float("nan")
    _each(L.attn_fwd_kv4, ok, [(0, NULL), (1, NULL), (2, NULL), (3, NULL), (5, NULL), (7, NULL), (18, NULL), (0, MIS),
                               (1, MIS), (5, MIS), (7, MIS), (8, MIS), (2, ODD), (3, ODD), (4, ODD), (6, ODD), (9, 0), (10, 0),
                               (10, 30), (11, 0), (12, 0), (13, 0), (15, 8), (15, 50), (16, 0), (17, 0), (16, 1 << 26),
                               (17, 1 << 26), (19, 0.0), (19, -1.0), (19, inf), (19, nan), (20, 2), (12, 1 << 27),
                               (4, NULL), (18, _arr(ctypes.c_longlong, 4096, 4, 4096, 128))], BAD)
    _each(L.attn_fwd_kv4, ok, [(14, 96), (14, 32)], UNSUP)
    w = L.attn_fwd_kv4_workspace_bytes
    good = [4, 32, 8, 40, 16, 128, 148]
    assert w(*good) > 0
    for idx, val in [(0, 0), (1, 0), (1, 30), (2, 0), (3, 0), (4, 0), (5, 96), (6, -1), (3, 1 << 27)]:
        a = list(good)
        a[idx] = val
        assert w(*a) == 0, (idx, val)


def test_binding_refuses_before_any_library_call(L):
    torch = pytest.importorskip("torch")
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    cache = torch.zeros(4, 2, 1, 18 * 64, dtype=torch.uint8)
    kv, q = torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    bad = [
        lambda: ea.attn_kv_tables(i32(2), i32(2), i32(2, 3), i32(4), i32(1), 16, 8),  # host memory
        lambda: ea.attn_kv_tables(i32(2), i32(3), i32(2, 3), i32(4), i32(1), 16, 8),
        lambda: ea.attn_kv_tables(i32(2), i32(2).long(), i32(2, 3), i32(4), i32(1), 16, 8),
        lambda: ea.attn_kv_tables(i32(2), i32(2), i32(2, 3), i32(4), i32(1), 16, -1),
        lambda: ea.attn_kv4_append(kv, kv, cache, i32(3)),
        lambda: ea.attn_kv4_append(kv, kv, cache, i32(2)),
        lambda: ea.attn_kv4_append(kv.float(), kv, cache, i32(3)),
        lambda: ea.attn_kv4_append(kv, kv, cache[..., :-1], i32(3)),
        lambda: ea.attn_kv4_read(cache, i32(3)),
        lambda: ea.attn_kv4_read(cache, i32(3), k=torch.zeros(3, 2, 64), v=kv),
        lambda: ea.attn_fwd_kv4(q, cache, i32(3, 1), i32(3)),
        lambda: ea.attn_fwd_kv4(q, cache, i32(2, 1), i32(2)),
        lambda: ea.attn_fwd_kv4(q, cache, i32(2, 1), i32(2), cu_seqlens_q=i32(2)),
        lambda: ea.attn_fwd_kv4(q[:, :3], cache, i32(3, 1), i32(3)),
        lambda: ea.attn_fwd_kv4(q.float(), cache, i32(3, 1), i32(3)),
        lambda: ea.attn_rope_axes(q, kv, torch.zeros(5, 32), torch.zeros(5, 32), i32(1, 3), [32]),
        lambda: ea.attn_rope_axes(q, kv, torch.zeros(5, 32), torch.zeros(5, 32), i32(1, 3), [16, 16]),
        lambda: ea.attn_rope_axes(q, kv, torch.zeros(5, 30), torch.zeros(5, 32), i32(1, 3), [32]),
        lambda: ea.attn_rope_axes(q, kv.float(), torch.zeros(5, 32), torch.zeros(5, 32), i32(1, 3), [32]),
        lambda: ea.attn_kv4_cache(4, 2, 24, 64),
        lambda: ea.attn_kv4_cache(4, 2, 16, 80),
    ]
    before = ea.attn_num_kernel_launches()
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(str(i))
    assert ea.attn_num_kernel_launches() == before
