"""The serving operators together: a prompt, then tokens one at a time, eagerly and as replays of one
captured graph."""

import numpy as np
import pytest
import torch

import exact_attention_100_b200 as ea
from exact_attention_100_b200 import build as ea_build
from exact_attention_100_b200.inputs import hadamard_signs, rope_tables
from kv_util import check, default_scale, held, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ea_build.build()


class Serving:
    """State of B requests on the device; step() is what a serving loop calls."""

    def __init__(self, B, Hq, Hk, d, page, blocks, width):
        self.B, self.Hq, self.Hk, self.d, self.page = B, Hq, Hk, d, page
        self.lens, self.cursor = i32(np.zeros(B)), i32([0])
        self.table = i32(np.full((B, width), -1))
        self.free = i32(np.random.default_rng(0).permutation(blocks))
        self.cache = ea.attn_kv4_cache(blocks, Hk, page, d)
        cos, sin = rope_tables(width * page, d)
        self.cos, self.sin = torch.from_numpy(cos).cuda(), torch.from_numpy(sin).cuda()
        self.signs = torch.from_numpy(hadamard_signs(d)).cuda()
        self.sections = [d // 8, d // 8, d // 4]

    def step(self, qkv, new, longest):
        slots, pos, cu, _, _, _ = ea.attn_kv_tables(self.lens, new, self.table, self.free, self.cursor, self.page,
                                                    qkv.shape[0], lens_out=self.lens, cursor_out=self.cursor)
        q, k, v = qkv[:, :self.Hq], qkv[:, self.Hq:self.Hq + self.Hk], qkv[:, self.Hq + self.Hk:]
        q, k = ea.attn_rope_axes(q, k, self.cos, self.sin, pos.expand(3, -1).contiguous(), self.sections)
        ea.attn_kv4_append(k, v, self.cache, slots, signs=self.signs)
        o, lse = ea.attn_fwd_kv4(q, self.cache, self.table, self.lens, cu, longest, signs=self.signs)
        return q, o, lse, cu


def _qkv(seed, rows, heads, d):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(rows, heads, d, device="cuda", generator=g).to(torch.bfloat16)


@pytest.mark.parametrize("Hq,Hk,d,page", [(8, 2, 128, 16), (6, 6, 64, 32), (4, 1, 256, 64)])
def test_prompt_then_tokens(Hq, Hk, d, page):
    prompts = [37, 1, 130]
    s = Serving(3, Hq, Hk, d, page, blocks=64, width=20)
    new, lens = np.array(prompts), np.zeros(3, int)
    for step in range(4):
        # two rows more than the requests have: their slots are -1 and no request's cache changes
        qkv = _qkv(step, int(new.sum()) + 2, Hq + 2 * Hk, d)
        q, o, lse, cu = s.step(qkv, i32(new), int(new.max()))
        assert ea.attn_device_status() == ea.ATTN_OK
        lens = lens + new
        assert s.lens.tolist() == lens.tolist()
        ks, vs = held(s.cache, lens, s.table.cpu().numpy(), page)
        check(o, lse, q, ks, vs, cu.tolist(), lens, default_scale(d), True, s.signs)
        new = np.array([1, 1, 1]) if step else np.array([1, 0, 3])


def test_replays_of_a_captured_step_equal_eager_steps():
    B, Hq, Hk, d, page = 5, 8, 2, 128, 16
    prompts = [3, 40, 16, 0, 95]
    a, b = (Serving(B, Hq, Hk, d, page, 64, 16) for _ in range(2))
    for s in (a, b):
        s.step(_qkv(0, sum(prompts), Hq + 2 * Hk, d), i32(prompts), max(prompts))
    ones = i32(np.ones(B))
    inp = torch.empty(B, Hq + 2 * Hk, d, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, o, lse, _ = b.step(inp, ones, 1)
    for i in range(20):  # crosses pages
        x = _qkv(i + 1, B, Hq + 2 * Hk, d)
        _, oe, le, _ = a.step(x, ones, 1)
        inp.copy_(x)
        graph.replay()
        assert torch.equal(o, oe) and torch.equal(lse, le) and torch.equal(a.lens, b.lens)
    assert torch.equal(a.table, b.table) and torch.equal(a.cache, b.cache)
    assert ea.attn_device_status() == ea.ATTN_OK


def test_two_streams_at_once():
    """Two requests' steps on two streams, each with its own state and workspace, equal to one after the other."""
    kw = dict(B=2, Hq=8, Hk=2, d=128, page=16, blocks=300, width=140)
    states = [Serving(**kw) for _ in range(4)]
    prompt = [2000, 1500]
    x = [_qkv(i, sum(prompt), 12, 128) for i in range(2)]
    y = [_qkv(i + 5, 2, 12, 128) for i in range(2)]
    want = []
    for i in range(2):
        states[i].step(x[i], i32(prompt), max(prompt))
        want.append(states[i].step(y[i], i32([1, 1]), 1)[1])
    news = [i32(prompt), i32([1, 1])]
    torch.cuda.synchronize()
    got, streams = [None, None], [torch.cuda.Stream() for _ in range(2)]
    for i in range(2):
        with torch.cuda.stream(streams[i]):
            states[2 + i].step(x[i], news[0], max(prompt))
            got[i] = states[2 + i].step(y[i], news[1], 1)[1]
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(got[i], want[i])
    assert ea.attn_device_status() == ea.ATTN_OK


def test_read_values_feed_the_dense_forward():
    """Attention over the cache agrees with attn_fwd_strided on the values read back from it (both within
    a few bf16 steps of unit values: 2^-8 each for the output, P in bf16 and V in bf16, over sums of
    weights 1 and |v| <= 4)."""
    Hk, d, page, n = 2, 128, 16, 100
    cache = ea.attn_kv4_cache(8, Hk, page, d)
    qkv = _qkv(3, n, 3 * Hk, d)
    slots = i32(np.arange(n))
    ea.attn_kv4_append(qkv[:, Hk:2 * Hk], qkv[:, 2 * Hk:], cache, slots)
    k, v = ea.attn_kv4_read(cache, slots)
    q = qkv[:, :Hk]
    dense, _ = ea.attn_fwd_strided(*(t.transpose(0, 1)[None] for t in (q, k, v)), causal=True)
    o, _ = ea.attn_fwd_kv4(q, cache, i32([np.arange(7)]), i32([n]), i32([0, n]), n)
    assert (o.float() - dense[0].transpose(0, 1).float()).abs().max() <= 4 * 3 * 2.0 ** -8
