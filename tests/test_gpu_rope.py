"""GPU: mx_rope_cache_write against the rotation in 64 bits, bit for bit: the
products of BF16 and FP32 values are exact there, so the rounded results are
the only ones that the formula has; the cache against the oracle's quantizer."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_scaled_precision_mm_amd as mx
import oracle
from tests import servingref as sr

pytestmark = pytest.mark.gpu


def rotated(x, table, positions, rot, inter):
    """bfloat16 [tokens][heads][dim] on the CPU, by the formula."""
    n = table.shape[0]
    at = table.cpu().double().numpy()[np.clip(positions, 0, n - 1)]
    at[(positions < 0) | (positions >= n)] = np.nan
    c, s = at[:, None, :, 0], at[:, None, :, 1]
    v = sr.f64(x)
    a, b = (v[..., 0:rot:2], v[..., 1:rot:2]) if inter else (v[..., :rot // 2], v[..., rot // 2:rot])
    with np.errstate(invalid="ignore"):
        a2, b2 = a * c - b * s, b * c + a * s
    y = np.stack((a2, b2), -1).reshape(a.shape[:-1] + (rot,)) if inter else np.concatenate((a2, b2), -1)
    with np.errstate(over="ignore"):
        y = torch.from_numpy(y.astype(np.float32)).to(torch.bfloat16)
    return torch.cat((y, x.cpu()[..., rot:]), -1)


def same(a, b):
    """Equal bits, but for the bits of NaNs."""
    a, b = a.cpu(), b.cpu()
    nan = torch.isnan(b)
    return torch.equal(torch.isnan(a), nan) and torch.equal(torch.where(nan, 0, a).view(torch.int16), torch.where(nan, 0, b).view(torch.int16))


class Case:
    def __init__(self, tokens, q_heads=8, heads=2, dim=128, rot=128, inter=False, fmt="fp8", page=16, pad=0, seed=1, positions=4096):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.heads, self.dim, self.rot, self.inter, self.fmt, self.page = heads, dim, rot, inter, fmt, page
        qkv = torch.randn((tokens, (q_heads + 2 * heads) * dim + pad), generator=g, device="cuda").bfloat16()
        qkv *= torch.exp2(torch.randint(-6, 7, qkv.shape, generator=g, device="cuda")).bfloat16()
        self.qkv = qkv
        self.q, self.k, self.v = (t.unflatten(1, (-1, dim)) for t in
                                  qkv[:, :(q_heads + 2 * heads) * dim].split((q_heads * dim, heads * dim, heads * dim), dim=1))
        self.table = mx.rope_table(positions, rot)
        self.positions = torch.randint(0, positions, (tokens,), generator=g, device="cuda")
        pages = tokens // page + 3
        self.slots = torch.randperm(pages * page, generator=g, device="cuda")[:tokens]
        self.cache = mx.KVCache.empty(pages, page, heads, dim, fmt)
        for t in self.parts():
            t.random_(0, 256, generator=g)
        self.before = [t.cpu() for t in self.parts()]

    def parts(self):
        return self.cache.k_codes, self.cache.k_scales, self.cache.v_codes, self.cache.v_scales

    def want(self):
        """Queries and the whole cache."""
        pos = self.positions.cpu().numpy()
        q = rotated(self.q, self.table, pos, self.rot, self.inter)
        parts = [t.clone() for t in self.before]
        slots = self.slots.cpu().numpy()
        n = len(slots)
        ok = (slots >= 0) & (slots < parts[0].shape[0] * self.page)
        for i, x in ((0, rotated(self.k, self.table, pos, self.rot, self.inter)), (2, self.v.cpu())):
            if n:
                codes, scales = oracle.quantize(self.fmt, sr.bits(x.reshape(n * self.heads, self.dim)), n * self.heads, self.dim)
                at = slots[ok] // self.page, slots[ok] % self.page
                for part, new in ((parts[i], codes), (parts[i + 1], scales)):
                    part.numpy()[at[0], :, at[1]] = new.reshape(n, self.heads, -1)[ok]
        return q, parts

    def check(self, what="", in_place=False, stream=None):
        print("rope", what, tuple(self.q.shape), self.heads, self.dim, self.rot, self.inter, self.fmt, self.page, flush=True)
        q, parts = self.want()
        rest = self.qkv.clone()
        out = None if in_place else torch.full(self.q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        mx.mx_rope_cache_write(self.cache, self.q, self.k, self.v, self.positions, self.slots, self.table, out,
                               interleaved=self.inter, stream=stream)
        torch.cuda.synchronize()
        assert same(self.q if in_place else out, q)
        for got, want in zip(self.parts(), parts):
            assert torch.equal(got.cpu(), want)
        kept = self.q.shape[1] * self.dim if in_place else 0
        assert torch.equal(self.qkv[:, kept:].view(torch.int16), rest[:, kept:].view(torch.int16))


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dim,rot", [(32, 16), (32, 32), (64, 32), (64, 48), (64, 64), (96, 96), (128, 16), (128, 64), (128, 112),
                                     (128, 128), (160, 80), (256, 256), (1024, 1024)])
def test_widths(fmt, inter, dim, rot):
    Case(5, dim=dim, rot=rot, inter=inter, fmt=fmt).check("widths")


@pytest.mark.parametrize("tokens", [1, 2, 3, 17, 64, 255, 1000])
@pytest.mark.parametrize("q_heads,heads", [(1, 1), (5, 5), (14, 2), (32, 8), (33, 3)])
def test_tokens_and_heads(tokens, q_heads, heads):
    Case(tokens, q_heads, heads, dim=64, rot=64).check("tokens")


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot", [48, 128])
def test_in_place_in_wide_rows(rot, inter):
    Case(300, 32, 8, rot=rot, inter=inter, pad=24).check("in place", in_place=True)


@pytest.mark.parametrize("page", [1, 2, 256])
def test_pages(page):
    Case(100, page=page, fmt="fp4").check("pages")


def test_keys_alone_and_no_tokens():
    c = Case(33)
    _, parts = c.want()
    mx.mx_rope_cache_write(c.cache, None, c.k, c.v, c.positions, c.slots, c.table)
    torch.cuda.synchronize()
    assert all(torch.equal(a.cpu(), b) for a, b in zip(c.parts(), parts))
    c = Case(0)
    c.check("no tokens")


def test_keys_are_those_of_a_cache_write():
    c = Case(200, rot=64)
    other = Case(200, rot=64)
    k = rotated(c.k, c.table, c.positions.cpu().numpy(), 64, False).cuda()
    mx.mx_kv_cache_write(other.cache, k, c.v, c.slots)
    c.check("against a cache write")
    assert all(torch.equal(a, b) for a, b in zip(c.parts(), other.parts()))


def test_padding_tokens_and_positions_outside_the_table():
    c = Case(64, positions=100)
    c.slots[5:20] = -1
    c.slots[21] = c.cache.pages * c.page
    c.slots[22] = -(1 << 62)
    c.slots[23] = 1 << 62
    c.positions[7] = -1
    c.positions[30] = 100
    c.positions[31] = -(1 << 40)
    c.positions[32] = (1 << 62) + 5
    c.check("padding")
    at = int(c.slots[30])
    assert (c.cache.k_scales[at // c.page, :, at % c.page] == 255).all()


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("inter", [False, True])
def test_values_out_of_the_ordinary(fmt, inter):
    c = Case(40, fmt=fmt, inter=inter, rot=64)
    odd = torch.tensor([np.inf, -np.inf, np.nan, 1e-40, -1e-40, 0.0, -0.0, 3e38, -3e38, 2.0 ** -126], device="cuda").bfloat16()
    g = torch.Generator(device="cuda").manual_seed(2)
    for t in (c.q, c.k, c.v):
        at = torch.rand(t.shape, generator=g, device="cuda") < 0.03
        t[at] = odd[torch.randint(0, len(odd), (int(at.sum()),), generator=g, device="cuda")]
    c.k[3] = 0
    c.k[4] = 1e-39
    c.check("odd values")


def test_far_positions():
    c = Case(50, dim=64, rot=64, positions=1 << 20)
    c.positions += 0
    c.positions[0] = (1 << 20) - 1
    c.check("far")


def test_slots_past_32_bits():
    # 2^20 pages of 16 tokens of 8 heads of 32: codes of 2^32 bytes a side
    g = torch.Generator(device="cuda").manual_seed(1)
    cache = mx.KVCache.empty(1 << 20, 16, 8, 32, "fp8")
    last = (1 << 24) - 1
    slots = torch.tensor([last, 3, last - 16], device="cuda")
    k, v, q = (torch.randn((3, 8, 32), generator=g, device="cuda").bfloat16() for _ in "kvq")
    table = mx.rope_table(64, 32)
    pos = torch.tensor([1, 2, 63], device="cuda")
    out = torch.empty_like(q)
    mx.mx_rope_cache_write(cache, q, k, v, pos, slots, table, out)
    rk, rv = torch.empty_like(k), torch.empty_like(v)
    mx.mx_kv_cache_read(cache, rk, rv, slots)
    small = mx.KVCache.empty(1, 4, 8, 32, "fp8")
    mx.mx_kv_cache_write(small, rotated(k, table, pos.cpu().numpy(), 32, False).cuda(), v, torch.arange(3, device="cuda"))
    sk, sv = torch.empty_like(k), torch.empty_like(v)
    mx.mx_kv_cache_read(small, sk, sv, torch.arange(3, device="cuda"))
    torch.cuda.synchronize()
    assert same(rk, sk) and same(rv, sv)
    assert int(cache.k_codes.view(-1, 32).any(1).sum()) == 24


def test_other_stream_and_replays():
    c = Case(70, 8, 2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.check("stream", stream=s)
    out = torch.empty(c.q.shape, dtype=torch.bfloat16, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mx.mx_rope_cache_write(c.cache, c.q, c.k, c.v, c.positions, c.slots, c.table, out)
    for i in range(3):
        c.qkv.normal_()
        c.positions.random_(0, 4096)
        c.slots.copy_(torch.randperm(c.cache.pages * c.page, device="cuda")[:70])
        c.before = [t.cpu() for t in c.parts()]
        q, parts = c.want()
        g.replay()
        torch.cuda.synchronize()
        assert same(out, q)
        assert all(torch.equal(a.cpu(), b) for a, b in zip(c.parts(), parts))


# (past 2^19 pieces a thread has four heads)
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("fmt,inter,rot", [("fp8", False, 128), ("fp8", True, 128), ("fp4", False, 48), ("fp4", True, 16)])
@pytest.mark.parametrize("tokens,q_heads,heads", [(1100, 32, 8), (1777, 33, 3), (2500, 9, 9)])
def test_many_tokens(tokens, q_heads, heads, fmt, inter, rot, in_place):
    assert tokens * (q_heads * 8 + 2 * heads * 16) > 1 << 19
    Case(tokens, q_heads, heads, rot=rot, inter=inter, fmt=fmt, pad=8).check("many tokens", in_place=in_place)


def test_many_keys_alone():
    c = Case(9000, 1, 2)
    assert 9000 * 2 * 2 * 16 > 1 << 19
    _, parts = c.want()
    mx.mx_rope_cache_write(c.cache, None, c.k, c.v, c.positions, c.slots, c.table)
    torch.cuda.synchronize()
    assert all(torch.equal(a.cpu(), b) for a, b in zip(c.parts(), parts))
