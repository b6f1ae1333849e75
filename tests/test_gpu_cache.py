"""GPU: the paged MX key/value cache (mx_kv_cache_write, mx_kv_cache_read)
against the oracle's quantizer and decoder, bit for bit."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_scaled_precision_mm_amd as mx
import oracle
from tests import servingref as sr

pytestmark = pytest.mark.gpu


def _filled(pages, page, heads, dim, fmt, byte=0xEE):
    c = mx.KVCache.empty(pages, page, heads, dim, fmt)
    for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales):
        t.fill_(byte)
    return c


def _parts(c):
    torch.cuda.synchronize()
    return [t.cpu().numpy() for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales)]


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("tokens,page,heads,dim", [(1, 1, 1, 32), (1, 16, 8, 128), (3, 2, 3, 96), (65, 16, 1, 64),
                                                   (257, 64, 5, 160), (1000, 256, 2, 128), (17, 8, 7, 1024)])
def test_write_and_read(fmt, tokens, page, heads, dim):
    print("cache", fmt, tokens, page, heads, dim, flush=True)
    rng = np.random.default_rng(tokens + dim)
    pages = -(-tokens // page) + 3
    c = _filled(pages, page, heads, dim, fmt)
    slots = rng.permutation(pages * page)[:tokens]
    # tokens are parts of wider rows, as a joint QKV product writes them
    wide = sr.bf16(rng.standard_normal((tokens, 4 * heads * dim)) * np.exp2(rng.integers(-20, 20, (tokens, 1)))).cuda()
    k = wide[:, heads * dim:2 * heads * dim].unflatten(1, (heads, dim))
    v = wide[:, 3 * heads * dim:].unflatten(1, (heads, dim))
    ds = torch.from_numpy(slots).cuda()
    mx.mx_kv_cache_write(c, k, v, ds)
    parts = _parts(c)
    want = [np.full_like(p, 0xEE) for p in parts]
    for x, codes, scales in ((k, want[0], want[1]), (v, want[2], want[3])):
        oc, os_ = oracle.quantize(fmt, sr.bits(x).reshape(tokens * heads, dim), tokens * heads, dim)
        codes[slots // page, :, slots % page] = oc.reshape(tokens, heads, -1)
        scales[slots // page, :, slots % page] = os_.reshape(tokens, heads, -1)
    for name, a, b in zip(("k codes", "k scales", "v codes", "v scales"), parts, want):
        assert np.array_equal(a, b), name
    # back, into parts of wider rows
    back = torch.full((tokens, 3 * heads * dim), 5.0, dtype=torch.bfloat16, device="cuda")
    rk, rv = back[:, :heads * dim].unflatten(1, (heads, dim)), back[:, 2 * heads * dim:].unflatten(1, (heads, dim))
    mx.mx_kv_cache_read(c, rk, rv, ds)
    torch.cuda.synchronize()
    for got, codes, scales in ((rk, parts[0], parts[1]), (rv, parts[2], parts[3])):
        ref = sr.rows_of(fmt, codes[slots // page, :, slots % page], scales[slots // page, :, slots % page])
        assert np.array_equal(sr.f64(got), ref)
    assert (back[:, heads * dim:2 * heads * dim] == 5).all()


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_read_every_code_under_every_scale(fmt):
    # 256 scales x every element code: BF16 rounds (to nearest even) where
    # the value is below its subnormals, and overflows to infinity
    n = 256
    c = mx.KVCache.empty(n, 1, 1, 256 if fmt == "fp8" else 32, fmt)
    row = torch.arange(256, dtype=torch.uint8) if fmt == "fp8" else \
        torch.tensor([i + 16 * ((i + 1) % 16) for i in range(16)], dtype=torch.uint8)
    c.k_codes.copy_(row.expand(n, -1).view(c.k_codes.shape))
    c.v_codes.copy_(row.flip(0).expand(n, -1).view(c.k_codes.shape))
    for t in (c.k_scales, c.v_scales):
        t.copy_(torch.arange(n, dtype=torch.uint8)[:, None].expand(n, t.shape[-1]).reshape(t.shape))
    k = torch.empty((n, 1, c.head_dim), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    mx.mx_kv_cache_read(c, k, v, torch.arange(n, device="cuda"))
    parts = _parts(c)
    for got, codes, scales in ((k, parts[0], parts[1]), (v, parts[2], parts[3])):
        ref = torch.from_numpy(sr.rows_of(fmt, codes[:, :, 0], scales[:, :, 0])).to(torch.float32).to(torch.bfloat16)
        got = got.cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(ref))
        diff = (got.view(torch.int16) != ref.view(torch.int16)) & ~torch.isnan(ref)
        assert not diff.any(), (diff.nonzero()[:5], got[diff][:5], ref[diff][:5])


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_slots_outside_are_skipped_and_read_zeros(fmt):
    pages, page, heads, dim = 3, 4, 2, 64
    c = _filled(pages, page, heads, dim, fmt)
    x = torch.randn(6, heads, dim, device="cuda").bfloat16()
    slots = torch.tensor([-1, 11, 12, 1 << 40, -(1 << 40), 0], device="cuda")
    mx.mx_kv_cache_write(c, x, x, slots)
    parts = _parts(c)
    for p in parts:
        p = p.reshape(pages, heads, page, -1).transpose(0, 2, 1, 3).reshape(pages * page, -1)
        assert (p[1:11] == 0xEE).all() and not (p[0] == 0xEE).all() and not (p[11] == 0xEE).all()
    k, v = torch.full_like(x, 9), torch.full_like(x, 9)
    mx.mx_kv_cache_read(c, k, v, slots)
    assert (k[[0, 2, 3, 4]] == 0).all() and (v[[0, 2, 3, 4]] == 0).all() and (k[1] != 9).any() and (k[5] != 9).any()


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_special_blocks(fmt):
    x = torch.zeros(1, 1, 160)
    x[0, 0, 3] = float("nan")
    x[0, 0, 40] = float("-inf")
    x[0, 0, 70] = 1e-39                 # a BF16 subnormal
    x[0, 0, 100] = 3.38e38
    x = x.bfloat16().cuda()
    c = mx.KVCache.empty(1, 1, 1, 160, fmt)
    mx.mx_kv_cache_write(c, x, x, torch.zeros(1, dtype=torch.int64, device="cuda"))
    k, v = torch.empty_like(x), torch.empty_like(x)
    mx.mx_kv_cache_read(c, k, v, torch.zeros(1, dtype=torch.int64, device="cuda"))
    k = k.cpu()[0, 0]
    assert torch.isnan(k[:64]).all() and not torch.isnan(k[64:]).any() and k[100] > 2.5e38 and (k[101:] == 0).all()
    assert torch.equal(k.view(torch.int16), v.cpu()[0, 0].view(torch.int16))


def test_offsets_past_32_bits():
    # 6 GiB of codes on each side; tokens at both ends and around 4 GiB
    pages, page, heads, dim = 6144, 1024, 8, 128
    c = mx.KVCache.empty(pages, page, heads, dim, "fp8")
    slots = torch.tensor([0, 4194303, 4194304, 4194305, pages * page - 1], device="cuda")
    x = torch.randn(5, heads, dim, device="cuda").bfloat16()
    mx.mx_kv_cache_write(c, x, -x, slots)
    k, v = torch.empty_like(x), torch.empty_like(x)
    mx.mx_kv_cache_read(c, k, v, slots)
    oc, os_ = oracle.quantize("fp8", sr.bits(x).reshape(40, 128), 40, 128)
    ref = sr.rows_of("fp8", oc, os_).reshape(5, heads, dim)
    assert np.array_equal(sr.f64(k), ref) and np.array_equal(sr.f64(v), -ref)
    p, o = pages - 1, page - 1
    assert np.array_equal(c.k_codes[p, :, o].cpu().numpy(), oc.reshape(5, heads, dim)[4])
    assert int(c.k_codes[1:4096].count_nonzero()) <= 2 * heads * dim


def test_no_tokens():
    c = mx.KVCache.empty(2, 16, 2, 64, "fp8")
    x = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    mx.mx_kv_cache_write(c, x, x, torch.empty(0, dtype=torch.int64, device="cuda"))
    mx.mx_kv_cache_read(c, x, x, torch.empty(0, dtype=torch.int64, device="cuda"))
