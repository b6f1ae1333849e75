"""Host checks of the operators around the products: every invalid argument
is refused with its status before any HIP call (no GPU needed), workspace
sizes, and the binding's checks of tensors."""
from __future__ import annotations

import ctypes

import pytest
import torch

import block_scaled_precision_mm_amd as mx

A = 0x10000     # aligned, never dereferenced
L = mx._lib


def norm(x=A, res=A, w=A, h=A, y=A, ys=A, rows=4, K=64, eps=1e-6, kind=3):
    return L.mx_rmsnorm(x, res, w, h, y, ys, rows, K, eps, kind, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=0), -1), (dict(y=0), -1), (dict(ys=0), -1), (dict(ys=0, kind=4), -1),
    (dict(kind=5), -5), (dict(kind=-1), -5),
    (dict(rows=-1), -2), (dict(rows=1 << 31), -2), (dict(K=0), -2), (dict(K=65568), -2), (dict(K=48), -3),
    (dict(eps=-1e-6), -9), (dict(eps=float("nan")), -9), (dict(eps=float("inf")), -9),
    (dict(x=A + 8), -4), (dict(res=A + 2), -4), (dict(w=A + 4), -4), (dict(h=A + 8), -4), (dict(y=A + 8), -4),
])
def test_norm_refusals(kw, status):
    assert norm(**kw) == status


def cache(pages=8, page=16, heads=2, dim=128, fp4=0, kc=A, ks=A, vc=A, vs=A):
    return mx._KVCacheStruct(kc, ks, vc, vs, pages, page, heads, dim, fp4)


CACHES = [
    (dict(kc=0), -1), (dict(ks=0), -1), (dict(vc=0), -1), (dict(vs=0), -1),
    (dict(pages=0), -2), (dict(pages=1 << 31), -2), (dict(page=0), -2), (dict(page=24), -2), (dict(page=131072), -2),
    (dict(heads=0), -2), (dict(heads=4097), -2), (dict(dim=0), -2), (dict(dim=2048), -2), (dict(dim=80), -3),
    (dict(pages=(1 << 31) - 1, page=65536), -2),
    (dict(kc=A + 8), -4), (dict(vc=A + 1), -4), (dict(ks=A + 2), -4), (dict(vs=A + 1), -4),
]


def tokens(c, k=A, v=A, kst=256, vst=256, slots=A, n=5, fn="mx_kv_cache_write"):
    return getattr(L, fn)(ctypes.addressof(c), k, v, kst, vst, slots, n, None)


@pytest.mark.parametrize("fn", ["mx_kv_cache_write", "mx_kv_cache_read"])
@pytest.mark.parametrize("kw,status", CACHES)
def test_cache_refusals(fn, kw, status):
    assert tokens(cache(**kw), fn=fn) == status
    assert getattr(L, fn)(None, A, A, 256, 256, A, 5, None) == -1


@pytest.mark.parametrize("fn", ["mx_kv_cache_write", "mx_kv_cache_read"])
@pytest.mark.parametrize("kw,status", [
    (dict(k=0), -1), (dict(v=0), -1), (dict(slots=0), -1), (dict(n=-1), -2), (dict(n=1 << 40), -2),
    (dict(kst=248), -2), (dict(vst=0), -2), (dict(kst=1 << 31), -2), (dict(kst=260), -3), (dict(vst=257), -3),
    (dict(k=A + 8), -4), (dict(v=A + 2), -4), (dict(slots=A + 4), -4),
])
def test_token_refusals(fn, kw, status):
    assert tokens(cache(), fn=fn, **kw) == status


def attend(c=None, q=A, qst=1024, ends=A, lens=A, table=A, width=4, seqs=3, n=7, heads=8, most=7, scale=0.1, causal=1,
           window=0, out=A, kind=0, lse=0, ws=0, wsb=0):
    c = c or cache()
    return L.mx_paged_attention(ctypes.addressof(c), q, qst, ends, lens, table, width, seqs, n, heads, most, scale, causal,
                                window, out, kind, lse, ws, wsb, None)


@pytest.mark.parametrize("kw,status", CACHES)
def test_attention_cache_refusals(kw, status):
    assert attend(cache(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(kind=3), -5), (dict(kind=-1), -5),
    (dict(seqs=-1), -2), (dict(seqs=65537), -2), (dict(n=-1), -2), (dict(n=1 << 28), -2), (dict(heads=7), -2), (dict(heads=0), -2),
    (dict(heads=1), -2), (dict(most=-1), -2), (dict(width=-1), -2), (dict(width=1 << 27), -2), (dict(qst=1016), -2),
    (dict(qst=1 << 31), -2), (dict(window=-1), -2), (dict(c=cache(dim=96)), -2), (dict(c=cache(dim=256), qst=2048), -2),
    (dict(c=cache(heads=256), qst=256 * 128, seqs=65536, n=65536, heads=256, most=1), -2),     # 2^24 row tiles and more
    (dict(q=0), -1), (dict(ends=0), -1), (dict(lens=0), -1), (dict(table=0), -1), (dict(out=0), -1),
    (dict(qst=1028), -3),
    (dict(scale=0.0), -9), (dict(scale=-1.0), -9), (dict(scale=float("nan")), -9), (dict(scale=float("inf")), -9), (dict(causal=2), -9),
    (dict(q=A + 8), -4), (dict(out=A + 8), -4), (dict(ws=A + 8), -4), (dict(ends=A + 2), -4), (dict(lens=A + 1), -4),
    (dict(table=A + 2), -4), (dict(lse=A + 2), -4),
])
def test_attention_refusals(kw, status):
    assert attend(**kw) == status


def test_workspace_sizes():
    size = lambda c, *a: L.mx_paged_attention_workspace_bytes(ctypes.addressof(c), *a)  # noqa: E731
    for dim in (64, 128):
        c = cache(dim=dim, heads=8)
        for a in ((1, 1, 32, 1), (64, 64, 32, 1), (1, 4096, 32, 4096), (20, 700, 32, 300)):
            n = size(c, *a)
            assert n == 0 or n > 65536
        assert size(c, 1, 1, 32, 1) > 0
        assert size(c, 1, 1, 33, 1) == 0            # not a multiple of the KV heads
        assert size(c, 65536, 65536, 8, 1) == 0     # enough row tiles without splitting
    assert size(cache(dim=96), 1, 1, 8, 1) == 0
    assert L.mx_paged_attention_workspace_bytes(None, 1, 1, 8, 1) == 0


def test_binding_refuses_tensors_before_the_library():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):                 # not on a GPU
        mx.mx_rmsnorm(x, None, None, None, x, None, 4, 64, 1e-6)
    with pytest.raises(ValueError):
        mx.mx_rmsnorm(A, None, None, None, A, None, 4, 64, 1e-6)    # no out_kind
    t = torch.zeros(2, 2, 16, 128, dtype=torch.uint8)
    s = torch.zeros(2, 2, 16, 4, dtype=torch.uint8)
    for args, kw in (((t, s, t, s), {}), ((t, s, t, s), dict(fmt="fp6")), ((t[0], s, t, s), {})):
        with pytest.raises(ValueError):
            mx.KVCache(*args, **kw)
