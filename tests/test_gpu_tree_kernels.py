"""GPU: mx_tree_attention by each of its kernels.  Which one runs goes by the
rows and the most keys that the page table could hold, so a table that is wider
than its sequences need takes small inputs to the kernels of large ones."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_scaled_precision_mm_amd as mx
from tests import servingref as sr
from tests import test_gpu_tree as base

pytestmark = pytest.mark.gpu

KEYS = {"16 rows": 0, "32 rows": 1, "tiles": 2}


def widen(c, kernel):
    """The case with a table of as many columns as take it to a kernel: 32 rows
    from 400000 (row tiles of 32) x keys on, tiles of 128 or 256 rows (more than
    64, 128 rows a sequence on average) from 2500000 on."""
    rows = sum(n for n, _ in c.seqs) * c.group
    tiles = c.heads * -(-rows // 32)
    keys = (0, 500000, 2600000)[KEYS[kernel]]
    width = -(-keys // tiles) // c.page + 2
    if width > c.table.shape[1]:
        c.table = np.pad(c.table, ((0, 0), (0, width - c.table.shape[1])), constant_values=-1)
    return c


@pytest.mark.parametrize("kernel", KEYS)
@pytest.mark.parametrize("fmt,dim", [("fp8", 64), ("fp8", 128), ("fp4", 64), ("fp4", 128)])
@pytest.mark.parametrize("seqs", [[(20, 20), (33, 300), (25, 26)], [(40, 333), (30, 31), (64, 130)], [(130, 500), (70, 70), (100, 611)]])
def test_sizes(kernel, fmt, dim, seqs):
    widen(base.Case(seqs, fmt, dim, heads=2), kernel).check(kernel)


@pytest.mark.parametrize("kernel", KEYS)
@pytest.mark.parametrize("page", [1, 4, 64])
def test_pages(kernel, page):
    widen(base.Case([(30, 250), (70, 177)], page=page, heads=1), kernel).check(kernel)


@pytest.mark.parametrize("kernel", KEYS)
@pytest.mark.parametrize("window", [1, 5, 64, 100, 5000])
def test_windows(kernel, window):
    c = base.Case([(40, 500), (90, 91), (33, 260)], heads=1)
    widen(c, kernel)
    if kernel != "16 rows":         # (a window bounds the keys too)
        window += 1 << 22
        c.check(kernel, window=window)
        window -= 1 << 22
    c.check(kernel, window=window)


@pytest.mark.parametrize("kernel", KEYS)
@pytest.mark.parametrize("seqs", [[(40, 6000)], [(50, 5000), (45, 300), (60, 61)], [(100, 9000), (70, 2000)]])
def test_parts(kernel, seqs):
    c = widen(base.Case(seqs, heads=1), kernel)
    split, _ = c.check(kernel)
    whole, _ = c.check(kernel, workspace=None)
    assert torch.allclose(split, whole, rtol=2.0 ** -6, atol=2.0 ** -6)


@pytest.mark.parametrize("kernel", KEYS)
def test_many_parts(kernel):
    """More than 16 parts of a row tile, joined in two steps, and many sequences of unequal lengths."""
    widen(base.Case([(5, 17000)], heads=1), kernel).check(kernel)
    widen(base.Case([(33, 30000)], heads=1, group=2), kernel).check(kernel)
    rng = np.random.default_rng(2)
    seqs = [(int(rng.integers(15, 30)), int(np.exp(rng.uniform(np.log(30), np.log(4000))))) for _ in range(30)]
    widen(base.Case(seqs, heads=1, group=4), kernel).check(kernel)


@pytest.mark.parametrize("kernel", KEYS)
def test_masks_that_are_no_trees(kernel):
    rng = np.random.default_rng(4)
    seqs = [(40, 90), (75, 75), (32, 32), (30, 240)]
    sees = [rng.random((n, n)) < 0.3 for n, _ in seqs]
    sees[2][:] = False
    sees[2][4, 7] = True
    for junk in (False, True):
        c = widen(base.Case(seqs, heads=1, sees=[s.copy() for s in sees], words=3, junk=junk), kernel)
        out, lse = c.check(kernel)
        assert (out[115:119] == 0).all() and (lse[115:119] == -np.inf).all()


@pytest.mark.parametrize("kernel", KEYS)
@pytest.mark.parametrize("what", ["nan", "inf"])
@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_unseen_nodes_hold_anything(kernel, what, fmt):
    seqs = [(40, 300), (30, 130), (35, 35)]
    c = widen(base.Case(seqs, fmt, heads=1), kernel)
    for s, (n, L) in enumerate(seqs):
        j = n // 2
        c.sees[s][:, j] = False
        c.sees[s][n - 1, j] = True
        key = L - n + j
        page = int(c.table[s, key // c.page])
        c.parts[3][page, :, key % c.page] = 255 if what == "nan" else 254
        if what == "inf":
            c.parts[2][page, :, key % c.page] = 0x77 if fmt == "fp4" else 0x78
        c.v[s][key] = np.nan if what == "nan" else np.inf
    c.mask.copy_(torch.from_numpy(np.concatenate([base.words_of(s, c.words) for s in c.sees])))
    c.upload()
    out, lse = c.run()
    at, q = 0, sr.f64(c.q)
    for s, (n, L) in enumerate(seqs):
        last = out[at + n - 1]
        assert torch.isnan(last).all() if what == "nan" else (last == np.inf).all()
        mask = base.seen(c.sees[s], n, L, 0)
        v = np.where(np.isfinite(c.v[s]), c.v[s], 0.0)
        parts = [sr.attention(q[at + i:at + i + 1], c.k[s], v, c.dim ** -0.5, False, 0, 1, mask[i]) for i in range(n - 1)]
        sr.check_attention(out[at:at + n - 1], lse[at:at + n - 1], [np.concatenate(t) for t in zip(*parts)], L, what)
        at += n


@pytest.mark.parametrize("kernel", KEYS)
def test_pages_outside_the_cache(kernel):
    seqs = [(40, 100), (60, 260)]
    c = widen(base.Case(seqs, heads=1), kernel)
    here = []
    for s, (n, L) in enumerate(seqs):
        ok = np.ones(L, bool)
        for page, bad in ((1, -1), ((L - n) // c.page, 1 << 30), ((L - 1) // c.page, c.cache.pages)):
            c.table[s, page] = bad
            ok[page * c.page:(page + 1) * c.page] = False
        here.append(ok)
    c.check(kernel, here=here)


@pytest.mark.parametrize("kernel", KEYS)
def test_replays(kernel):
    c = widen(base.Case([(40, 3000), (45, 200)], heads=1), kernel)
    want, wl = c.check(kernel)
    args = [torch.from_numpy(t).cuda() for t in (c.ends, c.lens, c.table)]
    out, lse = torch.empty_like(want), torch.empty_like(wl)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(2):
            mx.mx_tree_attention(c.cache, c.q, *args, c.mask, out, lse=lse, max_new=45)
    for i in range(3):
        out.fill_(-7)
        base.Case([(40, 900)], seed=5 + i).run()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("kernel", KEYS)
def test_offsets_past_32_bits(kernel):
    """The pages at the end of a cache of 2^33 codes a side."""
    c = base.Case([(40, 300), (30, 130)], heads=1, dim=64)
    want, wl = widen(c, kernel).check(kernel)
    pages = 1 << 23
    big = mx.KVCache.empty(pages, c.page, 1, 64, "fp8")
    n = c.cache.pages
    for t, s in zip((big.k_codes, big.k_scales, big.v_codes, big.v_scales),
                    (c.cache.k_codes, c.cache.k_scales, c.cache.v_codes, c.cache.v_scales)):
        t[pages - n:] = s
    c.table = np.where(c.table >= 0, c.table + pages - n, -1).astype(np.int32)
    c.cache = big
    out, lse = c.run()
    assert torch.equal(out, want) and torch.equal(lse, wl)
