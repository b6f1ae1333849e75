"""GPU: mx_tree_attention under windows, over contexts in parts and in many
parts, by the kernel that each input is named by (treecases.py, held to the
plan by test_tree_plan_host.py)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import servingref as sr
from tests import test_gpu_tree as base
from tests import treecases as tc

pytestmark = pytest.mark.gpu

ROWS = [16, 32, 128, 256]
FORMATS = [("fp8", 64), ("fp8", 128), ("fp4", 64), ("fp4", 128)]


def make(case, fmt="fp8", dim=128, page=16, **kw):
    """The case, with its table's width, and the max_new of its calls."""
    seqs, _, most = case
    c = base.Case(seqs, fmt, dim, page, heads=1, **kw)
    c.table = np.pad(c.table, ((0, 0), (0, max(0, tc.width(case, page) - c.table.shape[1]))), constant_values=-1)
    assert c.table.shape[1] == tc.width(case, page)
    return c, max(n for n, _ in seqs) if most is None else most


def chain(n):
    return np.tril(np.ones((n, n), bool))


@pytest.mark.parametrize("page", [2, 16])
@pytest.mark.parametrize("fmt,dim", FORMATS)
@pytest.mark.parametrize("rows", ROWS)
def test_windows(rows, fmt, dim, page):
    """Shallow and deep nodes, deeper than the window too: the second sequence is a chain."""
    case = tc.WINDOWED[rows]
    rng = np.random.default_rng(7)
    c, most = make(case, fmt, dim, page, sees=[chain(n) if s == 1 else base.tree(n, rng) for s, (n, _) in enumerate(case[0])])
    for window in tc.WINDOWS:
        c.check("windows by %d rows" % rows, window=window, max_new=most)


@pytest.mark.parametrize("rows", ROWS)
def test_windows_with_any_masks(rows):
    """Rows that see no node, or nothing but some of the context, and bits of nodes that are not there."""
    case = tc.WINDOWED[rows]
    rng = np.random.default_rng(8)
    sees = [rng.random((n, n)) < 0.2 for n, _ in case[0]]
    sees[0][3] = False
    sees[1][:, ::2] = False
    c, most = make(case, sees=sees, junk=True, words=3)
    for window in (1, 64, 450):
        c.check("any masks by %d rows" % rows, window=window, max_new=most)


@pytest.mark.parametrize("window", tc.LONG_WINDOWS)
@pytest.mark.parametrize("fmt,page", [("fp8", 16), ("fp4", 2)])
@pytest.mark.parametrize("rows", ROWS)
def test_parts(rows, fmt, page, window):
    """Parts that begin inside a context, where the window does."""
    case = tc.LONG[rows]
    c, most = make(case, fmt, page=page)
    split, _ = c.check("parts by %d rows" % rows, window=window, max_new=most)
    whole, _ = c.run(window=window, max_new=most, workspace=None)
    assert torch.allclose(split, whole, rtol=2.0 ** -6, atol=2.0 ** -6)


@pytest.mark.parametrize("page", [2, 16])
@pytest.mark.parametrize("rows", ROWS)
def test_many_parts(rows, page):
    c, most = make(tc.MANY[rows], page=page)
    c.check("many parts by %d rows" % rows, max_new=most)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("rows", ROWS)
def test_keys_that_the_window_hides_from_deeper_nodes_hold_anything(rows, fmt):
    """NaN values at the window's edge reach the nodes that are shallow enough to see them, and no other."""
    case = tc.WINDOWED[rows]
    c, most = make(case, fmt)
    window, reached = 64, []
    for s, (n, L) in enumerate(case[0]):
        depth = c.sees[s].sum(1) - 1
        # seen where j > L - n + depth - window: by depths below 1 and below 4 (the second sequence has no context there)
        for j in (L - n - window + 1, L - n - window + 4):
            if j >= 0:
                c.parts[3][int(c.table[s, j // c.page]), :, j % c.page] = 255
                c.v[s][j] = np.nan
        reached.append(depth < 4 if L - n >= window else np.zeros(n, bool))
    c.upload()
    out, _ = c.check("hidden keys by %d rows" % rows, window=window, max_new=most)
    nan = torch.isnan(out).flatten(1)
    want = torch.from_numpy(np.concatenate(reached))
    assert torch.equal(nan.any(1).cpu(), want) and torch.equal(nan.all(1).cpu(), want) and 0 < int(want.sum()) < len(want)


@pytest.mark.parametrize("rows", ROWS)
def test_context_that_the_window_hides_holds_anything(rows):
    """Keys before the window of every node, NaN and infinite, keys and values."""
    case = tc.WINDOWED[rows]
    c, most = make(case)
    window = 70
    want, wl = c.check("window by %d rows" % rows, window=window, max_new=most)
    for s, (n, L) in enumerate(case[0]):
        for j in range(0, max(0, L - n - window + 1)):
            page, at = int(c.table[s, j // c.page]), j % c.page
            for side in (0, 2):         # codes, and their scales: NaN, or past FP32's range
                c.parts[side][page, :, at] = 0x78
                c.parts[side + 1][page, :, at] = 255 if j % 2 else 254
    c.upload()
    out, lse = c.run(window=window, max_new=most)
    assert torch.equal(out, want) and torch.equal(lse, wl)
