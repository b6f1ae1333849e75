"""GPU: trees deeper than a window.  With the bits of the ancestors that the window
is to hide left out of the masks, mx_tree_attention gives a window of positions:
node i at depth d is position L - n + d, and sees positions above that less the
window, among its ancestors and the context."""
from __future__ import annotations

import numpy as np
import pytest

import block_scaled_precision_mm_amd as mx
from tests import servingref as sr
from tests import test_gpu_tree as base
from tests import treecases as tc
from tests.test_gpu_tree_windows import ROWS, make

pytestmark = pytest.mark.gpu


def parents_of(n, rng):
    """A tree of branches that are many nodes deep."""
    return [-1] + [int(rng.integers(max(0, i - 3), i)) for i in range(1, n)]


@pytest.mark.parametrize("window", [1, 4, 11, 40])
@pytest.mark.parametrize("rows", ROWS)
def test_masks_without_the_ancestors_that_a_window_hides(rows, window):
    case = tc.WINDOWED[rows]
    rng = np.random.default_rng(5)
    sees, positions = [], []
    for n, L in case[0]:
        parents = parents_of(n, rng)
        words = mx.tree_mask(parents).numpy().view(np.uint64)
        full = np.array([[bool(int(words[i, j // 64]) >> (j % 64) & 1) for j in range(n)] for i in range(n)])
        depth = full.sum(1) - 1
        sees.append(full & (depth[None, :] > depth[:, None] - window))
        j = np.arange(L)
        at = np.zeros((n, L), bool)
        for i in range(n):
            context = j < L - n
            at[i] = context & (j > L - n + depth[i] - window)
            for a in np.flatnonzero(full[i]):
                at[i, L - n + a] = depth[a] > depth[i] - window
        positions.append(at)
    if window <= 11:        # the trees are deeper: some node has as many as the window leaves, itself among them
        assert max(s.sum(1).max() for s in sees) == window
    c, most = make(case, sees=sees)
    out, lse = c.run(window=window, max_new=most)
    q, at = sr.f64(c.q), 0
    for s, (n, L) in enumerate(case[0]):
        parts = [sr.attention(q[at + i:at + i + 1], c.k[s], c.v[s], c.dim ** -0.5, False, 0, 1, positions[s][i]) for i in range(n)]
        sr.check_attention(out[at:at + n], lse[at:at + n], [np.concatenate(t) for t in zip(*parts)], L, "sequence %d" % s)
        assert np.array_equal(base.seen(c.sees[s], n, L, window), positions[s])
        at += n
