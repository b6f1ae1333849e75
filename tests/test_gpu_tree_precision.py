"""GPU: mx_tree_attention's FP32 and FP16 outputs, whose weights p are not rounded to
BF16 but taken in two BF16 parts: within bounds that the rounded ones miss.  In
tiles of 16 rows BF16 outputs have them too."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import servingref as sr
from tests import test_gpu_tree as base
from tests import treecases as tc
from tests.test_gpu_tree_windows import FORMATS, ROWS, make

pytestmark = pytest.mark.gpu

# small scores, so that their own FP32 errors stay far below those of the weights
SCALE = 0.01


def bounds(c, s, at, window):
    """64-bit outputs of sequence s (rows at ..), and how far an FP32 sum of weights in two parts may be off.

    A weight's BF16 part is off by at most 2^-8 of it, the rest is exact in FP32 and rounded to BF16 by at most 2^-8 of
    itself: 2^-16 in all (a rest below BF16's normal range: 2^-126).  Both parts of each of the n keys that a row sees are
    added in FP32, n weights in the divisor: 2 n and n steps of 2^-24; scores, as in check_attention, move a weight and its
    reference by 2 err each."""
    n, L = c.seqs[s]
    mask = base.seen(c.sees[s], n, L, window)
    q = sr.f64(c.q)[at:at + n]
    parts = [sr.attention(q[i:i + 1], c.k[s], c.v[s], SCALE, False, 0, 1, mask[i]) for i in range(n)]
    out, lse, spread, err = [np.concatenate(t) for t in zip(*parts)]
    keys = mask.sum(1)[:, None, None]
    return out, spread * (2.0 ** -16 + 4 * err[..., None] + 3 * keys * 2.0 ** -24) * 1.01 + 1e-30, spread


def weights_in_one_part(c, s, at, window):
    """What rounding the weights to BF16 gives, else in 64 bits."""
    n, L = c.seqs[s]
    mask, q, out = base.seen(c.sees[s], n, L, window), sr.f64(c.q)[at:at + n], []
    for i in range(n):
        row = np.zeros((c.heads * c.group, c.dim))
        for h in range(c.heads * c.group if mask[i].any() else 0):
            x = SCALE * (c.k[s][mask[i], h // c.group] @ q[i, h])
            p = np.exp(x - x.max())
            row[h] = sr.f64(sr.bf16(p)) @ c.v[s][mask[i], h // c.group] / p.sum()
        out.append(row)
    return np.stack(out)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("fmt,dim", FORMATS)
@pytest.mark.parametrize("rows", ROWS)
def test_weights_keep_their_bits(rows, fmt, dim, dtype):
    case = tc.SHORT[rows]
    c, most = make(case, fmt, dim)
    for window in (0, 5):
        print("precision", rows, fmt, dim, dtype, window, flush=True)
        out, _ = c.run(dtype=dtype, scale=SCALE, window=window, max_new=most)
        got, at = sr.f64(out), 0
        for s, (n, _) in enumerate(case[0]):
            want, tol, _ = bounds(c, s, at, window)
            # (FP16 below its normal range: half of 2^-24)
            tol = tol + np.abs(want) * sr.HALF[dtype] * 1.01 + (2.0 ** -25 if dtype is torch.float16 else 0.0)
            off = np.abs(got[at:at + n] - want)
            assert (off <= tol).all(), "off by %.3g where %.3g is allowed" % ((off - tol).max(), tol.flat[(off - tol).argmax()])
            # the bound is one that weights of a single part miss
            assert (np.abs(weights_in_one_part(c, s, at, window) - want) > tol).any()
            at += n


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows", ROWS)
def test_long_contexts_whole_and_in_parts(rows, dtype):
    case = tc.LONG[rows]
    c, most = make(case)
    c.check("by %d rows" % rows, max_new=most, dtype=dtype)
    c.check("whole by %d rows" % rows, max_new=most, dtype=dtype, workspace=None)


@pytest.mark.parametrize("fmt,dim", FORMATS)
def test_bf16_outputs_of_few_rows_are_the_fp32_ones_rounded_once(fmt, dim):
    for case in (tc.SHORT[16], tc.LONG[16], tc.WINDOWED[16]):
        c, most = make(case, fmt, dim)
        for window in (0, 70):
            wide, _ = c.run(window=window, max_new=most)
            half, _ = c.run(dtype=torch.bfloat16, window=window, max_new=most)
            assert torch.equal(half, wide.bfloat16())
