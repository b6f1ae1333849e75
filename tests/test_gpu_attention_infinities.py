"""GPU: values of the cache that are infinities in BF16 (a code under a scale
that takes it past the range) reach the rows that see their key, as that
infinity, and no other row: in the kernel of few rows, and in the one of many
rows with tiles of 128 and of 256."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_scaled_precision_mm_amd as mx
from tests import servingref as sr
from tests import test_gpu_attention as base

pytestmark = pytest.mark.gpu

BIG = {"fp8": 0x7E, "fp4": 0x7}         # 448 and 6
SIGN = {"fp8": 0x80, "fp4": 0x8}


def _plant(c, s, j, head, d, sign):
    """An infinity (sign +1, -1; 0: a NaN, by its scale) as value d of a key, zeros in the rest of its block."""
    page, off, b = c.table[s, j // c.page], j % c.page, d // 32
    codes, scales = c.parts[2][page, head, off], c.parts[3][page, head, off]
    if c.fmt == "fp8":
        codes[32 * b:32 * b + 32] = 0
    else:
        codes[16 * b:16 * b + 16] = 0
    c.v[s][j, head, 32 * b:32 * b + 32] = 0
    if sign == 0:
        scales[b] = 255
        c.v[s][j, head, 32 * b:32 * b + 32] = np.nan
        return
    scales[b] = 254
    code = BIG[c.fmt] | (SIGN[c.fmt] if sign < 0 else 0)
    if c.fmt == "fp8":
        codes[d] = code
    else:
        codes[d // 2] = code << (4 * (d % 2))
    c.v[s][j, head, d] = sign * np.inf


def _check(c, what, **kw):
    """As Case.check, with the places of the infinities compared too."""
    out, lse = c.check(what, **kw)
    q, at = sr.f64(c.q), 0
    for s, (n, L) in enumerate(c.seqs):
        ref = sr.attention(q[at:at + n], c.k[s], c.v[s], c.dim ** -0.5, kw.get("causal", True), kw.get("window", 0), n)[0]
        got = sr.f64(out[at:at + n])
        odd = ~np.isfinite(ref)
        assert np.array_equal(np.isfinite(got), ~odd), "%s, sequence %d: finite elsewhere" % (what, s)
        assert np.array_equal(got[odd], ref[odd], equal_nan=True), "%s, sequence %d" % (what, s)
        at += n
    return out, lse


# new tokens and heads of a group: rows of the kernel of few rows (16 and 32 a
# tile) and of the kernel of many; `empty` sequences without new tokens lower
# the average, for tiles of 128 rows
SHAPES = [(1, 3, 0), (3, 2, 0), (20, 2, 0), (60, 16, 0), (60, 16, 12)]


@pytest.mark.parametrize("fmt,dim", [("fp8", 64), ("fp8", 128), ("fp4", 64), ("fp4", 128)])
@pytest.mark.parametrize("new,group,empty", SHAPES)
@pytest.mark.parametrize("window", [0, 40])
def test_infinities_reach_only_rows_that_see_them(fmt, dim, new, group, empty, window):
    L = 300
    c = base.Case([(new, L), (new, 70)] + [(0, 20)] * empty, fmt, dim, heads=2, group=group)
    _plant(c, 0, L - 1, 0, 5, +1)                       # a future key for all tokens but the last
    _plant(c, 0, L - max(new // 2, 1), 0, 40, -1)
    _plant(c, 0, L - new - 35, 1, 33, -1)               # before some tokens' window
    _plant(c, 0, L - new - 5, 1, 2, +1)
    _plant(c, 1, 0, 0, 6, -1)                           # the first tile's first key
    _plant(c, 1, 69, 1, 6, +1)
    c.upload()
    _check(c, "infinities", window=window)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("new,group,empty", SHAPES)
def test_infinities_that_every_row_sees(fmt, new, group, empty):
    # whole tiles: the first one, one in the middle, and both infinities or a NaN and one in a column
    L = 700
    c = base.Case([(new, L)] + [(0, 20)] * empty, fmt, heads=1, group=group)
    _plant(c, 0, 3, 0, 5, +1)
    _plant(c, 0, 17, 0, 41, -1)
    _plant(c, 0, 300, 0, 70, -1)
    _plant(c, 0, 301, 0, 71, +1)
    _plant(c, 0, 310, 0, 71, -1)                        # +inf and -inf: NaN
    _plant(c, 0, 320, 0, 100, +1)
    _plant(c, 0, 321, 0, 100, 0)                        # and a block of NaNs
    c.upload()
    a = _check(c, "seen infinities")
    b = _check(c, "seen infinities, not split", workspace=None)
    for t, u in zip(a, b):
        assert torch.equal(torch.isnan(t), torch.isnan(u))


@pytest.mark.parametrize("new,group", [(1, 2), (20, 2), (60, 16)])
def test_an_infinity_whose_weight_underflows(new, group):
    # its key's score lies so far below the others' that its weight is 0 in FP32,
    # in its own tile and in another one: the sums that see it are infinite still
    L, D = 6000, 128
    c = base.Case([(new, L)], dim=D, heads=1, group=group, page=64)
    c.q.fill_(16.0)
    for j, kcode in [(j, 0x38) for j in range(L)] + [(10, 0xC8), (4000, 0xC8)]:        # 1.0, and -4.0
        page, off = c.table[0, j // 64], j % 64
        c.parts[0][page, 0, off] = kcode
        c.parts[1][page, 0, off] = 127
    c.k[0][:] = 1.0
    c.k[0][[10, 4000]] = -4.0                           # scores 181 and -724
    _plant(c, 0, 10, 0, 9, +1)
    _plant(c, 0, 4000, 0, 64, -1)
    c.upload()
    for workspace in ("auto", None):
        out, _ = c.run(workspace=workspace)
        o = sr.f64(out)
        assert (o[:, :, 9] == np.inf).all() and (o[:, :, 64] == -np.inf).all()
        rest = np.delete(np.arange(D), np.r_[np.arange(0, 32), np.arange(64, 96)])
        assert np.isfinite(o[:, :, rest]).all() and np.isfinite(np.delete(o, [9, 64], axis=2)).all()
    assert base.counters_are_zero()


@pytest.mark.parametrize("new,group", [(1, 2), (20, 2), (60, 16)])
def test_a_nan_score_beside_an_infinity(new, group):
    c = base.Case([(new, 100)], heads=1, group=group)
    _plant(c, 0, 0, 0, 5, +1)
    c.upload()
    c.q[new - 1, 1, 3] = float("nan")
    out, lse = c.run()
    o = sr.f64(out)
    assert np.isnan(o[new - 1, 1]).all() and torch.isnan(lse[new - 1, 1])
    rows = np.ones(o.shape[:2], bool)
    rows[new - 1, 1] = False
    assert (o[rows][:, 5] == np.inf).all() and np.isfinite(np.delete(o[rows], 5, axis=1)).all()


def test_infinities_as_they_are_read_back():
    # the cache's own reading takes the same values past the range
    c = mx.KVCache.empty(1, 1, 1, 32, "fp8")
    c.k_codes.view(-1)[:3] = torch.tensor([0x7E, 0xFE, 0x38], dtype=torch.uint8, device="cuda")
    c.k_scales.fill_(247)
    k, v = (torch.empty(1, 1, 32, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    mx.mx_kv_cache_read(c, k, v, torch.zeros(1, dtype=torch.int64, device="cuda"))
    assert k[0, 0, :3].tolist() == [float("inf"), float("-inf"), 2.0 ** 120]
