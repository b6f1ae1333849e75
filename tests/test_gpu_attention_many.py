"""GPU: long keys split over workgroups in calls of more than 64 sequences,
which the plan walks 64 at a time: split ones before and behind places 64 and
128, others without new tokens or of few keys between them, in the kernel of
few rows (with both of its part counts) and in the one of many rows with its
join."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import test_gpu_attention as base

pytestmark = pytest.mark.gpu

# places of the sequences with thousands of keys
LONG = (3, 62, 63, 64, 65, 100, 127, 128, 129, 131)


def _seqs(count, new, long_keys, seed, least=0):
    """Short sequences of `least` to `new` tokens, long ones of `new` tokens at LONG."""
    rng = np.random.default_rng(seed)
    seqs = []
    for s in range(count):
        if s in LONG:
            seqs.append((new, int(rng.integers(long_keys // 2, long_keys))))
        else:
            n = int(rng.integers(least, new + 1))
            seqs.append((n, n + int(rng.integers(0, 40))))
    return seqs


def _split(c):
    """Two runs, bit for bit the same, near the 64-bit form and near the run
    that does not split; counters at zero at the end."""
    a = c.check("split past 64 sequences")
    again = c.run()
    assert torch.equal(a[0], again[0]) and torch.equal(a[1], again[1]), "another run, other bits"
    assert base.counters_are_zero()
    whole = c.run(workspace=None)
    # the long ones were split: joining the parts rounds differently somewhere
    assert not torch.equal(a[0], whole[0])
    return a


@pytest.mark.parametrize("fmt,dim", [("fp8", 64), ("fp8", 128), ("fp4", 128)])
@pytest.mark.parametrize("count", [66, 132, 200])
def test_few_rows(fmt, dim, count):
    _split(base.Case(_seqs(count, 2, 3000, count), fmt, dim, heads=1, group=3, page=32))


def test_few_rows_of_many_heads():
    # 560 (sequence, head) pairs: parts for 1024 workgroups
    _split(base.Case(_seqs(70, 1, 3000, 5, least=1), "fp8", 64, heads=8, group=2, page=64))


@pytest.mark.parametrize("count,new,group", [(66, 3, 100), (132, 3, 49), (132, 6, 180)])
def test_many_rows(count, new, group):
    # tiles of 128 rows, and of 256 where a sequence has many on average; the second kernel joins the parts
    _split(base.Case(_seqs(count, new, 2500, count + new), "fp8", 64, heads=1, group=group, page=32))


def test_few_and_many_rows_in_one_call():
    seqs = _seqs(140, 2, 2500, 9)
    for s in (10, 64, 90, 130):
        seqs[s] = (40, 1800)
    _split(base.Case(seqs, "fp8", 64, heads=2, group=14, page=16))
