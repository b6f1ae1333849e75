"""GPU: the attention's hazards again with head groups so wide that the
sequences' rows go to the kernel of many rows: tiles of 256 rows, and tiles of
128 where sequences without new tokens lower the average."""
from __future__ import annotations

import pytest
import torch

import block_scaled_precision_mm_amd as mx
from tests import test_gpu_attention as base

pytestmark = pytest.mark.gpu


@pytest.fixture(params=[0, 12])
def wide(request, monkeypatch):
    class Wide(base.Case):
        def __init__(self, seqs, fmt="fp8", dim=128, page=16, heads=2, group=4, **kw):
            super().__init__(list(seqs) + [(0, 20)] * request.param, fmt, dim, page, heads, 12 * group + 1, **kw)

    monkeypatch.setattr(base, "Case", Wide)
    return Wide


@pytest.mark.parametrize("fmt,dim", [("fp8", 64), ("fp8", 128), ("fp4", 64), ("fp4", 128)])
@pytest.mark.parametrize("page", [1, 8, 16, 64, 1024])
def test_pages(wide, fmt, dim, page):
    base.test_pages(fmt, dim, page)


@pytest.mark.parametrize("fmt,dim", [("fp8", 64), ("fp8", 128), ("fp4", 64), ("fp4", 128)])
@pytest.mark.parametrize("new", [11, 31, 100])
def test_chunks(wide, fmt, dim, new):
    base.test_chunks(fmt, dim, new)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 1, 17, 64, 100])
def test_windows(wide, causal, window):
    base.test_windows(causal, window)


def test_empty_rows(wide):
    base.test_empty_rows()


@pytest.mark.parametrize("max_new", ["known", 1, None])
def test_max_new(wide, max_new):
    base.test_max_new_changes_nothing_but_speed(max_new)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_output_types(wide, dtype):
    base.test_output_types(dtype)


def test_split_and_whole(wide):
    c = wide([(20, 1500)], heads=1, group=3, page=64)
    a = c.check("split")
    c.check("whole", workspace=None)
    again = c.run()
    assert torch.equal(a[0], again[0]) and torch.equal(a[1], again[1]), "another run, other bits"
    assert base.counters_are_zero()


@pytest.mark.parametrize("sigma,scale", [(30.0, None), (0.01, None), (1.0, 3.0)])
def test_score_ranges(wide, sigma, scale):
    base.test_score_ranges(sigma, scale)


def test_strided_queries(wide):
    base.test_strided_queries(40)


@pytest.mark.parametrize("wide", [0], indirect=True)
def test_pages_outside_the_cache(wide):
    base.test_pages_outside_the_cache(45)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("window", [0, 20])
def test_nan_values(wide, fmt, window):
    base.test_nan_values_reach_only_rows_that_see_them(fmt, 60, window)


def test_nan_keys_and_query(wide):
    base.test_nan_keys_reach_only_rows_that_see_them(60)
    base.test_nan_query_row_stays_alone()


@pytest.mark.parametrize("wide", [0], indirect=True)
def test_any_lengths_stay_in_bounds(wide):
    base.test_any_lengths_stay_in_bounds()


def test_graph_replays(wide):
    c = wide([(1, 2000), (60, 400)], heads=1)
    want = c.run()
    out, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    args = [torch.from_numpy(t).cuda() for t in (c.ends, c.lens, c.table)]
    size = mx.mx_paged_attention_workspace_bytes(c.cache, len(c.seqs), 61, c.group, 60)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    call = lambda: mx.mx_paged_attention(c.cache, c.q, *args, out, lse=lse, max_new=60, workspace=ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(4):
        out.zero_()
        lse.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        c.run()
