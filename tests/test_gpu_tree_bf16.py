"""GPU: mx_tree_attention into BF16, whose weights are of one part in tiles of 32
rows and more: the tests of FP32 outputs by each of these kernels, with the
outputs' own rounding allowed for (servingref.check_attention)."""
from __future__ import annotations

import pytest
import torch

from tests import test_gpu_tree as base
from tests import test_gpu_tree_kernels as kernels
from tests import test_gpu_tree_windows as windows
from tests import treecases as tc

pytestmark = pytest.mark.gpu

KERNELS = ["32 rows", "tiles"]
ROWS = [32, 128, 256]


@pytest.fixture(autouse=True)
def bf16_outputs(monkeypatch):
    assert base.Case.run.__defaults__[0] is torch.float32
    monkeypatch.setattr(base.Case.run, "__defaults__", (torch.bfloat16,) + base.Case.run.__defaults__[1:])


def test_the_outputs_are_bf16():
    assert base.Case([(3, 40)]).run()[0].dtype is torch.bfloat16


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("fmt,dim", windows.FORMATS)
@pytest.mark.parametrize("seqs", [[(40, 333), (30, 31), (64, 130)], [(130, 500), (70, 70), (100, 611)]])
def test_sizes(kernel, fmt, dim, seqs):
    kernels.test_sizes(kernel, fmt, dim, seqs)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("page", [1, 64])
def test_pages(kernel, page):
    kernels.test_pages(kernel, page)


@pytest.mark.parametrize("kernel", KERNELS)
def test_masks_that_are_no_trees(kernel):
    kernels.test_masks_that_are_no_trees(kernel)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("what", ["nan", "inf"])
@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_unseen_nodes_hold_anything(kernel, what, fmt):
    kernels.test_unseen_nodes_hold_anything(kernel, what, fmt)


@pytest.mark.parametrize("kernel", KERNELS)
def test_pages_outside_the_cache(kernel):
    kernels.test_pages_outside_the_cache(kernel)


@pytest.mark.parametrize("kernel", KERNELS)
def test_replays(kernel):
    kernels.test_replays(kernel)


@pytest.mark.parametrize("fmt,dim", windows.FORMATS)
@pytest.mark.parametrize("rows", ROWS)
def test_windows(rows, fmt, dim):
    windows.test_windows(rows, fmt, dim, 16)


@pytest.mark.parametrize("rows", ROWS)
def test_windows_with_any_masks(rows):
    windows.test_windows_with_any_masks(rows)


@pytest.mark.parametrize("window", tc.LONG_WINDOWS)
@pytest.mark.parametrize("rows", ROWS)
def test_parts(rows, window):
    windows.test_parts(rows, "fp8", 16, window)


@pytest.mark.parametrize("rows", ROWS)
def test_many_parts(rows):
    windows.test_many_parts(rows, 16)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("rows", ROWS)
def test_keys_that_the_window_hides_from_deeper_nodes_hold_anything(rows, fmt):
    windows.test_keys_that_the_window_hides_from_deeper_nodes_hold_anything(rows, fmt)


@pytest.mark.parametrize("rows", ROWS)
def test_context_that_the_window_hides_holds_anything(rows):
    windows.test_context_that_the_window_hides_holds_anything(rows)
