"""Host checks of the limits of the operators around the products (no GPU
needed): arguments whose own products leave FP32's range."""
from __future__ import annotations

import ctypes

import pytest

import block_scaled_precision_mm_amd as mx
from tests.test_serving_host import attend


@pytest.mark.parametrize("scale", [2.4e38, 3.4e38])
def test_a_scale_whose_exponents_are_not_finite_is_refused(scale):
    # the kernels take scale * log2 e: an infinity would make NaN of a score of 0
    assert ctypes.c_float(scale).value < float("inf")
    assert attend(scale=scale) == -9


def test_the_largest_scale_is_taken():
    # up to the device check, which a host without a GPU does not pass
    assert attend(scale=2.3e38, n=0) in (0, -7, -8)
    assert mx.mx_status_string(-9)
