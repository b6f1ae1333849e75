"""GPU: mx_rmsnorm against the formula in 64 bits, and its MX outputs against
the oracle's quantizer on its own BF16 output (bit for bit)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_scaled_precision_mm_amd as mx
import oracle
from tests import servingref as sr

pytestmark = pytest.mark.gpu


def _run(x, res, w, eps, out, in_place=False):
    rows, K = x.shape
    d = [None if t is None else t.cuda() for t in (x, res, w)]
    h = None if res is None else (d[1] if in_place else torch.empty_like(d[0]))
    ys = None
    if out in ("fp8", "fp4"):
        y = torch.full((rows, K if out == "fp8" else K // 2), 0xAB, dtype=torch.uint8, device="cuda")
        ys = torch.full((rows, K // 32), 0xAB, dtype=torch.uint8, device="cuda")
    else:
        y = torch.full((rows, K), 7.0, dtype=out, device="cuda")
    mx.mx_rmsnorm(d[0], d[1], d[2], h, y, ys, rows, K, eps)
    torch.cuda.synchronize()
    return y.cpu(), None if ys is None else ys.cpu(), None if h is None else h.cpu()


def _check(x, res, w, eps, what):
    print("rmsnorm", what, tuple(x.shape), flush=True)
    h = x if res is None else (x.float() + res.float()).to(torch.bfloat16)
    ref = sr.rmsnorm(sr.f64(h), None if w is None else sr.f64(w), eps)
    got = {}
    for out in (torch.float32, torch.bfloat16, torch.float16):
        y, _, gh = _run(x, res, w, eps, out)
        if res is not None:
            assert np.array_equal(sr.bits(gh), sr.bits(h)), what + ": h"
        got[out] = y
        # r and two products are rounded to FP32, then the output: half a step
        # of it, or of its smallest subnormal
        tiny = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}[out]
        tol = np.abs(ref) * ((1 + 2.0 ** -24) ** 3 * (1 + sr.HALF[out]) - 1 + 2.0 ** -50) + tiny
        y64 = sr.f64(y)
        assert np.array_equal(np.isnan(y64), np.isnan(ref)), what
        fin = np.abs(ref) < (6e4 if out == torch.float16 else 1e38)
        assert (np.abs(y64 - ref)[fin] <= tol[fin]).all(), "%s %s: off by %.3g" % (what, out, np.nanmax(np.abs(y64 - ref)))
    for fmt in ("fp8", "fp4"):
        codes, scales, _ = _run(x, res, w, eps, fmt)
        oc, os_ = oracle.quantize(fmt, sr.bits(got[torch.bfloat16]), *x.shape)
        assert np.array_equal(scales.numpy(), os_), "%s %s: scales" % (what, fmt)
        assert np.array_equal(codes.numpy(), oc), "%s %s: codes" % (what, fmt)


@pytest.mark.parametrize("rows,K", [(1, 32), (3, 96), (2, 512), (5, 544), (7, 2048), (2, 2080), (3, 4128), (4, 6144),
                                    (33, 8192), (2, 9216), (2, 16384), (2, 16416), (1, 33024), (2, 65536)])
@pytest.mark.parametrize("residual", [False, True])
def test_shapes(rows, K, residual):
    rng = np.random.default_rng(rows * 131 + K)
    x = sr.bf16(rng.standard_normal((rows, K)))
    res = sr.bf16(rng.standard_normal((rows, K)) * 5) if residual else None
    w = sr.bf16(1 + 0.3 * rng.standard_normal(K))
    _check(x, res, w, 1e-6, "normal")


def test_without_weight_and_with_outliers():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((6, 1024))
    x[:, 17] *= 1000
    _check(sr.bf16(x), None, None, 1e-5, "outliers")


def test_zero_rows_and_extremes():
    x = np.zeros((7, 256))
    x[1] = 3e38                     # the squares overflow FP32, not FP64
    x[2] = 1e-38
    x[3, 5] = -2e19
    x[4] = np.linspace(-1, 1, 256)
    x[5] = 1e-20
    w = sr.bf16(np.linspace(-2, 2, 256))
    _check(sr.bf16(x), None, w, 1e-6, "extremes")
    _check(sr.bf16(x), None, None, 1e-30, "extremes, small eps")


def test_norms_beyond_the_normal_range():
    # 1 / norm is subnormal in FP32, or past its largest value
    x = np.stack([np.linspace(1, 3.3, 256) * 1e38, np.linspace(-3, 3.05, 256) * 1.1e38, np.full(256, 2.0 ** -133),
                  np.linspace(1, 120, 256).round() * 2.0 ** -133, np.linspace(-1, 1, 256)])
    _check(sr.bf16(x), None, sr.bf16(np.linspace(-2, 2, 256)), 0.0, "beyond the normal range")


def test_more_rows_than_a_launch_holds():
    # 64 threads a row: 2^26 - 1 rows are a launch's most
    rows, K = 2 ** 26 + 5, 32
    x = torch.ones(1, 1, dtype=torch.bfloat16, device="cuda").expand(rows, K).contiguous()
    tail = torch.randn(16, K, device="cuda").bfloat16()
    x[-16:] = tail
    y = torch.empty(rows, K // 2, dtype=torch.uint8, device="cuda")
    ys = torch.empty(rows, 1, dtype=torch.uint8, device="cuda")
    mx.mx_rmsnorm(x, None, None, None, y, ys, rows, K, 0.0)
    want, want_s, _ = mx.rmsnorm(tail, None, eps=0.0, out="fp4")
    assert torch.equal(y[-16:], want) and torch.equal(ys[-16:].view(-1), want_s.view(-1))
    one, one_s, _ = mx.rmsnorm(x[:1].contiguous(), None, eps=0.0, out="fp4")
    assert bool((y[:-16] == one).all()) and bool((ys[:-16] == one_s.view(-1)).all())


def test_nan_and_inf_rows_stay_apart():
    rng = np.random.default_rng(6)
    x = rng.standard_normal((5, 640))
    x[1, 3] = np.nan
    x[3, 600] = np.inf
    y, _, _ = _run(sr.bf16(x), None, None, 1e-6, torch.float32)
    n = torch.isnan(y)
    assert n[1].all() and n[3, 600] and not n[0].any() and not n[2].any() and not n[4].any()
    assert (y[3, :600] == 0).all()              # x / inf
    codes, scales, _ = _run(sr.bf16(x), None, None, 1e-6, "fp8")
    assert (scales[1] == 255).all() and (codes[1] == 0).all() and (scales[0] != 255).all()


def test_residual_stream_in_place():
    rng = np.random.default_rng(7)
    x, res = sr.bf16(rng.standard_normal((9, 4096))), sr.bf16(rng.standard_normal((9, 4096)))
    y0, s0, h0 = _run(x, res, None, 1e-6, "fp8")
    y1, s1, h1 = _run(x, res, None, 1e-6, "fp8", in_place=True)
    assert torch.equal(y0, y1) and torch.equal(s0, s1) and torch.equal(h0.view(torch.int16), h1.view(torch.int16))


def test_convenience_form_feeds_the_product():
    rng = np.random.default_rng(8)
    M, N, K = 24, 64, 512
    x = sr.bf16(rng.standard_normal((M, K))).cuda()
    w = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    codes, scales, h = mx.rmsnorm(x, w)
    b, sb = oracle.quantize("fp8", sr.bits(sr.bf16(rng.standard_normal((N, K)))), N, K)
    c = mx.scaled_mm(codes, torch.from_numpy(b).cuda(), scales, torch.from_numpy(sb).cuda(), fmt="fp8",
                     out_dtype=torch.float32)
    ref = sr.rows_of("fp8", codes.cpu().numpy(), scales.cpu().numpy()) @ sr.rows_of("fp8", b, sb).T
    assert h is x
    assert np.abs(sr.f64(c) - ref).max() <= 1e-4 * np.abs(ref).max()


def test_other_stream_and_empty():
    s = torch.cuda.Stream()
    x = torch.randn(64, 4096, device="cuda").bfloat16()
    want = mx.rmsnorm(x, None)
    s.wait_stream(torch.cuda.current_stream())
    y, ys = torch.empty_like(want[0]), torch.empty_like(want[1])
    mx.mx_rmsnorm(x, None, None, None, y, ys, 64, 4096, 1e-6, stream=s)
    s.synchronize()
    assert torch.equal(y, want[0]) and torch.equal(ys, want[1])
    mx.rmsnorm(x[:0], None)
