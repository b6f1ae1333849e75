"""GPU: the binding's convenience forms on a stream other than the current one."""
from __future__ import annotations

import pytest
import torch

import block_scaled_precision_mm_amd as mx
from tests import test_gpu_attention as base

pytestmark = pytest.mark.gpu


def test_convenience_forms_on_a_given_stream():
    s = torch.cuda.Stream()
    x, r = (torch.randn(64, 4096, device="cuda").bfloat16() for _ in "xr")
    w = (torch.randn(128, 4096, device="cuda") * 0.02).bfloat16()
    wc, ws, _ = mx.rmsnorm(w, None)
    c = base.Case([(1, 900), (50, 200)], heads=1)
    args = [torch.from_numpy(t).cuda() for t in (c.ends, c.lens, c.table)]

    def all_three(**kw):
        codes, scales, h = mx.rmsnorm(x, None, residual=r, **kw)
        return codes, scales, h, mx.scaled_mm(codes, wc, scales, ws, fmt="fp8", **kw), \
            mx.paged_attention(c.cache, c.q, *args, max_new=50, **kw)

    want = all_three()
    torch.cuda.synchronize()
    for _ in range(3):
        busy = torch.randn(4096, 4096, device="cuda")       # the current stream has work and free memory of its own
        for _ in range(4):
            busy = busy @ busy * 1e-3
        del busy
        got = all_three(stream=s)
        s.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        torch.cuda.synchronize()
