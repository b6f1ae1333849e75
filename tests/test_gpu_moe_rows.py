"""GPU: mx_moe_combine_grad where two assignments name one row: the weights'
gradients, the other rows and the memory behind them are as ever, and
mx_moe_combine takes such rows as any.  And mx_moe_dispatch around the number of
chunks that its workgroups add up."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_scaled_precision_mm_amd as mx
from tests import servingref as sr
from tests import test_gpu_moe as base

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out", ["same", "fp8", "fp4"])
@pytest.mark.parametrize("tokens,top_k,N", [(40, 4, 96), (33, 6, 2080)])
def test_gradient_of_rows_that_are_named_twice(tokens, top_k, N, out):
    y, pos, w = base.inputs(tokens, top_k, N, torch.bfloat16, drop=0.0)
    twice = int(pos[3, 1])
    pos[3, 2] = twice           # by one token, and by another
    pos[17, 0] = twice
    d_out = torch.randn((tokens, N), device="cuda", generator=torch.Generator(device="cuda").manual_seed(4)).bfloat16()
    rows = y.shape[0]
    if out == "same":
        d_y, d_s = torch.full_like(y, 9.0), None
    else:
        d_y, d_s = base.buffers(rows, N, out)
    d_w = torch.empty((tokens, top_k), device="cuda")
    mx.mx_moe_combine_grad(d_out, y, pos, w, d_y, d_s, d_w)
    torch.cuda.synchronize()
    p, here = pos.cpu().numpy(), np.ones((tokens, top_k), bool)
    prod = sr.f64(d_out)[:, None, :] * sr.f64(y)[p]
    steps = 8 * -(-N // 2048) + 10
    assert (np.abs(sr.f64(d_w) - prod.sum(-1)) <= np.abs(prod).sum(-1) * steps * 2.0 ** -24 * 1.01).all()
    # the other rows: those of the same call without the two that name it again
    here[3, 2] = here[17, 0] = False
    alone = pos.clone()
    alone[torch.from_numpy(~here).cuda()] = -1
    want_y, want_s = torch.full_like(d_y, 9.0) if out == "same" else base.buffers(rows, N, out)[0], base.buffers(rows, N, out)[1] if out != "same" else None
    mx.mx_moe_combine_grad(d_out, y, alone, w, want_y, want_s, None)
    torch.cuda.synchronize()
    keep = torch.arange(rows, device="cuda") != twice
    assert torch.equal(d_y[keep], want_y[keep]) and (d_s is None or torch.equal(d_s[keep], want_s[keep]))


def test_combine_of_rows_that_are_named_twice():
    y, pos, w = base.inputs(20, 3, 264, torch.float32, drop=0.0)
    pos[:, 1] = pos[:, 0]
    pos[7:] = pos[0]
    want, size = base.combined(y, pos, w)
    got = sr.f64(mx.moe_combine(y, pos, w, torch.float32))
    assert (np.abs(got - want) <= size * 4 * 2.0 ** -24 * 1.01).all()


@pytest.mark.parametrize("tokens", [16384, 32767, 32768, 32769, 33000])
def test_dispatch_at_the_most_chunks_that_each_workgroup_adds_up(tokens):
    base.check_dispatch(tokens, 8, 40, 32)
    base.check_dispatch(tokens * 8, 1, 1024, 32, "bf16")
