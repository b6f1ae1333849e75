"""GPU: the operators around the products as a served attention block runs
them (examples/attention_block.py), against the same block in 64 bits whose
only roundings are those that the block's formats define."""
from __future__ import annotations

import importlib.util
import os

import numpy as np
import pytest
import torch

import oracle
from tests import servingref as sr

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("attention_block", os.path.join(ROOT, "examples", "attention_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _mx(fmt, x):
    """Values of the MX blocks of BF16 rows."""
    rows, K = x.shape
    return sr.rows_of(fmt, *oracle.quantize(fmt, sr.bits(x), rows, K))


def _bf16(x):
    return torch.from_numpy(x).to(torch.float32).to(torch.bfloat16)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_prompt_and_decode(fmt):
    ex = _example()
    seqs, hidden, H, K, D, page = 3, 256, 8, 2, 64, 16
    torch.manual_seed(1)
    block = ex.AttentionBlock(hidden, H, K, D, seqs * 6, page, fmt)
    batch = ex.Batch(seqs, 6, page)
    wq, wo = _mx("fp8", block.w_qkv), _mx("fp8", block.w_out)
    keys = [np.zeros((0, K, D)) for _ in range(seqs)]
    values = [np.zeros((0, K, D)) for _ in range(seqs)]
    for new in (33, 17, 1, 1, 1):
        x = torch.randn(seqs * new, hidden).bfloat16()
        stream = torch.randn(seqs * new, hidden).bfloat16()
        y, h = block.forward(x.cuda(), stream.cuda(), *batch.add(new))
        h_ref = (x.float() + stream.float()).bfloat16()
        assert torch.equal(h.cpu(), h_ref)
        a = _mx("fp8", _bf16(sr.rmsnorm(sr.f64(h_ref), sr.f64(block.norm), 1e-6)))
        qkv = _bf16(a @ wq.T)
        q, k, v = (t.reshape(seqs * new, -1, D) for t in qkv.split((H * D, K * D, K * D), dim=1))
        out = np.zeros((seqs * new, H, D))
        for s in range(seqs):
            rows = slice(s * new, (s + 1) * new)
            for held, t in ((keys, k), (values, v)):
                held[s] = np.concatenate([held[s], _mx(fmt, t[rows].reshape(new * K, D)).reshape(new, K, D)])
            out[rows] = sr.attention(sr.f64(q[rows]), keys[s], values[s], D ** -0.5, True, 0, new)[0]
        ref = _mx("fp8", _bf16(out.reshape(seqs * new, H * D))) @ wo.T
        # A BF16 value that rounds the other way (the products sum in another
        # order, p is rounded to BF16) can move a code by one step, 2^-3 of an
        # E4M3 value (2^-1 of an E2M1 one in the cache); a few per cent of the
        # codes do, so the block is off by a part of that in the 2-norm.
        off = np.linalg.norm(sr.f64(y) - ref) / np.linalg.norm(ref)
        print("block", fmt, "new", new, "off by %.4f" % off, flush=True)
        assert off < (0.04 if fmt == "fp8" else 0.08)
