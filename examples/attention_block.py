"""The attention half of a transformer layer in MX formats, served: a prompt in
chunks, then one token at a time for a batch of sequences.

    RMSNorm with the residual's addition -> MX codes      mx_rmsnorm
    joint QKV product                                     mx_scaled_mm_fp8
    keys and values into the paged MX cache               mx_kv_cache_write
    attention of the new tokens over the cache            mx_paged_attention
    MX codes of its output                                mx_quantize_bf16
    output product                                        mx_scaled_mm_fp8

Random weights and inputs.  Run from the repository's root:

    python examples/attention_block.py [--fmt fp8|fp4] [--seqs N] [--prompt N] [--steps N]
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_precision_mm_amd as mx  # noqa: E402


def quantize(x):
    """BF16 [rows][K] -> E4M3 codes, E8M0 scales."""
    rows, K = x.shape
    codes = torch.empty((rows, K), dtype=torch.uint8, device=x.device)
    scales = torch.empty((rows, K // 32), dtype=torch.uint8, device=x.device)
    mx.mx_quantize_bf16(x, codes, scales, rows, K, False)
    return codes, scales


class AttentionBlock:
    """Weights in MXFP8; a paged cache in MXFP8 or MXFP4."""

    def __init__(self, hidden, q_heads, kv_heads, head_dim, pages, page_size, fmt="fp8", seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        width = (q_heads + 2 * kv_heads) * head_dim
        normal = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
        self.w_qkv = normal(width, hidden) * hidden ** -0.5
        self.w_out = normal(hidden, q_heads * head_dim) * (q_heads * head_dim) ** -0.5
        self.norm = (1 + 0.1 * normal(hidden)).bfloat16()
        self.qkv, self.out = quantize(self.w_qkv), quantize(self.w_out)
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        self.cache = mx.KVCache.empty(pages, page_size, kv_heads, head_dim, fmt)

    def forward(self, x, residual, slots, ends, lens, table, max_new):
        """x: what the layer below added, residual: the stream it belongs to
        (both bfloat16 [tokens][hidden]).  Returns this block's x and the
        stream that it belongs to."""
        T, (H, K, D) = x.shape[0], (self.q_heads, self.kv_heads, self.head_dim)
        a, sa, h = mx.rmsnorm(x, self.norm, residual)
        qkv = mx.scaled_mm(a, self.qkv[0], sa, self.qkv[1], fmt="fp8")
        q, k, v = qkv.split((H * D, K * D, K * D), dim=1)
        mx.mx_kv_cache_write(self.cache, k.unflatten(1, (K, D)), v.unflatten(1, (K, D)), slots)
        y = mx.paged_attention(self.cache, q.unflatten(1, (H, D)), ends, lens, table, max_new=max_new)
        a, sa = quantize(y.view(T, H * D))
        return mx.scaled_mm(a, self.out[0], sa, self.out[1], fmt="fp8"), h


class Batch:
    """Sequences of a fixed set of pages each: where their next tokens go."""

    def __init__(self, seqs, pages_each, page_size):
        self.page_size = page_size
        self.table = torch.randperm(seqs * pages_each, device="cuda").int().view(seqs, pages_each)
        self.lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")

    def add(self, new):
        """`new` tokens more per sequence: (slots, ends, lens, table, max_new)."""
        seqs = self.lens.shape[0]
        pos = self.lens.long()[:, None] + torch.arange(new, device="cuda")
        pages = torch.gather(self.table.long(), 1, pos // self.page_size)
        self.lens += new
        ends = torch.arange(1, seqs + 1, dtype=torch.int32, device="cuda") * new
        return (pages * self.page_size + pos % self.page_size).view(-1), ends, self.lens, self.table, new


def main():
    a = argparse.ArgumentParser()
    a.add_argument("--fmt", default="fp8", choices=("fp8", "fp4"))
    a.add_argument("--seqs", type=int, default=16)
    a.add_argument("--prompt", type=int, default=2048)
    a.add_argument("--chunk", type=int, default=512)
    a.add_argument("--steps", type=int, default=50)
    a = a.parse_args()
    hidden, page = 4096, 64
    each = -(-(a.prompt + a.steps) // page)
    block = AttentionBlock(hidden, 32, 8, 128, a.seqs * each, page, a.fmt)
    batch = Batch(a.seqs, each, page)

    def step(new):
        x = torch.randn(a.seqs * new, hidden, device="cuda").bfloat16()
        stream = torch.randn(a.seqs * new, hidden, device="cuda").bfloat16()
        where = batch.add(new)
        torch.cuda.synchronize()
        t = time.perf_counter()
        y, _ = block.forward(x, stream, *where)
        torch.cuda.synchronize()
        assert torch.isfinite(y).all()
        return time.perf_counter() - t

    took = sum(step(min(a.chunk, a.prompt - at)) for at in range(0, a.prompt, a.chunk))
    print("prompt: %d x %d tokens in chunks of %d: %.2f ms" % (a.seqs, a.prompt, a.chunk, took * 1e3))
    times = sorted(step(1) for _ in range(a.steps))
    if times:
        print("decode: %d sequences of %d keys: %.1f us a step (median of %d)"
              % (a.seqs, int(batch.lens[0]), times[len(times) // 2] * 1e6, a.steps))


if __name__ == "__main__":
    main()
