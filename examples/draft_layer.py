"""A transformer layer with experts in MX formats, served with drafted tokens:
a prompt in chunks, then trees of drafts, of which one path is accepted.

    RMSNorm with the residual's addition -> MX codes      mx_rmsnorm
    joint QKV product                                     mx_scaled_mm_fp8
    rotation of queries and keys, keys and values into
    the paged MX cache                                    mx_rope_cache_write
    attention of the chunk, or of the trees               mx_paged_attention, mx_tree_attention
    MX codes of its output, output product                mx_quantize_bf16, mx_scaled_mm_fp8
    RMSNorm, router product                               mx_rmsnorm, mx_dense_gemm
    tokens sorted by expert -> MX codes                   mx_moe_dispatch
    the experts' products                                 mx_grouped_mm_fp8
    rows back to their tokens with the router's weights   mx_moe_combine
    an accepted path's keys and values to their places    mx_kv_cache_read, mx_kv_cache_write

Random weights and inputs.  Run from the repository's root:

    python examples/draft_layer.py [--fmt fp8|fp4] [--seqs N] [--prompt N] [--nodes N] [--steps N]
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
    """BF16 [..][K] -> E4M3 codes, E8M0 scales."""
    K = x.shape[-1]
    codes = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    scales = torch.empty(x.shape[:-1] + (K // 32,), dtype=torch.uint8, device=x.device)
    mx.mx_quantize_bf16(x, codes, scales, x.numel() // K, K, False)
    return codes, scales


class DraftLayer:
    """Weights in MXFP8; a paged cache in MXFP8 or MXFP4."""

    def __init__(self, hidden, q_heads, kv_heads, head_dim, experts, top_k, ffn, pages, page_size, fmt="fp8", positions=4096,
                 seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        normal = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        self.experts, self.top_k, self.ffn = experts, top_k, ffn
        self.w_qkv = normal((q_heads + 2 * kv_heads) * head_dim, hidden) * hidden ** -0.5
        self.w_out = normal(hidden, q_heads * head_dim) * (q_heads * head_dim) ** -0.5
        self.w_router = normal(experts, hidden) * hidden ** -0.5
        self.w_up = normal(experts, 2 * ffn, hidden) * hidden ** -0.5
        self.w_down = normal(experts, hidden, ffn) * ffn ** -0.5
        self.norms = [(1 + 0.1 * normal(hidden)).bfloat16() for _ in range(2)]
        self.qkv, self.out, self.up, self.down = (quantize(w) for w in (self.w_qkv, self.w_out, self.w_up, self.w_down))
        self.cache = mx.KVCache.empty(pages, page_size, kv_heads, head_dim, fmt)
        self.rope = mx.rope_table(positions, head_dim)

    def attention(self, x, residual, step):
        """x: what the layer below added, residual: the stream it belongs to
        (both bfloat16 [tokens][hidden]).  What this half adds, and its stream."""
        T, (H, K, D) = x.shape[0], (self.q_heads, self.kv_heads, self.head_dim)
        a, sa, h = mx.rmsnorm(x, self.norms[0], residual)
        q, k, v = (t.unflatten(1, (-1, D)) for t in
                   mx.scaled_mm(a, self.qkv[0], sa, self.qkv[1], fmt="fp8").split((H * D, K * D, K * D), dim=1))
        mx.mx_rope_cache_write(self.cache, q, k, v, step.positions, step.slots, self.rope)      # q in place
        if step.mask is None:
            y = mx.paged_attention(self.cache, q, step.ends, step.lens, step.table, max_new=step.new)
        else:
            y = mx.tree_attention(self.cache, q, step.ends, step.lens, step.table, step.mask, max_new=step.new)
        a, sa = quantize(y.view(T, H * D))
        return mx.scaled_mm(a, self.out[0], sa, self.out[1], fmt="fp8"), h

    def route(self, b):
        """(weights, experts) of normed tokens."""
        T, hidden = b.shape
        logits = torch.empty((T, self.experts), dtype=torch.float32, device="cuda")
        mx.mx_dense_gemm(b, self.w_router, logits, T, self.experts, hidden, trans_b=1)
        top = logits.topk(self.top_k, dim=1)
        return top.values.softmax(1), top.indices

    def mixture(self, x, residual):
        """The experts' half, as attention."""
        T, hidden = x.shape
        b, _, h = mx.rmsnorm(x, self.norms[1], residual, out=torch.bfloat16)
        weights, ids = self.route(b)
        a, sa, offs, pos = mx.moe_dispatch(b, ids, self.experts)
        rows, E, F = T * self.top_k, self.experts, self.ffn
        u = torch.empty((rows, 2 * F), dtype=torch.bfloat16, device="cuda")
        mx.mx_grouped_mm_fp8(a, self.up[0], sa, self.up[1], u, offs, E, rows, 2 * F, hidden)
        a, sa = quantize(torch.nn.functional.silu(u[:, :F]) * u[:, F:])
        d = torch.empty((rows, hidden), dtype=torch.bfloat16, device="cuda")
        mx.mx_grouped_mm_fp8(a, self.down[0], sa, self.down[1], d, offs, E, rows, hidden, F)
        return mx.moe_combine(d, pos, weights), h

    def forward(self, x, residual, step):
        return self.mixture(*self.attention(x, residual, step))


class Step:
    """Where a step's tokens go: a chunk of the prompt, or a tree per sequence."""

    def __init__(self, batch, new, parents=None):
        seqs = batch.lens.shape[0]
        node = torch.arange(new, device="cuda")
        places = batch.lens.long()[:, None] + node
        self.slots = batch.slots(places).view(-1)
        self.mask, depth = None, node
        if parents is not None:
            mask = mx.tree_mask(parents)
            self.mask = mask.repeat(seqs, 1).cuda()
            depth = torch.tensor([sum(bin(w & (1 << 64) - 1).count("1") for w in row) - 1 for row in mask.tolist()], device="cuda")
        # a node's position is that of its depth, whatever its place in the cache
        self.positions = (batch.lens.long()[:, None] + depth).view(-1)
        self.lens = batch.lens + new
        self.ends = torch.arange(1, seqs + 1, dtype=torch.int32, device="cuda") * new
        self.table, self.new = batch.table, new


class Batch:
    """Sequences of a fixed set of pages each."""

    def __init__(self, seqs, pages_each, page_size):
        self.page_size = page_size
        self.table = torch.randperm(seqs * pages_each, device="cuda").int().view(seqs, pages_each)
        self.lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")

    def slots(self, places):
        return torch.gather(self.table.long(), 1, places // self.page_size) * self.page_size + places % self.page_size

    def accept(self, cache, path):
        """Keep the nodes of a path (the same for every sequence) of the last
        tree, in the order of their depths."""
        seqs, n = self.lens.shape[0], len(path)
        base = self.lens.long()[:, None]
        held = [torch.empty((seqs * n, cache.kv_heads, cache.head_dim), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
        mx.mx_kv_cache_read(cache, *held, self.slots(base + torch.tensor(path, device="cuda")).view(-1))
        mx.mx_kv_cache_write(cache, *held, self.slots(base + torch.arange(n, device="cuda")).view(-1))
        self.lens += n


def main():
    a = argparse.ArgumentParser()
    a.add_argument("--fmt", default="fp8", choices=("fp8", "fp4"))
    a.add_argument("--seqs", type=int, default=16)
    a.add_argument("--prompt", type=int, default=2048)
    a.add_argument("--chunk", type=int, default=512)
    a.add_argument("--nodes", type=int, default=15)
    a.add_argument("--steps", type=int, default=30)
    a = a.parse_args()
    hidden, page = 4096, 64
    parents = [-1] + [(i - 1) // 2 for i in range(1, a.nodes)]
    path = [0]      # the first child's line
    while 2 * path[-1] + 1 < a.nodes:
        path.append(2 * path[-1] + 1)
    longest = a.prompt + a.steps * len(path) + a.nodes
    each = -(-longest // page)
    layer = DraftLayer(hidden, 32, 8, 128, 16, 2, 2048, a.seqs * each, page, a.fmt, positions=longest)
    batch = Batch(a.seqs, each, page)

    def run(new, parents=None):
        x = torch.randn(a.seqs * new, hidden, device="cuda").bfloat16()
        stream = torch.randn(a.seqs * new, hidden, device="cuda").bfloat16()
        step = Step(batch, new, parents)
        torch.cuda.synchronize()
        t = time.perf_counter()
        y, _ = layer.forward(x, stream, step)
        torch.cuda.synchronize()
        assert torch.isfinite(y).all()
        return time.perf_counter() - t

    took = 0.0
    for at in range(0, a.prompt, a.chunk):
        new = min(a.chunk, a.prompt - at)
        took += run(new)
        batch.lens += new
    print("prompt: %d x %d tokens in chunks of %d: %.2f ms" % (a.seqs, a.prompt, a.chunk, took * 1e3))
    times = []
    for _ in range(a.steps):
        times.append(run(a.nodes, parents))
        batch.accept(layer.cache, path)
    if times:
        print("trees: %d of %d nodes, %d accepted a step: %.1f us a step (median of %d)"
              % (a.seqs, a.nodes, len(path), sorted(times)[len(times) // 2] * 1e6, a.steps))


if __name__ == "__main__":
    main()
