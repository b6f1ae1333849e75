"""GPU: the binding's own workspaces (workspace="auto") in captured graphs:
every replay gives the eager result, whatever the stream's later calls need
and in whichever order the graphs are replayed."""
from __future__ import annotations

import pytest
import torch

import block_scaled_precision_mm_amd as mx
from tests import test_gpu_attention as base

pytestmark = pytest.mark.gpu


class Call:
    """An attention call on fixed buffers, and its eager result without splitting's help from another workspace."""

    def __init__(self, seqs, seed, **kw):
        self.c = base.Case(seqs, heads=1, seed=seed, **kw)
        self.args = [torch.from_numpy(t).cuda() for t in (self.c.ends, self.c.lens, self.c.table)]
        self.most = max(n for n, _ in seqs)
        self.out = torch.empty(self.c.q.shape, device="cuda")
        assert self.need() > 0, "a call that splits"
        ws = torch.zeros(self.need(), dtype=torch.uint8, device="cuda")
        self.run(ws)
        torch.cuda.synchronize()
        self.want = self.out.clone()

    def need(self):
        return mx.mx_paged_attention_workspace_bytes(self.c.cache, len(self.c.seqs), self.c.q.shape[0], self.c.group, self.most)

    def run(self, workspace="auto"):
        mx.mx_paged_attention(self.c.cache, self.c.q, *self.args, self.out, max_new=self.most, workspace=workspace)

    def capture(self, stream):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            self.run()
            self.run()
        return g

    def same(self):
        torch.cuda.synchronize()
        ok = torch.equal(self.out, self.want)
        self.out.fill_(-7)
        torch.cuda.synchronize()
        return ok


def _calls():
    # few rows (their counters), then tiles of many rows (a larger workspace)
    return Call([(1, 3000)], 1, group=4), Call([(3, 2000), (1, 900)], 2, group=2), Call([(60, 1500)], 3, group=12)


def test_replays_after_larger_calls_of_the_stream():
    small, _, large = _calls()
    assert large.need() > small.need()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        small.run()                         # the stream's own workspace is there before the capture
    assert small.same()
    g = small.capture(s)
    with torch.cuda.stream(s):
        large.run()                         # and replaced by a larger one
        junk = [torch.full((1 << 20,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(40)]
    assert large.same()
    for _ in range(4):
        g.replay()
        assert small.same()
        with torch.cuda.stream(s):
            large.run()
        assert large.same()
    assert all(bool((t == 0xFF).all()) for t in junk)


def test_graphs_of_one_stream_in_any_order():
    calls = _calls()
    s = torch.cuda.Stream()
    graphs = [c.capture(s) for c in calls]
    for c in calls:
        c.out.fill_(-7)
    torch.cuda.synchronize()
    for order in ((2, 1, 0), (0, 1, 2), (1, 1, 2, 0, 2)):
        for i in order:
            graphs[i].replay()
            assert calls[i].same(), order
    with torch.cuda.stream(s):
        calls[1].run()
    assert calls[1].same()


def test_a_captured_product_that_splits():
    M, N, K = 128, 4096, 14336
    g = torch.Generator(device="cuda").manual_seed(1)
    a, b = (torch.randint(0, 256, (n, K // 2), dtype=torch.uint8, device="cuda", generator=g) for n in (M, N))
    sa, sb = (torch.randint(120, 134, (n, K // 32), dtype=torch.uint8, device="cuda", generator=g) for n in (M, N))
    assert mx.mx_scaled_mm_workspace_bytes(True, M, N, K) > 0
    c = torch.empty(M, N, device="cuda")
    mx.mx_scaled_mm_fp4(a, b, sa, sb, c, M, N, K)
    torch.cuda.synchronize()
    want = c.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mx.mx_scaled_mm_fp4(a, b, sa, sb, c, M, N, K)
    for _ in range(3):
        c.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c, want)
        mx.mx_scaled_mm_fp4(a, b, sa, sb, c, M, N, K)
        torch.cuda.synchronize()
