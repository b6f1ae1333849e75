"""GPU: the operators for drafted tokens and for experts called side by side:
from two host threads on one stream, on two streams, and in graphs that are
replayed in any order between eager calls, all with the binding's own
workspaces."""
from __future__ import annotations

import threading

import pytest
import torch

import block_scaled_precision_mm_amd as mx
from tests import test_gpu_tree as base
from tests.test_gpu_tree_kernels import widen

pytestmark = pytest.mark.gpu


class Tree:
    """A call that splits key ranges, on fixed buffers, and its result alone."""

    def __init__(self, seqs, seed, kernel="16 rows"):
        self.c = widen(base.Case(seqs, heads=1, seed=seed), kernel)
        self.args = [torch.from_numpy(t).cuda() for t in (self.c.ends, self.c.lens, self.c.table)]
        self.out = torch.empty(self.c.q.shape, device="cuda")
        self.run()
        torch.cuda.synchronize()
        self.want = self.out.clone()

    def run(self, stream=None):
        mx.mx_tree_attention(self.c.cache, self.c.q, *self.args, self.c.mask, self.out, max_new=self.c.seqs[0][0], stream=stream)

    def same(self):
        ok = torch.equal(self.out, self.want)
        self.out.fill_(-7)
        return ok


class Experts:
    """A dispatch that counts in chunks, and the way back."""

    def __init__(self, tokens, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.x = torch.randn((tokens, 256), generator=g, device="cuda").bfloat16()
        self.ids = torch.randint(-1, 33, (tokens, 4), generator=g, device="cuda")
        self.w = torch.rand((tokens, 4), generator=g, device="cuda")
        self.y = torch.zeros((tokens * 4, 256), dtype=torch.bfloat16, device="cuda")
        self.offs = torch.zeros(32, dtype=torch.int32, device="cuda")
        self.pos = torch.zeros((tokens, 4), dtype=torch.int32, device="cuda")
        self.out = torch.zeros_like(self.x)
        self.run()
        torch.cuda.synchronize()
        self.want = [t.clone() for t in self.results()]

    def results(self):
        return self.y, self.offs, self.pos, self.out

    def run(self, stream=None):
        mx.mx_moe_dispatch(self.x, self.ids, self.y, None, self.offs, self.pos, stream=stream)
        mx.mx_moe_combine(self.y, self.pos, self.w, self.out, stream=stream)

    def same(self):
        ok = all(torch.equal(a, b) for a, b in zip(self.results(), self.want))
        for t in self.results():
            t.zero_()
        return ok


def calls():
    return [Tree([(12, 9000)], 1), Experts(5000, 2), Tree([(70, 5000), (60, 3000)], 3, "tiles"), Experts(30000, 4)]


def test_two_host_threads_on_one_stream():
    work = calls()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    errors = []

    def many(which):
        try:
            for _ in range(30):
                for c in which:
                    c.run(stream=s)
        except Exception as e:      # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=many, args=(work[i::2],)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors and all(c.same() for c in work)
    assert base.base.counters_are_zero()


def test_two_streams():
    work = calls()
    streams = [torch.cuda.Stream() for _ in work]
    torch.cuda.synchronize()
    for _ in range(10):
        for c, s in zip(work, streams):
            c.run(stream=s)
    torch.cuda.synchronize()
    assert all(c.same() for c in work)
    assert base.base.counters_are_zero()


def test_graphs_replayed_in_any_order():
    work = calls()
    graphs = []
    for c in work:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run()
            c.run()
        graphs.append(g)
    for order in ([0, 1, 2, 3], [3, 1, 0, 2], [2, 2, 0, 1, 3]):
        for i in order:
            graphs[i].replay()
            work[(i + 1) % 4].run()
            torch.cuda.synchronize()
            assert work[i].same() and work[(i + 1) % 4].same()
