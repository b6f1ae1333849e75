"""GPU: mx_tree_attention against attention in 64 bits over the cache's decoded
values, with the bounds of mx_paged_attention's tests."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_scaled_precision_mm_amd as mx
from tests import servingref as sr
from tests import test_gpu_attention as base

pytestmark = pytest.mark.gpu


def tree(n, rng):
    """bool [n][n] of a random tree (or forest): what each node sees."""
    sees = np.eye(n, dtype=bool)
    for i in range(1, n):
        parent = int(rng.integers(max(-1, i - 9), i))
        if parent >= 0:
            sees[i] |= sees[parent]
    return sees


def words_of(sees, words):
    """int64 [n][words] of bool [n][m], m <= 64 words; what lies past the m is ones where `junk`."""
    n, m = sees.shape
    bits = np.zeros((n, 64 * words), np.uint64)
    bits[:, :m] = sees
    return (bits.reshape(n, words, 64) << np.arange(64, dtype=np.uint64)).sum(-1, dtype=np.uint64).view(np.int64)


def seen(sees, n, L, window):
    """bool [n][L]: the keys that each node sees."""
    at = np.zeros((n, max(L, 1)), bool)
    for i in range(n):
        depth = max(int(sees[i].sum()) - 1, 0)
        for j in range(L):
            node = j - (L - n)
            at[i, j] = sees[i, node] if node >= 0 else not window or j > L - n + depth - window
    return at[:, :L]


class Case(base.Case):
    """seqs = [(nodes, keys)]; sees: what the nodes of each see, random trees if None."""

    def __init__(self, seqs, *args, words=None, sees=None, junk=False, **kw):
        super().__init__(seqs, *args, **kw)
        rng = np.random.default_rng(kw.get("seed", 1) + 100)
        self.sees = [tree(n, rng) for n, _ in seqs] if sees is None else sees
        need = max(1, -(-max(n for n, _ in seqs) // 64))
        self.words = need if words is None else words
        rows = []
        for s in self.sees:
            n = s.shape[0]
            wide = np.zeros((n, 64 * self.words), bool)
            m = min(n, 64 * self.words)
            wide[:, :m] = s[:, :m]
            if junk:        # bits of nodes that the sequence does not have
                wide[:, n:] = rng.random((n, 64 * self.words - n)) < 0.5
            rows.append(words_of(wide, self.words))
            s[:, m:] = False
        self.mask = torch.from_numpy(np.concatenate(rows) if rows else np.zeros((0, self.words), np.int64)).cuda()

    def run(self, dtype=torch.float32, scale=None, window=0, max_new="known", workspace="auto", lse=True):
        out = torch.full(tuple(self.q.shape), 123.0, dtype=dtype, device="cuda")
        ls = torch.full((self.q.shape[0], self.heads * self.group), 123.0, device="cuda") if lse else None
        if max_new == "known":
            max_new = max(n for n, _ in self.seqs)
        mx.mx_tree_attention(self.cache, self.q, *(torch.from_numpy(t).cuda() for t in (self.ends, self.lens, self.table)),
                             self.mask, out, lse=ls, scale=scale, window=window, max_new=max_new, workspace=workspace)
        torch.cuda.synchronize()
        return out, ls

    def check(self, what, here=None, **kw):
        print("tree", what, self.fmt, self.dim, self.page, self.heads, self.group, self.seqs[:6], self.words, kw, flush=True)
        out, lse = self.run(**kw)
        scale = kw.get("scale") or self.dim ** -0.5
        q, at = sr.f64(self.q), 0
        for s, (n, L) in enumerate(self.seqs):
            mask = seen(self.sees[s], n, L, kw.get("window", 0))
            if here is not None:
                mask = mask & here[s]
            # one row at a time, of the keys that it sees
            parts = [sr.attention(q[at + i:at + i + 1], self.k[s], self.v[s], scale, False, 0, 1, mask[i]) for i in range(n)]
            if n:
                ref = [np.concatenate(t) for t in zip(*parts)]
                if out.dtype == torch.float16:
                    # below 2^-14 FP16's steps are 2^-24, so its rounding is off by up to
                    # 2^-25 whatever the value: 2^-17 of spread, of which 2^-8 is allowed
                    ref[2] = ref[2] + 2.0 ** -17
                sr.check_attention(out[at:at + n], None if lse is None else lse[at:at + n], ref, max(L, 1), "%s, sequence %d" % (what, s))
            at += n
        assert base.counters_are_zero()
        return out, lse


@pytest.mark.parametrize("fmt,dim", [("fp8", 64), ("fp8", 128), ("fp4", 64), ("fp4", 128)])
@pytest.mark.parametrize("nodes,keys", [(1, 1), (1, 200), (2, 2), (5, 37), (16, 16), (16, 300), (27, 1051), (33, 64)])
def test_one_sequence(fmt, dim, nodes, keys):
    Case([(nodes, keys)], fmt, dim).check("one sequence")


@pytest.mark.parametrize("fmt,dim", [("fp8", 64), ("fp8", 128), ("fp4", 64), ("fp4", 128)])
@pytest.mark.parametrize("nodes", [63, 64, 65, 128, 130, 200])
def test_many_nodes(fmt, dim, nodes):
    Case([(nodes, nodes + 111)], fmt, dim, heads=1, group=2).check("many nodes")


@pytest.mark.parametrize("group,nodes", [(1, 300), (4, 140), (8, 70), (16, 40)])
@pytest.mark.parametrize("dim", [64, 128])
def test_tiles_of_many_rows(group, nodes, dim):
    """Several sequences of many rows."""
    Case([(nodes, nodes + 90), (nodes, nodes + 700), (nodes, nodes), (nodes, nodes + 33)], dim=dim, heads=1, group=group).check("tiles")


@pytest.mark.parametrize("page", [1, 4, 16, 64, 512])
def test_pages(page):
    Case([(7, 300), (20, 77), (1, 1), (70, 210)], page=page).check("pages")
    Case([(70, 300), (100, 177)], page=page, heads=1).check("pages, many rows", max_new=100)


@pytest.mark.parametrize("heads,group", [(1, 1), (1, 17), (3, 5), (8, 1), (2, 7), (1, 64)])
def test_heads(heads, group):
    Case([(9, 200), (2, 65), (5, 129)], heads=heads, group=group).check("heads")


@pytest.mark.parametrize("window", [1, 2, 5, 31, 64, 100, 5000])
@pytest.mark.parametrize("seqs", [[(9, 400), (30, 210)], [(140, 500), (80, 81)]])
def test_windows(window, seqs):
    Case(seqs, heads=1).check("window", window=window)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_output_types_without_lse(dtype):
    Case([(9, 300)]).check("types", dtype=dtype, lse=False)
    Case([(9, 300)]).check("types", dtype=dtype, scale=0.3)


def test_a_chain_is_causal_attention():
    """Each node seeing all nodes before it: the rows of mx_paged_attention, with its own bounds."""
    for seqs in ([(6, 300), (40, 90)], [(130, 400)]):
        c = Case(seqs, sees=[np.tril(np.ones((n, n), bool)) for n, _ in seqs])
        out, lse = c.check("chain")
        causal, clse = base.Case.run(c)
        for a, b in ((out, causal), (lse, clse)):
            assert torch.allclose(a, b, rtol=2.0 ** -6, atol=2.0 ** -6)


def test_masks_that_are_no_trees():
    rng = np.random.default_rng(4)
    seqs = [(20, 90), (75, 75), (12, 12), (3, 40)]
    sees = [rng.random((n, n)) < 0.3 for n, _ in seqs]      # later nodes too, not always itself
    sees[2][:] = False                                      # rows that see nothing
    sees[2][4, 7] = True
    for junk in (False, True):
        out, lse = Case(seqs, sees=[s.copy() for s in sees], words=3, junk=junk).check("any bits")
        empty = slice(95, 99)
        assert (out[empty] == 0).all() and (lse[empty] == -np.inf).all()


def test_many_rows_that_see_nothing():
    n = 150
    sees = [np.zeros((n, n), bool) for _ in range(4)]
    sees[1][10, 3] = True
    out, lse = Case([(n, n)] * 4, heads=1, sees=sees).check("nothing seen")
    assert (out[:n] == 0).all() and (lse[:n] == -np.inf).all()


def test_nodes_past_the_words_are_seen_by_none():
    Case([(100, 160), (30, 45)], words=1).check("one word for 100 nodes")


def test_long_contexts_in_parts():
    for seqs in ([(13, 5000)], [(60, 9000), (3, 200)], [(80, 6000)]):
        c = Case(seqs, heads=1)
        split, lse = c.check("parts")
        whole, _ = c.check("no parts", workspace=None)
        assert torch.allclose(split, whole, rtol=2.0 ** -6, atol=2.0 ** -6)


def test_more_sequences_than_lanes():
    rng = np.random.default_rng(3)
    seqs = [(int(rng.integers(0, 6)), int(rng.integers(6, 90))) for _ in range(130)] + [(4, 3000)]
    Case(seqs, heads=1, group=2).check("131 sequences", max_new=6)


def test_few_and_many_nodes_in_a_call():
    Case([(1, 50), (150, 400), (3, 900), (90, 100)], heads=2, group=4).check("mixed")


@pytest.mark.parametrize("seqs", [[(10, 64), (7, 200)], [(150, 300), (100, 260), (90, 350)]])
@pytest.mark.parametrize("what", ["nan", "inf"])
@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_unseen_nodes_hold_anything(seqs, what, fmt):
    """A node's values are NaN or infinite: only the rows that see it have them."""
    c = Case(seqs, fmt, heads=1, group=4)
    bad = []
    for s, (n, L) in enumerate(seqs):
        j = n // 2
        c.sees[s][:, j] = False
        c.sees[s][n - 1, j] = True      # the last node sees it and no other does
        key = L - n + j
        page = int(c.table[s, key // c.page])
        if what == "nan":
            c.parts[3][page, :, key % c.page] = 255
            c.v[s][key] = np.nan
        else:                           # codes under a scale past BF16's range
            c.parts[3][page, :, key % c.page] = 254
            c.parts[2][page, :, key % c.page] = 0x77 if fmt == "fp4" else 0x78
            c.v[s][key] = np.inf
        bad.append(key)
    c.mask.copy_(torch.from_numpy(np.concatenate([words_of(s, c.words) for s in c.sees])))
    c.upload()
    out, lse = c.run()
    at, q = 0, sr.f64(c.q)
    for s, (n, L) in enumerate(seqs):
        last = out[at + n - 1]
        assert torch.isnan(last).all() if what == "nan" else (last == np.inf).all()
        assert torch.isfinite(out[at:at + n - 1]).all() and torch.isfinite(lse[at:at + n]).all()
        mask = seen(c.sees[s], n, L, 0)
        v = np.where(np.isfinite(c.v[s]), c.v[s], 0.0)
        parts = [sr.attention(q[at + i:at + i + 1], c.k[s], v, c.dim ** -0.5, False, 0, 1, mask[i]) for i in range(n - 1)]
        sr.check_attention(out[at:at + n - 1], lse[at:at + n - 1], [np.concatenate(t) for t in zip(*parts)], L, what)
        at += n


def test_unseen_keys_hold_anything():
    """NaN keys among the nodes reach the rows that see them alone."""
    for seqs in ([(10, 64)], [(150, 300), (100, 260)]):
        c = Case(seqs, heads=1)
        for s, (n, L) in enumerate(seqs):
            j = n // 3
            c.sees[s][:, j] = False
            c.sees[s][j, j] = True
            key = L - n + j
            c.parts[1][int(c.table[s, key // c.page]), :, key % c.page] = 255
            c.k[s][key] = np.nan
        c.mask.copy_(torch.from_numpy(np.concatenate([words_of(s, c.words) for s in c.sees])))
        c.upload()
        out, lse = c.check("NaN keys")
        at = 0
        for n, _ in seqs:
            rows = torch.isnan(out[at:at + n]).flatten(1).all(1)
            assert rows[n // 3] and int(rows.sum()) == 1
            at += n


def test_pages_outside_the_cache():
    for seqs in ([(10, 100)], [(150, 300), (100, 260)]):
        c = Case(seqs, heads=1)
        here = []
        for s, (n, L) in enumerate(seqs):
            ok = np.ones(L, bool)
            for page, bad in ((1, -1), ((L - n) // c.page, 1 << 30), ((L - 1) // c.page, c.cache.pages)):
                c.table[s, page] = bad
                ok[page * c.page:(page + 1) * c.page] = False
            here.append(ok)
        c.check("pages outside", here=here)


def test_lengths_of_any_content():
    """Fewer keys than nodes, none, and ends that decrease or pass the rows: the rows of the clamped ends."""
    c = Case([(8, 40), (6, 50), (5, 30)], heads=1)
    c.lens[:] = (5, 0, 30)
    c.ends[:] = (8, 3, 90)
    out, lse = c.run()
    q = sr.f64(c.q)
    # sequence 0: 8 nodes over 5 keys, node i is key i - 3
    for i in range(8):
        mask = np.array([c.sees[0][i, j + 3] for j in range(5)])
        ref = sr.attention(q[i:i + 1], c.k[0][:5], c.v[0][:5], c.dim ** -0.5, False, 0, 1, mask)
        sr.check_attention(out[i:i + 1], lse[i:i + 1], ref, 5, "fewer keys than nodes")
    # sequence 1 has no rows, sequence 2 all the rest: 11 nodes over 30 keys
    bits = c.mask[8:].cpu().numpy().view(np.uint64)[:, 0]
    for i in range(11):
        mask = np.array([j < 19 or bool(int(bits[i]) >> (j - 19) & 1) for j in range(30)])
        ref = sr.attention(q[8 + i:9 + i], c.k[2], c.v[2], c.dim ** -0.5, False, 0, 1, mask)
        sr.check_attention(out[8 + i:9 + i], lse[8 + i:9 + i], ref, 30, "the rest")


def test_rows_past_the_last_end_stay():
    c = Case([(8, 40), (6, 50)], heads=1)
    c.ends[1] = 11
    c.lens[1] = 47
    c.seqs[1] = (3, 47)
    out, lse = c.run()
    assert (out[11:] == 123).all() and (lse[11:] == 123).all() and (out[:11] != 123).all()


def test_other_stream_and_replays():
    c = Case([(9, 3000), (12, 200)], heads=1)
    want, wl = c.check("eager")
    args = [torch.from_numpy(t).cuda() for t in (c.ends, c.lens, c.table)]
    out, lse = torch.empty_like(want), torch.empty_like(wl)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    mx.mx_tree_attention(c.cache, c.q, *args, c.mask, out, lse=lse, max_new=12, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wl)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mx.mx_tree_attention(c.cache, c.q, *args, c.mask, out, lse=lse, max_new=12)
    for i in range(3):
        out.fill_(-7)
        junk = Case([(40, 900)], seed=5 + i).run()      # an eager call between, with the stream's own workspace
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wl)
        del junk


def test_the_convenience_form():
    c = Case([(9, 300)])
    want, _ = c.run(dtype=torch.bfloat16)
    args = [torch.from_numpy(t).cuda() for t in (c.ends, c.lens, c.table)]
    assert torch.equal(mx.tree_attention(c.cache, c.q, *args, c.mask, max_new=9), want)
