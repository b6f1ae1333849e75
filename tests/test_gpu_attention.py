"""GPU: mx_paged_attention against attention in 64 bits over the cache's
decoded values, with bounds counted from the kernels' roundings."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_scaled_precision_mm_amd as mx
import oracle
from tests import servingref as sr

pytestmark = pytest.mark.gpu


class Case:
    """A cache whose unused places hold NaN codes and scales, and the inputs
    of seqs = [(new tokens, keys)] over it."""

    def __init__(self, seqs, fmt="fp8", dim=128, page=16, heads=2, group=4, seed=1, sigma=1.0, extra=3, q_pad=0):
        rng = np.random.default_rng(seed)
        self.seqs, self.fmt, self.dim, self.page, self.heads, self.group = seqs, fmt, dim, page, heads, group
        per = [-(-L // page) for _, L in seqs]
        pages = max(1, sum(per) + extra)
        self.cache = mx.KVCache.empty(pages, page, heads, dim, fmt)
        self.table = np.full((len(seqs), max(per + [1]) + 1), -1, np.int32)
        order, at = rng.permutation(pages), 0
        self.k, self.v = [], []
        parts = [np.full(tuple(t.shape), 0xFF, np.uint8) for t in
                 (self.cache.k_codes, self.cache.k_scales, self.cache.v_codes, self.cache.v_scales)]
        for s, (n, L) in enumerate(seqs):
            mine = order[at:at + per[s]]
            at += per[s]
            self.table[s, :per[s]] = mine
            j = np.arange(L)
            for side, c, e in ((self.k, 0, 1), (self.v, 2, 3)):
                x = sr.bf16(rng.standard_normal((L * heads, dim)) * sigma * np.exp2(rng.integers(-2, 3, (L * heads, 1))))
                codes, scales = oracle.quantize(fmt, sr.bits(x), L * heads, dim)
                if L:
                    parts[c][mine[j // page], :, j % page] = codes.reshape(L, heads, -1)
                    parts[e][mine[j // page], :, j % page] = scales.reshape(L, heads, -1)
                    side.append(sr.rows_of(fmt, codes.reshape(L, heads, -1), scales.reshape(L, heads, -1)))
                else:
                    side.append(np.zeros((0, heads, dim)))
        self.parts = parts
        tokens = sum(n for n, _ in seqs)
        Hq = heads * group
        wide = sr.bf16(rng.standard_normal((tokens, Hq * dim + q_pad)) * sigma)
        self.q = wide.cuda()[:, :Hq * dim].unflatten(1, (Hq, dim))
        self.ends = np.cumsum([n for n, _ in seqs]).astype(np.int32)
        self.lens = np.array([L for _, L in seqs], np.int32)
        self.upload()

    def upload(self):
        for t, p in zip((self.cache.k_codes, self.cache.k_scales, self.cache.v_codes, self.cache.v_scales), self.parts):
            t.copy_(torch.from_numpy(p))

    def run(self, dtype=torch.float32, scale=None, causal=True, window=0, max_new="known", workspace="auto", lse=True):
        tokens = self.q.shape[0]
        out = torch.full(tuple(self.q.shape), 123.0, dtype=dtype, device="cuda")
        ls = torch.full((tokens, self.heads * self.group), 123.0, device="cuda") if lse else None
        if max_new == "known":
            max_new = max(n for n, _ in self.seqs)
        mx.mx_paged_attention(self.cache, self.q, *(torch.from_numpy(t).cuda() for t in (self.ends, self.lens, self.table)),
                              out, lse=ls, scale=scale, causal=causal, window=window, max_new=max_new, workspace=workspace)
        torch.cuda.synchronize()
        return out, ls

    def check(self, what, here=None, **kw):
        print("attention", what, self.fmt, self.dim, self.page, self.heads, self.group, self.seqs[:6], kw, flush=True)
        out, lse = self.run(**kw)
        scale = kw.get("scale") or self.dim ** -0.5
        q = sr.f64(self.q)
        at = 0
        for s, (n, L) in enumerate(self.seqs):
            ref = sr.attention(q[at:at + n], self.k[s], self.v[s], scale, kw.get("causal", True), kw.get("window", 0), n,
                               None if here is None else here[s])
            sr.check_attention(out[at:at + n], None if lse is None else lse[at:at + n], ref, max(L, 1), "%s, sequence %d" % (what, s))
            at += n
        return out, lse


def counters_are_zero():
    return all(int(w[:65536].count_nonzero()) == 0 for w in mx._WORKSPACES.values())


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("L", [1, 2, 31, 32, 33, 127, 128, 129, 640, 1025])
def test_one_token(fmt, dim, L):
    Case([(1, L)], fmt, dim).check("one token")
    assert counters_are_zero()


@pytest.mark.parametrize("fmt,dim", [("fp8", 64), ("fp8", 128), ("fp4", 64), ("fp4", 128)])
@pytest.mark.parametrize("page", [1, 2, 8, 16, 64, 256, 1024])
def test_pages(fmt, dim, page):
    Case([(1, 300), (3, 77), (40, 210)], fmt, dim, page).check("pages")


@pytest.mark.parametrize("heads,group", [(1, 1), (1, 16), (1, 17), (3, 5), (8, 1), (2, 7), (1, 33), (2, 64)])
def test_heads(heads, group):
    Case([(1, 200), (2, 65), (5, 129)], heads=heads, group=group).check("heads")


@pytest.mark.parametrize("fmt,dim", [("fp8", 64), ("fp8", 128), ("fp4", 64), ("fp4", 128)])
@pytest.mark.parametrize("new", [2, 4, 5, 8, 9, 31, 32, 33, 100, 257])
def test_chunks(fmt, dim, new):
    Case([(new, new + 150)], fmt, dim, heads=1).check("chunk behind a context")
    Case([(new, new)], fmt, dim, heads=1).check("chunk alone")


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 1, 17, 64, 100])
def test_windows(causal, window):
    c = Case([(1, 400), (6, 300), (80, 333), (3, 2)], dim=64, heads=1, group=4)
    c.check("window", causal=causal, window=window)


def test_empty_rows():
    # no keys; more new tokens than keys (the first see none); no new tokens
    for seqs in ([(1, 0)], [(5, 0), (1, 3)], [(7, 3)], [(0, 50), (2, 50), (0, 0)], [(200, 150)], [(140, 0), (1, 9)]):
        c = Case(seqs, heads=1)
        out, lse = c.check("empty rows")
        if seqs[0][1] == 0:
            assert (out[0] == 0).all() and (lse[0] == -torch.inf).all()


@pytest.mark.parametrize("max_new", ["known", 1, None, 10 ** 6])
def test_max_new_changes_nothing_but_speed(max_new):
    Case([(1, 500), (90, 200), (9, 9), (0, 4), (4, 1000)], heads=2, group=2).check("max_new", max_new=max_new)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_output_types(dtype):
    Case([(1, 100), (2, 70), (70, 100)]).check("types", dtype=dtype)


@pytest.mark.parametrize("new", [1, 3, 70])
def test_split_and_whole(new):
    # long keys for few rows: split over workgroups with a workspace, not without
    c = Case([(new, 6000), (new, 70)], heads=1, group=3, page=64)
    a = c.check("split")
    b = c.check("whole", workspace=None)
    again = c.run()
    assert torch.equal(a[0], again[0]) and torch.equal(a[1], again[1]), "another run, other bits"
    assert counters_are_zero()
    small = torch.zeros(65536, dtype=torch.uint8, device="cuda")
    d = c.run(workspace=small)
    assert torch.equal(b[0], d[0]) and int(small.count_nonzero()) == 0


def test_many_sequences():
    rng = np.random.default_rng(3)
    seqs = [(int(rng.integers(0, 4)), int(rng.integers(0, 90))) for _ in range(200)]
    Case(seqs, dim=64, heads=1, group=2).check("200 sequences")
    Case([(n * 9, L + 9) for n, L in seqs[:70]], dim=64, heads=1, group=2).check("70 sequences")


@pytest.mark.parametrize("sigma,scale", [(30.0, None), (0.01, None), (1.0, 3.0), (1.0, 1e-3)])
def test_score_ranges(sigma, scale):
    Case([(1, 700), (33, 300)], sigma=sigma, heads=1).check("scores", scale=scale)


@pytest.mark.parametrize("new", [1, 2, 40])
def test_strided_queries(new):
    Case([(new, 90), (new, 41)], q_pad=256).check("strided")


@pytest.mark.parametrize("new", [1, 4, 45])
def test_pages_outside_the_cache(new):
    # an unmapped page's keys are as if they were not there
    c = Case([(new, 300), (new, 200)], heads=1, page=32)
    here = [np.ones(300, bool), np.ones(200, bool)]
    c.table[0, 2], c.table[0, 5], c.table[1, 0] = -1, c.cache.pages, 2 ** 31 - 1
    here[0][64:96] = False
    here[0][160:192] = False
    here[1][:32] = False
    c.check("unmapped pages", here=here)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("new,window", [(1, 0), (1, 9), (3, 0), (3, 5), (60, 0), (60, 20)])
def test_nan_values_reach_only_rows_that_see_them(fmt, new, window):
    L = 110
    c = Case([(new, L), (new, 64)], fmt, heads=2, group=2)
    for j in (L - 2, L - 1, 50, 3):
        page, off = c.table[0, j // 16], j % 16
        c.parts[3][page, 1, off, 1] = 255          # one block of the second head's values
        c.v[0][j, 1, 32:64] = np.nan
    if fmt == "fp8":                               # and a single NaN element
        c.parts[2][c.table[0, 100 // 16], 0, 100 % 16, 7] = 0x7F
        c.v[0][100, 0, 7] = np.nan
    c.upload()
    c.check("NaN values", window=window)


@pytest.mark.parametrize("new", [1, 3, 60])
def test_nan_keys_reach_only_rows_that_see_them(new):
    L = 100
    c = Case([(new, L)], heads=1, group=2)
    for j in (L - 1, 70):
        c.parts[1][c.table[0, j // 16], 0, j % 16, 0] = 255
        c.k[0][j, 0, :32] = np.nan
    c.upload()
    c.check("NaN keys", window=25)


def test_nan_query_row_stays_alone():
    c = Case([(40, 80)], heads=1, group=2)
    c.q[11, 1, 5] = float("nan")
    c.check("NaN query")


def test_any_lengths_stay_in_bounds():
    c = Case([(3, 50), (40, 60), (2, 30)], heads=1)
    good = c.run()
    for ends, lens in (([45, 3, 2], [50, 60, 30]), ([-7, 2 ** 31 - 1, 5], [50, 60, 30]), ([3, 43, 45], [-5, 2 ** 31 - 1, -2 ** 31]),
                       ([0, 0, 0], [50, 60, 30])):
        c.ends, c.lens = np.array(ends, np.int32), np.array(lens, np.int32)
        c.run()
        assert counters_are_zero()
    c.ends, c.lens = np.array([3, 43, 45], np.int32), np.array([50, 60, 30], np.int32)
    again = c.run()
    assert torch.equal(good[0], again[0])
    # rows past the last end are not written
    c.ends = np.array([3, 20, 20], np.int32)
    out, lse = c.run()
    assert (out[20:] == 123).all() and (lse[20:] == 123).all()


def test_cache_past_32_bits():
    pages, page, heads, dim = 5000, 1024, 8, 128
    cache = mx.KVCache.empty(pages, page, heads, dim, "fp8")
    L = 1500
    table = torch.tensor([[pages - 1, 4096]], dtype=torch.int32, device="cuda")
    slots = table[0].long()[torch.arange(L, device="cuda") // page] * page + torch.arange(L, device="cuda") % page
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(L, heads, dim, generator=g).bfloat16().cuda() for _ in "kv")
    mx.mx_kv_cache_write(cache, k, v, slots)
    rk, rv = torch.empty_like(k), torch.empty_like(v)
    mx.mx_kv_cache_read(cache, rk, rv, slots)
    for n in (1, 40):
        q = torch.randn(n, heads, dim, generator=g).bfloat16().cuda()
        lse = torch.empty(n, heads, device="cuda")
        out = torch.empty_like(q)
        mx.mx_paged_attention(cache, q, torch.tensor([n], dtype=torch.int32, device="cuda"),
                              torch.tensor([L], dtype=torch.int32, device="cuda"), table, out, lse=lse)
        ref = sr.attention(sr.f64(q), sr.f64(rk), sr.f64(rv), dim ** -0.5, True, 0, n)
        sr.check_attention(out, lse, ref, L, "far pages")


def test_other_stream():
    c = Case([(1, 3000), (50, 200)], heads=1)
    want = c.run()
    s = torch.cuda.Stream()
    out = torch.empty_like(want[0])
    args = [torch.from_numpy(t).cuda() for t in (c.ends, c.lens, c.table)]
    s.wait_stream(torch.cuda.current_stream())
    mx.mx_paged_attention(c.cache, c.q, *args, out, max_new=50, stream=s)
    s.synchronize()
    assert torch.equal(out, want[0])


def test_graph_replays():
    c = Case([(1, 2000), (60, 100)], heads=1)
    want = c.run()
    out, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    args = [torch.from_numpy(t).cuda() for t in (c.ends, c.lens, c.table)]
    ws = torch.zeros(mx.mx_paged_attention_workspace_bytes(c.cache, 2, 61, 4, 60), dtype=torch.uint8, device="cuda")
    call = lambda: mx.mx_paged_attention(c.cache, c.q, *args, out, lse=lse, max_new=60, workspace=ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(4):
        out.zero_()
        lse.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        c.run()
    # the lengths are read on the device: a replay takes the new ones
    args[1].copy_(torch.tensor([7, 80], dtype=torch.int32))
    g.replay()
    c.lens = np.array([7, 80], np.int32)
    assert torch.equal(out, c.run()[0])


def test_no_tokens():
    c = Case([(1, 10)])
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    mx.mx_paged_attention(c.cache, c.q[:0], e, e, torch.empty(0, 1, dtype=torch.int32, device="cuda"), c.q[:0].float())
