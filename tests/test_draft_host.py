"""Host checks of the operators for drafted tokens and for experts: every
invalid argument is refused with its status before any HIP call (no GPU
needed), workspace sizes, tables and masks, and the binding's checks."""
from __future__ import annotations

import ctypes
import math

import pytest
import torch

import block_scaled_precision_mm_amd as mx
from tests.test_serving_host import CACHES, cache

A = 0x10000     # aligned, never dereferenced
L = mx._lib
BF, U8, I32, I64, F32 = torch.bfloat16, torch.uint8, torch.int32, torch.int64, torch.float32


def rope(c=None, q=A, qo=A, k=A, v=A, heads=4, qst=512, qost=512, kst=256, vst=256, pos=A, slots=A, table=A, npos=100, rot=128,
         inter=0, n=5):
    c = c or cache()
    return L.mx_rope_cache_write(ctypes.addressof(c), q, qo, k, v, heads, qst, qost, kst, vst, pos, slots, table, npos, rot, inter,
                                 n, None)


@pytest.mark.parametrize("kw,status", CACHES)
def test_rope_cache_refusals(kw, status):
    assert rope(cache(**kw)) == status
    assert L.mx_rope_cache_write(None, A, A, A, A, 4, 512, 512, 256, 256, A, A, A, 100, 128, 0, 5, None) == -1


@pytest.mark.parametrize("kw,status", [
    (dict(q=0), -1), (dict(qo=0), -1), (dict(k=0), -1), (dict(v=0), -1), (dict(pos=0), -1), (dict(slots=0), -1), (dict(table=0), -1),
    (dict(n=-1), -2), (dict(n=1 << 40), -2), (dict(n=1 << 25), -2), (dict(heads=-1), -2), (dict(heads=65537), -2), (dict(npos=0), -2),
    (dict(npos=1 << 31), -2), (dict(rot=0), -2), (dict(rot=-16), -2), (dict(rot=144), -2), (dict(qst=504), -2), (dict(qost=504), -2),
    (dict(kst=248), -2), (dict(vst=0), -2), (dict(qst=1 << 31), -2), (dict(qost=1 << 31), -2), (dict(kst=1 << 31), -2),
    (dict(rot=24), -3), (dict(rot=100), -3), (dict(qst=516), -3), (dict(qost=513), -3), (dict(kst=260), -3), (dict(vst=257), -3),
    (dict(inter=2), -9), (dict(inter=-1), -9), (dict(qst=1024), -9),
    (dict(q=A + 8), -4), (dict(qo=A + 8), -4), (dict(k=A + 8), -4), (dict(v=A + 2), -4), (dict(table=A + 8), -4),
    (dict(pos=A + 4), -4), (dict(slots=A + 4), -4),
])
def test_rope_refusals(kw, status):
    assert rope(**kw) == status


def tree(c=None, q=A, qst=1024, ends=A, lens=A, table=A, width=4, mask=A, words=1, seqs=3, n=7, heads=8, most=7, scale=0.1,
         window=0, out=A, kind=0, lse=0, ws=0, wsb=0):
    c = c or cache()
    return L.mx_tree_attention(ctypes.addressof(c), q, qst, ends, lens, table, width, mask, words, seqs, n, heads, most, scale,
                               window, out, kind, lse, ws, wsb, None)


@pytest.mark.parametrize("kw,status", CACHES)
def test_tree_cache_refusals(kw, status):
    assert tree(cache(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(mask=0), -1), (dict(mask=A + 4), -4), (dict(words=0), -2), (dict(words=-1), -2), (dict(words=1025), -2),
    (dict(kind=3), -5), (dict(kind=-1), -5), (dict(seqs=-1), -2), (dict(seqs=65537), -2), (dict(n=-1), -2), (dict(n=1 << 28), -2),
    (dict(heads=7), -2), (dict(heads=1), -2), (dict(most=-1), -2), (dict(width=-1), -2), (dict(width=1 << 27), -2),
    (dict(qst=1016), -2), (dict(qst=1 << 31), -2), (dict(window=-1), -2), (dict(c=cache(dim=96)), -2),
    (dict(q=0), -1), (dict(ends=0), -1), (dict(lens=0), -1), (dict(table=0), -1), (dict(out=0), -1), (dict(qst=1028), -3),
    (dict(scale=0.0), -9), (dict(scale=float("nan")), -9), (dict(scale=float("inf")), -9),
    (dict(q=A + 8), -4), (dict(out=A + 8), -4), (dict(ws=A + 8), -4), (dict(ends=A + 2), -4), (dict(lens=A + 1), -4),
    (dict(table=A + 2), -4), (dict(lse=A + 2), -4),
])
def test_tree_refusals(kw, status):
    assert tree(**kw) == status


def test_tree_workspace_sizes():
    size = lambda c, *a: L.mx_tree_attention_workspace_bytes(ctypes.addressof(c), *a)  # noqa: E731
    for dim in (64, 128):
        c = cache(dim=dim, heads=8)
        assert size(c, 1, 27, 32, 27) > 65536
        assert size(c, 1, 27, 33, 27) == 0
        for a in ((64, 64, 32, 1), (1, 4096, 32, 4096), (20, 700, 32, 300)):
            n = size(c, *a)
            assert n == 0 or n > 65536
    assert size(cache(dim=96), 1, 1, 8, 1) == 0 and L.mx_tree_attention_workspace_bytes(None, 1, 1, 8, 1) == 0


def dispatch(x=A, ids=A, n=9, k=2, groups=8, K=64, y=A, ys=A, kind=3, offs=A, pos=A, ws=0, wsb=0):
    return L.mx_moe_dispatch(x, ids, n, k, groups, K, y, ys, kind, offs, pos, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=0), -1), (dict(ids=0), -1), (dict(y=0), -1), (dict(ys=0), -1), (dict(offs=0), -1), (dict(pos=0), -1),
    (dict(n=0, offs=0), -1), (dict(kind=1), -5), (dict(kind=2), -5), (dict(kind=5), -5), (dict(kind=-1), -5),
    (dict(n=-1), -2), (dict(n=1 << 24), -2), (dict(n=1 << 21, k=64), -2), (dict(n=1 << 62, k=64), -2), (dict(k=0), -2), (dict(k=65), -2),
    (dict(groups=0), -2), (dict(groups=1025), -2), (dict(K=0), -2), (dict(K=(1 << 20) + 32), -2), (dict(K=48), -3),
    (dict(K=36, kind=0), -3), (dict(n=5000, ws=0), -6), (dict(n=5000, ws=A, wsb=65536), -6),
    (dict(x=A + 8), -4), (dict(y=A + 8), -4), (dict(ws=A + 8), -4), (dict(ids=A + 4), -4), (dict(offs=A + 2), -4), (dict(pos=A + 1), -4),
])
def test_dispatch_refusals(kw, status):
    assert dispatch(**kw) == status


def test_dispatch_workspace_sizes():
    size = L.mx_moe_dispatch_workspace_bytes
    assert size(2048, 2, 8) == 0 and size(2049, 2, 8) > 65536
    for n, k in ((4097, 1), (65536, 8), (1 << 20, 64), ((1 << 24) - 1, 4)):
        assert 65536 < size(n, k, 1024) <= 65536 + 8192 * 1024 * 4
    assert size(1 << 24, 1, 8) == 0 and size(1 << 23, 64, 8) == 0 and size(5000, 0, 8) == 0 and size(5000, 2, 0) == 0
    assert size(-1, 2, 8) == 0 and size(5000, 2, 1025) == 0


def combine(y=A, yd=0, pos=A, w=A, n=9, k=2, rows=18, N=64, out=A, od=0):
    return L.mx_moe_combine(y, yd, pos, w, n, k, rows, N, out, od, None)


SIZES = [(dict(n=-1), -2), (dict(n=1 << 24), -2), (dict(k=0), -2), (dict(k=65), -2), (dict(rows=-1), -2), (dict(rows=1 << 31), -2),
         (dict(N=0), -2), (dict(N=(1 << 20) + 8), -2), (dict(n=1 << 20, N=1 << 14), -2), (dict(N=60), -3)]


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(y=0), -1), (dict(pos=0), -1), (dict(out=0), -1), (dict(yd=3), -5), (dict(yd=-1), -5), (dict(od=3), -5), (dict(od=-1), -5),
    (dict(y=A + 8), -4), (dict(out=A + 8), -4), (dict(pos=A + 2), -4), (dict(w=A + 2), -4),
])
def test_combine_refusals(kw, status):
    assert combine(**kw) == status


def grad(d=A, y=A, dt=0, pos=A, w=A, n=9, k=2, rows=18, N=64, dy=A, ds=A, kind=0, dw=A):
    return L.mx_moe_combine_grad(d, y, dt, pos, w, n, k, rows, N, dy, ds, kind, dw, None)


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(d=0), -1), (dict(y=0), -1), (dict(pos=0), -1), (dict(dy=0), -1), (dict(kind=3, ds=0), -1), (dict(kind=4, ds=0), -1),
    (dict(dt=3), -5), (dict(dt=-1), -5), (dict(dt=0, kind=1), -5), (dict(dt=2, kind=0), -5), (dict(kind=5), -5),
    (dict(N=72, kind=3), -3), (dict(d=A + 8), -4), (dict(y=A + 8), -4), (dict(dy=A + 8), -4), (dict(pos=A + 2), -4), (dict(w=A + 1), -4),
    (dict(dw=A + 2), -4),
])
def test_gradient_refusals(kw, status):
    assert grad(**kw) == status


def test_masks_from_parents():
    m = mx.tree_mask([-1, 0, 0, 1, -1])
    assert m.tolist() == [[0b1], [0b11], [0b101], [0b1011], [0b10000]]
    chain = mx.tree_mask(range(-1, 129), words=4)
    assert chain.shape == (130, 4) and chain[63].tolist() == [-1, 0, 0, 0] and chain[129].tolist() == [-1, -1, 3, 0]
    assert mx.tree_mask([]).shape == (0, 1)
    for bad in ([0], [-1, 1], [-1, -2], [-1, 5]):
        with pytest.raises(ValueError):
            mx.tree_mask(bad)
    with pytest.raises(ValueError):
        mx.tree_mask(range(-1, 64), words=1)


def test_rope_table():
    t = mx.rope_table(1000, 64, base=500.0, device="cpu")
    assert t.shape == (1000, 32, 2) and t.dtype is F32 and t.is_contiguous()
    for p, i in ((0, 0), (999, 0), (999, 31), (500, 7)):
        a = p * 500.0 ** (-2 * i / 64)
        assert abs(float(t[p, i, 0]) - math.cos(a)) < 2.0 ** -24 and abs(float(t[p, i, 1]) - math.sin(a)) < 2.0 ** -24


class OnGpu(torch.Tensor):
    """A CPU tensor that says it is on a GPU."""

    is_cuda = True
    index = 0

    def get_device(self):
        return self.index

    @property
    def device(self):
        return torch.device("cuda", self.index)


def gpu(shape, dtype, index=0):
    t = torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)
    t.index = index
    return t


def _cache(index):
    return mx.KVCache(*(gpu((2, 2, 16, n), U8, index) for n in (128, 4, 128, 4)))


# name: (call of the operands by name, operands: shape and type, or a maker; another shape for each that is refused)
CALLS = {
    "mx_rope_cache_write": (
        lambda t: mx.mx_rope_cache_write(t["c"], t["q"], t["k"], t["v"], t["p"], t["s"], t["r"], t["o"]),
        dict(c=_cache, q=((3, 4, 128), BF), k=((3, 2, 128), BF), v=((3, 2, 128), BF), p=((3,), I64), s=((3,), I64), r=((9, 64, 2), F32),
             o=((3, 4, 128), BF))),
    "mx_tree_attention": (
        lambda t: mx.mx_tree_attention(t["c"], t["q"], t["e"], t["l"], t["t"], t["m"], t["o"], lse=t["ls"], workspace=t["ws"]),
        dict(c=_cache, q=((3, 4, 128), BF), e=((1,), I32), l=((1,), I32), t=((1, 2), I32), m=((3, 1), I64), o=((3, 4, 128), BF),
             ls=((3, 4), F32), ws=((1 << 24,), U8))),
    "mx_moe_dispatch": (
        lambda t: mx.mx_moe_dispatch(t["x"], t["e"], t["y"], t["ys"], t["o"], t["p"], workspace=t["ws"]),
        dict(x=((3000, 64), BF), e=((3000, 2), I64), y=((6000, 64), U8), ys=((6000, 2), U8), o=((4,), I32), p=((3000, 2), I32),
             ws=((1 << 18,), U8))),
    "mx_moe_combine": (
        lambda t: mx.mx_moe_combine(t["y"], t["p"], t["w"], t["o"]),
        dict(y=((7, 64), BF), p=((3, 2), I32), w=((3, 2), F32), o=((3, 64), F32))),
    "mx_moe_combine_grad": (
        lambda t: mx.mx_moe_combine_grad(t["d"], t["y"], t["p"], t["w"], t["dy"], t["ds"], t["dw"]),
        dict(d=((3, 64), BF), y=((7, 64), BF), p=((3, 2), I32), w=((3, 2), F32), dy=((7, 64), U8), ds=((7, 2), U8), dw=((3, 2), F32))),
}


@pytest.fixture
def called(monkeypatch):
    log = []
    monkeypatch.setattr(mx, "_current_device", lambda: 0)
    monkeypatch.setattr(mx, "_raw_stream", lambda device: 7)
    for name in CALLS:
        monkeypatch.setattr(mx._lib, name, lambda *args, name=name: log.append(name) or 0)
    return log


@pytest.mark.parametrize("name", CALLS)
def test_operands_of_another_device_shape_type_or_order_are_refused(called, name):
    call, operands = CALLS[name]

    def make(n, index=0):
        how = operands[n]
        return how(index) if callable(how) else gpu(*how, index)

    call({n: make(n) for n in operands})
    assert called == [name]
    for other in operands:
        with pytest.raises(ValueError):         # another device
            call({n: make(n, int(n == other)) for n in operands})
        if callable(operands[other]):
            continue
        shape, dtype = operands[other]
        if other == "ws":
            continue
        wrong = [gpu(shape + (1,), dtype)]      # another number of dimensions
        if other != "r":                        # (a table may hold any number of positions)
            wrong.append(gpu((shape[0] + 1,) + shape[1:], dtype))
        wrong.append(gpu(shape, torch.float64))
        if len(shape) > 1:                      # not contiguous
            wrong.append(gpu(shape[:-2] + (shape[-1], shape[-2]), dtype).transpose(-1, -2).as_subclass(OnGpu))
        for t in wrong:
            if name == "mx_moe_dispatch" and other == "o" and t.dim() == 1 and t.dtype is I32:
                continue                        # (any number of experts)
            if name == "mx_moe_combine_grad" and other == "dy" and t.shape == (8, 64):
                pass                            # y disagrees
            if name == "mx_moe_combine" and other == "y" and t.shape == (8, 64):
                continue                        # (any number of rows)
            if min(shape[-2:]) == 1 and t.shape == shape and t.dtype is dtype:
                continue                        # (contiguous all the same)
            with pytest.raises(ValueError):
                call({n: t if n == other else make(n) for n in operands})
    assert called == [name]


def test_more_refusals_of_the_binding(called):
    c = _cache(0)
    k, pos, table = gpu((3, 2, 128), BF), gpu((3,), I64), gpu((9, 64, 2), F32)
    q = gpu((3, 4, 128), BF)
    with pytest.raises(ValueError):
        mx.mx_rope_cache_write(c, None, k, k, pos, pos, table, q)           # q_out without q
    with pytest.raises(ValueError):
        mx.mx_rope_cache_write(c, gpu((3, 512), BF), k, k, pos, pos, table)
    mx.mx_rope_cache_write(c, None, k, k, pos, pos, table)
    mx.mx_rope_cache_write(c, q, k, k, pos, pos, table)
    i32 = lambda *s: gpu(s, I32)  # noqa: E731
    with pytest.raises(ValueError):
        mx.mx_tree_attention(c, q, i32(1), i32(1), i32(1, 2), None, q)
    x, ids = gpu((3, 64), BF), gpu((3, 2), I64)
    for y, ys in ((gpu((6, 64), U8), None), (gpu((6, 32), U8), None), (gpu((6, 48), U8), gpu((6, 2), U8)), (gpu((6, 64), F32), None),
                  (gpu((6, 64), torch.float16), None), (gpu((6, 64), U8), gpu((6, 2), I32))):
        with pytest.raises(ValueError):
            mx.mx_moe_dispatch(x, ids, y, ys, i32(4), i32(3, 2))
    with pytest.raises(ValueError):
        mx.moe_dispatch(x, ids, 4, torch.float32)
    w = gpu((3, 2), F32)
    for d_y, ds in ((gpu((6, 64), F32), None), (gpu((6, 64), U8), None)):
        with pytest.raises(ValueError):
            mx.mx_moe_combine_grad(x, gpu((6, 64), BF), i32(3, 2), w, d_y, ds, w)
    with pytest.raises(ValueError):
        mx.mx_moe_combine_grad(x, None, i32(3, 2), w, gpu((6, 64), BF), None, w)
    with pytest.raises(ValueError):
        mx.mx_moe_combine(gpu((6, 64), torch.int16), i32(3, 2), w, x)


def test_tensors_are_refused_where_there_is_no_gpu(monkeypatch):
    def none():
        raise RuntimeError("no GPU")

    monkeypatch.setattr(mx, "_current_device", none)
    x = torch.zeros(4, 64, dtype=BF)
    p = torch.zeros(4, 1, dtype=I32)
    with pytest.raises(ValueError):
        mx.mx_moe_dispatch(x, torch.zeros(4, 1, dtype=I64), x, None, torch.zeros(2, dtype=I32), p)
    with pytest.raises(ValueError):
        mx.mx_moe_combine(x, p, None, x)


class Stream:
    cuda_stream = 9


@pytest.mark.parametrize("stream,want", [(None, 7), (9, 9), (Stream(), 9), (0, 0)])
def test_outputs_are_made_on_the_stream_that_writes_them(monkeypatch, stream, want):
    import contextlib
    log, now = [], [7]
    empty, zeros = torch.empty, torch.zeros

    @contextlib.contextmanager
    def use(s):
        before, now[0] = now[0], s if isinstance(s, int) else s.cuda_stream
        yield
        now[0] = before

    made = lambda f: lambda *a, device=None, **kw: (log.append(now[0]), f(*a, **kw).as_subclass(OnGpu))[1]  # noqa: E731
    q, ids, x, c = gpu((3, 4, 128), BF), gpu((3, 2), I64), gpu((3, 64), BF), _cache(0)
    i32 = {s: gpu(s, I32) for s in ((1,), (1, 2), (3, 2))}
    m, w, y = gpu((3, 1), I64), gpu((3, 2), F32), gpu((6, 64), BF)
    monkeypatch.setattr(torch, "empty", made(empty))
    monkeypatch.setattr(torch, "zeros", made(zeros))
    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda ptr, **kw: ptr)
    monkeypatch.setattr(mx, "_current_device", lambda: 0)
    monkeypatch.setattr(mx, "_raw_stream", lambda device: now[0])
    for fn in CALLS:
        monkeypatch.setattr(mx._lib, fn, lambda *args: log.append(args[-1]) or 0)
    mx.tree_attention(c, q, i32[1,], i32[1,], i32[1, 2], m, workspace=None, stream=stream)
    mx.moe_dispatch(x, ids, 4, workspace=None, stream=stream)
    mx.moe_dispatch(x, ids, 4, BF, workspace=None, stream=stream)
    mx.moe_combine(y, i32[3, 2], w, stream=stream)
    mx.moe_combine_grad(x, y, i32[3, 2], w, stream=stream)
    assert len(log) > 10 and set(log) == {want}, log
