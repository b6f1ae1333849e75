"""GPU: mx_moe_dispatch, mx_moe_combine and mx_moe_combine_grad against plain
forms in 64 bits: rows and codes bit for bit, sums within the bounds of FP32
sums in the order of their terms, gradients against the formula and against
differences of the calls themselves (both are linear in each argument)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_scaled_precision_mm_amd as mx
import oracle
from tests import servingref as sr

pytestmark = pytest.mark.gpu


def sort(ids, groups):
    """(offs, pos) by a stable sort."""
    flat = ids.reshape(-1)
    held = (flat >= 0) & (flat < groups)
    order = np.argsort(np.where(held, flat, groups), kind="stable")
    pos = np.empty(len(flat), np.int64)
    pos[order] = np.arange(len(flat))
    offs = np.cumsum(np.bincount(flat[held].astype(np.int64), minlength=groups)[:groups])
    return offs.astype(np.int32), np.where(held, pos, -1).reshape(ids.shape).astype(np.int32)


def buffers(rows, K, out):
    if out == "bf16":
        return torch.full((rows, K), 7.0, dtype=torch.bfloat16, device="cuda"), None
    y = torch.full((rows, K if out == "fp8" else K // 2), 0xA5, dtype=torch.uint8, device="cuda")
    return y, torch.full((rows, K // 32), 0x5A, dtype=torch.uint8, device="cuda")


def check_dispatch(tokens, top_k, groups, K, out="fp8", seed=1, ids=None, **kw):
    print("dispatch", tokens, top_k, groups, K, out, flush=True)
    rng = np.random.default_rng(seed)
    if ids is None:
        ids = rng.integers(-1, groups + 1, (tokens, top_k))
    x = torch.from_numpy(rng.standard_normal((tokens, K)).astype(np.float32)).bfloat16()
    y, ys = buffers(tokens * top_k, K, out)
    offs = torch.full((groups,), -9, dtype=torch.int32, device="cuda")
    pos = torch.full((tokens, top_k), -9, dtype=torch.int32, device="cuda")
    mx.mx_moe_dispatch(x.cuda(), torch.from_numpy(ids.astype(np.int64)).cuda(), y, ys, offs, pos, **kw)
    torch.cuda.synchronize()
    want_offs, want_pos = sort(ids, groups)
    assert np.array_equal(offs.cpu().numpy(), want_offs)
    assert np.array_equal(pos.cpu().numpy(), want_pos)
    n = int(want_offs[-1])
    row_token = np.zeros(n, np.int64)
    t, j = np.nonzero(want_pos >= 0)
    row_token[want_pos[t, j]] = t
    if out == "bf16":
        assert torch.equal(y[:n].cpu().view(torch.int16), x[row_token].view(torch.int16))
        assert (y[n:] == 7).all()
    else:
        if tokens:
            codes, scales = oracle.quantize(out, sr.bits(x), tokens, K)
            assert np.array_equal(y[:n].cpu().numpy(), codes.reshape(tokens, -1)[row_token])
            assert np.array_equal(ys[:n].cpu().numpy(), scales.reshape(tokens, -1)[row_token])
        assert (y[n:] == 0xA5).all() and (ys[n:] == 0x5A).all()
    return offs, pos


@pytest.mark.parametrize("out", ["fp8", "fp4", "bf16"])
@pytest.mark.parametrize("tokens,top_k,groups,K", [
    (1, 1, 1, 32), (1, 8, 128, 2048), (2, 2, 8, 4096), (7, 3, 5, 96), (64, 8, 128, 2048), (64, 64, 64, 64), (33, 6, 60, 1056),
    (511, 8, 256, 160), (513, 8, 256, 64), (5000, 1, 8, 32), (3000, 4, 1024, 64), (1300, 64, 100, 32), (3, 2, 4, 32768)])
def test_dispatch(tokens, top_k, groups, K, out):
    check_dispatch(tokens, top_k, groups, K, out)


def test_dispatch_of_many_assignments():
    """More chunks than a pass of the last workgroup's threads."""
    check_dispatch(70000, 8, 256, 32)
    check_dispatch(262144, 2, 3, 32, "bf16")
    check_dispatch(9000, 64, 1000, 32)


@pytest.mark.parametrize("K", [8, 24, 40, 264])
def test_dispatch_of_odd_bf16_rows(K):
    check_dispatch(37, 3, 9, K, "bf16")
    check_dispatch(5000, 2, 9, K, "bf16")


@pytest.mark.parametrize("tokens", [50, 6000])
def test_dispatch_of_any_ids(tokens):
    rng = np.random.default_rng(3)
    ids = rng.integers(-3, 20, (tokens, 4))
    check_dispatch(tokens, 4, 16, 64, ids=ids)
    check_dispatch(tokens, 4, 16, 64, ids=np.full((tokens, 4), 5))              # one expert, every choice of every token
    check_dispatch(tokens, 4, 16, 64, ids=np.full((tokens, 4), -1))             # none held
    ids[::3] = 1 << 40
    ids[1::3] = -(1 << 62)
    check_dispatch(tokens, 4, 16, 64, ids=ids)
    check_dispatch(tokens, 4, 16, 64, ids=np.tile([2, 2, 1 << 32, 2], (tokens, 1)))


def test_dispatch_of_no_tokens():
    offs, _ = check_dispatch(0, 2, 7, 64)
    assert (offs == 0).all()


def test_dispatch_values_out_of_the_ordinary():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    x[0, 3], x[1, 40], x[2] = np.inf, np.nan, 1e-40
    ids = torch.tensor([[0, 1], [1, 0], [1, 1], [0, 0]])
    for out in ("fp8", "fp4"):
        y, ys, offs, pos = mx.moe_dispatch(x.cuda(), ids.cuda(), 2, out)
        codes, scales = oracle.quantize(out, sr.bits(x), 4, 64)
        for t in range(4):
            for j in range(2):
                assert np.array_equal(y[int(pos[t, j])].cpu().numpy(), codes.reshape(4, -1)[t])
                assert np.array_equal(ys[int(pos[t, j])].cpu().numpy(), scales.reshape(4, -1)[t])


def test_dispatch_workspaces():
    need = mx.mx_moe_dispatch_workspace_bytes(6000, 4, 64)
    assert need > 65536 and mx.mx_moe_dispatch_workspace_bytes(1024, 4, 64) == 0
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    ws[65536:] = 0xEE
    for seed in (1, 2, 3):
        check_dispatch(6000, 4, 64, 32, seed=seed, workspace=ws)
        assert int(ws[:65536].count_nonzero()) == 0
    check_dispatch(1000, 4, 64, 32, workspace=None)
    with pytest.raises(mx.MxGemmError) as e:
        check_dispatch(6000, 4, 64, 32, workspace=None)
    assert e.value.status == -6
    with pytest.raises(mx.MxGemmError) as e:
        check_dispatch(6000, 4, 64, 32, workspace=ws[:need - 16])
    assert e.value.status == -6
    check_dispatch(6000, 4, 64, 32)
    assert all(int(w[:65536].count_nonzero()) == 0 for w in mx._WORKSPACES.values())


@pytest.mark.parametrize("tokens", [40, 5000])
def test_dispatch_on_another_stream_and_replayed(tokens):
    g0 = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((tokens, 256), generator=g0, device="cuda").bfloat16()
    ids = torch.randint(-1, 17, (tokens, 4), generator=g0, device="cuda")
    want = mx.moe_dispatch(x, ids, 16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = mx.moe_dispatch(x, ids, 16, stream=s)
    torch.cuda.synchronize()
    n = int(want[2][-1])
    for a, b in zip(got, want):
        assert torch.equal(a[:n] if a.shape[0] == tokens * 4 else a, b[:n] if b.shape[0] == tokens * 4 else b)
    out = [torch.empty_like(t) for t in want]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mx.mx_moe_dispatch(x, ids, out[0], out[1], out[2], out[3])
    for i in range(3):
        x.normal_(generator=g0)
        ids.random_(0, 20, generator=g0)
        want = mx.moe_dispatch(x, ids, 16)          # the stream's own workspace, between replays
        g.replay()
        torch.cuda.synchronize()
        n = int(want[2][-1])
        assert torch.equal(out[2], want[2]) and torch.equal(out[3], want[3])
        assert torch.equal(out[0][:n], want[0][:n]) and torch.equal(out[1][:n], want[1][:n])


# ------------------------------------------------------------------ combine
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
SHAPES = [(1, 1, 32), (1, 8, 2048), (3, 2, 8), (64, 8, 2048), (65, 6, 264), (17, 64, 96), (1000, 2, 4096), (129, 3, 40), (31, 4, 20000),
          (9, 9, 512)]


def inputs(tokens, top_k, N, dtype, seed=1, rows=None, drop=0.2):
    rng = np.random.default_rng(seed)
    rows = tokens * top_k + 3 if rows is None else rows
    y = torch.from_numpy(rng.standard_normal((rows, N)).astype(np.float32)).to(dtype).cuda()
    pos = rng.permutation(rows)[:tokens * top_k].reshape(tokens, top_k).astype(np.int32)
    gone = rng.random(pos.shape) < drop
    pos[gone] = rng.choice([-1, -(1 << 31), rows, (1 << 31) - 1], int(gone.sum()))
    w = torch.from_numpy(rng.random((tokens, top_k)).astype(np.float32)).cuda()
    return y, torch.from_numpy(pos).cuda(), w


def combined(y, pos, w):
    """The sums in 64 bits, and of the magnitudes."""
    y, pos = sr.f64(y), pos.cpu().numpy()
    here = (pos >= 0) & (pos < y.shape[0])
    w = np.where(here, 1.0 if w is None else sr.f64(w), 0.0)
    rows = y[np.where(here, pos, 0)]
    return np.einsum("tj,tjn->tn", w, rows), np.einsum("tj,tjn->tn", np.abs(w), np.abs(rows))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,top_k,N", SHAPES)
def test_combine(tokens, top_k, N, dtype):
    y, pos, w = inputs(tokens, top_k, N, dtype)
    for weights in (w, None):
        want, size = combined(y, pos, weights)
        for out_dtype in DTYPES:
            print("combine", tokens, top_k, N, dtype, out_dtype, weights is not None, flush=True)
            out = torch.full((tokens, N), 9.0, dtype=out_dtype, device="cuda")
            mx.mx_moe_combine(y, pos, weights, out)
            torch.cuda.synchronize()
            # top_k fused steps, each half an FP32 step of a partial sum; then
            # the output's rounding (FP16 below its normal range: half of 2^-24)
            tol = size * top_k * 2.0 ** -24 * 1.01 + np.abs(want) * sr.HALF[out_dtype] * 1.01 + 2.0 ** -25
            assert (np.abs(sr.f64(out) - want) <= tol).all()


def test_combine_gives_zeros_without_rows_and_keeps_what_is_special():
    y, pos, w = inputs(6, 2, 64, torch.float32, drop=0.0)
    pos[2] = -1
    y[int(pos[0, 0]), 5] = np.inf
    y[int(pos[1, 1]), 6] = np.nan
    w[3, 0] = 0.0
    y[int(pos[3, 0]), 7] = np.inf            # 0 * inf
    out = mx.moe_combine(y, pos, w, torch.float32)
    assert (out[2] == 0).all()
    assert out[0, 5] == np.inf and torch.isnan(out[1, 6]) and torch.isnan(out[3, 7])
    assert int((~torch.isfinite(out)).sum()) == 3
    none = mx.moe_combine(torch.empty((0, 64), device="cuda"), pos, w, torch.float32)
    assert (none == 0).all()
    assert mx.moe_combine(y, pos[:0], w[:0]).shape == (0, 64)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,top_k,N", SHAPES)
def test_gradient(tokens, top_k, N, dtype):
    print("gradient", tokens, top_k, N, dtype, flush=True)
    y, pos, w = inputs(tokens, top_k, N, dtype)
    d_out = torch.from_numpy(np.random.default_rng(2).standard_normal((tokens, N)).astype(np.float32)).to(dtype).cuda()
    d_y = torch.full_like(y, 9.0)
    d_w = torch.full((tokens, top_k), 9.0, device="cuda")
    mx.mx_moe_combine_grad(d_out, y, pos, w, d_y, None, d_w)
    torch.cuda.synchronize()
    p, rows = pos.cpu().numpy(), y.shape[0]
    here = (p >= 0) & (p < rows)
    t, j = np.nonzero(here)
    # one FP32 product, rounded to the type
    want = torch.full((rows, N), 9.0).to(dtype)
    want[p[t, j]] = (d_out.cpu().float()[t] * w.cpu()[t, j][:, None]).to(dtype)
    assert torch.equal(d_y.cpu(), want)
    prod = sr.f64(d_out)[t] * sr.f64(y)[p[t, j]]
    exact, size = np.zeros((tokens, top_k)), np.zeros((tokens, top_k))
    exact[t, j], size[t, j] = prod.sum(1), np.abs(prod).sum(1)
    # a thread's 8 values of every 256th piece, 6 steps over lanes, 4 over waves
    steps = 8 * -(-N // 2048) + 10
    assert (np.abs(sr.f64(d_w) - exact) <= size * steps * 2.0 ** -24 * 1.01).all()
    # without the weights' gradient, and without weights
    d_y2 = torch.full_like(y, 9.0)
    mx.mx_moe_combine_grad(d_out, None, pos, None, d_y2)
    want[p[t, j]] = d_out.cpu()[t]
    assert torch.equal(d_y2.cpu(), want)


@pytest.mark.parametrize("out", ["fp8", "fp4"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,top_k,N", [(1, 1, 32), (40, 8, 2048), (33, 3, 96), (9, 5, 8224)])
def test_gradient_in_mx_blocks(tokens, top_k, N, dtype, out):
    y, pos, w = inputs(tokens, top_k, N, dtype)
    d_out = torch.from_numpy(np.random.default_rng(2).standard_normal((tokens, N)).astype(np.float32)).to(dtype).cuda()
    rows = y.shape[0]
    d_y, d_s = buffers(rows, N, out)
    d_w = torch.empty((tokens, top_k), device="cuda")
    mx.mx_moe_combine_grad(d_out, y, pos, w, d_y, d_s, d_w)
    torch.cuda.synchronize()
    p = pos.cpu().numpy()
    t, j = np.nonzero((p >= 0) & (p < rows))
    codes = np.full(tuple(d_y.shape), 0xA5, np.uint8)
    scales = np.full(tuple(d_s.shape), 0x5A, np.uint8)
    v = (d_out.cpu().float()[t] * w.cpu()[t, j][:, None]).bfloat16()
    if len(t):
        c, s = oracle.quantize(out, sr.bits(v), len(t), N)
        codes[p[t, j]], scales[p[t, j]] = c.reshape(len(t), -1), s.reshape(len(t), -1)
    assert np.array_equal(d_y.cpu().numpy(), codes) and np.array_equal(d_s.cpu().numpy(), scales)
    plain = torch.empty_like(d_w)
    mx.mx_moe_combine_grad(d_out, y, pos, w, torch.empty_like(y), None, plain)
    assert torch.equal(plain, d_w)


def test_gradients_against_differences():
    """<d_out, combine(y + a, w) - combine(y, w)> = <d_y, a>, and the same for
    the weights and for the dispatch, whose gradient is a combine without
    weights.  Differences are of FP32 outputs, off by top_k fused steps each."""
    tokens, top_k, N, E = 50, 4, 256, 8
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    y, pos, w = inputs(tokens, top_k, N, torch.float32)
    d_out, a, b = rnd(tokens, N), rnd(*y.shape), rnd(tokens, top_k)
    d_y, d_w = mx.moe_combine_grad(d_out, y, pos, w)
    f = lambda y, w: mx.moe_combine(y, pos, w, torch.float32).double()  # noqa: E731
    size = lambda y, w: torch.from_numpy(combined(y, pos, w)[1]).cuda()  # noqa: E731
    # (y + a and w + b are rounded too: the differences taken are of what was passed)
    ya, wb = y + a, w + b
    for diff, grad, step, s in ((f(ya, w) - f(y, w), d_y, ya.double() - y.double(), size(ya, w) + size(y, w)),
                                (f(y, wb) - f(y, w), d_w, wb.double() - w.double(), size(y, wb) + size(y, w))):
        off = float((d_out.double() * diff).sum() - (grad.double() * step).sum())
        # outputs' steps, and the gradient's own (d_w: 18 steps)
        tol = float((d_out.abs().double() * s).sum()) * (top_k + 19) * 2.0 ** -24
        assert abs(off) <= tol, (off, tol)
    x, ids = rnd(tokens, N).bfloat16(), torch.randint(-1, E + 1, (tokens, top_k), generator=g, device="cuda")
    rows, _, offs, at = mx.moe_dispatch(x, ids, E, torch.bfloat16)
    n = int(offs[-1])
    d_rows = rnd(tokens * top_k, N)
    d_x = mx.moe_combine(d_rows[:n], at, None, torch.float32)
    off = float((rows[:n].double() * d_rows[:n].double()).sum() - (x.double() * d_x.double()).sum())
    tol = float((rows[:n].double() * d_rows[:n].double()).abs().sum()) * top_k * 2.0 ** -24
    assert abs(off) <= tol, (off, tol)


def test_there_and_back_on_another_stream_and_replayed():
    tokens, top_k, N, E = 300, 4, 512, 16
    g0 = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((tokens, N), generator=g0, device="cuda").bfloat16()
    ids = torch.randint(0, E, (tokens, top_k), generator=g0, device="cuda")
    w = torch.rand((tokens, top_k), generator=g0, device="cuda")

    def both(stream=None):
        y, _, offs, pos = mx.moe_dispatch(x, ids, E, torch.bfloat16, stream=stream)
        out = mx.moe_combine(y, pos, w, stream=stream)
        return (out,) + mx.moe_combine_grad(x, y, pos, w, stream=stream)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    want, got = both(), both(s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = both()
    for _ in range(3):
        x.normal_(generator=g0)
        ids.random_(0, E, generator=g0)
        w.uniform_(generator=g0)
        want = both()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, held))


def test_offsets_past_32_bits():
    """Rows of more than 2^32 codes and 2^33 bytes: dispatched, combined, and their gradient, at rows throughout."""
    tokens, top_k, K, E = 560000, 8, 1024, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((tokens, K), generator=g, device="cuda", dtype=torch.bfloat16)
    ids = torch.randint(0, E, (tokens, top_k), generator=g, device="cuda")
    y, ys, offs, pos = mx.moe_dispatch(x, ids, E)
    assert y.numel() > 1 << 32 and int(offs[-1]) == tokens * top_k
    codes, scales = torch.empty((tokens, K), dtype=torch.uint8, device="cuda"), torch.empty((tokens, K // 32), dtype=torch.uint8, device="cuda")
    mx.mx_quantize_bf16(x, codes, scales, tokens, K, False)
    for j in (0, 7):
        at = pos[:, j].long()
        assert int(at.max()) * K > 1 << 32
        for part in range(0, tokens, 70000):
            rows = at[part:part + 70000]
            assert torch.equal(y[rows], codes[part:part + 70000]) and torch.equal(ys[rows], scales[part:part + 70000])
    del y, ys, codes, scales
    rows, _, _, pos2 = mx.moe_dispatch(x, ids, E, torch.bfloat16)
    assert torch.equal(pos, pos2)
    # powers of two: every product and sum of eight like values is exact
    w = torch.full((tokens, top_k), 0.125, device="cuda")
    out = mx.moe_combine(rows, pos, w)
    assert torch.equal(out, x)
    d_y, d_w = mx.moe_combine_grad(x, rows, pos, w)
    torch.cuda.synchronize()
    assert torch.equal(d_w, d_w[:, :1].expand(-1, top_k))
    for part in range(0, tokens, 70000):
        at = pos[part:part + 70000, 3].long()
        assert torch.equal(d_y[at], x[part:part + 70000] * 0.125)


@pytest.mark.parametrize("tokens", [8191, 8192, 8193, 8320])
def test_dispatch_at_the_most_chunks_that_are_added_up_by_each_workgroup(tokens):
    check_dispatch(tokens, 8, 40, 32)
    check_dispatch(tokens * 8, 1, 1024, 32, "bf16")
