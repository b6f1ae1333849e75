"""GPU: the operators for drafted tokens and for experts as a served layer runs
them (examples/draft_layer.py), against the same layer in 64 bits whose only
roundings are those that the layer's formats define; and the backward pass of
the experts' rows through the dispatch, against differences."""
from __future__ import annotations

import importlib.util
import os

import numpy as np
import pytest
import torch

import block_scaled_precision_mm_amd as mx
import oracle
from tests import servingref as sr
from tests.test_gpu_rope import rotated
from tests.test_gpu_tree import seen

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("draft_layer", os.path.join(ROOT, "examples", "draft_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _mx(fmt, x):
    """Values of the MX blocks of BF16 rows."""
    rows, K = x.shape
    return sr.rows_of(fmt, *oracle.quantize(fmt, sr.bits(x), rows, K))


def _bf16(x):
    return torch.from_numpy(x).to(torch.float32).to(torch.bfloat16)


def _off(y, ref):
    return np.linalg.norm(sr.f64(y) - ref) / np.linalg.norm(ref)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_prompt_and_trees(fmt):
    ex = _example()
    seqs, hidden, H, K, D, page, E, k, F = 3, 256, 8, 2, 64, 16, 6, 2, 128
    torch.manual_seed(1)
    layer = ex.DraftLayer(hidden, H, K, D, E, k, F, seqs * 8, page, fmt, positions=128)
    batch = ex.Batch(seqs, 8, page)
    wq, wo = _mx("fp8", layer.w_qkv), _mx("fp8", layer.w_out)
    up = _mx("fp8", layer.w_up.view(-1, hidden)).reshape(E, 2 * F, hidden)
    down = _mx("fp8", layer.w_down.view(-1, F)).reshape(E, hidden, F)
    keys = [np.zeros((0, K, D)) for _ in range(seqs)]
    values = [np.zeros((0, K, D)) for _ in range(seqs)]
    tree = [-1, 0, 0, 1, 1, 2, 3, -1, 7]
    for new, parents, path in ((33, None, None), (9, tree, [0, 1, 3, 6]), (9, tree, [0, 2]), (1, [-1], [0])):
        x = torch.randn(seqs * new, hidden).bfloat16()
        stream = torch.randn(seqs * new, hidden).bfloat16()
        step = ex.Step(batch, new, parents)
        y, h = layer.attention(x.cuda(), stream.cuda(), step)
        h_ref = (x.float() + stream.float()).bfloat16()
        assert torch.equal(h.cpu(), h_ref)
        a = _mx("fp8", _bf16(sr.rmsnorm(sr.f64(h_ref), sr.f64(layer.norms[0]), 1e-6)))
        q, kk, v = (t.reshape(seqs * new, -1, D) for t in _bf16(a @ wq.T).split((H * D, K * D, K * D), dim=1))
        pos = step.positions.cpu().numpy()
        q, kk = rotated(q, layer.rope, pos, D, False), rotated(kk, layer.rope, pos, D, False)
        sees = np.tril(np.ones((new, new), bool)) if parents is None else None
        if sees is None:
            sees = np.eye(new, dtype=bool)
            for i, p in enumerate(parents):
                if p >= 0:
                    sees[i] |= sees[p]
        out = np.zeros((seqs * new, H, D))
        for s in range(seqs):
            rows = slice(s * new, (s + 1) * new)
            held = [np.concatenate([old[s], _mx(fmt, t[rows].reshape(new * K, D)).reshape(new, K, D)])
                    for old, t in ((keys, kk), (values, v))]
            L = held[0].shape[0]
            assert L == int(step.lens[s])
            mask = seen(sees, new, L, 0)
            for i in range(new):
                out[s * new + i] = sr.attention(sr.f64(q[s * new + i:s * new + i + 1]), *held, D ** -0.5, False, 0, 1, mask[i])[0][0]
            keep = list(range(L - new)) + [L - new + j for j in (range(new) if path is None else path)]
            keys[s], values[s] = (t[keep] for t in held)
        ref = _mx("fp8", _bf16(out.reshape(seqs * new, H * D))) @ wo.T
        # as in the attention block's test: a few per cent of the codes round the
        # other way, each by a step of 2^-3 (2^-1 in an E2M1 cache) of its value
        off = _off(y, ref)
        # the experts, on what the first half gave
        m, h2 = layer.mixture(y, h)
        b_ref = _bf16(sr.rmsnorm(sr.f64(h2), sr.f64(layer.norms[1]), 1e-6))
        assert torch.equal(h2.cpu(), (y.cpu().float() + h.cpu().float()).bfloat16())
        weights, ids = layer.route(mx.rmsnorm(y, layer.norms[1], h, out=torch.bfloat16)[0])
        w, ids, b = sr.f64(weights), ids.cpu().numpy(), _mx("fp8", b_ref)
        ref = np.zeros((seqs * new, hidden))
        for t in range(seqs * new):
            for j in range(k):
                u = _bf16(up[ids[t, j]] @ b[t]).double()
                g = (torch.nn.functional.silu(u[:F]).float().bfloat16().float() * u[F:].float()).bfloat16()
                ref[t] += w[t, j] * sr.f64(_bf16(down[ids[t, j]] @ _mx("fp8", g[None])[0]))
        off2 = _off(m, ref)
        print("layer", fmt, "new", new, "attention off by %.4f, experts by %.4f" % (off, off2), flush=True)
        assert off < (0.04 if fmt == "fp8" else 0.08) and off2 < 0.04
        if path is None:
            batch.lens += new
        else:
            batch.accept(layer.cache, path)
        # the cache holds what is kept, in its order
        for s in range(seqs):
            n = keys[s].shape[0]
            assert n == int(batch.lens[s])
            got = [torch.empty((n, K, D), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
            mx.mx_kv_cache_read(layer.cache, *got, batch.slots(torch.arange(n, device="cuda")[None].expand(seqs, n))[s].contiguous())
            for t, r in zip(got, (keys[s], values[s])):
                assert _off(t, r) < (0.04 if fmt == "fp8" else 0.08)


def test_gradients_through_dispatch_and_combine():
    """out = sum_j w_j (x[t] * s[expert]) for scales s of each expert: the
    gradients of x and w through the calls, against the formula's in 64 bits."""
    T, k, E, N = 40, 3, 5, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((T, N), generator=g, device="cuda").bfloat16()
    w = torch.rand((T, k), generator=g, device="cuda")
    ids = torch.randint(-1, E + 1, (T, k), generator=g, device="cuda")
    scale = torch.exp2(torch.arange(E, device="cuda").float() - 2)     # powers of two: products are exact
    d_out = torch.randn((T, N), generator=g, device="cuda")
    rows, _, offs, pos = mx.moe_dispatch(x, ids, E, torch.bfloat16)
    n = int(offs[-1])
    expert = torch.bucketize(torch.arange(n, device="cuda"), offs, right=True)
    y = rows[:n].float() * scale[expert][:, None]
    out = mx.moe_combine(y, pos, w, torch.float32)
    d_y, d_w = mx.moe_combine_grad(d_out, y, pos, w)
    d_x = mx.moe_combine(d_y * scale[expert][:, None], pos, None, torch.float32)
    held = (ids >= 0) & (ids < E)
    s = torch.where(held, scale[ids.clamp(0, E - 1)], 0).double()
    want = (w.double() * s).sum(1, keepdim=True) * x.double()
    size = (w.double() * s).sum(1, keepdim=True) * x.double().abs()
    assert (torch.abs(out.double() - want) <= size * k * 2.0 ** -24 * 1.01).all()
    want = (w.double() * s).sum(1, keepdim=True) * d_out.double()
    size = (w.double() * s).sum(1, keepdim=True) * d_out.double().abs()
    # the product's rounding and k - 1 additions'
    assert (torch.abs(d_x.double() - want) <= size * k * 2.0 ** -24 * 1.01).all()
    want = (d_out.double() * x.double()).sum(1, keepdim=True) * s
    size = (d_out.double() * x.double()).abs().sum(1, keepdim=True) * s
    assert (torch.abs(d_w.double() - want) <= size * 18 * 2.0 ** -24 * 1.01).all()
