"""Plain 64-bit forms of the operators around the products, for their tests:
RMSNorm, the cache's rows from its codes (oracle decode), attention, and the
error bounds that the kernels' roundings give.  CPU, numpy."""
from __future__ import annotations

import numpy as np
import torch

import oracle

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def bf16(x) -> torch.Tensor:
    return torch.as_tensor(np.asarray(x, dtype=np.float32)).to(torch.bfloat16)


def bits(t: torch.Tensor) -> np.ndarray:
    return t.contiguous().cpu().view(torch.int16).numpy().view(np.uint16)


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().to(torch.float64).numpy()


def rmsnorm(h: np.ndarray, w, eps: float) -> np.ndarray:
    y = h / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    return y if w is None else y * w


def rows_of(fmt: str, codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """float64 values of a cache's rows: codes [..][bytes], scales [..][dim/32]."""
    lead = codes.shape[:-1]
    n = int(np.prod(lead)) if lead else 1
    dim = codes.shape[-1] * (2 if fmt == "fp4" else 1)
    v = oracle.decode(fmt, codes.reshape(n, -1), n, dim)
    s = oracle.decode_scale(scales.reshape(n, -1))
    with np.errstate(invalid="ignore"):
        return (v.reshape(n, -1, 32) * s[:, :, None]).reshape(lead + (dim,))


def attention(q, k, v, scale, causal, window, new, here=None):
    """q [new][Hq][D], k, v [L][H][D] float64; here [L]: keys that are there.
    Returns out, lse, spread = sum of weight * |v|, and the error of an FP32
    score relative to the largest one of its row."""
    L, H, D = k.shape
    n, Hq, _ = q.shape
    G = Hq // H
    out = np.zeros((n, Hq, D))
    lse = np.full((n, Hq), -np.inf)
    spread = np.zeros((n, Hq, D))
    err = np.zeros((n, Hq))
    for i in range(n):
        pos = L - n + i
        j = np.arange(L)
        see = np.ones(L, bool) if here is None else here.copy()
        if causal:
            see &= j <= pos
        if window:
            see &= j > pos - window
        if not see.any():
            continue
        for hq in range(Hq):
            kk, vv, qq = k[see, hq // G], v[see, hq // G], q[i, hq]
            x = scale * (kk @ qq)
            m = np.max(x)
            p = np.exp(x - m)
            out[i, hq] = p @ vv / p.sum()
            lse[i, hq] = m + np.log(p.sum())
            spread[i, hq] = p @ np.abs(vv) / p.sum()
            # FP32: D products accumulated, then x * log2 e - m and 2^that (each
            # within 2^-23 of what it works on, 2^-21 for the exponential)
            dot = scale * np.max(np.abs(kk) @ np.abs(qq))
            err[i, hq] = D * 2.0 ** -24 * dot + 4 * np.max(np.abs(x)) * 2.0 ** -23 + 2.0 ** -21
    return out, lse, spread, err


def check_attention(got, lse, ref, L, what):
    """Every p is off by 2 err (its own score's and the reference's) and half a
    BF16 step as an operand; sums of L terms in FP32; then the output's own
    rounding."""
    out, rl, spread, err = ref
    g = f64(got)
    sums = L * 2.0 ** -24
    tol = spread * (2.0 ** -8 + 4 * err[..., None] + 2 * sums) * 1.01 + np.abs(out) * HALF[got.dtype] * 1.01 + 1e-30
    nan = np.isnan(out)
    assert np.array_equal(np.isnan(g), nan), what + ": NaN elsewhere"
    bad = np.abs(g - out) > tol
    assert not (bad & ~nan).any(), "%s: off by %.3g where %.3g is allowed" % (
        what, np.abs(g - out)[bad & ~nan].max(), tol[bad & ~nan].min())
    if lse is not None:
        gl = f64(lse)
        fin = np.isfinite(rl)
        assert np.array_equal(np.isnan(gl), np.isnan(rl)), what + ": lse NaN elsewhere"
        assert np.array_equal(gl[~fin & ~np.isnan(rl)], rl[~fin & ~np.isnan(rl)]), what + ": lse of empty rows"
        t = 2 * err + 2 * sums + 4 * np.abs(np.where(fin, rl, 0)) * 2.0 ** -24 + 2.0 ** -21
        off = np.abs(gl[fin] - rl[fin])
        assert (off <= t[fin]).all(), "%s: lse off by %.3g" % (what, (off - t[fin]).max())
