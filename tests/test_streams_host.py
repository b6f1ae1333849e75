"""Host checks of the binding's convenience forms on a given stream: what they
allocate is made on the stream that writes it (no GPU needed: torch's streams,
its allocator and the library's entry points are replaced by stand-ins)."""
from __future__ import annotations

import contextlib

import pytest
import torch

import block_scaled_precision_mm_amd as mx

A = 0x10000


class OnGpu(torch.Tensor):
    """A CPU tensor that says it is on the GPU."""

    is_cuda = True

    def get_device(self):
        return 0


@pytest.fixture
def made(monkeypatch):
    """[(tensor's shape, stream that was current)] of what a call allocates."""
    log, now = [], [7]
    empty, empty_like = torch.empty, torch.empty_like

    @contextlib.contextmanager
    def stream(s):
        before, now[0] = now[0], s if isinstance(s, int) else s.cuda_stream
        yield
        now[0] = before

    def as_gpu(t):
        log.append((tuple(t.shape), now[0]))
        return t.as_subclass(OnGpu)

    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **kw: as_gpu(empty(*a, **kw)))
    monkeypatch.setattr(torch, "empty_like", lambda t, **kw: as_gpu(empty(t.shape, dtype=t.dtype)))
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda ptr, **kw: ptr)
    monkeypatch.setattr(mx, "_current_device", lambda: 0)
    monkeypatch.setattr(mx, "_raw_stream", lambda device: now[0])
    for fn in ("mx_rmsnorm", "mx_paged_attention", "mx_scaled_mm_fp8"):
        monkeypatch.setattr(mx._lib, fn, lambda *args, fn=fn: log.append((fn, args[-1])) or 0)
    return log


def gpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


class Stream:
    cuda_stream = 9


@pytest.mark.parametrize("stream,want", [(None, 7), (9, 9), (Stream(), 9), (0, 0)])
def test_outputs_are_made_on_the_stream_that_writes_them(made, stream, want):
    x = gpu(4, 64)
    mx.rmsnorm(x, None, residual=gpu(4, 64), stream=stream)
    mx.rmsnorm(x, None, out=torch.bfloat16, stream=stream)
    mx.scaled_mm(A, A, A, A, fmt="fp8", M=32, N=64, K=128, workspace=None, stream=stream)
    t = [torch.zeros(2, 2, 16, n, dtype=torch.uint8).as_subclass(OnGpu) for n in (128, 4, 128, 4)]
    cache = mx.KVCache(*t)
    i32 = lambda *s: gpu(*s, dtype=torch.int32)  # noqa: E731
    mx.paged_attention(cache, gpu(3, 4, 128), i32(1), i32(1), i32(1, 2), workspace=None, stream=stream)
    shapes = [s for s, _ in made]
    assert shapes.count("mx_rmsnorm") == 2 and "mx_scaled_mm_fp8" in shapes and "mx_paged_attention" in shapes
    assert {s for _, s in made} == {want}, made
