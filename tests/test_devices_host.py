"""Host checks: the binding launches on the current device, and refuses a
tensor that lies on another one before the library is called (no GPU needed:
the tensors are stand-ins, and so are the library's entry points)."""
from __future__ import annotations

import pytest
import torch

import block_scaled_precision_mm_amd as mx

BF, U8, I32 = torch.bfloat16, torch.uint8, torch.int32


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


# name: (call of the operands by name, operands: shape and type, or a maker)
CALLS = {
    "mx_rmsnorm": (lambda t: mx.mx_rmsnorm(t["x"], t["r"], t["w"], t["h"], t["y"], t["s"], 4, 64, 1e-6),
                   dict(x=((4, 64), BF), r=((4, 64), BF), w=((64,), BF), h=((4, 64), BF), y=((4, 64), U8), s=((4, 2), U8))),
    "mx_kv_cache_write": (lambda t: mx.mx_kv_cache_write(t["c"], t["k"], t["v"], t["at"]),
                          dict(c=_cache, k=((3, 2, 128), BF), v=((3, 2, 128), BF), at=((3,), torch.int64))),
    "mx_kv_cache_read": (lambda t: mx.mx_kv_cache_read(t["c"], t["k"], t["v"], t["at"]),
                         dict(c=_cache, k=((3, 2, 128), BF), v=((3, 2, 128), BF), at=((3,), torch.int64))),
    "mx_paged_attention": (lambda t: mx.mx_paged_attention(t["c"], t["q"], t["e"], t["l"], t["t"], t["o"], lse=t["ls"],
                                                           workspace=t["ws"]),
                           dict(c=_cache, q=((3, 4, 128), BF), e=((1,), I32), l=((1,), I32), t=((1, 2), I32),
                                o=((3, 4, 128), BF), ls=((3, 4), torch.float32), ws=((1 << 24,), U8))),
    "mx_scaled_mm_fp8": (lambda t: mx.mx_scaled_mm_fp8(t["a"], t["b"], t["sa"], t["sb"], t["c"], 32, 64, 128, workspace=None),
                         dict(a=((32, 128), U8), b=((64, 128), U8), sa=((32, 4), U8), sb=((64, 4), U8), c=((32, 64), BF))),
    "mx_scaled_mm_config": (lambda t: mx.mx_scaled_mm_config(False, t["a"], t["b"], t["sa"], t["sb"], t["c"], 32, 64, 128, 0,
                                                             workspace=None),
                            dict(a=((32, 128), U8), b=((64, 128), U8), sa=((32, 4), U8), sb=((64, 4), U8), c=((32, 64), BF))),
    "mx_scaled_mm_noalloc": (lambda t: mx.mx_scaled_mm_noalloc(False, t["a"], t["b"], t["sa"], t["sb"], t["c"], 32, 64, 128),
                             dict(a=((32, 128), U8), b=((64, 128), U8), sa=((32, 4), U8), sb=((64, 4), U8), c=((32, 64), BF))),
    "mx_scaled_mm_fused": (lambda t: mx.mx_scaled_mm_fused(False, t["a"], t["b"], t["sa"], t["sb"], t["bias"], 0, t["c"], None,
                                                           32, 64, 128),
                           dict(a=((32, 128), U8), b=((64, 128), U8), sa=((32, 4), U8), sb=((64, 4), U8), bias=((64,), BF),
                                c=((32, 64), BF))),
    "mx_grouped_mm_fp8": (lambda t: mx.mx_grouped_mm_fp8(t["a"], t["b"], t["sa"], t["sb"], t["c"], t["o"], 2, 32, 64, 128),
                          dict(a=((32, 128), U8), b=((2, 64, 128), U8), sa=((32, 4), U8), sb=((2, 64, 4), U8),
                               c=((32, 64), BF), o=((2,), I32))),
    "mx_quantize_bf16": (lambda t: mx.mx_quantize_bf16(t["x"], t["c"], t["s"], 4, 64, False),
                         dict(x=((4, 64), BF), c=((4, 64), U8), s=((4, 2), U8))),
    "mx_dense_gemm": (lambda t: mx.mx_dense_gemm(t["a"], t["b"], t["c"], 32, 64, 128),
                      dict(a=((32, 128), BF), b=((128, 64), BF), c=((32, 64), BF))),
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
def test_an_operand_on_another_device_is_refused(called, name):
    call, operands = CALLS[name]

    def make(n, index):
        how = operands[n]
        return how(index) if callable(how) else gpu(*how, index)

    call({n: make(n, 0) for n in operands})
    assert called == [name]
    for there in operands:
        with pytest.raises(ValueError):
            call({n: make(n, int(n == there)) for n in operands})
    assert called == [name]


def test_a_cache_lies_on_one_device():
    for there in range(4):
        with pytest.raises(ValueError):
            mx.KVCache(*(gpu((2, 2, 16, n), U8, int(i == there)) for i, n in enumerate((128, 4, 128, 4))))


def test_tensors_are_refused_where_there_is_no_gpu(monkeypatch):
    def none():
        raise RuntimeError("no GPU")

    monkeypatch.setattr(mx, "_current_device", none)
    x = torch.zeros(4, 64, dtype=BF)
    with pytest.raises(ValueError):
        mx.mx_rmsnorm(x, None, None, None, x, None, 4, 64, 1e-6)


@pytest.mark.parametrize("kind", [-1, 5, 7])
def test_an_output_kind_that_is_none_is_the_librarys_to_refuse(monkeypatch, kind):
    # a status, as with raw pointers, and no IndexError
    monkeypatch.setattr(mx, "_current_device", lambda: 0)
    monkeypatch.setattr(mx, "_raw_stream", lambda device: 0)
    with pytest.raises(mx.MxGemmError) as e:
        mx.mx_rmsnorm(gpu((4, 64), BF), None, None, None, gpu((4, 64), BF), None, 4, 64, 1e-6, out_kind=kind)
    assert e.value.status == -5
