"""Python binding of the gfx950 NT MX block-scaled GEMM library (libmxgemm.so).

Argument marshalling only: every step of the product runs in the HIP
kernels of ``csrc/``.  PyTorch supplies device memory and the stream.  The
functions carry the C ABI's names (see ``include/mxgemm.h``):

    mx_scaled_mm_fp4(a, b, a_scale, b_scale, c, M, N, K, out_dtype=None, workspace="auto", stream=None)
    mx_scaled_mm_fp8(...)
    mx_scaled_mm_workspace_bytes(is_fp4, M, N, K)
    mx_scaled_mm_config(is_fp4, a, b, a_scale, b_scale, c, M, N, K, variant, splits=1,
                        workspace="auto", out_dtype=None, stream=None)
    mx_default_config(is_fp4, M, N, K, with_workspace=True) -> (variant, splits)
    mx_default_variant(is_fp4, M, N, K)

``a``/``b`` are contiguous 1-byte CUDA tensors holding packed codes
([M, K/2] / [N, K/2] for MXFP4, [M, K] / [N, K] for MXFP8), the scales are
[M, K/32] / [N, K/32] E8M0 bytes, ``c`` is a contiguous [M, N] tensor of
the output dtype.  A non-zero status raises MxGemmError (the caller's cue to
fall back to another implementation).  There is no CPU fallback: if the
library is missing, importing this package raises.  Tensors lie on the current
device, on which the call is launched; others are refused (ValueError).

``scaled_mm`` is the convenience form that allocates C and returns it.  Given
a stream, the convenience forms allocate on it, as under torch.cuda.stream.

``workspace="auto"`` keeps one workspace per stream, which grows with the
largest call; host threads that call on one stream take turns at it.  A call that torch captures into a graph gets one of its own
from the graph's memory instead, which the graph clears before it (a fill of
64 KiB; with an explicit workspace, cleared once, there is none).  A graph
captured by other means than torch's takes an explicit workspace.

Around the products (see the same header):

    mx_rmsnorm(x, residual, weight, h, y, y_scale, rows, K, eps, out_kind=None, stream=None)
    KVCache(k_codes, k_scales, v_codes, v_scales, fmt), KVCache.empty(pages, page_size, kv_heads, head_dim, fmt)
    mx_kv_cache_write(cache, k, v, slots, stream=None)
    mx_kv_cache_read(cache, k, v, slots, stream=None)
    mx_paged_attention(cache, q, ends, lens, table, out, lse=None, scale=None, causal=True, window=0,
                       max_new=None, workspace="auto", stream=None)

Beside them, for drafted tokens and for experts:

    mx_rope_cache_write(cache, q, k, v, positions, slots, rope, q_out=None, interleaved=False, stream=None)
    mx_tree_attention(cache, q, ends, lens, table, mask, out, lse=None, scale=None, window=0, max_new=None,
                      workspace="auto", stream=None)
    mx_moe_dispatch(x, experts, y, y_scale, offs, pos, workspace="auto", stream=None)
    mx_moe_combine(y, pos, weights, out, stream=None)
    mx_moe_combine_grad(d_out, y, pos, weights, d_y, d_y_scale=None, d_weights=None, stream=None)

``rmsnorm``, ``paged_attention``, ``tree_attention``, ``moe_dispatch``,
``moe_combine`` and ``moe_combine_grad`` are their convenience forms;
``rope_table`` and ``tree_mask`` make the tables that the calls take.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading

import torch  # load torch's HIP runtime first so the library binds to the same one

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmxgemm.so")

OUT_BF16, OUT_F16, OUT_F32 = 0, 1, 2
_OUT_OF_DTYPE = {torch.bfloat16: OUT_BF16, torch.float16: OUT_F16, torch.float32: OUT_F32}
_DTYPE_OF_OUT = {v: k for k, v in _OUT_OF_DTYPE.items()}

if not os.path.exists(LIB_PATH):
    raise ImportError("libmxgemm.so is not built (%s); run __graft_entry__.build() or "
                      "python block_scaled_precision_mm_amd/build.py" % LIB_PATH)

_lib = ctypes.CDLL(LIB_PATH)
_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t
_INT = ctypes.c_int
_lib.mx_scaled_mm_fp4.argtypes = [_P, _P, _P, _P, _P, _I64, _I64, _I64, _INT, _P, _SZ, _P]
_lib.mx_scaled_mm_fp8.argtypes = _lib.mx_scaled_mm_fp4.argtypes
_lib.mx_scaled_mm_config.argtypes = [_INT, _P, _P, _P, _P, _P, _I64, _I64, _I64, _INT, _INT, _INT, _P, _SZ, _P]
_lib.mx_scaled_mm_workspace_bytes.argtypes = [_INT, _I64, _I64, _I64]
_lib.mx_scaled_mm_workspace_bytes.restype = _SZ
_lib.mx_config_workspace_bytes.argtypes = [_INT, _INT, _I64, _I64]
_lib.mx_config_workspace_bytes.restype = _SZ
_lib.mx_default_config.argtypes = [_INT, _I64, _I64, _I64, _INT, ctypes.POINTER(_INT)]
_lib.mx_default_variant.argtypes = [_INT, _I64, _I64, _I64]
_lib.mx_scaled_mm_noalloc.argtypes = [_INT, _P, _P, _P, _P, _P, _I64, _I64, _I64, _INT, _P]
_lib.mx_noalloc_scratch_bytes.restype = _SZ
_lib.mx_variant_max_k.argtypes = [_INT, _INT]
_lib.mx_variant_max_k.restype = _I64
_lib.mx_status_string.argtypes = [_INT]
_lib.mx_status_string.restype = ctypes.c_char_p
_lib.mx_variant_name.argtypes = [_INT]
_lib.mx_variant_name.restype = ctypes.c_char_p
_lib.mx_quantize_bf16.argtypes = [_P, _P, _P, _I64, _I64, _INT, _P]
_lib.mx_grouped_mm_fp4.argtypes = [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _INT, _P]
_lib.mx_grouped_mm_fp8.argtypes = _lib.mx_grouped_mm_fp4.argtypes
_lib.mx_grouped_mm_config.argtypes = [_INT, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _INT, _INT, _P]
_lib.mx_grouped_variant_name.argtypes = [_INT]
_lib.mx_grouped_variant_name.restype = ctypes.c_char_p
_lib.mx_grouped_default_variant.argtypes = [_I64, _I64, _I64]
_lib.mx_scaled_mm_fused.argtypes = [_INT, _P, _P, _P, _P, _P, _INT, _P, _P, _I64, _I64, _I64, _INT, _INT, _P]
_lib.mx_fused_variant_name.argtypes = [_INT]
_lib.mx_fused_variant_name.restype = ctypes.c_char_p
_lib.mx_fused_default_variant.argtypes = [_INT, _I64, _I64, _I64]
_lib.mx_fused_variant_max_k.argtypes = [_INT, _INT]
_lib.mx_fused_variant_max_k.restype = _I64
_lib.mx_dense_gemm.argtypes = [_INT, _INT, _INT, _P, _P, _P, _I64, _I64, _I64, _INT, _P]
_lib.mx_empty_like.argtypes = [_INT, _I64, _I64, _I64, _P]
_lib.mx_rmsnorm.argtypes = [_P, _P, _P, _P, _P, _P, _I64, _I64, ctypes.c_float, _INT, _P]
_lib.mx_kv_cache_write.argtypes = [_P, _P, _P, _I64, _I64, _P, _I64, _P]
_lib.mx_kv_cache_read.argtypes = _lib.mx_kv_cache_write.argtypes
_lib.mx_paged_attention.argtypes = [_P, _P, _I64, _P, _P, _P, _I64, _I64, _I64, _I64, _I64, ctypes.c_float,
                                    _INT, _I64, _P, _INT, _P, _P, _SZ, _P]
_lib.mx_paged_attention_workspace_bytes.argtypes = [_P, _I64, _I64, _I64, _I64]
_lib.mx_paged_attention_workspace_bytes.restype = _SZ
_lib.mx_rope_cache_write.argtypes = [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _I64, _P, _P, _P, _I64, _I64, _INT,
                                     _I64, _P]
_lib.mx_tree_attention.argtypes = [_P, _P, _I64, _P, _P, _P, _I64, _P, _I64, _I64, _I64, _I64, _I64, ctypes.c_float,
                                   _I64, _P, _INT, _P, _P, _SZ, _P]
_lib.mx_tree_attention_workspace_bytes.argtypes = [_P, _I64, _I64, _I64, _I64]
_lib.mx_tree_attention_workspace_bytes.restype = _SZ
_lib.mx_moe_dispatch.argtypes = [_P, _P, _I64, _I64, _I64, _I64, _P, _P, _INT, _P, _P, _P, _SZ, _P]
_lib.mx_moe_dispatch_workspace_bytes.argtypes = [_I64, _I64, _I64]
_lib.mx_moe_dispatch_workspace_bytes.restype = _SZ
_lib.mx_moe_combine.argtypes = [_P, _INT, _P, _P, _I64, _I64, _I64, _I64, _P, _INT, _P]
_lib.mx_moe_combine_grad.argtypes = [_P, _P, _INT, _P, _P, _I64, _I64, _I64, _I64, _P, _P, _INT, _P, _P]
for _f in ("mx_rmsnorm", "mx_kv_cache_write", "mx_kv_cache_read", "mx_paged_attention", "mx_rope_cache_write",
           "mx_tree_attention", "mx_moe_dispatch", "mx_moe_combine", "mx_moe_combine_grad", "mx_scaled_mm_fp4", "mx_scaled_mm_fp8", "mx_scaled_mm_config", "mx_num_variants",
           "mx_default_config", "mx_scaled_mm_noalloc",
           "mx_last_hip_error", "mx_abi_version", "mx_default_variant", "mx_quantize_bf16",
           "mx_grouped_mm_fp4", "mx_grouped_mm_fp8", "mx_grouped_mm_config",
           "mx_grouped_num_variants", "mx_grouped_default_variant", "mx_scaled_mm_fused",
           "mx_fused_num_variants", "mx_fused_default_variant", "mx_dense_gemm", "mx_empty_like"):
    getattr(_lib, _f).restype = _INT

# every symbol include/mxgemm.h declares
EXPORTS = ("mx_scaled_mm_fp4", "mx_scaled_mm_fp8", "mx_scaled_mm_config", "mx_num_variants",
           "mx_scaled_mm_workspace_bytes", "mx_config_workspace_bytes", "mx_default_config",
           "mx_scaled_mm_noalloc", "mx_noalloc_scratch_bytes",
           "mx_variant_max_k", "mx_variant_name", "mx_default_variant", "mx_status_string",
           "mx_last_hip_error", "mx_abi_version", "mx_quantize_bf16",
           "mx_grouped_mm_fp4", "mx_grouped_mm_fp8", "mx_grouped_mm_config",
           "mx_grouped_num_variants", "mx_grouped_variant_name", "mx_grouped_default_variant",
           "mx_scaled_mm_fused", "mx_fused_num_variants", "mx_fused_variant_name",
           "mx_fused_default_variant", "mx_fused_variant_max_k", "mx_dense_gemm", "mx_empty_like",
           "mx_rmsnorm", "mx_kv_cache_write", "mx_kv_cache_read", "mx_paged_attention",
           "mx_paged_attention_workspace_bytes", "mx_rope_cache_write", "mx_tree_attention",
           "mx_tree_attention_workspace_bytes", "mx_moe_dispatch", "mx_moe_dispatch_workspace_bytes",
           "mx_moe_combine", "mx_moe_combine_grad")


class MxGemmError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib.mx_status_string(status).decode()
        if status == -8:
            msg += " (hipError %d)" % _lib.mx_last_hip_error()
        super().__init__("%s: %s (status %d)" % (where, msg, status))


def _ptr(t) -> int:
    if t is None:
        return 0
    if isinstance(t, int):
        return t
    return t.data_ptr()


# the current stream's handle without the Stream object around it (3 us a
# call), and whether it is being captured
_raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
_is_capturing = torch._C._cuda_isCurrentStreamCapturing


def _here() -> int:
    """The current device, whose streams the calls run on: tensors have to lie
    on it.  Without a GPU a number that is no tensor's (-1 is the CPU's)."""
    try:
        return _current_device()
    except RuntimeError:
        return -2


def _stream(stream, device=None) -> int:
    if stream is None:
        return _raw_stream(_current_device() if device is None else device)
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check_tensors(is_fp4, a, b, sa, sb, c, M, N, K):
    """Shape/contiguity checks on torch tensors (ints pass through as raw pointers)."""
    eb, dev = K // 2 if is_fp4 else K, _here()
    for name, t, rows, cols in (("a", a, M, eb), ("b", b, N, eb), ("a_scale", sa, M, K // 32),
                                ("b_scale", sb, N, K // 32)):
        if isinstance(t, torch.Tensor):
            if t.get_device() != dev or not t.is_contiguous() or t.element_size() != 1:
                raise ValueError("%s must be a contiguous 1-byte CUDA tensor on the current device" % name)
            if t.numel() != rows * cols:
                raise ValueError("%s has %d bytes, expected %d x %d" % (name, t.numel(), rows, cols))
    if isinstance(c, torch.Tensor):
        if c.get_device() != dev or not c.is_contiguous() or c.numel() != M * N:
            raise ValueError("c must be a contiguous CUDA tensor with M*N elements on the current device")


def _out_code(c, out_dtype):
    if out_dtype is not None:
        return out_dtype
    if isinstance(c, torch.Tensor):
        return _OUT_OF_DTYPE[c.dtype]
    raise ValueError("out_dtype is required when c is a raw pointer")


_WORKSPACES, _WORKSPACE_LOCKS = {}, {}      # by (device, stream)
_COUNTER_BYTES = 65536          # of a workspace, at its start: zero before every call


def _on_stream(stream_ptr):
    """The context in which tensors are made, filled and, later, given back to
    the allocator on that stream."""
    return torch.cuda.stream(torch.cuda.ExternalStream(stream_ptr))


def _made_on(stream):
    """The context for a convenience form's outputs: memory of the stream that
    writes them (memory of the current stream may still be in use there)."""
    return contextlib.nullcontext() if stream is None else _on_stream(_stream(stream))


def _auto_workspace(key, nbytes):
    """The stream's workspace, or one for this call alone where it is captured:
    a graph may be replayed after any later call of the stream, and before any
    graph that was captured earlier."""
    stream_ptr = key[1]
    if stream_ptr == _raw_stream(key[0]):
        captured = _is_capturing()
    else:
        with _on_stream(stream_ptr):
            captured = _is_capturing()
    if captured:
        with _on_stream(stream_ptr):
            held = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
            held[:_COUNTER_BYTES].zero_()
        return held
    held = _WORKSPACES.get(key)
    if held is None or held.numel() < nbytes:
        with _on_stream(stream_ptr):
            held = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
        _WORKSPACES[key] = held
    return held


def _call(name, fn, args, workspace, nbytes, dev, stream_ptr):
    """fn(*args, workspace, its bytes, stream) with the workspace argument of
    the call (see the module doc), nbytes being what the call splits with."""
    if workspace is None or nbytes == 0:
        st = fn(*args, 0, 0, stream_ptr)
    elif isinstance(workspace, torch.Tensor):
        if workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor on the current device")
        st = fn(*args, workspace.data_ptr(), workspace.numel() * workspace.element_size(), stream_ptr)
    elif workspace == "auto":
        # one thread at a time from the lookup to the last launch: a call's second
        # kernel reads what its first left in the workspace
        key = (dev, stream_ptr)
        lock = _WORKSPACE_LOCKS.get(key) or _WORKSPACE_LOCKS.setdefault(key, threading.RLock())
        with lock:
            held = _auto_workspace(key, nbytes)
            st = fn(*args, held.data_ptr(), held.numel(), stream_ptr)
    else:
        raise ValueError("workspace must be a tensor, None or 'auto'")
    if st:
        raise MxGemmError(st, name)


def mx_scaled_mm_workspace_bytes(is_fp4, M, N, K) -> int:
    return int(_lib.mx_scaled_mm_workspace_bytes(int(bool(is_fp4)), M, N, K))


def mx_config_workspace_bytes(variant, splits, M, N) -> int:
    return int(_lib.mx_config_workspace_bytes(variant, splits, M, N))


def _default(is_fp4, a, b, a_scale, b_scale, c, M, N, K, out_dtype, workspace, stream, fn, name):
    _check_tensors(is_fp4, a, b, a_scale, b_scale, c, M, N, K)
    dev = _here()
    _call(name, fn, (_ptr(a), _ptr(b), _ptr(a_scale), _ptr(b_scale), _ptr(c), M, N, K, _out_code(c, out_dtype)),
          workspace, mx_scaled_mm_workspace_bytes(is_fp4, M, N, K), dev, _stream(stream, dev))


def mx_scaled_mm_fp4(a, b, a_scale, b_scale, c, M, N, K, out_dtype=None, workspace="auto",
                     stream=None) -> None:
    _default(True, a, b, a_scale, b_scale, c, M, N, K, out_dtype, workspace, stream,
             _lib.mx_scaled_mm_fp4, "mx_scaled_mm_fp4")


def mx_scaled_mm_fp8(a, b, a_scale, b_scale, c, M, N, K, out_dtype=None, workspace="auto",
                     stream=None) -> None:
    _default(False, a, b, a_scale, b_scale, c, M, N, K, out_dtype, workspace, stream,
             _lib.mx_scaled_mm_fp8, "mx_scaled_mm_fp8")


def mx_scaled_mm_config(is_fp4, a, b, a_scale, b_scale, c, M, N, K, variant, splits=1,
                        workspace="auto", out_dtype=None, stream=None) -> None:
    _check_tensors(bool(is_fp4), a, b, a_scale, b_scale, c, M, N, K)
    dev = _here()
    _call("mx_scaled_mm_config", _lib.mx_scaled_mm_config,
          (int(bool(is_fp4)), _ptr(a), _ptr(b), _ptr(a_scale), _ptr(b_scale), _ptr(c), M, N, K,
           _out_code(c, out_dtype), variant, splits),
          workspace, mx_config_workspace_bytes(variant, splits, M, N), dev, _stream(stream, dev))


def mx_default_config(is_fp4, M, N, K, with_workspace=True):
    """(variant, K parts) of the default entry points for this shape."""
    sp = _INT(0)
    v = int(_lib.mx_default_config(int(bool(is_fp4)), M, N, K, int(bool(with_workspace)), ctypes.byref(sp)))
    if v < 0:
        raise MxGemmError(v, "mx_default_config")
    return v, int(sp.value)


def mx_default_variant(is_fp4, M, N, K) -> int:
    v = int(_lib.mx_default_variant(int(bool(is_fp4)), M, N, K))
    if v < 0:
        raise MxGemmError(v, "mx_default_variant")
    return v


def mx_num_variants() -> int:
    return int(_lib.mx_num_variants())


def mx_variant_max_k(variant, is_fp4) -> int:
    v = int(_lib.mx_variant_max_k(variant, int(bool(is_fp4))))
    if v < 0:
        raise MxGemmError(v, "mx_variant_max_k")
    return v


def variants_for(is_fp4, K):
    """Every variant that accepts this format and K."""
    return [v for v in range(mx_num_variants()) if K <= mx_variant_max_k(v, is_fp4)]


def mx_variant_name(variant) -> str | None:
    r = _lib.mx_variant_name(variant)
    return None if r is None else r.decode()


def mx_status_string(status) -> str:
    return _lib.mx_status_string(status).decode()


def mx_last_hip_error() -> int:
    return int(_lib.mx_last_hip_error())


def mx_abi_version() -> int:
    return int(_lib.mx_abi_version())


def mx_quantize_bf16(x, codes, scales, rows: int, K: int, is_fp4: bool, stream=None) -> None:
    """MX-quantize BF16 rows along K on the GPU (C ABI mx_quantize_bf16).

    x: bfloat16 [rows][K] (or a raw device pointer); codes: uint8 [rows][K/2]
    (E2M1, two per byte, even k low nibble) or [rows][K] (E4M3); scales:
    uint8 [rows][K/32] E8M0.  Argument marshalling only.
    """
    dev = _here()
    if isinstance(x, torch.Tensor):
        if x.get_device() != dev or not x.is_contiguous() or x.element_size() != 2 or x.numel() != rows * K:
            raise ValueError("x must be a contiguous 2-byte CUDA tensor with rows*K elements on the current device")
    for name, t, n in (("codes", codes, rows * (K // 2 if is_fp4 else K)), ("scales", scales, rows * (K // 32))):
        if isinstance(t, torch.Tensor):
            if t.get_device() != dev or not t.is_contiguous() or t.element_size() != 1 or t.numel() != n:
                raise ValueError("%s must be a contiguous 1-byte CUDA tensor of %d elements on the current device" % (name, n))
    rc = _lib.mx_quantize_bf16(_ptr(x), _ptr(codes), _ptr(scales), rows, K, 1 if is_fp4 else 0,
                               _stream(stream))
    if rc != 0:
        raise MxGemmError(rc, "mx_quantize_bf16")


def _check_grouped(is_fp4, a, b, sa, sb, c, offs, groups, M, N, K):
    eb, dev = K // 2 if is_fp4 else K, _here()
    for name, t, n in (("a", a, M * eb), ("b", b, groups * N * eb), ("a_scale", sa, M * (K // 32)),
                       ("b_scale", sb, groups * N * (K // 32))):
        if isinstance(t, torch.Tensor):
            if t.get_device() != dev or not t.is_contiguous() or t.element_size() != 1 or t.numel() != n:
                raise ValueError("%s must be a contiguous 1-byte CUDA tensor of %d bytes on the current device" % (name, n))
    if isinstance(c, torch.Tensor):
        if c.get_device() != dev or not c.is_contiguous() or c.numel() != M * N:
            raise ValueError("c must be a contiguous CUDA tensor with M*N elements on the current device")
    if isinstance(offs, torch.Tensor):
        if offs.get_device() != dev or offs.dtype != torch.int32 or not offs.is_contiguous() or offs.numel() != groups:
            raise ValueError("offs must be a contiguous int32 CUDA tensor of `groups` elements on the current device")


def mx_grouped_mm_fp4(a, b, a_scale, b_scale, c, offs, groups, M, N, K, out_dtype=None,
                      stream=None) -> None:
    """Grouped MXFP4 product (C ABI mx_grouped_mm_fp4): rows [offs[g-1], offs[g])
    of a times b[g] (b is [groups][N][K/2]); offs is an int32 device tensor."""
    _check_grouped(True, a, b, a_scale, b_scale, c, offs, groups, M, N, K)
    st = _lib.mx_grouped_mm_fp4(_ptr(a), _ptr(b), _ptr(a_scale), _ptr(b_scale), _ptr(c), _ptr(offs),
                                groups, M, N, K, _out_code(c, out_dtype), _stream(stream))
    if st:
        raise MxGemmError(st, "mx_grouped_mm_fp4")


def mx_grouped_mm_fp8(a, b, a_scale, b_scale, c, offs, groups, M, N, K, out_dtype=None,
                      stream=None) -> None:
    """Grouped MXFP8 product (C ABI mx_grouped_mm_fp8); b is [groups][N][K]."""
    _check_grouped(False, a, b, a_scale, b_scale, c, offs, groups, M, N, K)
    st = _lib.mx_grouped_mm_fp8(_ptr(a), _ptr(b), _ptr(a_scale), _ptr(b_scale), _ptr(c), _ptr(offs),
                                groups, M, N, K, _out_code(c, out_dtype), _stream(stream))
    if st:
        raise MxGemmError(st, "mx_grouped_mm_fp8")


def mx_grouped_mm_config(is_fp4, a, b, a_scale, b_scale, c, offs, groups, M, N, K, variant,
                         out_dtype=None, stream=None) -> None:
    _check_grouped(bool(is_fp4), a, b, a_scale, b_scale, c, offs, groups, M, N, K)
    st = _lib.mx_grouped_mm_config(int(bool(is_fp4)), _ptr(a), _ptr(b), _ptr(a_scale), _ptr(b_scale),
                                   _ptr(c), _ptr(offs), groups, M, N, K, _out_code(c, out_dtype),
                                   variant, _stream(stream))
    if st:
        raise MxGemmError(st, "mx_grouped_mm_config")


def mx_grouped_num_variants() -> int:
    return _lib.mx_grouped_num_variants()


def mx_grouped_variant_name(variant) -> str | None:
    n = _lib.mx_grouped_variant_name(variant)
    return n.decode() if n is not None else None


def mx_grouped_default_variant(groups, M, N) -> int:
    return _lib.mx_grouped_default_variant(groups, M, N)


OUT_BF16, OUT_F16, OUT_F32, OUT_MXFP8, OUT_MXFP4 = 0, 1, 2, 3, 4
_SIZE_OF_OUT = {OUT_BF16: 2, OUT_F16: 2, OUT_F32: 4, OUT_MXFP8: 1, OUT_MXFP4: 1}
ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU_TANH = 0, 1, 2, 3


def mx_scaled_mm_fused(is_fp4, a, b, a_scale, b_scale, bias, act, c, c_scale, M, N, K,
                       out_kind=None, variant=-1, stream=None) -> None:
    """MX GEMM with a fused epilogue (C ABI mx_scaled_mm_fused):
    y = act(A B^T + bias) into c (BF16/FP16/FP32, the dtype of c unless
    out_kind is given) or, with out_kind OUT_MXFP8 / OUT_MXFP4, MX codes into
    c (uint8 [M][N] or [M][N/2]) and E8M0 codes into c_scale (uint8 [M][N/32]).
    bias: bfloat16 [N] tensor or None.  Argument marshalling only."""
    _check_tensors(bool(is_fp4), a, b, a_scale, b_scale, None, M, N, K)
    if out_kind is None:
        out_kind = _out_code(c, None)
    dev = _here()
    if isinstance(bias, torch.Tensor):
        if bias.get_device() != dev or bias.dtype != torch.bfloat16 or not bias.is_contiguous() or bias.numel() != N:
            raise ValueError("bias must be a contiguous bfloat16 CUDA tensor of N elements on the current device")
    if isinstance(c, torch.Tensor):
        n = M * N if out_kind in (OUT_BF16, OUT_F16, OUT_F32, OUT_MXFP8) else M * N // 2
        if c.get_device() != dev or not c.is_contiguous() or c.numel() != n:
            raise ValueError("c must be a contiguous CUDA tensor of %d elements on the current device" % n)
    if isinstance(c_scale, torch.Tensor) and c_scale.get_device() != dev:
        raise ValueError("c_scale must be a CUDA tensor on the current device")
    st = _lib.mx_scaled_mm_fused(int(bool(is_fp4)), _ptr(a), _ptr(b), _ptr(a_scale), _ptr(b_scale),
                                 _ptr(bias), act, _ptr(c), _ptr(c_scale), M, N, K, out_kind, variant,
                                 _stream(stream))
    if st:
        raise MxGemmError(st, "mx_scaled_mm_fused")


def mx_fused_num_variants() -> int:
    return _lib.mx_fused_num_variants()


def mx_fused_default_variant(is_fp4, M, N, K) -> int:
    return _lib.mx_fused_default_variant(int(bool(is_fp4)), M, N, K)


def mx_fused_variant_max_k(variant, is_fp4) -> int:
    v = _lib.mx_fused_variant_max_k(variant, int(bool(is_fp4)))
    if v < 0:
        raise MxGemmError(v, "mx_fused_variant_max_k")
    return v


def mx_fused_variant_name(variant) -> str | None:
    n = _lib.mx_fused_variant_name(variant)
    return n.decode() if n is not None else None


def mx_dense_gemm(a, b, c, M, N, K, trans_a=0, trans_b=0, dtype=None, out_dtype=None,
                  stream=None) -> None:
    """Dense BF16 / FP16 product C = A B (C ABI mx_dense_gemm): a stored
    [M][K] (trans_a 0) or [K][M] (1), b stored [K][N] (trans_b 0) or [N][K]
    (1); dtype 0 BF16 / 1 FP16 (default: from a's torch dtype)."""
    if dtype is None:
        if not isinstance(a, torch.Tensor):
            raise ValueError("dtype is required when a is a raw pointer")
        dtype = {torch.bfloat16: 0, torch.float16: 1}[a.dtype]
    dev = _here()
    for name, t, n in (("a", a, M * K), ("b", b, N * K), ("c", c, M * N)):
        if isinstance(t, torch.Tensor):
            if t.get_device() != dev or not t.is_contiguous() or t.numel() != n:
                raise ValueError("%s must be a contiguous CUDA tensor of %d elements on the current device" % (name, n))
    st = _lib.mx_dense_gemm(dtype, trans_a, trans_b, _ptr(a), _ptr(b), _ptr(c), M, N, K,
                            _out_code(c, out_dtype), _stream(stream))
    if st:
        raise MxGemmError(st, "mx_dense_gemm")


# ------------------------------------------------------------- convenience
_FMT_OF_DTYPE = {}
for _name, _fmt in (("float4_e2m1fn_x2", "fp4"), ("float8_e4m3fn", "fp8")):
    if hasattr(torch, _name):
        _FMT_OF_DTYPE[getattr(torch, _name)] = _fmt


def _nk_storage(t):
    """A 2-D operand given as stored [rows][cols] (contiguous), or as the
    column-major [cols][rows] view of that storage (what F.scaled_mm takes as
    its second operand): the contiguous [rows][cols] tensor."""
    if t.dim() != 2:
        raise ValueError("operands must be 2-D")
    if t.is_contiguous():
        return t
    if t.t().is_contiguous():
        return t.t()
    raise ValueError("operand must be contiguous or the transpose of a contiguous tensor")


def scaled_mm_shapes(a, b, a_scale, b_scale, fmt=None):
    """(fmt, M, N, K, a, b, a_scale, b_scale) of a scaled_mm call with 2-D
    operands: a [M][K/2] (E2M1 pairs) or [M][K] (E4M3) bytes, row-major; b
    [N][K/2] / [N][K] bytes, or its column-major [K/2][N] / [K][N] view; the
    scales [M][K/32] and [N][K/32] (or that one's transpose view).  fmt
    'fp4' / 'fp8', or None to take it from a's dtype."""
    if fmt is None:
        fmt = _FMT_OF_DTYPE.get(a.dtype)
        if fmt is None:
            raise ValueError("fmt is required unless a is float4_e2m1fn_x2 or float8_e4m3fn")
    if fmt not in ("fp4", "fp8"):
        raise ValueError("fmt must be 'fp4' or 'fp8'")
    a, b = _nk_storage(a), _nk_storage(b)
    a_scale, b_scale = _nk_storage(a_scale), _nk_storage(b_scale)
    M, kb = a.shape
    N = b.shape[0]
    K = kb * 2 if fmt == "fp4" else kb
    if b.shape[1] != kb:
        raise ValueError("a and b disagree on K")
    if tuple(a_scale.shape) != (M, K // 32) or tuple(b_scale.shape) != (N, K // 32):
        raise ValueError("scales must be [M][K/32] and [N][K/32]")
    return fmt, int(M), int(N), int(K), a, b, a_scale, b_scale


def scaled_mm(a, b, a_scale, b_scale, fmt=None, M=None, N=None, K=None,
              out_dtype=torch.bfloat16, workspace="auto", stream=None) -> torch.Tensor:
    """C = MX scaled GEMM of packed operands; returns a new [M, N] tensor.

    With M, N and K given, the operands are any 1-byte CUDA tensors (or raw
    pointers) laid out as mx_scaled_mm_fp4 / mx_scaled_mm_fp8 take them and
    fmt ('fp4' or 'fp8') is required.  Without them, the operands are 2-D
    tensors whose shapes give the sizes (scaled_mm_shapes): torch's
    float4_e2m1fn_x2 / float8_e4m3fn codes and float8_e8m0fnu scales, or
    uint8 with fmt, B either stored [N][K] or as F.scaled_mm's column-major
    [K][N] view of that storage."""
    if M is None or N is None or K is None:
        fmt, M, N, K, a, b, a_scale, b_scale = scaled_mm_shapes(a, b, a_scale, b_scale, fmt)
    elif fmt not in ("fp4", "fp8"):
        raise ValueError("fmt must be 'fp4' or 'fp8'")
    dev = a.device if isinstance(a, torch.Tensor) else torch.device("cuda")
    with _made_on(stream):
        c = torch.empty((M, N), dtype=out_dtype, device=dev)
    fn = mx_scaled_mm_fp4 if fmt == "fp4" else mx_scaled_mm_fp8
    fn(a, b, a_scale, b_scale, c, M, N, K, workspace=workspace, stream=stream)
    return c


def mx_empty_like(is_fp4, M, N, K, stream=None) -> None:
    """Enqueue an empty kernel on the grid the default product would use for
    this shape (C ABI mx_empty_like; measurement of the launch cost)."""
    st = _lib.mx_empty_like(int(bool(is_fp4)), M, N, K, _stream(stream))
    if st:
        raise MxGemmError(st, "mx_empty_like")


def mx_scaled_mm_noalloc(is_fp4, a, b, a_scale, b_scale, c, M, N, K, out_dtype=None, stream=None) -> None:
    """The default product with the library's built-in split-K scratch
    (C ABI mx_scaled_mm_noalloc): no workspace argument and no allocation.
    Calls that may overlap on one GPU race on that scratch."""
    _check_tensors(bool(is_fp4), a, b, a_scale, b_scale, c, M, N, K)
    st = _lib.mx_scaled_mm_noalloc(int(bool(is_fp4)), _ptr(a), _ptr(b), _ptr(a_scale), _ptr(b_scale),
                                   _ptr(c), M, N, K, _out_code(c, out_dtype), _stream(stream))
    if st:
        raise MxGemmError(st, "mx_scaled_mm_noalloc")


def mx_noalloc_scratch_bytes() -> int:
    return int(_lib.mx_noalloc_scratch_bytes())


# ------------------------------------------------- around the products
_BF16 = torch.bfloat16


def _bf16_ptr(name, t, n, dev):
    """Address of a contiguous bfloat16 CUDA tensor of n elements, a raw pointer itself, 0 for None."""
    if t is None:
        return 0
    if t.__class__ is int:
        return t
    if t.dtype is not _BF16 or t.get_device() != dev or not t.is_contiguous() or t.numel() != n:
        raise ValueError("%s must be a contiguous bfloat16 CUDA tensor of %d elements on the current device" % (name, n))
    return t.data_ptr()


def mx_rmsnorm(x, residual, weight, h, y, y_scale, rows, K, eps, out_kind=None, stream=None) -> None:
    """RMSNorm with the residual's addition (C ABI mx_rmsnorm): x, residual
    (or None) and h (or None) bfloat16 [rows][K], weight bfloat16 [K] or None.
    y: the output in its own dtype (BF16 / FP16 / FP32), or 1-byte E4M3 codes
    [rows][K] or E2M1 pairs [rows][K/2] with y_scale uint8 [rows][K/32]; a
    1-byte y takes its format from its size unless out_kind is given."""
    n, dev = rows * K, _here()
    px, pr, ph = _bf16_ptr("x", x, n, dev), _bf16_ptr("residual", residual, n, dev), _bf16_ptr("h", h, n, dev)
    pw = _bf16_ptr("weight", weight, K, dev)
    if y.__class__ is int:
        if out_kind is None:
            raise ValueError("out_kind is required when y is a raw pointer")
        py = y
    else:
        size = y.element_size()
        if out_kind is None:
            out_kind = _OUT_OF_DTYPE.get(y.dtype)
            if out_kind is None:
                out_kind = OUT_MXFP8 if y.numel() == n else OUT_MXFP4
        if y.get_device() != dev or not y.is_contiguous() or size != _SIZE_OF_OUT.get(out_kind, size) or \
                y.numel() != (n // 2 if out_kind == OUT_MXFP4 else n):
            raise ValueError("y must be a contiguous CUDA tensor of rows*K values of its output kind on the current device")
        py = y.data_ptr()
    if y_scale is None or y_scale.__class__ is int:
        ps = y_scale or 0
    else:
        if y_scale.get_device() != dev or not y_scale.is_contiguous() or y_scale.element_size() != 1 or \
                y_scale.numel() != rows * (K // 32):
            raise ValueError("y_scale must be a contiguous 1-byte CUDA tensor of rows*K/32 elements on the current device")
        ps = y_scale.data_ptr()
    st = _lib.mx_rmsnorm(px, pr, pw, ph, py, ps, rows, K, eps, out_kind, _stream(stream, dev))
    if st:
        raise MxGemmError(st, "mx_rmsnorm")


def rmsnorm(x, weight, residual=None, eps=1e-6, out="fp8", stream=None):
    """(y, y_scale, h) of mx_rmsnorm on bfloat16 [..., K] tensors: out 'fp8'
    or 'fp4' (codes and E8M0 scales, uint8) or a torch dtype (y_scale None);
    h the sum with the residual (x itself without one)."""
    K = x.shape[-1]
    rows = x.numel() // K if K else 0
    lead = x.shape[:-1]
    ys = None
    with _made_on(stream):
        h = torch.empty_like(x) if residual is not None else None
        if out in ("fp8", "fp4"):
            y = torch.empty(lead + (K if out == "fp8" else K // 2,), dtype=torch.uint8, device=x.device)
            ys = torch.empty(lead + (K // 32,), dtype=torch.uint8, device=x.device)
            kind = OUT_MXFP8 if out == "fp8" else OUT_MXFP4
        else:
            y = torch.empty(x.shape, dtype=out, device=x.device)
            kind = _OUT_OF_DTYPE[out]
    mx_rmsnorm(x, residual, weight, h, y, ys, rows, K, eps, out_kind=kind, stream=stream)
    return y, ys, x if residual is None else h


class _KVCacheStruct(ctypes.Structure):
    _fields_ = [("k_codes", _P), ("k_scales", _P), ("v_codes", _P), ("v_scales", _P), ("pages", _I64),
                ("page_size", _I64), ("kv_heads", _I64), ("head_dim", _I64), ("is_fp4", _INT)]


class KVCache:
    """A paged key/value cache in MX formats (C ABI mxg_kv_cache_t): codes
    [pages][kv_heads][page_size][head_dim] E4M3 bytes (fmt 'fp8') or
    [..][head_dim/2] E2M1 pairs ('fp4'), scales [..][head_dim/32] E8M0 bytes."""

    __slots__ = ("k_codes", "k_scales", "v_codes", "v_scales", "fmt", "pages", "page_size", "kv_heads", "head_dim",
                 "device", "_struct", "_ref")

    def __init__(self, k_codes, k_scales, v_codes, v_scales, fmt="fp8"):
        if fmt not in ("fp4", "fp8"):
            raise ValueError("fmt must be 'fp4' or 'fp8'")
        if k_codes.dim() != 4:
            raise ValueError("codes must be [pages][kv_heads][page_size][bytes of a row]")
        pages, heads, size, row = (int(n) for n in k_codes.shape)
        dim, dev = row * 2 if fmt == "fp4" else row, k_codes.get_device()
        for name, t, last in (("k_codes", k_codes, row), ("k_scales", k_scales, dim // 32),
                              ("v_codes", v_codes, row), ("v_scales", v_scales, dim // 32)):
            if dev < 0 or t.get_device() != dev or not t.is_contiguous() or t.element_size() != 1 or \
                    tuple(t.shape) != (pages, heads, size, last):
                raise ValueError("%s must be a contiguous 1-byte CUDA tensor [%d][%d][%d][%d], all on one device"
                                 % (name, pages, heads, size, last))
        self.k_codes, self.k_scales, self.v_codes, self.v_scales, self.fmt = k_codes, k_scales, v_codes, v_scales, fmt
        self.pages, self.kv_heads, self.page_size, self.head_dim, self.device = pages, heads, size, dim, dev
        self._struct = _KVCacheStruct(k_codes.data_ptr(), k_scales.data_ptr(), v_codes.data_ptr(),
                                      v_scales.data_ptr(), pages, size, heads, dim, int(fmt == "fp4"))
        self._ref = ctypes.addressof(self._struct)

    @classmethod
    def empty(cls, pages, page_size, kv_heads, head_dim, fmt="fp8", device="cuda"):
        """A cache whose slots hold zeros."""
        row = head_dim // 2 if fmt == "fp4" else head_dim
        shape = (pages, kv_heads, page_size)
        t = [torch.zeros(shape + (n,), dtype=torch.uint8, device=device) for n in (row, head_dim // 32) * 2]
        return cls(*t, fmt=fmt)


def _cache_device(cache) -> int:
    """The current device, which has to be the cache's."""
    dev = _here()
    if cache.device != dev:
        raise ValueError("the cache lies on cuda:%d and not on the current device" % cache.device)
    return dev


def _token_rows(name, t, tokens, heads, dim, dev):
    """Stride between the tokens of a bfloat16 [tokens][heads][dim] tensor
    whose tokens may be apart (a part of the rows of a joint product)."""
    if t.dtype is not _BF16 or t.get_device() != dev or t.shape != (tokens, heads, dim):
        raise ValueError("%s must be a bfloat16 CUDA tensor [%d][%d][%d] on the current device" % (name, tokens, heads, dim))
    if tokens == 0:
        return heads * dim
    s0, s1, s2 = t.stride()
    if (s2 != 1 and dim > 1) or (s1 != dim and heads > 1):
        raise ValueError("%s must hold each token's values contiguously" % name)
    return s0 if tokens > 1 else heads * dim


def _cache_call(fn, name, cache, k, v, slots, stream):
    dev = _cache_device(cache)
    if slots.dtype is not torch.int64 or slots.get_device() != dev or slots.dim() != 1 or not slots.is_contiguous():
        raise ValueError("slots must be a contiguous one-dimensional int64 CUDA tensor on the current device")
    n = slots.shape[0]
    ks = _token_rows("k", k, n, cache.kv_heads, cache.head_dim, dev)
    vs = _token_rows("v", v, n, cache.kv_heads, cache.head_dim, dev)
    st = fn(cache._ref, k.data_ptr(), v.data_ptr(), ks, vs, slots.data_ptr(), n, _stream(stream, dev))
    if st:
        raise MxGemmError(st, name)


def mx_kv_cache_write(cache, k, v, slots, stream=None) -> None:
    """Quantize tokens into cache slots (C ABI mx_kv_cache_write): k and v
    bfloat16 [tokens][kv_heads][head_dim], tokens may be apart; slots int64
    [tokens], -1 to skip one, the others distinct."""
    _cache_call(_lib.mx_kv_cache_write, "mx_kv_cache_write", cache, k, v, slots, stream)


def mx_kv_cache_read(cache, k, v, slots, stream=None) -> None:
    """Read cache slots back (C ABI mx_kv_cache_read) into k and v, laid out
    as for mx_kv_cache_write; a slot outside the cache reads zeros."""
    _cache_call(_lib.mx_kv_cache_read, "mx_kv_cache_read", cache, k, v, slots, stream)


def mx_paged_attention_workspace_bytes(cache, seqs, tokens, q_heads, max_new) -> int:
    return int(_lib.mx_paged_attention_workspace_bytes(cache._ref, seqs, tokens, q_heads, max_new))


def _int32(name, t, shape, dev):
    if t.dtype is not torch.int32 or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        raise ValueError("%s must be a contiguous int32 CUDA tensor of shape %s on the current device" % (name, tuple(shape)))


_F32, _I32, _I64T = torch.float32, torch.int32, torch.int64


def _attention_args(cache, q, ends, lens, table, out, lse):
    """The checks of an attention call's tensors: device, sequences, q's shape and stride between tokens, out's kind."""
    tokens, heads, dim = q.shape
    if dim != cache.head_dim:
        raise ValueError("q has head_dim %d, the cache %d" % (dim, cache.head_dim))
    dev = _cache_device(cache)
    qs = _token_rows("q", q, tokens, heads, dim, dev)
    seqs = ends.shape[0]
    _int32("ends", ends, (seqs,), dev)
    _int32("lens", lens, (seqs,), dev)
    if table.dim() != 2:
        raise ValueError("table must be [seqs][pages of a sequence]")
    _int32("table", table, (seqs, table.shape[1]), dev)
    kind = _OUT_OF_DTYPE.get(out.dtype)
    if kind is None or out.get_device() != dev or out.shape != q.shape or not out.is_contiguous():
        raise ValueError("out must be a contiguous CUDA tensor of q's shape in BF16, FP16 or FP32 on the current device")
    if lse is not None and (lse.dtype is not _F32 or lse.get_device() != dev or lse.shape != (tokens, heads) or
                            not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous float32 CUDA tensor [tokens][q_heads] on the current device")
    return dev, seqs, tokens, heads, dim, qs, kind


def mx_paged_attention(cache, q, ends, lens, table, out, lse=None, scale=None, causal=True, window=0,
                       max_new=None, workspace="auto", stream=None) -> None:
    """Attention of new tokens over the paged cache (C ABI
    mx_paged_attention): q bfloat16 [tokens][q_heads][head_dim], tokens may be
    apart; ends and lens int32 [seqs]; table int32 [seqs][pages of a
    sequence]; out contiguous [tokens][q_heads][head_dim] in BF16 / FP16 /
    FP32; lse float32 [tokens][q_heads] or None.  scale: 1/sqrt(head_dim) if
    None; max_new: the most new tokens of a sequence, if known (for speed)."""
    dev, seqs, tokens, heads, dim, qs, kind = _attention_args(cache, q, ends, lens, table, out, lse)
    if max_new is None:
        max_new = tokens
    need = _lib.mx_paged_attention_workspace_bytes(cache._ref, seqs, tokens, heads, max_new) if workspace is not None else 0
    _call("mx_paged_attention", _lib.mx_paged_attention,
          (cache._ref, q.data_ptr(), qs, ends.data_ptr(), lens.data_ptr(), table.data_ptr(), table.shape[1], seqs,
           tokens, heads, max_new, dim ** -0.5 if scale is None else scale, int(causal), window, out.data_ptr(),
           kind, 0 if lse is None else lse.data_ptr()), workspace, need, dev, _stream(stream, dev))


def paged_attention(cache, q, ends, lens, table, out_dtype=torch.bfloat16, stream=None, **kw) -> torch.Tensor:
    """mx_paged_attention into a new tensor, which it returns.  Rows of q past
    the last end are not written."""
    with _made_on(stream):
        out = torch.empty(q.shape, dtype=out_dtype, device=q.device)
    mx_paged_attention(cache, q, ends, lens, table, out, stream=stream, **kw)
    return out


def mx_tree_attention_workspace_bytes(cache, seqs, tokens, q_heads, max_new) -> int:
    return int(_lib.mx_tree_attention_workspace_bytes(cache._ref, seqs, tokens, q_heads, max_new))


def mx_tree_attention(cache, q, ends, lens, table, mask, out, lse=None, scale=None, window=0, max_new=None,
                      workspace="auto", stream=None) -> None:
    """Attention of trees of drafted tokens over the paged cache (C ABI
    mx_tree_attention): mask int64 [tokens][words], bit j % 64 of word j / 64
    of a token's row set where it sees the j-th new token of its sequence,
    itself included (tree_mask makes it from parents); all else as for
    mx_paged_attention, but that FP16 and FP32 outputs take the weights in two
    BF16 parts."""
    dev, seqs, tokens, heads, dim, qs, kind = _attention_args(cache, q, ends, lens, table, out, lse)
    if mask is None or mask.dtype is not _I64T or mask.get_device() != dev or mask.dim() != 2 or mask.shape[0] != tokens or \
            not mask.is_contiguous():
        raise ValueError("mask must be a contiguous int64 CUDA tensor [tokens][words] on the current device")
    if max_new is None:
        max_new = tokens
    need = _lib.mx_tree_attention_workspace_bytes(cache._ref, seqs, tokens, heads, max_new) if workspace is not None else 0
    _call("mx_tree_attention", _lib.mx_tree_attention,
          (cache._ref, q.data_ptr(), qs, ends.data_ptr(), lens.data_ptr(), table.data_ptr(), table.shape[1], mask.data_ptr(),
           mask.shape[1], seqs, tokens, heads, max_new, dim ** -0.5 if scale is None else scale, window, out.data_ptr(),
           kind, 0 if lse is None else lse.data_ptr()), workspace, need, dev, _stream(stream, dev))


def tree_attention(cache, q, ends, lens, table, mask, out_dtype=torch.bfloat16, stream=None, **kw) -> torch.Tensor:
    """mx_tree_attention into a new tensor, which it returns.  Rows of q past
    the last end are not written."""
    with _made_on(stream):
        out = torch.empty(q.shape, dtype=out_dtype, device=q.device)
    mx_tree_attention(cache, q, ends, lens, table, mask, out, stream=stream, **kw)
    return out


def tree_mask(parents, words=None) -> torch.Tensor:
    """The mask rows of one sequence's tree: parents a list, for each node the
    earlier node that it continues, or -1 for one that continues the context.
    int64 [nodes][words] on the CPU.  All ancestors are in it: a window hides
    none of them by itself."""
    rows = []
    for i, parent in enumerate(parents):
        if not -1 <= parent < i:
            raise ValueError("node %d: its parent %d is not an earlier node or -1" % (i, parent))
        rows.append((rows[parent] if parent >= 0 else 0) | 1 << i)
    need = max(1, -(-len(rows) // 64))
    words = need if words is None else words
    if words < need:
        raise ValueError("%d nodes need %d words" % (len(rows), need))
    signed = lambda w: w - (1 << 64) if w >> 63 else w  # noqa: E731
    return torch.tensor([[signed(r >> 64 * w & (1 << 64) - 1) for w in range(words)] for r in rows],
                        dtype=torch.int64).view(len(rows), words)


def rope_table(positions, rot, base=10000.0, device="cuda") -> torch.Tensor:
    """float32 [positions][rot / 2][2]: cosine and sine of p * base^(-2 i / rot)
    for mx_rope_cache_write, from angles in 64 bits."""
    p = torch.arange(positions, dtype=torch.float64, device=device)
    angle = p[:, None] * float(base) ** (torch.arange(0, rot, 2, dtype=torch.float64, device=device) / -rot)
    return torch.stack((angle.cos(), angle.sin()), -1).float()


def _int64(name, t, shape, dev):
    if t.dtype is not torch.int64 or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        raise ValueError("%s must be a contiguous int64 CUDA tensor of shape %s on the current device" % (name, tuple(shape)))


def mx_rope_cache_write(cache, q, k, v, positions, slots, rope, q_out=None, interleaved=False, stream=None) -> None:
    """Rotate queries and keys by their positions and quantize keys and values
    into cache slots (C ABI mx_rope_cache_write): q bfloat16
    [tokens][q_heads][head_dim] (or None: keys and values only) into q_out, q
    itself if None; k and v [tokens][kv_heads][head_dim]; the tokens of each may
    be apart; positions and slots int64 [tokens]; rope float32
    [positions][rot / 2][2] (rope_table)."""
    dev = _cache_device(cache)
    if slots.dim() != 1:
        raise ValueError("slots must be a contiguous one-dimensional int64 CUDA tensor on the current device")
    n, dim = slots.shape[0], cache.head_dim
    _int64("slots", slots, (n,), dev)
    _int64("positions", positions, (n,), dev)
    ks = _token_rows("k", k, n, cache.kv_heads, dim, dev)
    vs = _token_rows("v", v, n, cache.kv_heads, dim, dev)
    if rope.dtype is not torch.float32 or rope.get_device() != dev or rope.dim() != 3 or rope.shape[2] != 2 or \
            not rope.is_contiguous():
        raise ValueError("rope must be a contiguous float32 CUDA tensor [positions][rot / 2][2] on the current device")
    heads = qs = os_ = pq = po = 0
    if q is not None:
        if q_out is None:
            q_out = q
        heads = q.shape[1] if q.dim() == 3 else 0
        qs, os_ = _token_rows("q", q, n, heads, dim, dev), _token_rows("q_out", q_out, n, heads, dim, dev)
        pq, po = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    st = _lib.mx_rope_cache_write(cache._ref, pq, po, k.data_ptr(), v.data_ptr(), heads, qs, os_, ks, vs,
                                  positions.data_ptr(), slots.data_ptr(), rope.data_ptr(), rope.shape[0], 2 * rope.shape[1],
                                  int(interleaved), n, _stream(stream, dev))
    if st:
        raise MxGemmError(st, "mx_rope_cache_write")


def mx_moe_dispatch_workspace_bytes(tokens, top_k, groups) -> int:
    return int(_lib.mx_moe_dispatch_workspace_bytes(tokens, top_k, groups))


def _rows(name, t, rows, width, dev):
    """A contiguous [rows][width] CUDA tensor."""
    if t.shape != (rows, width) or t.get_device() != dev or not t.is_contiguous():
        raise ValueError("%s must be a contiguous CUDA tensor [%d][%d] on the current device" % (name, rows, width))


def _of_type(name, t, dtype):
    if t.dtype is not dtype:
        raise ValueError("%s must be %s" % (name, str(dtype).replace("torch.", "")))


def _mx_kind(name, y, y_scale, rows, width, dev):
    """Output kind of y [rows][..] by its type and size: BF16 (y_scale ignored), or MX codes with y_scale."""
    if y.dtype is _BF16:
        _rows(name, y, rows, width, dev)
        return OUT_BF16
    if y.element_size() != 1 or y.dim() != 2:
        raise ValueError("%s must be bfloat16, or 1-byte codes with scales" % name)
    kind = OUT_MXFP8 if y.shape[1] == width else OUT_MXFP4
    _rows(name, y, rows, width if kind == OUT_MXFP8 else width // 2, dev)
    if y_scale is None or y_scale.element_size() != 1:
        raise ValueError("%s_scale must be a contiguous 1-byte CUDA tensor [rows][%d] on the current device" % (name, width // 32))
    _rows(name + "_scale", y_scale, rows, width // 32, dev)
    return kind


def mx_moe_dispatch(x, experts, y, y_scale, offs, pos, workspace="auto", stream=None) -> None:
    """Tokens sorted by expert into the grouped product's A operand (C ABI
    mx_moe_dispatch): x bfloat16 [tokens][K]; experts int64 [tokens][top_k],
    ids outside [0, groups) without a row; y [tokens * top_k][..] bfloat16, or
    1-byte E4M3 codes or E2M1 pairs with y_scale [tokens * top_k][K / 32];
    offs int32 [groups] and pos int32 [tokens][top_k] are written."""
    dev = _here()
    tokens, K = x.shape
    _rows("x", x, tokens, K, dev)
    _of_type("x", x, _BF16)
    if experts.dim() != 2 or offs.dim() != 1:
        raise ValueError("experts must be [tokens][top_k] and offs [groups]")
    top_k, groups = experts.shape[1], offs.shape[0]
    _int64("experts", experts, (tokens, top_k), dev)
    kind = _mx_kind("y", y, y_scale, tokens * top_k, K, dev)
    _int32("offs", offs, (groups,), dev)
    _int32("pos", pos, (tokens, top_k), dev)
    need = _lib.mx_moe_dispatch_workspace_bytes(tokens, top_k, groups)
    _call("mx_moe_dispatch", _lib.mx_moe_dispatch,
          (x.data_ptr(), experts.data_ptr(), tokens, top_k, groups, K, y.data_ptr(), 0 if kind == OUT_BF16 else y_scale.data_ptr(),
           kind, offs.data_ptr(), pos.data_ptr()), workspace, need, dev, _stream(stream, dev))


def moe_dispatch(x, experts, groups, out="fp8", workspace="auto", stream=None):
    """(y, y_scale, offs, pos) of mx_moe_dispatch in new tensors: out 'fp8',
    'fp4' (codes and E8M0 scales, uint8) or torch.bfloat16 (y_scale None)."""
    tokens, K = x.shape
    rows = tokens * experts.shape[1]
    ys = None
    with _made_on(stream):
        if out in ("fp8", "fp4"):
            y = torch.empty((rows, K if out == "fp8" else K // 2), dtype=torch.uint8, device=x.device)
            ys = torch.empty((rows, K // 32), dtype=torch.uint8, device=x.device)
        elif out is _BF16:
            y = torch.empty((rows, K), dtype=out, device=x.device)
        else:
            raise ValueError("out must be 'fp8', 'fp4' or torch.bfloat16")
        offs = torch.empty((groups,), dtype=torch.int32, device=x.device)
        pos = torch.empty((tokens, experts.shape[1]), dtype=torch.int32, device=x.device)
    mx_moe_dispatch(x, experts, y, ys, offs, pos, workspace=workspace, stream=stream)
    return y, ys, offs, pos


def _combine_args(pos, weights, dev):
    if pos.dim() != 2:
        raise ValueError("pos must be [tokens][top_k]")
    tokens, top_k = pos.shape
    _int32("pos", pos, (tokens, top_k), dev)
    if weights is not None:
        _rows("weights", weights, tokens, top_k, dev)
        _of_type("weights", weights, _F32)
    return tokens, top_k, 0 if weights is None else weights.data_ptr()


def _float_kind(name, t):
    kind = _OUT_OF_DTYPE.get(t.dtype)
    if kind is None or t.dim() != 2:
        raise ValueError("%s must be a two-dimensional tensor in BF16, FP16 or FP32" % name)
    return kind


def mx_moe_combine(y, pos, weights, out, stream=None) -> None:
    """The experts' rows back to their tokens (C ABI mx_moe_combine): y
    [rows][N], pos int32 [tokens][top_k], weights float32 [tokens][top_k] or
    None for ones, out [tokens][N]; y and out each BF16, FP16 or FP32.  Without
    weights it is the gradient of mx_moe_dispatch."""
    dev = _here()
    tokens, top_k, pw = _combine_args(pos, weights, dev)
    ky, ko = _float_kind("y", y), _float_kind("out", out)
    rows, N = y.shape
    _rows("y", y, rows, N, dev)
    _rows("out", out, tokens, N, dev)
    st = _lib.mx_moe_combine(y.data_ptr(), ky, pos.data_ptr(), pw, tokens, top_k, rows, N, out.data_ptr(), ko,
                             _stream(stream, dev))
    if st:
        raise MxGemmError(st, "mx_moe_combine")


def moe_combine(y, pos, weights=None, out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """mx_moe_combine into a new tensor, which it returns."""
    with _made_on(stream):
        out = torch.empty((pos.shape[0], y.shape[1]), dtype=out_dtype, device=y.device)
    mx_moe_combine(y, pos, weights, out, stream=stream)
    return out


def mx_moe_combine_grad(d_out, y, pos, weights, d_y, d_y_scale=None, d_weights=None, stream=None) -> None:
    """The gradients of mx_moe_combine (C ABI mx_moe_combine_grad): d_out
    [tokens][N] and y [rows][N] of one type; d_y [rows][N] of that type, or
    1-byte E4M3 codes or E2M1 pairs with d_y_scale [rows][N / 32]; d_weights
    float32 [tokens][top_k] or None (then y may be None).  The rows that pos
    names are distinct."""
    dev = _here()
    tokens, top_k, pw = _combine_args(pos, weights, dev)
    dtype = _float_kind("d_out", d_out)
    N, rows = d_out.shape[1], d_y.shape[0]
    _rows("d_out", d_out, tokens, N, dev)
    if d_y.dtype is d_out.dtype:
        _rows("d_y", d_y, rows, N, dev)
        kind = dtype
    elif d_y.element_size() == 1:
        kind = _mx_kind("d_y", d_y, d_y_scale, rows, N, dev)
    else:
        raise ValueError("d_y must be of d_out's type, or 1-byte codes with scales")
    if d_weights is not None:
        _rows("d_weights", d_weights, tokens, top_k, dev)
        _of_type("d_weights", d_weights, _F32)
        if y is None:
            raise ValueError("y is needed for d_weights")
    if y is not None:
        _rows("y", y, rows, N, dev)
        _of_type("y", y, d_out.dtype)
    st = _lib.mx_moe_combine_grad(d_out.data_ptr(), 0 if y is None else y.data_ptr(), dtype, pos.data_ptr(), pw, tokens, top_k,
                                  rows, N, d_y.data_ptr(), 0 if kind == dtype else d_y_scale.data_ptr(), kind,
                                  0 if d_weights is None else d_weights.data_ptr(), _stream(stream, dev))
    if st:
        raise MxGemmError(st, "mx_moe_combine_grad")


def moe_combine_grad(d_out, y, pos, weights=None, stream=None):
    """(d_y, d_weights) of mx_moe_combine_grad in new tensors; rows of d_y that
    no token has are zeros."""
    with _made_on(stream):
        d_y = torch.zeros(y.shape, dtype=y.dtype, device=y.device)
        d_w = torch.empty(pos.shape, dtype=torch.float32, device=y.device)
    mx_moe_combine_grad(d_out, y, pos, weights, d_y, None, d_w, stream=stream)
    return d_y, d_w
