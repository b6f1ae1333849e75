// mxserve.hip -- host side of the operators around the products: RMSNorm into
// the next product's A operand, the paged key/value cache in MX formats and
// the attention over it.  Argument validation, configuration choice and
// launches behind the C ABI declared in include/mxgemm.h.
#include <hip/hip_runtime.h>

#include "mx_attn_host.hpp"

using namespace mxg;

namespace {

// ------------------------------------------------------------------- RMSNorm
// Longest row: 1024 threads hold 64 values each.
constexpr int64_t kMaxNormK = 65536;

template <int THR, int NV>
int launch_norm(NormArgs a, int64_t rows, int out_kind, hipStream_t stream)
{
    const bool fp4 = out_kind == MXG_OUT_MXFP4, mx = fp4 || out_kind == MXG_OUT_MXFP8;
    const int64_t y_row = fp4 ? a.K / 2 : mx ? a.K : out_kind == MXG_OUT_F32 ? 4 * (int64_t)a.K : 2 * (int64_t)a.K;

    void (*fn)(NormArgs) = nullptr;
    switch (out_kind) {
    case MXG_OUT_BF16: fn = &mx_rmsnorm_rows<THR, NV, OUT_BF16>; break;
    case MXG_OUT_F16: fn = &mx_rmsnorm_rows<THR, NV, OUT_F16>; break;
    case MXG_OUT_F32: fn = &mx_rmsnorm_rows<THR, NV, OUT_F32>; break;
    case MXG_OUT_MXFP8: fn = &mx_rmsnorm_rows<THR, NV, OUT_MX8>; break;
    default: fn = &mx_rmsnorm_rows<THR, NV, OUT_MX4>; break;
    }
    for (;;) {
        const int64_t n = std::min(rows, kMaxThreads / THR);
        hipLaunchKernelGGL(fn, dim3((unsigned)n), dim3(THR), 0, stream, a);
        const int rc = host_hip_status(hipGetLastError());
        rows -= n;
        if (rc || rows == 0)
            return rc;
        a.x += n * a.K;
        if (a.res)
            a.res += n * a.K;
        if (a.h)
            a.h += n * a.K;
        a.y = (uint8_t *)a.y + n * y_row;
        if (mx)
            a.scales += n * (a.K / 32);
    }
}

int run_norm(const void *x, const void *residual, const void *weight, void *h, void *y, void *y_scale,
             int64_t rows, int64_t K, float eps, int out_kind, hipStream_t stream)
{
    if (rows != 0 && (!x || !y))
        return MXG_ERR_NULL;
    if (out_kind < MXG_OUT_BF16 || out_kind > MXG_OUT_MXFP4)
        return MXG_ERR_DTYPE;
    const bool mx = out_kind == MXG_OUT_MXFP8 || out_kind == MXG_OUT_MXFP4;
    if (rows != 0 && mx && !y_scale)
        return MXG_ERR_NULL;
    if (rows < 0 || rows > INT32_MAX || K < 1 || K > kMaxNormK)
        return MXG_ERR_SHAPE;
    if (K % 32)
        return MXG_ERR_K_ALIGN;
    if (!(eps >= 0.0f) || !isfinite(eps))
        return MXG_ERR_CONFIG;
    if (((uintptr_t)x | (uintptr_t)residual | (uintptr_t)weight | (uintptr_t)h | (uintptr_t)y) & 15)
        return MXG_ERR_PTR_ALIGN;
    int rc = host_check_device();
    if (rc || rows == 0)
        return rc;
    const NormArgs a = {(const uint16_t *)x, (const uint16_t *)residual, (const uint16_t *)weight,
                        (uint16_t *)h, y, (uint8_t *)y_scale, (int)K, eps};
    // One workgroup per row, with up to four 16-byte pieces per thread (eight
    // past 32768 values): a wave up to 512 values (16384 rows of them 14 us,
    // with 256 threads 23), 256 threads up to 6144, 512 up to 16384 and 1024
    // beyond.  Rows with residual and E4M3 output, 256 / 512 / 1024 threads:
    // 8192 of 4096 values 41 / 47 / - us, of 5120 54 / 59 / 74, of 8192
    // 79 / 79 / 98 (but 129 of them 6.0 / 4.9 / 4.9), 4096 of 16384
    // 136 / 78 / 82.
    const int64_t pieces = K / 8;
    if (pieces <= 64)
        return launch_norm<64, 1>(a, rows, out_kind, stream);
    switch (cdiv(pieces, 256)) {
    case 1: return launch_norm<256, 1>(a, rows, out_kind, stream);
    case 2: return launch_norm<256, 2>(a, rows, out_kind, stream);
    case 3: return launch_norm<256, 3>(a, rows, out_kind, stream);
    case 4: return launch_norm<512, 2>(a, rows, out_kind, stream);
    case 5: case 6: return launch_norm<512, 3>(a, rows, out_kind, stream);
    case 7: case 8: return launch_norm<512, 4>(a, rows, out_kind, stream);
    }
    return pieces <= 4096 ? launch_norm<1024, 4>(a, rows, out_kind, stream)
                          : launch_norm<1024, 8>(a, rows, out_kind, stream);
}

// --------------------------------------------------------------------- cache

int run_cache(bool write, const mxg_kv_cache_t *c, const void *k, const void *v, int64_t k_stride,
              int64_t v_stride, const int64_t *slots, int64_t tokens, hipStream_t stream)
{
    int rc = validate_cache(c);
    if (rc)
        return rc;
    if (tokens < 0)
        return MXG_ERR_SHAPE;
    if (tokens > 0 && (!k || !v || !slots))
        return MXG_ERR_NULL;
    const int64_t width = c->kv_heads * c->head_dim;
    if (tokens > ((int64_t)1 << 30) / (width / 8) || k_stride < width || v_stride < width ||
        k_stride > INT32_MAX || v_stride > INT32_MAX)
        return MXG_ERR_SHAPE;
    if ((k_stride | v_stride) % 8)
        return MXG_ERR_K_ALIGN;
    if (((uintptr_t)k | (uintptr_t)v) & 15 || ((uintptr_t)slots & 7))
        return MXG_ERR_PTR_ALIGN;
    rc = host_check_device();
    if (rc || tokens == 0)
        return rc;
    CacheArgs a;
    a.codes[0] = (uint8_t *)c->k_codes;
    a.codes[1] = (uint8_t *)c->v_codes;
    a.scales[0] = (uint8_t *)c->k_scales;
    a.scales[1] = (uint8_t *)c->v_scales;
    a.in[0] = (const uint16_t *)k;
    a.in[1] = (const uint16_t *)v;
    a.out[0] = (uint16_t *)k;
    a.out[1] = (uint16_t *)v;
    a.stride[0] = k_stride;
    a.stride[1] = v_stride;
    a.slots = (const long long *)slots;
    a.nslots = c->pages * c->page_size;
    a.n = (int)(tokens * (width / 8));
    a.heads = (int)c->kv_heads;
    a.dim = (int)c->head_dim;
    a.page_shift = log2_of(c->page_size);
    a.per_token = fast_div((unsigned)(width / 8));
    a.per_head = fast_div((unsigned)(c->head_dim / 8));
    void (*fn)(CacheArgs) = write ? (c->is_fp4 ? &mx_cache_write<FMT_FP4> : &mx_cache_write<FMT_FP8>)
                                  : (c->is_fp4 ? &mx_cache_read<FMT_FP4> : &mx_cache_read<FMT_FP8>);
    hipLaunchKernelGGL(fn, dim3((unsigned)cdiv(a.n, 256 * kCachePieces), 2), dim3(256), 0, stream, a);
    return host_hip_status(hipGetLastError());
}

}  // namespace

extern "C" {

int mx_rmsnorm(const void *x, const void *residual, const void *weight, void *h, void *y, void *y_scale,
               int64_t rows, int64_t K, float eps, int out_kind, mxg_stream_t stream)
{
    return run_norm(x, residual, weight, h, y, y_scale, rows, K, eps, out_kind, (hipStream_t)stream);
}

int mx_kv_cache_write(const mxg_kv_cache_t *cache, const void *k, const void *v, int64_t k_stride,
                      int64_t v_stride, const int64_t *slots, int64_t tokens, mxg_stream_t stream)
{
    return run_cache(true, cache, k, v, k_stride, v_stride, slots, tokens, (hipStream_t)stream);
}

int mx_kv_cache_read(const mxg_kv_cache_t *cache, void *k, void *v, int64_t k_stride, int64_t v_stride,
                     const int64_t *slots, int64_t tokens, mxg_stream_t stream)
{
    return run_cache(false, cache, k, v, k_stride, v_stride, slots, tokens, (hipStream_t)stream);
}

size_t mx_paged_attention_workspace_bytes(const mxg_kv_cache_t *cache, int64_t seqs, int64_t tokens,
                                          int64_t q_heads, int64_t max_new)
{
    if (validate_cache(cache) || !attn_shape_ok(cache, seqs, tokens, q_heads, max_new))
        return 0;
    return attn_workspace(attn_plan(seqs, tokens, cache->kv_heads, q_heads / cache->kv_heads, cache->head_dim, max_new));
}

int mx_paged_attention(const mxg_kv_cache_t *cache, const void *q, int64_t q_stride, const int32_t *ends,
                       const int32_t *lens, const int32_t *table, int64_t table_width, int64_t seqs,
                       int64_t tokens, int64_t q_heads, int64_t max_new, float scale, int causal,
                       int64_t window, void *out, int out_dtype, float *lse, void *workspace,
                       size_t workspace_bytes, mxg_stream_t stream)
{
    return run_attention<0>(cache, q, q_stride, ends, lens, table, table_width, seqs, tokens, q_heads, max_new, scale,
                            causal, nullptr, 1, window, out, out_dtype, lse, workspace, workspace_bytes, stream);
}

}  // extern "C"
