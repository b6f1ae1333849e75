// mxserve.hip -- host side of the operators around the products: RMSNorm into
// the next product's A operand, the paged key/value cache in MX formats and
// the attention over it.  Argument validation, configuration choice and
// launches behind the C ABI declared in include/mxgemm.h.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/mxgemm.h"
#include "mx_attn.hpp"
#include "mx_host.hpp"
#include "mx_norm.hpp"

using namespace mxg;

namespace {

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

FastDiv fast_div(unsigned d)
{
    FastDiv f = {d, 0, 0};
    if (d > 1) {
        while ((2ull << f.s) < d)
            ++f.s;
        f.m = (unsigned)(((1ull << (32 + f.s)) + d - 1) / d);
    }
    return f;
}

// ------------------------------------------------------------------- RMSNorm
// Longest row: 1024 threads hold 64 values each.
constexpr int64_t kMaxNormK = 65536;

// A launch has fewer than 2^32 threads.
constexpr int64_t kMaxThreads = UINT32_MAX;

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
int log2_of(int64_t v)
{
    int s = 0;
    while (((int64_t)1 << s) < v)
        ++s;
    return s;
}

constexpr int64_t kMaxPage = 65536, kMaxHeads = 4096, kMaxHeadDim = 1024;

int validate_cache(const mxg_kv_cache_t *c)
{
    if (!c || !c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales)
        return MXG_ERR_NULL;
    if (c->pages < 1 || c->pages > INT32_MAX || c->page_size < 1 || c->page_size > kMaxPage ||
        (c->page_size & (c->page_size - 1)) || c->kv_heads < 1 || c->kv_heads > kMaxHeads ||
        c->head_dim < 1 || c->head_dim > kMaxHeadDim)
        return MXG_ERR_SHAPE;
    if (c->head_dim % 32)
        return MXG_ERR_K_ALIGN;
    // (codes and element offsets within 2^62: far past any memory)
    if (c->pages * c->page_size > ((int64_t)1 << 40))
        return MXG_ERR_SHAPE;
    if (((uintptr_t)c->k_codes | (uintptr_t)c->v_codes) & 15)
        return MXG_ERR_PTR_ALIGN;
    if (((uintptr_t)c->k_scales | (uintptr_t)c->v_scales) & 3)
        return MXG_ERR_PTR_ALIGN;
    return MXG_OK;
}

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

// ----------------------------------------------------------------- attention
typedef void (*AttnFn)(AttnArgs);

// Row tiles of 16 or 32 rows in mx_attn_rows, of 128 or 256 in mx_attn_tile.
enum { ROWS_16 = 0, ROWS_32 = 1, ROWS_128 = 2, ROWS_256 = 3 };
constexpr int kAttnBM[4] = {16, 32, 128, 256};
constexpr int kAttnThreads[4] = {256, 256, 256, 512};
// Parts that the key tiles are cut into: about as many as run at once on 256
// CUs.  (mx_attn_rows: with few row tiles each has many parts, whose join
// costs: one sequence of 100000 keys 47 us cut into 512 parts, 54 into 1024;
// 32 sequences of 16 rows over 4096 keys 50 and 57.  With 512 row tiles they
// balance ragged lengths: 64 sequences of 100 to 16000 keys 100 and 95 us.
// Nothing between 256 and 512 row tiles was measured: the step may lie lower.)
int attn_target(int which, int64_t pairs)      // (sequence, head) pairs
{
    switch (which) {
    case ROWS_16: return pairs < 512 ? 512 : 1024;
    case ROWS_128: return 384;
    case ROWS_256: return 256;
    default: return 512;
    }
}

// The kernel that joins the parts of row tiles of many rows.
AttnFn attn_join_fn(int which, int64_t dim)
{
    if (which == ROWS_128)
        return dim == 64 ? &mx_attn_join<64, 128> : &mx_attn_join<128, 128>;
    return dim == 64 ? &mx_attn_join<64, 256> : &mx_attn_join<128, 256>;
}

template <int F, int D, int PAGED>
AttnFn attn_fn(int which)
{
    switch (which) {
    case ROWS_16: return &mx_attn_rows<F, D, 1, PAGED>;
    case ROWS_32: return &mx_attn_rows<F, D, 2, PAGED>;
    case ROWS_128: return &mx_attn_tile<F, D, 4, PAGED>;
    default: return &mx_attn_tile<F, D, 8, PAGED>;
    }
}

template <int F, int D>
AttnFn attn_fn(int which, int64_t page_size)
{
    // mx_attn_rows takes tiles of two pages, mx_attn_tile loads of one wave
    // (64 chunks of 16 bytes)
    const bool paged = page_size >= (which <= ROWS_32 ? 16 : 64 / AttnGeom<F, D>::CH);
    return paged ? attn_fn<F, D, 1>(which) : attn_fn<F, D, 0>(which);
}

AttnFn attn_fn(int which, bool fp4, int64_t dim, int64_t page_size)
{
    if (dim == 64)
        return fp4 ? attn_fn<FMT_FP4, 64>(which, page_size) : attn_fn<FMT_FP8, 64>(which, page_size);
    return fp4 ? attn_fn<FMT_FP4, 128>(which, page_size) : attn_fn<FMT_FP8, 128>(which, page_size);
}

// Most rows (new tokens x heads of a group) of a sequence for mx_attn_rows,
// which takes 32 at a time and so reads and expands a key once for each 32,
// but cuts its keys finer and joins the parts itself, without a second
// kernel.  By the number of row tiles it gains more than it loses (8 KV heads
// of 128, E4M3):
//     row tiles  sequences, rows, keys   us, in tiles of 128
//          32    1 of 128 over 2048       16   27
//         128    1 of 512 over 2048       22   33  (over 32768 keys 110 and 92)
//         200    2 of 400 over 4096       46   41
//         256    4 of 256 over 4096       40   43
//         512    32 of 64 over 4096       66   94  (E2M1 54 and 86)
//        1024    32 of 128 over 4096     120  112
//        4096    128 of 128 over 1024    165  107
// and for 64 rows with 2048 row tiles 93 and 88.  So the rule gives away 20% for
// 512 rows over 32768 keys and 6% there; the keys' numbers are on the device,
// and only their bound, table_width * page_size, is known here.
int attn_few_rows(int64_t row_tiles)        // of 32 rows, all heads
{
    return row_tiles <= 128 ? 512 : row_tiles <= 256 ? 256 : 64;
}

// What a call launches: one kernel for all sequences, or one for those of
// few rows and one for the others.
struct AttnPlan {
    int n;
    int which[2];
    int above[2], upto[2];
    int64_t base[2];        // most row tiles
    int target[2];          // parts
    size_t bytes[2];        // of the workspace for splitting; 0: none
};

AttnPlan attn_plan(int64_t seqs, int64_t tokens, int64_t heads, int64_t group, int64_t dim, int64_t max_new)
{
    AttnPlan p = {};
    const int64_t most = max_new * group;       // rows of the longest
    // 256 rows where sequences fill several such tiles (4096 tokens of 4 heads
    // a group behind 12204 keys 825 us against 935, 512 tokens 85 against 92),
    // else 128 (24 sequences of 1 to 600 tokens 52 us against 65)
    const int tile = tokens * group >= 512 * seqs ? ROWS_256 : ROWS_128;
    const int few = attn_few_rows(heads * cdiv(tokens * group, 32));
    if (most <= few || tokens == seqs * max_new) {
        p.n = 1;
        p.which[0] = most <= 16 ? ROWS_16 : most <= few ? ROWS_32 : tile;
        p.above[0] = 0;
        p.upto[0] = INT32_MAX;
    } else {
        p.n = 2;
        p.which[0] = tile;
        p.above[0] = few;
        p.upto[0] = INT32_MAX;
        p.which[1] = ROWS_32;
        p.above[1] = 0;
        p.upto[1] = few;
    }
    for (int i = 0; i < p.n; ++i) {
        const int bm = kAttnBM[p.which[i]];
        const int64_t some = std::min(seqs, tokens);        // sequences with a new token
        p.base[i] = heads * std::min(tokens * group / bm + some, cdiv(p.upto[i], bm) * some);
        p.target[i] = attn_target(p.which[i], heads * some);
        // (one sequence with a row tile per part or more is never split)
        const bool whole = seqs == 1 && heads * cdiv(tokens * group, bm) >= p.target[i];
        p.bytes[i] = p.base[i] <= kSplitCounters && !whole ? (size_t)2 * p.target[i] * attn_slot_bytes(bm, (int)dim) : 0;
    }
    return p;
}

bool attn_shape_ok(const mxg_kv_cache_t *c, int64_t seqs, int64_t tokens, int64_t q_heads, int64_t max_new)
{
    return seqs >= 0 && seqs <= 65536 && tokens >= 0 && q_heads >= c->kv_heads && q_heads <= 65536 &&
           q_heads % c->kv_heads == 0 && tokens <= ((int64_t)1 << 30) / q_heads && max_new >= 0 &&
           max_new <= INT32_MAX && (c->head_dim == 64 || c->head_dim == 128);
}

size_t attn_workspace(const AttnPlan &p)
{
    size_t most = 0;
    for (int i = 0; i < p.n; ++i)
        most = std::max(most, p.bytes[i]);
    return most ? most + kSplitCounters * sizeof(unsigned) : 0;
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
    int rc = validate_cache(cache);
    if (rc)
        return rc;
    if (out_dtype < MXG_OUT_BF16 || out_dtype > MXG_OUT_F32)
        return MXG_ERR_DTYPE;
    if (!attn_shape_ok(cache, seqs, tokens, q_heads, max_new) || table_width < 0 ||
        table_width > ((int64_t)1 << 30) / cache->page_size || q_stride < q_heads * cache->head_dim ||
        q_stride > INT32_MAX || window < 0)
        return MXG_ERR_SHAPE;
    if (tokens > 0 && seqs > 0 && (!q || !ends || !lens || !out || (table_width > 0 && !table)))
        return MXG_ERR_NULL;
    if (q_stride % 8)
        return MXG_ERR_K_ALIGN;
    const float c = scale * 1.4426950408889634f;        // exponents of 2
    if (!(scale > 0.0f) || !isfinite(c) || (causal != 0 && causal != 1))
        return MXG_ERR_CONFIG;
    if (((uintptr_t)q | (uintptr_t)out | (uintptr_t)workspace) & 15)
        return MXG_ERR_PTR_ALIGN;
    if (((uintptr_t)ends | (uintptr_t)lens | (uintptr_t)table | (uintptr_t)lse) & 3)
        return MXG_ERR_PTR_ALIGN;
    const int64_t group = q_heads / cache->kv_heads;
    const AttnPlan plan = attn_plan(seqs, tokens, cache->kv_heads, group, cache->head_dim, max_new);
    for (int i = 0; i < plan.n; ++i)        // (split ones are far below)
        if (plan.base[i] > kMaxThreads / kAttnThreads[plan.which[i]])
            return MXG_ERR_SHAPE;
    rc = host_check_device();
    if (rc || tokens == 0 || seqs == 0)
        return rc;
    const bool split = workspace && workspace_bytes >= attn_workspace(plan);
    AttnArgs a;
    a.codes[0] = (const uint8_t *)cache->k_codes;
    a.codes[1] = (const uint8_t *)cache->v_codes;
    a.scales[0] = (const uint8_t *)cache->k_scales;
    a.scales[1] = (const uint8_t *)cache->v_scales;
    a.q = (const uint16_t *)q;
    a.ends = ends;
    a.lens = lens;
    a.table = table;
    a.out = out;
    a.lse = lse;
    a.q_stride = q_stride;
    a.table_stride = table_width;
    a.c = c;
    a.seqs = (int)seqs;
    a.tokens = (int)tokens;
    a.heads = (int)cache->kv_heads;
    a.group = (int)group;
    a.by_heads = fast_div((unsigned)a.heads);
    a.by_group = fast_div((unsigned)a.group);
    a.page_shift = log2_of(cache->page_size);
    a.pages = (int)cache->pages;
    a.table_width = (int)table_width;
    a.causal = causal;
    a.window = (int)std::min<int64_t>(window, 1 << 30);
    a.out_kind = out_dtype;
    for (int i = 0; i < plan.n; ++i) {
        const int which = plan.which[i];
        const bool parts = split && plan.bytes[i] > 0;
        a.counters = parts ? (unsigned *)workspace : nullptr;
        a.parts = parts ? (uint8_t *)workspace + kSplitCounters * sizeof(unsigned) : nullptr;
        a.rows_above = plan.above[i];
        a.rows_upto = plan.upto[i];
        a.per_target = (float)a.heads / (float)plan.target[i];
        const int64_t grid = plan.base[i] + (parts ? plan.target[i] : 0);
        hipLaunchKernelGGL(attn_fn(which, cache->is_fp4 != 0, cache->head_dim, cache->page_size), dim3((unsigned)grid),
                           dim3(kAttnThreads[which]), 0, (hipStream_t)stream, a);
        rc = host_hip_status(hipGetLastError());
        if (rc)
            return rc;
        if (parts && which >= ROWS_128) {
            const int64_t join = std::min<int64_t>(plan.base[i], plan.target[i]) * attn_join_blocks(kAttnBM[which], (int)cache->head_dim);
            hipLaunchKernelGGL(attn_join_fn(which, cache->head_dim), dim3((unsigned)join), dim3(256), 0,
                               (hipStream_t)stream, a);
            rc = host_hip_status(hipGetLastError());
            if (rc)
                return rc;
        }
    }
    return MXG_OK;
}

}  // extern "C"
