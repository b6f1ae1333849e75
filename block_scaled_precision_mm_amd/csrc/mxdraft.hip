// mxdraft.hip -- host side of the cache's operators with positions and trees:
// the rotation of queries and keys on the way into the paged MX cache, and the
// attention of trees of drafted tokens over it.  Argument validation and
// launches behind the C ABI declared in include/mxgemm.h.
#include <hip/hip_runtime.h>

#include "mx_attn_host.hpp"
#include "mx_rope.hpp"

using namespace mxg;

namespace {

typedef void (*RopeFn)(RopeArgs);

template <int H>
RopeFn rope_fn(bool fp4, bool interleaved)
{
    return fp4 ? (interleaved ? &mx_rope_write<FMT_FP4, 1, H> : &mx_rope_write<FMT_FP4, 0, H>)
               : (interleaved ? &mx_rope_write<FMT_FP8, 1, H> : &mx_rope_write<FMT_FP8, 0, H>);
}

int run_rope(const mxg_kv_cache_t *c, const void *q, void *q_out, const void *k, const void *v, int64_t q_heads,
             int64_t q_stride, int64_t q_out_stride, int64_t k_stride, int64_t v_stride, const int64_t *positions,
             const int64_t *slots, const float *table, int64_t npositions, int64_t rot, int interleaved,
             int64_t tokens, hipStream_t stream)
{
    int rc = validate_cache(c);
    if (rc)
        return rc;
    if (tokens < 0 || q_heads < 0 || q_heads > 65536 || npositions < 1 || npositions > INT32_MAX)
        return MXG_ERR_SHAPE;
    if (tokens > 0 && (!k || !v || !positions || !slots || !table || (q_heads > 0 && (!q || !q_out))))
        return MXG_ERR_NULL;
    const int64_t dim = c->head_dim, width = c->kv_heads * dim, q_width = q_heads * dim;
    if (rot < 16 || rot > dim)
        return MXG_ERR_SHAPE;
    const int64_t most = cdiv(std::max(q_heads, c->kv_heads), kRopeHeads) * kRopeHeads * dim;
    if (tokens > ((int64_t)1 << 30) / (most / 8) || k_stride < width || v_stride < width || k_stride > INT32_MAX ||
        v_stride > INT32_MAX || q_stride < q_width || q_out_stride < q_width || q_stride > INT32_MAX ||
        q_out_stride > INT32_MAX)
        return MXG_ERR_SHAPE;
    if (rot % 16 || (k_stride | v_stride | q_stride | q_out_stride) % 8)
        return MXG_ERR_K_ALIGN;
    if (interleaved != 0 && interleaved != 1)
        return MXG_ERR_CONFIG;
    if (((uintptr_t)q | (uintptr_t)q_out | (uintptr_t)k | (uintptr_t)v | (uintptr_t)table) & 15 ||
        ((uintptr_t)positions | (uintptr_t)slots) & 7)
        return MXG_ERR_PTR_ALIGN;
    // (in place a thread reads what it writes, at the same addresses only)
    if (q_heads > 0 && q == q_out && q_stride != q_out_stride)
        return MXG_ERR_CONFIG;
    rc = host_check_device();
    if (rc || tokens == 0)
        return rc;
    RopeArgs a = {};
    a.kv.codes[0] = (uint8_t *)c->k_codes;
    a.kv.codes[1] = (uint8_t *)c->v_codes;
    a.kv.scales[0] = (uint8_t *)c->k_scales;
    a.kv.scales[1] = (uint8_t *)c->v_scales;
    a.kv.in[0] = (const uint16_t *)k;
    a.kv.in[1] = (const uint16_t *)v;
    a.kv.stride[0] = k_stride;
    a.kv.stride[1] = v_stride;
    a.kv.slots = (const long long *)slots;
    a.kv.nslots = c->pages * c->page_size;
    a.kv.heads = (int)c->kv_heads;
    a.kv.dim = (int)dim;
    a.kv.page_shift = log2_of(c->page_size);
    a.q = (const uint16_t *)q;
    a.q_out = (uint16_t *)q_out;
    a.q_stride = q_stride;
    a.q_out_stride = q_out_stride;
    a.positions = (const long long *)positions;
    a.table = table;
    a.npositions = npositions;
    a.rot = (int)rot;
    a.q_heads = (int)q_heads;
    // (pieces and units of one head each: the measured sides are at kRopeHeads)
    const bool many = tokens * (q_heads * (dim / 16) + 2 * c->kv_heads * (dim / 8)) > 1 << 19;
    a.q_groups = (int)(many ? cdiv(q_heads, kRopeHeads) : q_heads);
    a.kv_groups = (int)(many ? cdiv(c->kv_heads, kRopeHeads) : c->kv_heads);
    const int64_t q_token = a.q_groups * (dim / 16), kv_token = a.kv_groups * (dim / 8);
    a.units = (int)(tokens * q_token);
    a.kv.n = (int)(tokens * kv_token);
    a.per_token = fast_div((unsigned)std::max<int64_t>(q_token, 1));
    a.per_group = fast_div((unsigned)(dim / 16));
    a.kv_token = fast_div((unsigned)kv_token);
    a.kv_group = fast_div((unsigned)(dim / 8));
    a.q_blocks = (int)cdiv(a.units, 256);
    a.kv_blocks = (int)cdiv(a.kv.n, 256);
    const RopeFn fn = many ? rope_fn<kRopeHeads>(c->is_fp4 != 0, interleaved != 0) : rope_fn<1>(c->is_fp4 != 0, interleaved != 0);
    hipLaunchKernelGGL(fn, dim3((unsigned)(a.q_blocks + 2 * a.kv_blocks)), dim3(256), 0, stream, a);
    return host_hip_status(hipGetLastError());
}

}  // namespace

extern "C" {

int mx_rope_cache_write(const mxg_kv_cache_t *cache, const void *q, void *q_out, const void *k, const void *v,
                        int64_t q_heads, int64_t q_stride, int64_t q_out_stride, int64_t k_stride, int64_t v_stride,
                        const int64_t *positions, const int64_t *slots, const float *table, int64_t table_positions,
                        int64_t rot, int interleaved, int64_t tokens, mxg_stream_t stream)
{
    return run_rope(cache, q, q_out, k, v, q_heads, q_stride, q_out_stride, k_stride, v_stride, positions, slots, table,
                    table_positions, rot, interleaved, tokens, (hipStream_t)stream);
}

size_t mx_tree_attention_workspace_bytes(const mxg_kv_cache_t *cache, int64_t seqs, int64_t tokens,
                                         int64_t q_heads, int64_t max_new)
{
    if (validate_cache(cache) || !attn_shape_ok(cache, seqs, tokens, q_heads, max_new))
        return 0;
    // (for any number of keys)
    const int64_t group = q_heads / cache->kv_heads;
    size_t most = 0;
    for (const int64_t keys : {(int64_t)0, (int64_t)1 << 30})
        most = std::max(most, attn_workspace(tree_plan(seqs, tokens, cache->kv_heads, group, cache->head_dim, max_new, keys)));
    return most;
}

int mx_tree_attention(const mxg_kv_cache_t *cache, const void *q, int64_t q_stride, const int32_t *ends,
                      const int32_t *lens, const int32_t *table, int64_t table_width, const uint64_t *mask,
                      int64_t mask_words, int64_t seqs, int64_t tokens, int64_t q_heads, int64_t max_new, float scale,
                      int64_t window, void *out, int out_dtype, float *lse, void *workspace, size_t workspace_bytes,
                      mxg_stream_t stream)
{
    return run_attention<1>(cache, q, q_stride, ends, lens, table, table_width, seqs, tokens, q_heads, max_new, scale, 0,
                            mask, mask_words, window, out, out_dtype, lse, workspace, workspace_bytes, stream);
}

}  // extern "C"
