// mx_attn_host.hpp -- host side of the attention kernels (mx_attn.hpp): the
// choice of kernels and the launches, for mx_paged_attention (mxserve.hip) and
// mx_tree_attention (mxdraft.hip).
#pragma once

#include "mx_attn.hpp"
#include "mx_serve.hpp"

namespace mxg {
namespace {

// Words of a drafted token's mask: 64 nodes each.
constexpr int64_t kMaxMaskWords = 1024;

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
template <int TREE>
AttnFn attn_join_fn(int which, int64_t dim)
{
    if (which == ROWS_128)
        return dim == 64 ? &mx_attn_join<64, 128, TREE> : &mx_attn_join<128, 128, TREE>;
    return dim == 64 ? &mx_attn_join<64, 256, TREE> : &mx_attn_join<128, 256, TREE>;
}

template <int F, int D, int PAGED, int TREE, int P2>
AttnFn attn_fn(int which)
{
    switch (which) {
    // (trees: weights in two parts for every output, as it costs these next to nothing)
    case ROWS_16: return &mx_attn_rows<F, D, 1, PAGED, TREE, TREE ? 1 : P2>;
    case ROWS_32: return &mx_attn_rows<F, D, 2, PAGED, TREE, P2>;
    case ROWS_128: return &mx_attn_tile<F, D, 4, PAGED, TREE, P2>;
    default: return &mx_attn_tile<F, D, 8, PAGED, TREE, P2>;
    }
}

template <int F, int D, int TREE, int P2>
AttnFn attn_fn(int which, int64_t page_size)
{
    // mx_attn_rows takes tiles of two pages, mx_attn_tile loads of one wave
    // (64 chunks of 16 bytes)
    const bool paged = page_size >= (which <= ROWS_32 ? 16 : 64 / AttnGeom<F, D>::CH);
    return paged ? attn_fn<F, D, 1, TREE, P2>(which) : attn_fn<F, D, 0, TREE, P2>(which);
}

template <int TREE, int P2>
AttnFn attn_fn(int which, bool fp4, int64_t dim, int64_t page_size)
{
    if (dim == 64)
        return fp4 ? attn_fn<FMT_FP4, 64, TREE, P2>(which, page_size) : attn_fn<FMT_FP8, 64, TREE, P2>(which, page_size);
    return fp4 ? attn_fn<FMT_FP4, 128, TREE, P2>(which, page_size) : attn_fn<FMT_FP8, 128, TREE, P2>(which, page_size);
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
    int resident;           // (trees) workgroups that can run at once
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

// Trees: one launch, whatever the sequences' numbers of nodes.  keys: the most
// keys of a sequence, as far as the host knows.
//
// Rows per tile, by the work: `tiles` of 32 rows (all heads) times keys, and
// rows of a sequence on average.  Few rows per tile have more parts that run
// side by side, many read and expand a key less often.  us, 8 KV heads of 128
// with 4 query heads each, E4M3:
//                                               16    32   128   256 rows
//     1 sequence of 27 nodes over 1051 keys    12.7  14.9    27    28
//     1 of 16 over 4112                        16.5  23.5    27    29
//     32 of 16 over 256                        18.5  15.0    18    22
//     1 of 64 over 16064                         51    40    54    56
//     32 of 16 over 100 to 16000                112    77    90   151
//     8 of 64 over 4096                          92    57    62    65
//     32 of 32 over 4096                        181   118   112   128
//     1 of 200 over 16200                       165   108    87    84
//     32 of 64 over 4096                        344   230   171   152
//     16 of 64 over 300                          36    30    27    31
//     16 of 64 over 1000                         63    46    53    56
//     32 of 64 over 100                          54    49    28    30
//     32 of 64 over 1000                        119    89    60    57
//     8 of 200 over 300                          67    61    44    39
// The thresholds lie between these; near them the rule gives away up to 13%: 1 of
// 117 nodes with 5 query heads each over 32691 keys, 4 KV heads, 56.5 us where
// tiles of 128 take 49.9, 4 of 100 over 8000 43.9 and 38.8, 16 of 64 over 100 24.7
// and 22.1.  And the keys are those that the table has room for, as lengths are on
// the device: 27 nodes over 1051 keys take 13.0 us under a table of up to 4096 keys,
// 14.8 under one of 16384 or 32768, 24.9 under one of 131072.
AttnPlan tree_plan(int64_t seqs, int64_t tokens, int64_t heads, int64_t group, int64_t dim, int64_t max_new, int64_t keys)
{
    AttnPlan p = {};
    const int64_t some = std::min(seqs, tokens);        // sequences with a node
    const int64_t rows = tokens * group, mean = cdiv(rows, std::max<int64_t>(some, 1)), tiles = heads * cdiv(rows, 32);
    p.n = 1;
    // (256 rows in as many rounds of 256 items, 128 in as many of 512, 1.17 times
    // as long: 9 sequences of 880 rows over 500 keys, 288 items of 256 rows or 504
    // of 128, 48 and 35 us)
    const int64_t rounds256 = cdiv(heads * some * cdiv(mean, 256), 256), rounds128 = cdiv(heads * some * cdiv(mean, 128), 512);
    p.which[0] = max_new * group <= 16 || (tiles * keys < 400000 && heads * cdiv(rows, 16) <= 512) ? ROWS_16
                 : mean <= 64 || (tiles < 1400 && tiles * keys < 2500000)                         ? ROWS_32
                 : mean <= 128 || 117 * rounds128 < 100 * rounds256                               ? ROWS_128
                                                                                                  : ROWS_256;
    const int bm = kAttnBM[p.which[0]];
    p.upto[0] = INT32_MAX;
    p.base[0] = heads * (rows / bm + some);
    // (with 768 instead of 512 the parts' joins cost more than the parts gain:
    // 1 sequence of 27 nodes over 16027 keys 40 us instead of 31; with 256, 1 of
    // 200 over 4296 48 instead of 43.  Heads of 128; those of 64 have registers for
    // three waves a SIMD in tiles of 32 rows and the same 512: 24 sequences of 1 to
    // 200 nodes under a window of 1024, 476 row tiles of at most 11 key tiles, take
    // 23 to 25 us, and took 22.5 with other settings)
    p.resident = p.which[0] == ROWS_256 ? 256 : 512;
    p.target[0] = p.resident;
    p.bytes[0] = p.base[0] <= kTreeTiles ? (size_t)2 * p.target[0] * attn_slot_bytes(bm, (int)dim) : 0;
    return p;
}

// The most keys that a row of a tree may see, for tree_plan: what the table has
// room for, and with a window that many and the nodes.
int64_t tree_keys(int64_t table_width, int64_t page_size, int64_t window, int64_t max_new)
{
    return std::min(table_width * page_size, window > 0 ? std::min<int64_t>(window, 1 << 30) + max_new : (int64_t)INT32_MAX);
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

// mx_paged_attention and, TREE, mx_tree_attention (mask and mask_words in
// causal's place).
template <int TREE>
int run_attention(const mxg_kv_cache_t *cache, const void *q, int64_t q_stride, const int32_t *ends,
                  const int32_t *lens, const int32_t *table, int64_t table_width, int64_t seqs, int64_t tokens,
                  int64_t q_heads, int64_t max_new, float scale, int causal, const uint64_t *mask, int64_t mask_words,
                  int64_t window, void *out, int out_dtype, float *lse, void *workspace, size_t workspace_bytes,
                  mxg_stream_t stream)
{
    int rc = validate_cache(cache);
    if (rc)
        return rc;
    if (out_dtype < MXG_OUT_BF16 || out_dtype > MXG_OUT_F32)
        return MXG_ERR_DTYPE;
    if (!attn_shape_ok(cache, seqs, tokens, q_heads, max_new) || table_width < 0 ||
        table_width > ((int64_t)1 << 30) / cache->page_size || q_stride < q_heads * cache->head_dim ||
        q_stride > INT32_MAX || window < 0 || (TREE && (mask_words < 1 || mask_words > kMaxMaskWords)))
        return MXG_ERR_SHAPE;
    if (tokens > 0 && seqs > 0 && (!q || !ends || !lens || !out || (table_width > 0 && !table) || (TREE && !mask)))
        return MXG_ERR_NULL;
    if (q_stride % 8)
        return MXG_ERR_K_ALIGN;
    const float c = scale * 1.4426950408889634f;        // exponents of 2
    if (!(scale > 0.0f) || !isfinite(c) || (!TREE && causal != 0 && causal != 1))
        return MXG_ERR_CONFIG;
    if (((uintptr_t)q | (uintptr_t)out | (uintptr_t)workspace) & 15)
        return MXG_ERR_PTR_ALIGN;
    if (((uintptr_t)ends | (uintptr_t)lens | (uintptr_t)table | (uintptr_t)lse) & 3)
        return MXG_ERR_PTR_ALIGN;
    if ((uintptr_t)mask & 7)
        return MXG_ERR_PTR_ALIGN;
    const int64_t group = q_heads / cache->kv_heads;
    const AttnPlan plan = TREE ? tree_plan(seqs, tokens, cache->kv_heads, group, cache->head_dim, max_new,
                                           tree_keys(table_width, cache->page_size, window, max_new))
                               : attn_plan(seqs, tokens, cache->kv_heads, group, cache->head_dim, max_new);
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
    a.mask = (const unsigned long long *)mask;
    a.mask_words = (int)mask_words;
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
        a.resident = plan.resident;
        const int64_t grid = plan.base[i] + (parts ? plan.target[i] : 0);
        // (weights in two parts where the output has more bits than BF16;
        // tiles of 16 rows in any case)
        AttnFn fn = attn_fn<TREE, 0>(which, cache->is_fp4 != 0, cache->head_dim, cache->page_size);
        if constexpr (TREE)
            if (out_dtype != MXG_OUT_BF16)
                fn = attn_fn<TREE, 1>(which, cache->is_fp4 != 0, cache->head_dim, cache->page_size);
        hipLaunchKernelGGL(fn, dim3((unsigned)grid), dim3(kAttnThreads[which]), 0, (hipStream_t)stream, a);
        rc = host_hip_status(hipGetLastError());
        if (rc)
            return rc;
        if (parts && which >= ROWS_128) {
            const int64_t join = std::min<int64_t>(plan.base[i], plan.target[i]) * attn_join_blocks(kAttnBM[which], (int)cache->head_dim, TREE);
            hipLaunchKernelGGL(attn_join_fn<TREE>(which, cache->head_dim), dim3((unsigned)join), dim3(256), 0,
                               (hipStream_t)stream, a);
            rc = host_hip_status(hipGetLastError());
            if (rc)
                return rc;
        }
    }
    return MXG_OK;
}

}  // namespace
}  // namespace mxg
