// mx_rope.hpp -- the position rotation of a step's queries and keys, and its
// keys and values into the paged MX cache (mx_cache.hpp), in one launch,
// gfx950.
//
// The first `rot` values of every head of queries and keys are turned in
// pairs (a, b) by the token's angles: (i, i + rot / 2), or (2i, 2i + 1)
// interleaved:
//     a' = a cos - b sin,   b' = b cos + a sin
// with cosine and sine of (position, i) from a table that the caller keeps.
//
// Bound: HBM for many tokens: 8191 of 32 query and 8 key heads of 128 into
// E4M3 move 189 MB in 35 us, 5.4 TB/s, where a large copy reaches 5.1 to 5.2.  For
// a step's few the launch and a chain of dependent accesses (position, angles,
// slot): 64 tokens 2.8 us in a replayed graph.
//
// Roundings.  A BF16 value times an FP32 one is exact in FP64, so each result
// is rounded there once, then to FP32 and to BF16: it does not depend on how
// products are contracted, and the keys' codes are those of mx_kv_cache_write
// for the rotated BF16 keys, bit for bit.  The FP64 operations (two per value)
// stay hidden behind the memory accesses.
#pragma once

#include "mx_cache.hpp"

namespace mxg {

struct RopeArgs {
    CacheArgs kv;               // in: keys and values; n: 8-value pieces, one for each group of heads
    const uint16_t *q;
    uint16_t *q_out;            // may be q
    long long q_stride, q_out_stride;
    const long long *positions;
    const float *table;         // [npositions][rot / 2] (cosine, sine)
    long long npositions;
    int units;                  // of queries: tokens * q_groups * dim / 16
    int q_heads, q_groups, kv_groups;       // heads, and groups of at most H of them
    FastDiv per_token, per_group;           // units of a token, of a group (queries)
    FastDiv kv_token, kv_group;             // pieces of a token, of a group (keys, values)
    int rot, q_blocks, kv_blocks;           // workgroups of queries, of keys (as many of values)
};

// H heads of a token per thread (every q_groups-th), all their loads in flight
// together and the angles loaded once for them.  One head for few tokens, whose
// time is one thread's; four for many, and then past the caches, as nothing
// of a prompt's queries stays there until they are read (us, 32 and 8 heads of
// 128; with one head 1000 tokens 6.6 both ways):
//     tokens           64    512   1000   2000   4000   8000
//     1 head          2.9    4.4    6.6   11.1   22.9   41.1
//     4 heads         4.4    5.1    6.6    9.9   19.1   35.8
constexpr int kRopeHeads = 4;

template <int H>
__device__ __forceinline__ u4v rope_load(const uint16_t *at)
{
    const u4v *v = reinterpret_cast<const u4v *>(at);
    return H > 1 ? __builtin_nontemporal_load(v) : *v;
}

template <int H>
__device__ __forceinline__ void rope_store(uint16_t *at, u4v w)
{
    u4v *v = reinterpret_cast<u4v *>(at);
    if constexpr (H > 1)
        __builtin_nontemporal_store(w, v);
    else
        *v = w;
}

// (cos, sin) of the eight pairs 8u .. of a position, NaN for one that the table
// does not have.
struct RopeAngles {
    float c[8], s[8];
    __device__ __forceinline__ void load(const RopeArgs &p, long long position, int u)
    {
        const bool there = position >= 0 && position < p.npositions;
        const v4f *at = reinterpret_cast<const v4f *>(p.table + (there ? position : 0) * p.rot) + 4 * u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const v4f w = at[i];
            c[2 * i] = there ? w[0] : __builtin_nanf("");
            s[2 * i] = there ? w[1] : __builtin_nanf("");
            c[2 * i + 1] = there ? w[2] : __builtin_nanf("");
            s[2 * i + 1] = there ? w[3] : __builtin_nanf("");
        }
    }
};

// (contraction would fold the rounding to FP32 into the one to BF16)
__device__ __forceinline__ float rope_first(float a, float b, float c, float s)
{
#pragma clang fp contract(off)
    return (float)fma((double)a, (double)c, -((double)b * (double)s));
}

__device__ __forceinline__ float rope_second(float a, float b, float c, float s)
{
#pragma clang fp contract(off)
    return (float)fma((double)b, (double)c, (double)a * (double)s);
}

// Eight interleaved values, with angles at .. at + 3.
__device__ __forceinline__ u4v rope_adjacent(u4v w, const RopeAngles &t, int at)
{
    u4v y;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = bf16_lo(w[i]), b = bf16_hi(w[i]), c = t.c[at + i], s = t.s[at + i];
        y[i] = pack_bf16(rope_first(a, b, c, s), rope_second(a, b, c, s));
    }
    return y;
}

// Eight firsts (or seconds) of pairs, from both.
__device__ __forceinline__ u4v rope_firsts(u4v a, u4v b, const RopeAngles &t)
{
    u4v y;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        y[i] = pack_bf16(rope_first(bf16_lo(a[i]), bf16_lo(b[i]), t.c[2 * i], t.s[2 * i]),
                         rope_first(bf16_hi(a[i]), bf16_hi(b[i]), t.c[2 * i + 1], t.s[2 * i + 1]));
    return y;
}

__device__ __forceinline__ u4v rope_seconds(u4v a, u4v b, const RopeAngles &t)
{
    u4v y;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        y[i] = pack_bf16(rope_second(bf16_lo(a[i]), bf16_lo(b[i]), t.c[2 * i], t.s[2 * i]),
                         rope_second(bf16_hi(a[i]), bf16_hi(b[i]), t.c[2 * i + 1], t.s[2 * i + 1]));
    return y;
}

// Queries: a thread has unit u of 16 values, eight pairs: pieces u and
// u + rot / 16, or (interleaved, and past the rotated values) pieces 2u and
// 2u + 1, of every q_groups-th head.  Both pieces of a pair are one thread's,
// so q may be rotated in place.
template <int INTER, int H>
__device__ __forceinline__ void rope_queries(const RopeArgs &p)
{
    const int n = (int)blockIdx.x * 256 + (int)threadIdx.x;
    if (n >= p.units)
        return;
    const int t = p.per_token.div(n), in_token = n - t * (int)p.per_token.d;
    const int group = p.per_group.div(in_token), u = in_token - group * (int)p.per_group.d;
    const int dim = p.kv.dim, half = p.rot / 16;
    const bool turned = u < half, apart = !INTER && turned;
    const int first = 8 * (apart ? u : 2 * u), second = 8 * (apart ? u + half : 2 * u + 1);
    const uint16_t *src = p.q + t * p.q_stride;
    uint16_t *dst = p.q_out + t * p.q_out_stride;
    const long long position = p.positions[t];
    u4v a[H], b[H];
#pragma unroll
    for (int j = 0; j < H; ++j) {
        const int head = min(group + j * p.q_groups, p.q_heads - 1);
        a[j] = rope_load<H>(src + head * dim + first);
        b[j] = rope_load<H>(src + head * dim + second);
    }
    if (turned) {
        RopeAngles w;
        w.load(p, position, u);
#pragma unroll
        for (int j = 0; j < H; ++j) {
            if (INTER) {
                a[j] = rope_adjacent(a[j], w, 0);
                b[j] = rope_adjacent(b[j], w, 4);
            } else {
                const u4v x = a[j];
                a[j] = rope_firsts(x, b[j], w);
                b[j] = rope_seconds(x, b[j], w);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < H; ++j) {
        const int head = group + j * p.q_groups;
        if (head < p.q_heads) {
            rope_store<H>(dst + head * dim + first, a[j]);
            rope_store<H>(dst + head * dim + second, b[j]);
        }
    }
}

// Keys (kv 0) and values: a thread has one piece of every kv_groups-th head;
// the four lanes of a quad have a block of 32.  A key's piece takes the values
// that it is paired with from memory as well (a second time from the cache of
// the CU), so that blocks need not match pairs.
template <int F, int INTER, int H>
__device__ __forceinline__ void rope_keys(const RopeArgs &p, int kv, int block)
{
    const int n = block * 256 + (int)threadIdx.x;
    const int dim = p.kv.dim, half = p.rot / 16;
    const bool mine = n < p.kv.n;
    const int i = mine ? n : 0;
    const int t = p.kv_token.div(i), in_token = i - t * (int)p.kv_token.d;
    const int group = p.kv_group.div(in_token), piece = in_token - group * (int)p.kv_group.d;
    const bool turned = kv == 0 && piece < 2 * half, second = piece >= half;
    const int other = INTER ? piece : second ? piece - half : piece + half;
    const uint16_t *src = p.kv.in[kv] + t * p.kv.stride[kv];
    const long long slot = mine ? p.kv.slots[t] : -1;
    const long long position = turned ? p.positions[t] : 0;
    u4v a[H], b[H];
#pragma unroll
    for (int j = 0; j < H; ++j) {
        const int head = min(group + j * p.kv_groups, p.kv.heads - 1);
        a[j] = *reinterpret_cast<const u4v *>(src + head * dim + 8 * piece);
        if (!INTER)
            b[j] = turned ? *reinterpret_cast<const u4v *>(src + head * dim + 8 * other) : u4v{0u, 0u, 0u, 0u};
    }
    if (turned) {
        RopeAngles w;
        w.load(p, position, INTER ? piece >> 1 : second ? piece - half : piece);
#pragma unroll
        for (int j = 0; j < H; ++j) {
            if (INTER) {
                RopeAngles v = w;
                if (piece & 1)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        v.c[e] = w.c[4 + e];
                        v.s[e] = w.s[4 + e];
                    }
                a[j] = rope_adjacent(a[j], v, 0);
            } else {
                a[j] = second ? rope_seconds(b[j], a[j], w) : rope_firsts(a[j], b[j], w);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < H; ++j) {
        const int head = group + j * p.kv_groups;
        const unsigned s = mx_scale_code<F>(quad_max(amax8(a[j])));
        const u2v c = mx_encode8<F>(a[j], s);
        if (slot < 0 || slot >= p.kv.nslots || head >= p.kv.heads)
            continue;
        const long long at = cache_at(p.kv, slot, head, piece);
        if constexpr (F == FMT_FP4)
            *reinterpret_cast<unsigned *>(p.kv.codes[kv] + (at >> 1)) = c[0];
        else
            *reinterpret_cast<u2v *>(p.kv.codes[kv] + at) = c;
        if ((piece & 3) == 0)
            p.kv.scales[kv][at >> 5] = (uint8_t)s;
    }
}

template <int F, int INTER, int H>
__global__ __launch_bounds__(256)
void mx_rope_write(RopeArgs p)
{
    const int block = blockIdx.x;
    if (block < p.q_blocks)
        rope_queries<INTER, H>(p);
    else if (block < p.q_blocks + p.kv_blocks)
        rope_keys<F, INTER, H>(p, 0, block - p.q_blocks);
    else
        rope_keys<F, INTER, H>(p, 1, block - p.q_blocks - p.kv_blocks);
}

}  // namespace mxg
