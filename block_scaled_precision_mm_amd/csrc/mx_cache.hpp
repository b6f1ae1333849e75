// mx_cache.hpp -- the paged key/value cache in MX formats, gfx950: writing
// BF16 tokens into their slots (quantized as mx_quantize does, blocks of 32
// along the head dimension) and reading slots back as BF16.
//
// Layout.  A page holds page_size tokens of every KV head, head by head:
// codes [pages][kv_heads][page_size][head_dim] (E4M3 bytes, or E2M1 pairs),
// scales [pages][kv_heads][page_size][head_dim / 32].  So the rows that one
// head's attention reads from a page are contiguous, and slot t of the cache
// is token t % page_size of page t / page_size (page_size a power of two).
//
// Bound: HBM (and the launch, for one step's few tokens).  A lane moves 8
// values: 16 bytes of BF16 on one side, 8 (E4M3) or 4 (E2M1) bytes of codes on
// the other, so the lanes of a (token, head) row access contiguous bytes on
// both sides and the four lanes of a 32-value block are one quad.  8191
// tokens of 8 heads of 128 into E4M3 12.5 us (51 MB: 4.1 TB/s), 32769 of 8
// heads of 64 back from E2M1 15.4 us (85 MB: 5.5 TB/s), 64 tokens 3.0 us (the
// launch and three dependent accesses).
#pragma once

#include "mx_norm.hpp"

namespace mxg {

// n / d for 0 <= n < 2^31 by a multiplication: (n * m) >> (32 + s), exact for
// the host's m = ceil(2^(32 + s) / d), s = ceil(log2 d) - 1 (d = 1: m = 0).
struct FastDiv {
    unsigned d, m, s;
    __host__ __device__ int div(int n) const
    {
        return m ? (int)(((unsigned long long)(unsigned)n * m) >> 32 >> s) : n;
    }
};

struct CacheArgs {
    uint8_t *codes[2], *scales[2];      // keys, values
    const uint16_t *in[2];              // write: BF16 tokens
    uint16_t *out[2];                   // read
    long long stride[2];                // elements between tokens of in / out
    const long long *slots;
    long long nslots;                   // pages * page_size
    int n;                              // 8-value pieces: tokens * kv_heads * head_dim / 8
    int heads, dim, page_shift;
    FastDiv per_token, per_head;        // pieces of a token, of a head
};

// Element offset of piece `piece` of head `head` at a slot, in values.
__device__ __forceinline__ long long cache_at(const CacheArgs &p, long long slot, int head, int piece)
{
    const long long page = slot >> p.page_shift, off = slot & ((1 << p.page_shift) - 1);
    return (((page * p.heads + head) << p.page_shift) + off) * p.dim + 8 * piece;
}

// U pieces per thread, all their loads in flight together (one at a time: 8191
// tokens written in 13.3 us instead of 12.7, 32769 read in 21.5 instead of 15.4).
constexpr int kCachePieces = 4;

template <int F>
__global__ __launch_bounds__(256)
void mx_cache_write(CacheArgs p)
{
    constexpr int U = kCachePieces;
    const int kv = blockIdx.y, first = (int)blockIdx.x * U * 256 + (int)threadIdx.x;
    long long slot[U];
    u4v w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int i = first + u * 256;
        slot[u] = -1;
        w[u] = u4v{0u, 0u, 0u, 0u};
        if (i < p.n) {
            const int t = p.per_token.div(i);
            slot[u] = p.slots[t];
            w[u] = __builtin_nontemporal_load(
                reinterpret_cast<const u4v *>(p.in[kv] + t * p.stride[kv] + 8 * (i - t * (int)p.per_token.d)));
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int i = first + u * 256;
        const unsigned s = mx_scale_code<F>(quad_max(amax8(w[u])));
        const u2v c = mx_encode8<F>(w[u], s);
        if (slot[u] < 0 || slot[u] >= p.nslots)
            continue;
        const int in_token = i - p.per_token.div(i) * (int)p.per_token.d;
        const int head = p.per_head.div(in_token), piece = in_token - head * (int)p.per_head.d;
        const long long at = cache_at(p, slot[u], head, piece);
        if constexpr (F == FMT_FP4)
            *reinterpret_cast<unsigned *>(p.codes[kv] + (at >> 1)) = c[0];
        else
            *reinterpret_cast<u2v *>(p.codes[kv] + at) = c;
        if ((piece & 3) == 0)
            p.scales[kv][at >> 5] = (uint8_t)s;
    }
}

// Eight values of a block with E8M0 code s, as BF16 pairs: element times
// 2^(s - 127), rounded to nearest even where a BF16 cannot hold it (blocks
// of subnormal BF16 values; past its range, which takes scales that no block of
// finite values is written with, infinity); NaN for s = 255 and for E4M3 NaN
// codes.
// The conversions take s as an exponent field, 0 included, and give NaN for
// every code under the field 255 (checked on MI355X for all codes under all
// scales).
template <int F>
__device__ __forceinline__ u4v mx_decode8(u2v c, unsigned s)
{
    const float sc = __uint_as_float(s << 23);
    u4v w;
    if constexpr (F == FMT_FP4) {
        w[0] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[0], sc, 0));
        w[1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[0], sc, 1));
        w[2] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[0], sc, 2));
        w[3] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[0], sc, 3));
    } else {
        w[0] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[0], sc, false));
        w[1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[0], sc, true));
        w[2] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[1], sc, false));
        w[3] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[1], sc, true));
    }
    return w;
}

template <int F>
__global__ __launch_bounds__(256)
void mx_cache_read(CacheArgs p)
{
    constexpr int U = kCachePieces;
    const int kv = blockIdx.y, first = (int)blockIdx.x * U * 256 + (int)threadIdx.x;
    u2v c[U];
    unsigned s[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int i = first + u * 256;
        c[u] = u2v{0u, 0u};
        s[u] = 127u;                    // a slot outside the cache reads zeros
        if (i < p.n) {
            const int t = p.per_token.div(i), in_token = i - t * (int)p.per_token.d;
            const long long slot = p.slots[t];
            if (slot >= 0 && slot < p.nslots) {
                const int head = p.per_head.div(in_token), piece = in_token - head * (int)p.per_head.d;
                const long long at = cache_at(p, slot, head, piece);
                if constexpr (F == FMT_FP4)
                    c[u][0] = *reinterpret_cast<const unsigned *>(p.codes[kv] + (at >> 1));
                else
                    c[u] = *reinterpret_cast<const u2v *>(p.codes[kv] + at);
                s[u] = p.scales[kv][at >> 5];
            }
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int i = first + u * 256;
        if (i < p.n) {
            const int t = p.per_token.div(i), in_token = i - t * (int)p.per_token.d;
            __builtin_nontemporal_store(mx_decode8<F>(c[u], s[u]),
                                        reinterpret_cast<u4v *>(p.out[kv] + t * p.stride[kv] + 8 * in_token));
        }
    }
}

}  // namespace mxg
