// mx_moe.hpp -- tokens to their experts' rows and back, around the grouped
// product (mx_group.hpp), gfx950.
//
// Each token t has top_k assignments a = t * top_k + j to experts ids[a].
// Sorted by expert, and among one expert's by a (a stable counting sort, so
// that the order never depends on timing), assignment a has row
//     pos[a] = #{b : ids[b] < ids[a]} + #{b < a : ids[b] = ids[a]}
// over the assignments whose expert is in [0, groups); others have row -1.
//   dispatch   y[pos[a]] = x[t], as MX blocks or BF16;  offs[g] the end of g's rows
//   combine    out[t] = sum_j w[t,j] y[pos[t,j]]
//   gradient   d_y[pos[t,j]] = w[t,j] d_out[t],  d_w[t,j] = <d_out[t], y[pos[t,j]]>
//
// All three are bound by HBM for many tokens: 8191 tokens of 4096 with 4 choices
// each, half of them held here, into E4M3 137 MB in 32 us (4.3 TB/s, with the
// kernel that counts), back from all of them 336 MB in 63 us (5.3 TB/s), the
// gradients of 4095 with 2 choices 168 MB in 34.5 us (4.9 TB/s), calls back to back
// with inputs that change; and for a step's few by the launch and a chain of
// dependent accesses: ids, counts, rows (64 tokens with 8 choices 4.7 and 2.7 us
// in a replayed graph).
#pragma once

#include "mx_norm.hpp"
#include "mx_cache.hpp"

namespace mxg {

// Most experts (counters in LDS), most assignments of a token.
constexpr int kMoeGroups = 1024, kMoeTopK = 64;

struct MoeArgs {
    const uint16_t *x;
    const long long *ids;
    void *y;
    uint8_t *scales;
    int *offs, *pos;
    int *counts;                // [chunks][groups]: of each chunk's assignments, then rows before them; null: no chunks
    unsigned *arrived;          // zero, and left zero
    int tokens, top_k, groups, K;
    int each;                   // tokens per workgroup, each * top_k <= 64
    int chunk, chunks;          // assignments per chunk
    int summed;                 // counts become the rows before each chunk's (or stay counts, for few chunks)
    FastDiv per_row;            // pieces of eight values of a row
    int segments;               // workgroups that share a row's pieces
};

// The expert of assignment a, or -1 for one that is not held here.
__device__ __forceinline__ int moe_expert(const MoeArgs &p, int a)
{
    const long long e = p.ids[a];
    return e >= 0 && e < p.groups ? (int)e : -1;
}

// Exclusive sums of n counters in LDS, in place, by THR threads; returns the
// total.  `sums` holds THR / 64 words of LDS.
template <int THR>
__device__ __forceinline__ int moe_scan(int *count, int n, int *sums)
{
    const int tid = threadIdx.x, lane = tid & 63, each = (n + THR - 1) / THR;
    const int from = min(tid * each, n), upto = min(from + each, n);
    int mine = 0;
    for (int i = from; i < upto; ++i)
        mine += count[i];
    int inclusive = mine;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int u = __shfl_up(inclusive, d);
        inclusive += lane >= d ? u : 0;
    }
    if (lane == 63)
        sums[tid >> 6] = inclusive;
    __syncthreads();
    int before = inclusive - mine, total = 0;
#pragma unroll
    for (int w = 0; w < THR / 64; ++w) {
        before += w < tid >> 6 ? sums[w] : 0;
        total += sums[w];
    }
    for (int i = from; i < upto; ++i) {
        const int c = count[i];
        count[i] = before;
        before += c;
    }
    __syncthreads();
    return total;
}

// Many assignments, first kernel: each workgroup counts a chunk's; and with many
// chunks (summed) the one that arrives last turns the counts into the rows
// before each chunk's.  With few, up to kMoeChunks, the second kernel's
// workgroups add them up themselves, which is a round of loads for each but no
// chain of them in one workgroup while the GPU waits.  us on the GPU, 8 choices
// of each token, rows of 1024 into E4M3, added up by each / by the last:
//     chunks               64          128          256          512
//        8 experts    24.5  26.2   46.9  44.1   98.0  89.3   210  167
//       64            24.4  28.6   47.8  51.6    103   108   226  210
//      256            24.9  39.2   49.9  77.6    119   154   310  278
//     1024            35.3  74.2   83.2   142    224   292   702  581
// (4 choices of rows of 4096: up to 256 chunks by each always, 359 and 364 us
// with 8 experts, 469 and 558 with 1024; 2 choices of rows of 1024 from 128 chunks
// on up to 3% slower by each with 4 to 16 experts, and faster with 64.)
constexpr int kMoeChunks = 256;

template <int THR>
__global__ __launch_bounds__(THR)
void mx_moe_count(MoeArgs p)
{
    __shared__ int count[kMoeGroups], sums[THR / 64], part[THR];
    __shared__ unsigned arrived;
    const int tid = threadIdx.x, total = p.tokens * p.top_k;
    for (int g = tid; g < p.groups; g += THR)
        count[g] = 0;
    __syncthreads();
    const int from = (int)blockIdx.x * p.chunk, upto = min(from + p.chunk, total);
    for (int a = from + tid; a < upto; a += THR) {
        const int e = moe_expert(p, a);
        if (e >= 0)
            atomicAdd(&count[e], 1);
    }
    __syncthreads();
    int *row = p.counts + (long long)blockIdx.x * p.groups;
    for (int g = tid; g < p.groups; g += THR)
        __hip_atomic_store(row + g, count[g], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (!p.summed)
        return;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (tid == 0)
        arrived = __hip_atomic_fetch_add(p.arrived, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (arrived != (unsigned)(p.chunks - 1))
        return;
    // thread (s, g): expert g of the s-th of `segs` ranges of chunks
    int wide = 1;
    while (wide < p.groups)
        wide *= 2;
    wide = min(wide, THR);
    const int segs = THR / wide, s = tid / wide, g0 = tid % wide;
    const int each = (p.chunks + segs - 1) / segs, c0 = min(s * each, p.chunks), c1 = min(c0 + each, p.chunks);
    auto load = [&](int c, int g) {
        return __hip_atomic_load(p.counts + (long long)c * p.groups + g, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    };
    for (int g = tid; g < p.groups; g += THR)
        count[g] = 0;
    __syncthreads();
    for (int g = g0; g < p.groups; g += wide) {
        int n = 0;
        for (int c = c0; c < c1; ++c)
            n += load(c, g);
        atomicAdd(&count[g], n);
    }
    __syncthreads();
    moe_scan<THR>(count, p.groups, sums);
    // (experts of one thread in turn: those before it in the group's ranges of
    // chunks through `part`)
    for (int g1 = 0; g1 < p.groups; g1 += wide) {
        const int g = g1 + g0;
        int n = 0;
        if (g < p.groups)
            for (int c = c0; c < c1; ++c)
                n += load(c, g);
        part[tid] = n;
        __syncthreads();
        if (g < p.groups) {
            int before = count[g];
            for (int i = 0; i < s; ++i)
                before += part[i * wide + g0];
            if (s == segs - 1)
                p.offs[g] = before + n;
            for (int c = c0; c < c1; ++c) {
                const int m = load(c, g);
                __hip_atomic_store(p.counts + (long long)c * p.groups + g, before, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                before += m;
            }
        }
        __syncthreads();
    }
    if (tid == 0)
        __hip_atomic_store(p.arrived, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Eight values (BF16 pairs) to piece `piece` of row `row`: as they are, or as a
// part of an MX block, whose four lanes are a quad.  s: the block's scale code.
template <int OUT>
__device__ __forceinline__ void moe_store(void *y, uint8_t *scales, long long row, int K, int piece, const u4v &w, const u2v &c, unsigned s)
{
    if constexpr (OUT == OUT_BF16) {
        reinterpret_cast<u4v *>(reinterpret_cast<uint16_t *>(y) + row * K)[piece] = w;
    } else {
        uint8_t *codes = reinterpret_cast<uint8_t *>(y);
        if constexpr (OUT == OUT_MX4)
            reinterpret_cast<unsigned *>(codes + row * (K >> 1))[piece] = c[0];
        else
            reinterpret_cast<u2v *>(codes + row * K)[piece] = c;
        if ((piece & 3) == 0)
            scales[row * (K >> 5) + (piece >> 2)] = (uint8_t)s;
    }
}

// Each workgroup finds the rows of its tokens' assignments and writes the
// tokens there.  It counts the assignments of the same expert before its own:
// from the chunk's start, or where there are no chunks all of them, of every
// expert.  A token is read and quantized once, whatever top_k is; its next
// pieces are loaded before the last ones are written (8191 tokens 38.5 us
// without that, 35.3 with it).
template <int OUT, int THR>
__global__ __launch_bounds__(THR)
void mx_moe_dispatch_rows(MoeArgs p)
{
    constexpr int F = OUT == OUT_MX4 ? FMT_FP4 : FMT_FP8;
    constexpr int U = 4;            // pieces per thread in flight
    __shared__ int before[kMoeGroups], start[kMoeGroups], sums[THR / 64], rows[64];
    const int tid = threadIdx.x, segment = (int)blockIdx.x % p.segments;
    const int t0 = (int)blockIdx.x / p.segments * p.each, mine = min(p.each, p.tokens - t0);
    const int a0 = t0 * p.top_k, na = mine * p.top_k;
    const int pieces = (int)p.per_row.d, n = mine * pieces;
    // this workgroup's pieces: of a row's `segments` parts one (one token), or all
    const int part = (n + p.segments - 1) / p.segments, lo = min(segment * ((part + 3) & ~3), n), hi = min(lo + ((part + 3) & ~3), n);
    const u4v *x = reinterpret_cast<const u4v *>(p.x + (long long)t0 * p.K);
    u4v w[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (lo + tid + u * THR < hi)
            w[u] = __builtin_nontemporal_load(x + lo + tid + u * THR);
    const int own = tid < na ? moe_expert(p, a0 + tid) : -1;     // wave 0: the expert of assignment tid

    const bool chunks = p.counts != nullptr;
    const int chunk = chunks ? (int)((unsigned)a0 / (unsigned)p.chunk) : 0;
    for (int g = tid; g < p.groups; g += THR) {
        int all = 0, ahead = 0;
        if (chunks && !p.summed) {
#pragma unroll 8
            for (int c = 0; c < p.chunks; ++c) {
                const int n = p.counts[c * p.groups + g];
                all += n;
                ahead += c < chunk ? n : 0;
            }
        }
        start[g] = all;
        before[g] = ahead;
    }
    __syncthreads();
    if (chunks) {
        for (int a = chunk * p.chunk + tid; a < a0; a += THR) {
            const int e = moe_expert(p, a);
            if (e >= 0)
                atomicAdd(&before[e], 1);
        }
    } else {
        const int total = p.tokens * p.top_k;
        for (int a = tid; a < total; a += THR) {
            const int e = moe_expert(p, a);
            if (e >= 0) {
                atomicAdd(&start[e], 1);
                if (a < a0)
                    atomicAdd(&before[e], 1);
            }
        }
    }
    __syncthreads();
    const bool summed = chunks && p.summed;
    if (!summed) {
        const int all = moe_scan<THR>(start, p.groups, sums);
        if (blockIdx.x == 0)
            for (int g = tid; g < p.groups; g += THR)
                p.offs[g] = g + 1 < p.groups ? start[g + 1] : all;
    }
    if (tid < 64) {
        // the lanes with the same expert, a bit at a time
        unsigned long long same = __ballot(own >= 0);
#pragma unroll
        for (int b = 1; b < kMoeGroups; b *= 2) {
            const unsigned long long set = __ballot((own & b) != 0);
            same &= own & b ? set : ~set;
        }
        const int rank = __popcll(same & ~(~0ull << tid));
        int row = -1;
        if (own >= 0)
            row = rank + before[own] + (summed ? p.counts[(long long)chunk * p.groups + own] : start[own]);
        rows[tid] = row;
        if (tid < na && segment == 0)
            p.pos[a0 + tid] = row;
    }
    __syncthreads();
    for (int i = lo + tid; i - tid < hi; i += U * THR) {
        u4v v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            v[u] = w[u];
            if (i + (U + u) * THR < hi)
                w[u] = __builtin_nontemporal_load(x + i + (U + u) * THR);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = i + u * THR;
            if (at >= hi)
                continue;
            const int t = p.per_row.div(at), piece = at - t * pieces;
            unsigned s = 0;
            u2v c = {0u, 0u};
            if constexpr (OUT != OUT_BF16) {
                s = mx_scale_code<F>(quad_max(amax8(v[u])));
                c = mx_encode8<F>(v[u], s);
            }
            for (int j = 0; j < p.top_k; ++j) {
                const int row = rows[t * p.top_k + j];
                if (row >= 0)
                    moe_store<OUT>(p.y, p.scales, row, p.K, piece, v[u], c, s);
            }
        }
    }
}

// ------------------------------------------------------------ and back
// Eight values of a row of BF16, FP16 or FP32 (T: OUT_BF16, OUT_F16, OUT_F32).
template <int T>
struct MoeRow {
    u4v w[T == OUT_F32 ? 2 : 1];
    __device__ __forceinline__ void load(const void *base, long long row, int N, int piece)
    {
        if constexpr (T == OUT_F32) {
            const u4v *at = reinterpret_cast<const u4v *>(reinterpret_cast<const float *>(base) + row * N) + 2 * piece;
            w[0] = at[0];
            w[1] = at[1];
        } else {
            w[0] = reinterpret_cast<const u4v *>(reinterpret_cast<const uint16_t *>(base) + row * N)[piece];
        }
    }
    __device__ __forceinline__ float get(int e) const
    {
        if constexpr (T == OUT_F32)
            return __uint_as_float(w[e >> 2][e & 3]);
        else if constexpr (T == OUT_BF16)
            return e & 1 ? bf16_hi(w[0][e >> 1]) : bf16_lo(w[0][e >> 1]);
        else
            return (float)__builtin_bit_cast(_Float16, (unsigned short)(w[0][e >> 1] >> (16 * (e & 1))));
    }
};

template <int T>
__device__ __forceinline__ void moe_put(void *base, long long row, int N, int piece, const float (&f)[8])
{
    if constexpr (T == OUT_F32) {
        v4f *at = reinterpret_cast<v4f *>(reinterpret_cast<float *>(base) + row * N) + 2 * piece;
        at[0] = v4f{f[0], f[1], f[2], f[3]};
        at[1] = v4f{f[4], f[5], f[6], f[7]};
    } else {
        u4v *at = reinterpret_cast<u4v *>(reinterpret_cast<uint16_t *>(base) + row * N) + piece;
        if constexpr (T == OUT_BF16)
            *at = u4v{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])};
        else
            *at = u4v{pack_f16(f[0], f[1]), pack_f16(f[2], f[3]), pack_f16(f[4], f[5]), pack_f16(f[6], f[7])};
    }
}

struct CombineArgs {
    const void *y, *d_out;
    const int *pos;
    const float *w;             // null: ones
    void *out;                  // combine: [tokens][N]; gradient: d_y
    uint8_t *scales;            // of d_y
    float *d_w;                 // or null
    int tokens, top_k, rows, N;
    int n;                      // combine: pieces of out
    FastDiv per_row;
};

// A thread has a piece of a token; J of its rows are in flight at a time.
template <int T, int OUT, int J>
__global__ __launch_bounds__(256)
void mx_moe_combine_rows(CombineArgs p)
{
    const int i = (int)(blockIdx.x * 256 + threadIdx.x);
    if (i >= p.n)
        return;
    const int tok = p.per_row.div(i), piece = i - tok * (int)p.per_row.d;
    const long long t = tok;
    const int *pos = p.pos + t * p.top_k;
    const float *w = p.w ? p.w + t * p.top_k : nullptr;
    float f[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int j0 = 0; j0 < p.top_k; j0 += J) {
        int row[J];
        float g[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            row[j] = j0 + j < p.top_k ? pos[j0 + j] : -1;
            g[j] = w && j0 + j < p.top_k ? w[j0 + j] : 1.0f;
        }
        MoeRow<T> v[J];
#pragma unroll
        for (int j = 0; j < J; ++j)
            if ((unsigned)row[j] < (unsigned)p.rows)
                v[j].load(p.y, row[j], p.N, piece);
#pragma unroll
        for (int j = 0; j < J; ++j)
            if ((unsigned)row[j] < (unsigned)p.rows)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    f[e] = fmaf(g[j], v[j].get(e), f[e]);
    }
    moe_put<OUT>(p.out, t, p.N, piece, f);
}

// An FP32 product, as a register that holds it: the compiler would fold its
// rounding into the one to FP16 (v_fma_mixlo_f16).
__device__ __forceinline__ float moe_weighted(float w, float v)
{
    float f = w * v;
    asm("" : "+v"(f));
    return f;
}

// One workgroup per token: its row of d_out times each weight into d_y's rows,
// and the products with y's summed over the row: in a thread's own order, then
// over the lanes and the waves, in FP32.  Rows shorter than 2048 values leave some
// of its threads without any: 4095 tokens with 2 choices, BF16, of 512 values 9.0
// us for 21 MB, of 1024 11.4 for 42, of 2080 21.2 for 85, of 4096 34.5 for 168.
template <int T, int OUT, int THR>
__global__ __launch_bounds__(THR)
void mx_moe_combine_grad_rows(CombineArgs p)
{
    constexpr bool MX = OUT == OUT_MX8 || OUT == OUT_MX4;
    constexpr int F = OUT == OUT_MX4 ? FMT_FP4 : FMT_FP8;
    constexpr int J = 4;            // rows at a time
    __shared__ float sums[J][THR / 64];
    const int tid = threadIdx.x, pieces = (int)p.per_row.d;
    const long long t = blockIdx.x;
    for (int j0 = 0; j0 < p.top_k; j0 += J) {
        int row[J];
        float g[J], dot[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            row[j] = j0 + j < p.top_k ? p.pos[t * p.top_k + j0 + j] : -1;
            if ((unsigned)row[j] >= (unsigned)p.rows)
                row[j] = -1;
            g[j] = p.w && j0 + j < p.top_k ? p.w[t * p.top_k + j0 + j] : 1.0f;
            dot[j] = 0.0f;
        }
        for (int piece = tid; piece < pieces; piece += THR) {
            MoeRow<T> d, v[J];
            d.load(p.d_out, t, p.N, piece);
            if (p.d_w)
#pragma unroll
                for (int j = 0; j < J; ++j)
                    if (row[j] >= 0)
                        v[j].load(p.y, row[j], p.N, piece);
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if (row[j] < 0)
                    continue;
                float f[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    f[e] = moe_weighted(g[j], d.get(e));
                if constexpr (MX) {
                    const u4v b = {pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])};
                    const unsigned s = mx_scale_code<F>(quad_max(amax8(b)));
                    moe_store<OUT>(p.out, p.scales, row[j], p.N, piece, b, mx_encode8<F>(b, s), s);
                } else {
                    moe_put<OUT>(p.out, row[j], p.N, piece, f);
                }
                if (p.d_w)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        dot[j] = fmaf(d.get(e), v[j].get(e), dot[j]);
            }
        }
        if (p.d_w) {
#pragma unroll
            for (int j = 0; j < J; ++j) {
#pragma unroll
                for (int d = 1; d < 64; d *= 2)
                    dot[j] += __shfl_xor(dot[j], d);
                if ((tid & 63) == 0)
                    sums[j][tid >> 6] = dot[j];
            }
            __syncthreads();
            if (tid < J && j0 + tid < p.top_k) {
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < THR / 64; ++i)
                    sum += sums[tid][i];
                p.d_w[t * p.top_k + j0 + tid] = sum;
            }
            __syncthreads();
        }
    }
}

}  // namespace mxg
