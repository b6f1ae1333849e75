// mx_norm.hpp -- RMSNorm of BF16 rows with the residual's addition before it
// and the output as the next MX GEMM's A operand, gfx950.
//
// Per row of K values:
//     h = bf16(x + residual)                      (h = x without a residual)
//     r = 1 / sqrt(sum(h^2) / K + eps)
//     y = bf16((h * r) * weight)                  rounded to nearest even
// and for the MX outputs the blocks of 32 consecutive y quantized exactly as
// mx_quantize does (mx_quant.hpp).  The norm is that of the rounded h: it is
// what the residual stream holds, so the fused call gives what the addition
// and the norm give one after the other.
//
// Roundings.  The squares of BF16 values are exact in FP64, where they are
// summed: no row of finite values overflows (an FP32 sum would from
// |h| = 1.8e19 on) and r is the correctly rounded FP32 value but for sums
// next to a border, whatever the order of the sum.  r is rounded to FP32,
// the two products are FP32 operations.
#pragma once

#include "mx_quant.hpp"

namespace mxg {

struct NormArgs {
    const uint16_t *x, *res, *w;   // res and w may be null
    uint16_t *h;                   // may be null, x or res
    void *y;                       // values, or element codes
    uint8_t *scales;               // E8M0 codes of the MX outputs
    int K;
    float eps;
};

__device__ __forceinline__ float bf16_lo(unsigned v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(unsigned v) { return __uint_as_float(v & 0xFFFF0000u); }

__device__ __forceinline__ unsigned pack_bf16(float a, float b)
{
    return (unsigned)__builtin_bit_cast(unsigned short, (__bf16)a) |
           ((unsigned)__builtin_bit_cast(unsigned short, (__bf16)b) << 16);
}

__device__ __forceinline__ unsigned pack_f16(float a, float b)
{
    return (unsigned)__builtin_bit_cast(unsigned short, (_Float16)a) |
           ((unsigned)__builtin_bit_cast(unsigned short, (_Float16)b) << 16);
}

// E8M0 code of a block whose largest BF16 magnitude (bits) is amax, and the
// eight values of w (BF16 pairs) as codes of that block: 8 bytes (E4M3) or 4
// (E2M1, the second word unused).
template <int F>
__device__ __forceinline__ unsigned mx_scale_code(unsigned amax)
{
    constexpr int EMAX = F == FMT_FP4 ? 2 : 8;
    return amax >= 0x7F80u ? 255u : (unsigned)max((int)(amax >> 7) - EMAX, 0);
}

template <int F>
__device__ __forceinline__ u2v mx_encode8(const u4v &w, unsigned s)
{
    const float sc = __uint_as_float(s << 23);
    u2v d = {0u, 0u};
    if constexpr (F == FMT_FP4) {
        unsigned c = 0;
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, as_bf16x2(w[0]), sc, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, as_bf16x2(w[1]), sc, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, as_bf16x2(w[2]), sc, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, as_bf16x2(w[3]), sc, 3);
        d[0] = s == 255u ? 0u : c;
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            s16x2v o = {0, 0};
            o = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(o, as_bf16x2(w[2 * h]), sc, false);
            o = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(o, as_bf16x2(w[2 * h + 1]), sc, true);
            d[h] = s == 255u ? 0u : e4m3_saturate(__builtin_bit_cast(unsigned, o));
        }
    }
    return d;
}

// One workgroup of THR threads per row, NV 16-byte pieces (8 values) per
// thread, kept in registers between the sum and the output: the row is read
// once.  Piece j of thread t is piece t + j * THR of the row, so every access
// is contiguous and the four pieces of a 32-value block lie in one quad.
//
// Bound: HBM for many rows: 8192 rows of 8192 values with a residual, h and
// E4M3 output move 472 MB in 83 us, 5.7 TB/s.  A launch and the latency of
// a row's two passes for few: 1 row of 4096 3.1 us, 129 of 5120 5.0.
template <int THR, int NV, int OUT>
__global__ __launch_bounds__(THR)
void mx_rmsnorm_rows(NormArgs p)
{
    const int tid = threadIdx.x;
    const int npieces = p.K >> 3;
    const size_t row = blockIdx.x;
    const u4v *x = reinterpret_cast<const u4v *>(p.x + row * p.K);
    u4v v[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        v[j] = u4v{0u, 0u, 0u, 0u};
        if (tid + j * THR < npieces)
            v[j] = __builtin_nontemporal_load(x + tid + j * THR);
    }
    if (p.res) {
        const u4v *res = reinterpret_cast<const u4v *>(p.res + row * p.K);
        u4v a[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            a[j] = u4v{0u, 0u, 0u, 0u};
            if (tid + j * THR < npieces)
                a[j] = __builtin_nontemporal_load(res + tid + j * THR);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[j][i] = pack_bf16(bf16_lo(v[j][i]) + bf16_lo(a[j][i]), bf16_hi(v[j][i]) + bf16_hi(a[j][i]));
    }
    if (p.h) {
        u4v *h = reinterpret_cast<u4v *>(p.h + row * p.K);
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (tid + j * THR < npieces)
                h[tid + j * THR] = v[j];
    }
    double sum = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const double lo = bf16_lo(v[j][i]), hi = bf16_hi(v[j][i]);
            sum = fma(lo, lo, sum);
            sum = fma(hi, hi, sum);
        }
#pragma unroll
    for (int d = 1; d < 64; d *= 2)
        sum += __shfl_xor(sum, d);
    if constexpr (THR > 64) {
        __shared__ double part[THR / 64];
        if ((tid & 63) == 0)
            part[tid >> 6] = sum;
        __syncthreads();
        sum = 0;
#pragma unroll
        for (int i = 0; i < THR / 64; ++i)
            sum += part[i];
    }
    // (1 / r beyond FP32's normal range: both factors of h * r moved into it)
    const double rd = 1.0 / sqrt(sum / p.K + (double)p.eps);
    const float move = rd < 0x1p-126 ? 0x1p-32f : rd > 0x1p127 ? 0x1p32f : 1.0f;
    const float r = (float)(rd / move);
    const u4v *w = reinterpret_cast<const u4v *>(p.w);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int at = tid + j * THR;
        if (at >= npieces)
            break;
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = bf16_lo(v[j][i]) * move * r;
            f[2 * i + 1] = bf16_hi(v[j][i]) * move * r;
        }
        if (w) {
            const u4v g = w[at];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] *= bf16_lo(g[i]);
                f[2 * i + 1] *= bf16_hi(g[i]);
            }
        }
        if constexpr (OUT == OUT_F32) {
            v4f *y = reinterpret_cast<v4f *>(reinterpret_cast<float *>(p.y) + row * p.K) + 2 * at;
            y[0] = v4f{f[0], f[1], f[2], f[3]};
            y[1] = v4f{f[4], f[5], f[6], f[7]};
        } else if constexpr (OUT == OUT_F16) {
            reinterpret_cast<u4v *>(reinterpret_cast<uint16_t *>(p.y) + row * p.K)[at] =
                u4v{pack_f16(f[0], f[1]), pack_f16(f[2], f[3]), pack_f16(f[4], f[5]), pack_f16(f[6], f[7])};
        } else {
            const u4v b = {pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])};
            if constexpr (OUT == OUT_BF16) {
                reinterpret_cast<u4v *>(reinterpret_cast<uint16_t *>(p.y) + row * p.K)[at] = b;
            } else {
                constexpr int F = OUT == OUT_MX4 ? FMT_FP4 : FMT_FP8;
                const unsigned s = mx_scale_code<F>(quad_max(amax8(b)));
                const u2v c = mx_encode8<F>(b, s);
                uint8_t *codes = reinterpret_cast<uint8_t *>(p.y);
                if constexpr (F == FMT_FP4)
                    reinterpret_cast<unsigned *>(codes + row * (p.K >> 1))[at] = c[0];
                else
                    reinterpret_cast<u2v *>(codes + row * p.K)[at] = c;
                if ((tid & 3) == 0)
                    p.scales[row * (p.K >> 5) + (at >> 2)] = (uint8_t)s;
            }
        }
    }
}

}  // namespace mxg
