// mxmoe.hip -- host side of the operators around the grouped product: tokens
// sorted by expert into its A operand, the experts' rows back with the
// router's weights, and the gradients of that.  Argument validation and
// launches behind the C ABI declared in include/mxgemm.h.
#include <hip/hip_runtime.h>

#include "mx_moe.hpp"
#include "mx_serve.hpp"
#include "mx_splitk.hpp"

using namespace mxg;

namespace {

constexpr int64_t kMoeTokens = (1 << 24) - 1, kMoeAssignments = 1 << 26, kMoeRow = 1 << 20;

bool moe_sizes_ok(int64_t tokens, int64_t top_k)
{
    return tokens >= 0 && tokens <= kMoeTokens && top_k >= 1 && top_k <= kMoeTopK && tokens * top_k <= kMoeAssignments;
}

// ------------------------------------------------------------------ dispatch
struct MoePlan {
    int each, chunk, chunks;        // tokens per workgroup; assignments per chunk, 0 chunks: none
    size_t bytes;                   // of the workspace
};

MoePlan moe_plan(int64_t tokens, int64_t top_k, int64_t groups)
{
    MoePlan p = {};
    // As few tokens per workgroup as leave no more than 1024 workgroups, four per
    // CU, whose loads are all in flight (so 513 to 1024 of them for 1025 tokens
    // and more), and at most 64 assignments, past which there are more.  us on the
    // GPU, 4 choices of rows of 4096 into E4M3 / 8 choices of rows of 2048, by
    // tokens per workgroup:
    //     tokens         1            2            3            4            8
    //       1024    14.5  11.9   14.7  12.7   16.0  13.7   16.5  14.1
    //       1025    14.1  12.1   14.3  12.6   15.3  13.6   16.5  14.1
    //       1300    15.6  13.5   15.4  13.8   16.3  14.5   17.4  15.4
    //       1800    19.0  20.0   15.8  16.3   18.4  16.1   16.8  17.2   21.0  20.6
    //       2048    20.4  19.4   16.1  15.7   18.2  15.7   17.0  16.1   21.3  19.4
    //       4096    30.0  29.5   28.2  27.4   27.4  22.5   26.2  22.3   27.8  23.6
    //       8191    54.0  57.1   51.2  48.9   49.1  46.0   49.2  48.0   49.5  44.2
    // (2 choices of rows of 4096: 1100 tokens 11.6 and 10.8, 1800 19.4 and 15.1;
    // 9000 tokens of 4 choices, 8 per workgroup 58.4 and 4 54.2.)
    p.each = (int)std::max<int64_t>(1, std::min<int64_t>(cdiv(tokens, 1024), kMoeTopK / top_k));
    const int64_t total = tokens * top_k;
    // Up to 4096 assignments every workgroup goes through all of them (512
    // tokens with 8 choices 8.4 us, with a kernel that counts before it 9.3; 700
    // tokens 10.3 and 10.1).  Beyond, chunks of 1024 of them, at most 8192, of a
    // whole number of workgroups' assignments (4096 tokens with 2 choices 19.7
    // us, in chunks of 2048 21.6, of 4096 22.8).
    if (total > 4096) {
        const int64_t unit = p.each * top_k;
        p.chunk = (int)(cdiv(std::max<int64_t>(1024, cdiv(total, 8192)), unit) * unit);
        p.chunks = (int)cdiv(total, p.chunk);
        p.bytes = kSplitCounters * sizeof(unsigned) + (size_t)p.chunks * groups * sizeof(int);
    }
    return p;
}

int run_dispatch(const void *x, const int64_t *ids, int64_t tokens, int64_t top_k, int64_t groups, int64_t K, void *y,
                 void *y_scale, int out_kind, int32_t *offs, int32_t *pos, void *workspace, size_t workspace_bytes,
                 hipStream_t stream)
{
    const bool mx = out_kind == MXG_OUT_MXFP8 || out_kind == MXG_OUT_MXFP4;
    if (!offs || (tokens != 0 && (!x || !ids || !y || !pos || (mx && !y_scale))))
        return MXG_ERR_NULL;
    if (!mx && out_kind != MXG_OUT_BF16)
        return MXG_ERR_DTYPE;
    if (!moe_sizes_ok(tokens, top_k) || groups < 1 || groups > kMoeGroups || K < 1 || K > kMoeRow)
        return MXG_ERR_SHAPE;
    if (K % (mx ? 32 : 8))
        return MXG_ERR_K_ALIGN;
    if (((uintptr_t)x | (uintptr_t)y | (uintptr_t)workspace) & 15 || ((uintptr_t)ids & 7) ||
        ((uintptr_t)offs | (uintptr_t)pos) & 3)
        return MXG_ERR_PTR_ALIGN;
    const MoePlan plan = moe_plan(tokens, top_k, groups);
    if (plan.bytes && (!workspace || workspace_bytes < plan.bytes))
        return MXG_ERR_WORKSPACE;
    int rc = host_check_device();
    if (rc)
        return rc;
    MoeArgs a = {};
    a.x = (const uint16_t *)x;
    a.ids = (const long long *)ids;
    a.y = y;
    a.scales = (uint8_t *)y_scale;
    a.offs = offs;
    a.pos = pos;
    a.tokens = (int)tokens;
    a.top_k = (int)top_k;
    a.groups = (int)groups;
    a.K = (int)K;
    a.each = plan.each;
    a.chunk = plan.chunk;
    a.chunks = plan.chunks;
    a.summed = plan.chunks > kMoeChunks;
    a.per_row = fast_div((unsigned)(K / 8));
    // a few tokens' rows are shared by workgroups of 256 pieces
    a.segments = (int)std::max<int64_t>(1, std::min(cdiv(K / 8, 256), 256 / std::max<int64_t>(tokens, 1)));
    if (plan.bytes) {
        a.arrived = (unsigned *)workspace;
        a.counts = (int *)((uint8_t *)workspace + kSplitCounters * sizeof(unsigned));
        hipLaunchKernelGGL(mx_moe_count<1024>, dim3((unsigned)plan.chunks), dim3(1024), 0, stream, a);
        rc = host_hip_status(hipGetLastError());
        if (rc)
            return rc;
    }
    void (*fn)(MoeArgs) = out_kind == MXG_OUT_BF16    ? &mx_moe_dispatch_rows<OUT_BF16, 256>
                          : out_kind == MXG_OUT_MXFP8 ? &mx_moe_dispatch_rows<OUT_MX8, 256>
                                                      : &mx_moe_dispatch_rows<OUT_MX4, 256>;
    // (no tokens: one workgroup, for the experts' ends)
    const int64_t grid = std::max<int64_t>(1, cdiv(tokens, plan.each)) * a.segments;
    hipLaunchKernelGGL(fn, dim3((unsigned)grid), dim3(256), 0, stream, a);
    return host_hip_status(hipGetLastError());
}

// ------------------------------------------------------------------- combine
typedef void (*CombineFn)(CombineArgs);

template <int T, int OUT>
CombineFn combine_fn(int64_t top_k)
{
    return top_k == 1   ? &mx_moe_combine_rows<T, OUT, 1>
           : top_k == 2 ? &mx_moe_combine_rows<T, OUT, 2>
           : top_k <= 4 ? &mx_moe_combine_rows<T, OUT, 4>
                        : &mx_moe_combine_rows<T, OUT, 8>;
}

template <int T>
CombineFn combine_fn(int out_dtype, int64_t top_k)
{
    return out_dtype == MXG_OUT_BF16  ? combine_fn<T, OUT_BF16>(top_k)
           : out_dtype == MXG_OUT_F16 ? combine_fn<T, OUT_F16>(top_k)
                                      : combine_fn<T, OUT_F32>(top_k);
}

template <int T>
CombineFn grad_fn(int kind)
{
    return kind == MXG_OUT_MXFP8   ? &mx_moe_combine_grad_rows<T, OUT_MX8, 256>
           : kind == MXG_OUT_MXFP4 ? &mx_moe_combine_grad_rows<T, OUT_MX4, 256>
                                   : &mx_moe_combine_grad_rows<T, T, 256>;
}

CombineArgs combine_args(const void *y, const int32_t *pos, const float *weights, int64_t tokens, int64_t top_k,
                         int64_t rows, int64_t N, void *out)
{
    CombineArgs a = {};
    a.y = y;
    a.pos = pos;
    a.w = weights;
    a.out = out;
    a.tokens = (int)tokens;
    a.top_k = (int)top_k;
    a.rows = (int)rows;
    a.N = (int)N;
    a.n = (int)(tokens * (N / 8));
    a.per_row = fast_div((unsigned)(N / 8));
    return a;
}

bool combine_sizes_ok(int64_t tokens, int64_t top_k, int64_t rows, int64_t N)
{
    return moe_sizes_ok(tokens, top_k) && rows >= 0 && rows <= INT32_MAX && N >= 1 && N <= kMoeRow &&
           tokens * N < (int64_t)1 << 34;
}

int run_combine(const void *y, int y_dtype, const int32_t *pos, const float *weights, int64_t tokens, int64_t top_k,
                int64_t rows, int64_t N, void *out, int out_dtype, hipStream_t stream)
{
    if (tokens != 0 && (!pos || !out || (rows != 0 && !y)))
        return MXG_ERR_NULL;
    if (y_dtype < MXG_OUT_BF16 || y_dtype > MXG_OUT_F32 || out_dtype < MXG_OUT_BF16 || out_dtype > MXG_OUT_F32)
        return MXG_ERR_DTYPE;
    if (!combine_sizes_ok(tokens, top_k, rows, N))
        return MXG_ERR_SHAPE;
    if (N % 8)
        return MXG_ERR_K_ALIGN;
    if (((uintptr_t)y | (uintptr_t)out) & 15 || ((uintptr_t)pos | (uintptr_t)weights) & 3)
        return MXG_ERR_PTR_ALIGN;
    const int rc = host_check_device();
    if (rc || tokens == 0)
        return rc;
    const CombineArgs a = combine_args(y, pos, weights, tokens, top_k, rows, N, out);
    const CombineFn fn = y_dtype == MXG_OUT_BF16  ? combine_fn<OUT_BF16>(out_dtype, top_k)
                         : y_dtype == MXG_OUT_F16 ? combine_fn<OUT_F16>(out_dtype, top_k)
                                                  : combine_fn<OUT_F32>(out_dtype, top_k);
    hipLaunchKernelGGL(fn, dim3((unsigned)cdiv(a.n, 256)), dim3(256), 0, stream, a);
    return host_hip_status(hipGetLastError());
}

int run_combine_grad(const void *d_out, const void *y, int dtype, const int32_t *pos, const float *weights,
                     int64_t tokens, int64_t top_k, int64_t rows, int64_t N, void *d_y, void *d_y_scale, int d_y_kind,
                     float *d_weights, hipStream_t stream)
{
    const bool mx = d_y_kind == MXG_OUT_MXFP8 || d_y_kind == MXG_OUT_MXFP4;
    if (tokens != 0 && (!d_out || !pos || (rows != 0 && (!d_y || (d_weights && !y) || (mx && !d_y_scale)))))
        return MXG_ERR_NULL;
    if (dtype < MXG_OUT_BF16 || dtype > MXG_OUT_F32 || (!mx && d_y_kind != dtype))
        return MXG_ERR_DTYPE;
    if (!combine_sizes_ok(tokens, top_k, rows, N))
        return MXG_ERR_SHAPE;
    if (N % (mx ? 32 : 8))
        return MXG_ERR_K_ALIGN;
    if (((uintptr_t)d_out | (uintptr_t)y | (uintptr_t)d_y) & 15 ||
        ((uintptr_t)pos | (uintptr_t)weights | (uintptr_t)d_weights) & 3)
        return MXG_ERR_PTR_ALIGN;
    const int rc = host_check_device();
    if (rc || tokens == 0)
        return rc;
    CombineArgs a = combine_args(y, pos, weights, tokens, top_k, rows, N, d_y);
    a.d_out = d_out;
    a.scales = (uint8_t *)d_y_scale;
    a.d_w = d_weights;
    const CombineFn fn = dtype == MXG_OUT_BF16  ? grad_fn<OUT_BF16>(d_y_kind)
                         : dtype == MXG_OUT_F16 ? grad_fn<OUT_F16>(d_y_kind)
                                                : grad_fn<OUT_F32>(d_y_kind);
    hipLaunchKernelGGL(fn, dim3((unsigned)tokens), dim3(256), 0, stream, a);
    return host_hip_status(hipGetLastError());
}

}  // namespace

extern "C" {

size_t mx_moe_dispatch_workspace_bytes(int64_t tokens, int64_t top_k, int64_t groups)
{
    if (!moe_sizes_ok(tokens, top_k) || groups < 1 || groups > kMoeGroups)
        return 0;
    return moe_plan(tokens, top_k, groups).bytes;
}

int mx_moe_dispatch(const void *x, const int64_t *experts, int64_t tokens, int64_t top_k, int64_t groups, int64_t K,
                    void *y, void *y_scale, int out_kind, int32_t *offs, int32_t *pos, void *workspace,
                    size_t workspace_bytes, mxg_stream_t stream)
{
    return run_dispatch(x, experts, tokens, top_k, groups, K, y, y_scale, out_kind, offs, pos, workspace,
                        workspace_bytes, (hipStream_t)stream);
}

int mx_moe_combine(const void *y, int y_dtype, const int32_t *pos, const float *weights, int64_t tokens, int64_t top_k,
                   int64_t rows, int64_t N, void *out, int out_dtype, mxg_stream_t stream)
{
    return run_combine(y, y_dtype, pos, weights, tokens, top_k, rows, N, out, out_dtype, (hipStream_t)stream);
}

int mx_moe_combine_grad(const void *d_out, const void *y, int dtype, const int32_t *pos, const float *weights,
                        int64_t tokens, int64_t top_k, int64_t rows, int64_t N, void *d_y, void *d_y_scale,
                        int d_y_kind, float *d_weights, mxg_stream_t stream)
{
    return run_combine_grad(d_out, y, dtype, pos, weights, tokens, top_k, rows, N, d_y, d_y_scale, d_y_kind, d_weights,
                            (hipStream_t)stream);
}

}  // extern "C"
