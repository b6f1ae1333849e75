// mx_serve.hpp -- host helpers of the operators around the products, shared by
// their translation units: sizes, divisors, the checks of a cache.
#pragma once

#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/mxgemm.h"
#include "mx_cache.hpp"
#include "mx_host.hpp"

namespace mxg {
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

// A launch has fewer than 2^32 threads.
constexpr int64_t kMaxThreads = UINT32_MAX;

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

}  // namespace
}  // namespace mxg
