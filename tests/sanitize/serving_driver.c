/* Drives the host half of the operators around the products
 * (csrc/mxserve.hip) under AddressSanitizer and UndefinedBehaviorSanitizer,
 * linked against a build without device code, as abi_driver.c does for the
 * products: refusals, workspace sizes over a grid of shapes, and valid calls
 * up to the device check.  Built and run by tests/test_sanitize_serving.py. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "../../include/mxgemm.h"

#define CHECK(cond)                                                    \
    do {                                                               \
        if (!(cond)) {                                                 \
            fprintf(stderr, "check failed: %s (line %d)\n", #cond, __LINE__); \
            return 1;                                                  \
        }                                                              \
    } while (0)

#define STOPPED(rc) ((rc) == MXG_ERR_DEVICE || (rc) == MXG_ERR_HIP)

int main(void)
{
    void *a = (void *)0x10000;      /* aligned, never dereferenced on the host */
    /* RMSNorm: every output kind and thread count */
    const int64_t Ks[] = {32, 512, 544, 4096, 6144, 16384, 16416, 65536};
    for (size_t k = 0; k < sizeof Ks / sizeof Ks[0]; ++k)
        for (int kind = 0; kind < 5; ++kind)
            CHECK(STOPPED(mx_rmsnorm(a, a, a, a, a, a, 3, Ks[k], 1e-6f, kind, NULL)));
    CHECK(mx_rmsnorm(a, NULL, NULL, NULL, a, NULL, 3, 64, 0.0f, MXG_OUT_MXFP8, NULL) == MXG_ERR_NULL);
    CHECK(mx_rmsnorm(a, NULL, NULL, NULL, a, NULL, 3, 64, NAN, MXG_OUT_BF16, NULL) == MXG_ERR_CONFIG);
    CHECK(mx_rmsnorm(a, NULL, NULL, NULL, a, NULL, INT64_MAX, 64, 0.0f, MXG_OUT_BF16, NULL) == MXG_ERR_SHAPE);
    CHECK(mx_rmsnorm(a, NULL, NULL, NULL, a, NULL, INT64_MIN, 64, 0.0f, MXG_OUT_BF16, NULL) == MXG_ERR_SHAPE);
    /* the cache and attention over a grid of shapes */
    const int64_t pages[] = {1, 1000, INT32_MAX}, sizes[] = {1, 16, 256, 65536}, heads[] = {1, 3, 8, 4096};
    const int64_t dims[] = {32, 64, 128, 1024}, toks[] = {0, 1, 77, 4096, (int64_t)1 << 30, INT64_MAX};
    for (size_t i = 0; i < 3; ++i)
        for (size_t j = 0; j < 4; ++j)
            for (size_t h = 0; h < 4; ++h)
                for (size_t d = 0; d < 4; ++d)
                    for (size_t t = 0; t < 6; ++t)
                        for (int fp4 = 0; fp4 < 2; ++fp4) {
                            mxg_kv_cache_t c = {a, a, a, a, pages[i], sizes[j], heads[h], dims[d], fp4};
                            const int64_t st = heads[h] * dims[d];
                            int rc = mx_kv_cache_write(&c, a, a, st, st, (int64_t *)a, toks[t], NULL);
                            CHECK(STOPPED(rc) || rc == MXG_ERR_SHAPE);
                            rc = mx_kv_cache_read(&c, a, a, st, st, (int64_t *)a, toks[t], NULL);
                            CHECK(STOPPED(rc) || rc == MXG_ERR_SHAPE);
                            for (int64_t group = 1; group <= 16; group *= 4)
                                for (int64_t seqs = 1; seqs <= 65536; seqs *= 256) {
                                    const int64_t qh = heads[h] * group;
                                    const size_t need = mx_paged_attention_workspace_bytes(&c, seqs, toks[t], qh, toks[t]);
                                    CHECK(need < ((size_t)1 << 32));
                                    rc = mx_paged_attention(&c, a, qh * dims[d], (int32_t *)a, (int32_t *)a, (int32_t *)a, 4,
                                                            seqs, toks[t], qh, toks[t], 0.1f, 1, 0, a, MXG_OUT_BF16, NULL, a,
                                                            need, NULL);
                                    CHECK(STOPPED(rc) || rc == MXG_ERR_SHAPE);
                                }
                        }
    mxg_kv_cache_t c = {a, a, a, a, 10, 16, 2, 128, 0};
    CHECK(mx_paged_attention(&c, a, 256, (int32_t *)a, (int32_t *)a, (int32_t *)a, INT64_MAX, 1, 1, 2, 1, 0.1f, 1, 0, a, 0,
                             NULL, NULL, 0, NULL) == MXG_ERR_SHAPE);
    CHECK(mx_paged_attention(&c, a, 256, (int32_t *)a, (int32_t *)a, (int32_t *)a, 4, 1, 1, 2, 1, -INFINITY, 1, 0, a, 0,
                             NULL, NULL, 0, NULL) == MXG_ERR_CONFIG);
    CHECK(mx_paged_attention(NULL, a, 256, (int32_t *)a, (int32_t *)a, (int32_t *)a, 4, 1, 1, 2, 1, 0.1f, 1, 0, a, 0, NULL,
                             NULL, 0, NULL) == MXG_ERR_NULL);
    c.page_size = 48;
    CHECK(mx_kv_cache_write(&c, a, a, 256, 256, (int64_t *)a, 1, NULL) == MXG_ERR_SHAPE);
    puts("serving sanitizer run ok");
    return 0;
}
