/* Drives the host half of the operators for drafted tokens and for experts
 * (csrc/mxdraft.hip, csrc/mxmoe.hip) under AddressSanitizer and
 * UndefinedBehaviorSanitizer, linked against a build without device code, as
 * serving_driver.c does for the operators around the products.  Built and run
 * by tests/test_sanitize_draft.py. */
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
    const int64_t *i64 = a;
    int32_t *i32 = a;
    float *f32 = a;
    const int64_t pages[] = {1, INT32_MAX}, sizes[] = {1, 16, 65536}, heads[] = {1, 3, 8, 4096};
    const int64_t dims[] = {32, 64, 128, 1024}, toks[] = {0, 1, 77, 4096, (int64_t)1 << 24, (int64_t)1 << 30, INT64_MAX, INT64_MIN};
    for (size_t i = 0; i < 2; ++i)
        for (size_t j = 0; j < 3; ++j)
            for (size_t h = 0; h < 4; ++h)
                for (size_t d = 0; d < 4; ++d)
                    for (size_t t = 0; t < 8; ++t)
                        for (int64_t group = 0; group <= 16; group = group ? group * 4 : 1) {
                            mxg_kv_cache_t c = {a, a, a, a, pages[i], sizes[j], heads[h], dims[d], (int)(t & 1)};
                            const int64_t st = heads[h] * dims[d], qh = heads[h] * group, qs = qh * dims[d];
                            int rc = mx_rope_cache_write(&c, a, a, a, a, qh, qs, qs, st, st, i64, i64, f32, 4096, dims[d] / 2, 0,
                                                         toks[t], NULL);
                            CHECK(STOPPED(rc) || rc == MXG_ERR_SHAPE);
                            if (!group)
                                continue;
                            for (int64_t seqs = 1; seqs <= 65536; seqs *= 256) {
                                const size_t need = mx_tree_attention_workspace_bytes(&c, seqs, toks[t], qh, toks[t]);
                                CHECK(need < ((size_t)1 << 32));
                                rc = mx_tree_attention(&c, a, qs, i32, i32, i32, 4, a, 2, seqs, toks[t], qh, toks[t], 0.1f,
                                                       seqs > 1 ? INT64_MAX : 0, a, MXG_OUT_BF16, NULL, a, need, NULL);
                                CHECK(STOPPED(rc) || rc == MXG_ERR_SHAPE);
                            }
                        }
    const int64_t ks[] = {INT64_MIN, 0, 1, 7, 64, 65, INT64_MAX}, groups[] = {0, 1, 60, 1024, INT64_MAX};
    const int64_t widths[] = {0, 32, 4096, 1 << 20, INT64_MAX};
    for (size_t t = 0; t < 8; ++t)
        for (size_t k = 0; k < 7; ++k)
            for (size_t w = 0; w < 5; ++w) {
                for (size_t g = 0; g < 5; ++g) {
                    const size_t need = mx_moe_dispatch_workspace_bytes(toks[t], ks[k], groups[g]);
                    CHECK(need < ((size_t)1 << 32));
                    for (int kind = -1; kind < 6; ++kind) {
                        int rc = mx_moe_dispatch(a, i64, toks[t], ks[k], groups[g], widths[w], a, a, kind, i32, i32, a, need, NULL);
                        CHECK(STOPPED(rc) || rc == MXG_ERR_SHAPE || rc == MXG_ERR_DTYPE || rc == MXG_ERR_K_ALIGN);
                    }
                }
                for (int kind = -1; kind < 6; ++kind) {
                    int rc = mx_moe_combine(a, kind, i32, f32, toks[t], ks[k], INT32_MAX, widths[w], a, 2, NULL);
                    CHECK(STOPPED(rc) || rc == MXG_ERR_SHAPE || rc == MXG_ERR_DTYPE || rc == MXG_ERR_K_ALIGN || (rc == MXG_OK && toks[t] == 0));
                    rc = mx_moe_combine_grad(a, a, 1, i32, f32, toks[t], ks[k], INT32_MAX, widths[w], a, a, kind, f32, NULL);
                    CHECK(STOPPED(rc) || rc == MXG_ERR_SHAPE || rc == MXG_ERR_DTYPE || rc == MXG_ERR_K_ALIGN || (rc == MXG_OK && toks[t] == 0));
                }
            }
    CHECK(mx_moe_dispatch(a, i64, 6000, 2, 8, 64, a, a, MXG_OUT_MXFP8, i32, i32, NULL, 0, NULL) == MXG_ERR_WORKSPACE);
    CHECK(mx_rope_cache_write(NULL, a, a, a, a, 1, 128, 128, 128, 128, i64, i64, f32, 1, 16, 0, 1, NULL) == MXG_ERR_NULL);
    mxg_kv_cache_t c = {a, a, a, a, 10, 16, 2, 128, 0};
    CHECK(mx_tree_attention(&c, a, 256, i32, i32, i32, INT64_MAX, a, 1, 1, 1, 2, 1, 0.1f, 0, a, 0, NULL, NULL, 0, NULL) == MXG_ERR_SHAPE);
    CHECK(mx_tree_attention(&c, a, 256, i32, i32, i32, 4, a, INT64_MAX, 1, 1, 2, 1, 0.1f, 0, a, 0, NULL, NULL, 0, NULL) == MXG_ERR_SHAPE);
    CHECK(mx_tree_attention(&c, a, 256, i32, i32, i32, 4, a, 1, 1, 1, 2, 1, NAN, 0, a, 0, NULL, NULL, 0, NULL) == MXG_ERR_CONFIG);
    puts("draft sanitizer run ok");
    return 0;
}
