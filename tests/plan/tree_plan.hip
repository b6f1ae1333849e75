// Prints the rows per tile that mx_tree_attention takes for each line of sizes
// on its input, from the library's own plan (host code only; built and run by
// tests/test_tree_plan_host.py).
#include <hip/hip_runtime.h>
#include <stdio.h>

#include "../../block_scaled_precision_mm_amd/csrc/mx_attn_host.hpp"

int main(void)
{
    long long seqs, tokens, heads, group, dim, page, width, window, max_new;
    while (scanf("%lld %lld %lld %lld %lld %lld %lld %lld %lld", &seqs, &tokens, &heads, &group, &dim, &page, &width, &window, &max_new) == 9) {
        const mxg::AttnPlan p = mxg::tree_plan(seqs, tokens, heads, group, dim, max_new, mxg::tree_keys(width, page, window, max_new));
        printf("%d\n", mxg::kAttnBM[p.which[0]]);
    }
    return 0;
}
