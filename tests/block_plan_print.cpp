// block_plan_print.cpp -- prints what dense_gemm_06_amd/csrc/block_plan.h chooses (built by
// tests/test_block_plan.py as plain C++): a line of "mode rows products N K direct small tr
// may_split" on the input, a line of "kernel bm bn split rest" on the output.
#include <stdio.h>

#include "../dense_gemm_06_amd/csrc/block_plan.h"

int main() {
    long long mode, rows, n, N, K, direct, small, tr, may;
    while (scanf("%lld %lld %lld %lld %lld %lld %lld %lld %lld", &mode, &rows, &n, &N, &K, &direct, &small, &tr, &may) == 9) {
        const dg::BlockPlan p = dg::block_plan((dg::BlockMode)mode, rows, n, N, K, direct != 0, small != 0, (int)tr, may != 0);
        printf("%d %d %d %d %lld\n", p.kernel, p.bm, p.bn, p.split, mode == 0 ? (long long)dg::rest_rows(p, rows, N, K) : 0ll);
    }
    return 0;
}
