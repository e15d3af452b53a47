// Host build of the choice of kernel for e4m3 products (quantized_gemv_amd/csrc/
// qg_fp8_plan.h) for CPU tests: reads lines "m n k yt" from stdin and prints, for
// each, whether a stream runs, its kind, parts of k, columns of 256 x 256 tiles
// before the second kind takes over, and that kind.
#include <cstdio>

#include "../../quantized_gemv_amd/csrc/qg_fp8_plan.h"

int main() {
    long m, n, k;
    int yt;
    while (scanf("%ld %ld %ld %d", &m, &n, &k, &yt) == 4) {
        const qg::Fp8Plan p = qg::plan_fp8(m, n, k, yt);
        printf("%d %d %d %ld %d\n", p.stream ? 1 : 0, p.kind, p.parts, (long)p.cols, p.rest);
    }
    return 0;
}
