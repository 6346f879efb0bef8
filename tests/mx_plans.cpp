// The planner of the microscaled products on the host (no GPU).  Prints the compiled
// variants, one a line, as
//     variant <dtype> <index> <format> <gated> <few> <rows of the tile> <columns> <workgroups a CU>
// and then, for each line "<dtype> <format> <gated> <M> <N> <K>" of the input, the choice, as
//     plan <index> <splits> <threads of the launch>
// or "plan -1" where another way or no launch holds it.
#include "../software_pipelined_tiled_loop_amd/csrc/mx_abi.cpp"

int main() {
    for (int d : {PGEMM_F32, PGEMM_F16, PGEMM_BF16}) {
        const MxKernels k = kernels_for(d);
        for (int i = 0; i < k.n; ++i)
            std::printf("variant %d %d %d %d %d %d %d %d\n", d, i, k.v[i].format, k.v[i].gated, k.v[i].few, k.v[i].bm,
                        k.v[i].bn, k.v[i].per_cu);
    }
    int dtype, format, gated;
    long long M, N, K;
    while (std::scanf("%d %d %d %lld %lld %lld", &dtype, &format, &gated, &M, &N, &K) == 6) {
        Plan p;
        std::memset(&p, 0, sizeof(p));
        const int64_t need = product_workspace(M, N, K, format, dtype, gated ? 2 : 1, p);
        if (need < 0 || !p.v) {
            std::printf("plan -1\n");
            continue;
        }
        const long long grid = round_up(p.tiles_m * p.tiles_n * p.splits, 8);
        std::printf("plan %d %lld %lld\n", (int)(p.v - kernels_for(dtype).v), (long long)p.splits, grid * p.v->threads);
    }
    return 0;
}
