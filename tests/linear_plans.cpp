// The planner of the feed-forward operators on the host (no GPU).  Prints the
// compiled variants, one a line, as
//     variant <dtype> <index> <layout> <gated> <few> <rows of the tile> <columns> <workgroups a CU>
// and then, for each line "<dtype> <product> <M> <N> <K>" of the input, the choice, as
//     plan <index> <splits> <threads of the launch>
// or "plan -1" where no launch holds it.
// Products: 0 1 linear, W [K][N] or W [N][K]; 2 3 gated; 4 5 dX of linear; 6 7 of gated;
// 8 9 dW of linear, stored K x N or N x K; 10 11 of gated.
#include "../software_pipelined_tiled_loop_amd/csrc/linear_abi.cpp"

static Shape product(int kind, int64_t M, int64_t N, int64_t K) {
    const int order = kind & 1, pair = (kind >> 1) & 1;
    return kind < 4 ? forward_shape(M, N, K, order, pair)
           : kind < 8 ? dx_shape(M, N, K, order, 1 + pair)
                      : dw_shape(M, N, K, order, 1 + pair);
}

int main() {
    for (int d : {PGEMM_F32, PGEMM_F16, PGEMM_BF16}) {
        const LinKernels k = kernels_for(d);
        for (int i = 0; i < k.n; ++i)
            std::printf("variant %d %d %d %d %d %d %d %d\n", d, i, k.v[i].lay, k.v[i].gated, k.v[i].few, k.v[i].bm,
                        k.v[i].bn, k.v[i].per_cu);
    }
    int dtype, kind;
    long long M, N, K;
    while (std::scanf("%d %d %lld %lld %lld", &dtype, &kind, &M, &N, &K) == 5) {
        const Plan p = search_plan(product(kind, M, N, K), dtype);
        if (!p.v) {
            std::printf("plan -1\n");
            continue;
        }
        const long long grid = round_up(p.tiles_m * p.tiles_n * product(kind, M, N, K).outs * p.splits, 8);
        std::printf("plan %d %lld %lld\n", (int)(p.v - kernels_for(dtype).v), (long long)p.splits, grid * p.v->threads);
    }
    return 0;
}
