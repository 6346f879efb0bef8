// linear_variants.hpp -- the compiled kernels of the feed-forward operators (host side).
#pragma once

#include <hip/hip_runtime.h>
#include "linear_kernel.hpp"

namespace pgemm {

typedef hipError_t (*LinLaunch)(const LinArgs&, int grid, hipStream_t);

// Operand layouts of a product: activations times W [K][N] or W [N][K], and
// X^T times dZ.
enum LinLay : int { LIN_KX = 0, LIN_KK = 1, LIN_XX = 2 };

struct LinVariant {
    int lay, gated;
    int bm, bn, bk;  // bn: output columns of the tile
    int threads;     // of a workgroup
    int few;         // waves that share the K tiles of a few-rows kernel, else 0
    int per_cu;      // workgroups whose LDS a CU holds
    int (*ring_tiles)(int64_t K, int64_t rows, int64_t lda, int64_t cols, int64_t ldb);
    LinLaunch launch;
};

struct LinKernels {
    const LinVariant* v;
    int n;
    LinLaunch join, join_gated;
    hipError_t (*slope)(const SlopeArgs&, bool gated, int pass, int grid, hipStream_t);
    hipError_t (*colsum)(const SumArgs&, int grid, hipStream_t);
};

template <class Args>
hipError_t lin_launch(void (*kernel)(Args), const Args& a, dim3 grid, int threads, hipStream_t s) {
    Args arg = a;
    void* args[] = {&arg};
    return hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, dim3(threads), args, 0, s);
}

template <class C>
hipError_t lin_launch_tile(const LinArgs& a, int grid, hipStream_t s) {
    return lin_launch<LinArgs>(&linear_kernel<C>, a, dim3(grid), C::NT, s);
}
template <class C>
hipError_t lin_launch_few(const LinArgs& a, int grid, hipStream_t s) {
    return lin_launch<LinArgs>(&linear_few<C>, a, dim3(grid), C::NT, s);
}
template <class C>
int lin_ring_tiles(int64_t K, int64_t rows, int64_t lda, int64_t cols, int64_t ldb) {
    const int a = C::OA::ring_tiles(K, rows, lda), b = C::OB::ring_tiles(K, cols, ldb);
    return a < b ? a : b;
}
template <int D, bool GATED>
hipError_t lin_launch_join(const LinArgs& a, int grid, hipStream_t s) {
    return lin_launch<LinArgs>(&linear_join<D, GATED>, a, dim3(grid), kJoinCols / 8, s);
}
template <int D, int PASS>
hipError_t lin_launch_pass(const SlopeArgs& a, bool gated, int grid, hipStream_t s) {
    return gated ? lin_launch<SlopeArgs>(&linear_slope<D, true, PASS>, a, dim3(grid), 256, s)
                 : lin_launch<SlopeArgs>(&linear_slope<D, false, PASS>, a, dim3(grid), 256, s);
}
template <int D>
hipError_t lin_launch_slope(const SlopeArgs& a, bool gated, int pass, int grid, hipStream_t s) {
    if constexpr (D != DT_F16)  // bf16 and fp32 have the range of the values
        return lin_launch_pass<D, SLOPE_PLAIN>(a, gated, grid, s);
    else if (pass == SLOPE_SCALED)
        return lin_launch_pass<D, SLOPE_SCALED>(a, gated, grid, s);
    else
        return lin_launch_pass<D, SLOPE_RANGE>(a, gated, grid, s);
}
template <int D>
hipError_t lin_launch_colsum(const SumArgs& a, int grid, hipStream_t s) {
    return lin_launch<SumArgs>(&linear_colsum<D>, a, dim3(grid, a.planes + (a.rows ? 1 : 0)), 1024, s);
}

constexpr int lin_la(int lay) { return lay == LIN_XX ? LAY_X : LAY_K; }
constexpr int lin_lb(int lay) { return lay == LIN_KK ? LAY_K : LAY_X; }

#define LIN_CFG(D, LAY, GATED, BM, BN, BK, S, WGM, WGN) \
    LinCfg<D, lin_la(LAY), lin_lb(LAY), BM, BN, BK, S, WGM, WGN, GATED != 0>
#define LIN_VARIANT(D, LAY, GATED, BM, BN, BK, S, WGM, WGN)                                 \
    LinVariant {                                                                            \
        LAY, GATED, BM, GATED ? BN / 2 : BN, BK, 64 * WGM * WGN, 0,                         \
            163840 / LIN_CFG(D, LAY, GATED, BM, BN, BK, S, WGM, WGN)::LDS,                  \
            &lin_ring_tiles<LIN_CFG(D, LAY, GATED, BM, BN, BK, S, WGM, WGN)>,               \
            &lin_launch_tile<LIN_CFG(D, LAY, GATED, BM, BN, BK, S, WGM, WGN)>               \
    }
// A tile class in every layout.
#define LIN_CLASS(D, BM, BN, BK, S, WGM, WGN)                                                           \
    LIN_VARIANT(D, LIN_KX, 0, BM, BN, BK, S, WGM, WGN), LIN_VARIANT(D, LIN_KK, 0, BM, BN, BK, S, WGM, WGN), \
        LIN_VARIANT(D, LIN_KX, 1, BM, BN, BK, S, WGM, WGN), LIN_VARIANT(D, LIN_KK, 1, BM, BN, BK, S, WGM, WGN), \
        LIN_VARIANT(D, LIN_XX, 0, BM, BN, BK, S, WGM, WGN)
// A few-rows kernel of 16 FM rows by NCOL columns (gated: of both weights), NW
// waves with rings of S stages.
#define LIN_FEW_CFG(D, LAY, GATED, FM, NCOL, NW, S) FewCfg<D, lin_la(LAY), lin_lb(LAY), FM, NCOL, NW, S, GATED != 0>
#define LIN_FEW(D, LAY, GATED, FM, NCOL, NW, S)                                                      \
    LinVariant {                                                                                     \
        LAY, GATED, 16 * FM, GATED ? NCOL / 2 : NCOL, LIN_FEW_CFG(D, LAY, GATED, FM, NCOL, NW, S)::BK, 64 * NW, NW, \
            163840 / LIN_FEW_CFG(D, LAY, GATED, FM, NCOL, NW, S)::LDS,                               \
            &lin_ring_tiles<LIN_FEW_CFG(D, LAY, GATED, FM, NCOL, NW, S)>,                            \
            &lin_launch_few<LIN_FEW_CFG(D, LAY, GATED, FM, NCOL, NW, S)>                             \
    }
// The few-rows kernels of every layout, of 16, 32 and 64 rows.  Rings of 64 to
// 128 KiB a workgroup: measured on one token to 16384 x 4096 gated, two
// workgroups a CU with short rings stream faster (5.0 TB/s) than one with all
// of the CU's LDS (4.2 TB/s).  Sixteen columns a tile (W [N][K] only, where they
// are whole rows) give 256 workgroups at N = 4096 without splitting K: 8.2 us
// for one token by 4096 x 4096, 11.9 us on 64 columns in four splits.
#define LIN_FEW_CLASSES(D)                                                                                    \
    LIN_FEW(D, LIN_KK, 0, 1, 16, 8, 3), LIN_FEW(D, LIN_KK, 0, 2, 16, 4, 4), LIN_FEW(D, LIN_KK, 0, 4, 16, 4, 3), \
        LIN_FEW(D, LIN_KK, 0, 1, 64, 4, 2), LIN_FEW(D, LIN_KK, 0, 2, 64, 4, 2),                               \
        LIN_FEW(D, LIN_KK, 0, 4, 64, 4, 2), LIN_FEW(D, LIN_KX, 0, 1, 64, 4, 2),                               \
        LIN_FEW(D, LIN_KX, 0, 2, 64, 4, 2), LIN_FEW(D, LIN_KX, 0, 4, 64, 4, 2),                               \
        LIN_FEW(D, LIN_KK, 1, 1, 128, 2, 2), LIN_FEW(D, LIN_KK, 1, 1, 64, 4, 2),                              \
        LIN_FEW(D, LIN_KK, 1, 2, 64, 4, 2), LIN_FEW(D, LIN_KK, 1, 4, 64, 4, 2),                               \
        LIN_FEW(D, LIN_KX, 1, 1, 64, 4, 2), LIN_FEW(D, LIN_KX, 1, 1, 128, 2, 2),                              \
        LIN_FEW(D, LIN_KX, 1, 2, 64, 4, 2), LIN_FEW(D, LIN_KX, 1, 4, 64, 4, 2), LIN_FEW(D, LIN_XX, 0, 4, 64, 4, 2)
#define LIN_KERNELS(D, table)                                                                              \
    LinKernels {                                                                                           \
        table, (int)(sizeof(table) / sizeof(table[0])), &lin_launch_join<D, false>, &lin_launch_join<D, true>, \
            &lin_launch_slope<D>, &lin_launch_colsum<D>                                                    \
    }

// Per-dtype kernels, each in its own translation unit.
LinKernels linear_kernels_f32();
LinKernels linear_kernels_f16();
LinKernels linear_kernels_bf16();

}  // namespace pgemm
