// mx_variants.hpp -- the compiled kernels of the norm and of the microscaled operators (host side).
#pragma once

#include <hip/hip_runtime.h>

#include "linear_variants.hpp"
#include "mx_large.hpp"
#include "norm_kernel.hpp"

namespace pgemm {

// The norm's kernels by the groups of eight columns that they hold: threads of a row, groups a thread.
template <class Args>
struct NormVariant {
    int threads, groups;  // no groups: rows of any length
    hipError_t (*launch)(const Args&, int grid, hipStream_t);
};
template <class Args>
struct NormTable {
    const NormVariant<Args>* v;  // by what they hold
    int n;
};

// A kernel of the products.
struct MxVariant {
    int format, gated;
    int bm, bn, bk;  // bn: output columns of the tile
    int threads;
    int few;         // waves that share the contraction of a few-rows kernel, else 0
    int per_cu;      // workgroups that a CU holds
    hipError_t (*launch)(const MxArgs&, int grid, hipStream_t);
};

struct MxKernels {
    NormTable<NormArgs> norm;
    NormTable<NormGradArgs> norm_grad;
    hipError_t (*norm_join)(const NormSumArgs&, int grid, hipStream_t);
    hipError_t (*quantize)(const MxCopyArgs&, int format, bool columns, int grid, hipStream_t);
    hipError_t (*dequantize)(const MxCopyArgs&, int format, int grid, hipStream_t);
    const MxVariant* v;
    int n;
    LinLaunch join, join_gated;
    hipError_t (*rest)(const MxRestArgs&, bool gated, int grid, hipStream_t);
};

template <int D, int TPR, int CH>
hipError_t launch_norm(const NormArgs& a, int grid, hipStream_t s) {
    return lin_launch<NormArgs>(&rms_norm_rows<D, TPR, CH>, a, dim3(grid), norm_threads<TPR>, s);
}
template <int D, int TPR, int CH>
hipError_t launch_norm_grad(const NormGradArgs& a, int grid, hipStream_t s) {
    return lin_launch<NormGradArgs>(&rms_norm_grad<D, TPR, CH>, a, dim3(grid), norm_grad_threads<TPR>, s);
}
template <int D>
hipError_t launch_norm_join(const NormSumArgs& a, int grid, hipStream_t s) {
    return lin_launch<NormSumArgs>(&rms_norm_join<D>, a, dim3(grid), 1024, s);
}
template <int D>
hipError_t launch_norm_long(const NormArgs& a, int grid, hipStream_t s) {
    return lin_launch<NormArgs>(&rms_norm_long<D>, a, dim3(grid), 1024, s);
}
template <int D>
hipError_t launch_norm_grad_long(const NormGradArgs& a, int grid, hipStream_t s) {
    return lin_launch<NormGradArgs>(&rms_norm_grad_long<D>, a, dim3(grid), 1024, s);
}
template <int D, int F>
hipError_t launch_quantize(const MxCopyArgs& a, bool columns, int grid, hipStream_t s) {
    return columns ? lin_launch<MxCopyArgs>(&mx_quantize_columns<D, F>, a, dim3(grid), 512, s)
                   : lin_launch<MxCopyArgs>(&mx_quantize_rows<D, F>, a, dim3(grid), 256, s);
}
template <int D>
hipError_t launch_quantize_any(const MxCopyArgs& a, int format, bool columns, int grid, hipStream_t s) {
    return format == MX8 ? launch_quantize<D, MX8>(a, columns, grid, s) : launch_quantize<D, MX4>(a, columns, grid, s);
}
template <int D>
hipError_t launch_dequantize(const MxCopyArgs& a, int format, int grid, hipStream_t s) {
    return format == MX8 ? lin_launch<MxCopyArgs>(&mx_dequantize_rows<D, MX8>, a, dim3(grid), 256, s)
                         : lin_launch<MxCopyArgs>(&mx_dequantize_rows<D, MX4>, a, dim3(grid), 256, s);
}
inline hipError_t launch_mx_rest(const MxRestArgs& a, bool gated, int grid, hipStream_t s) {
    return gated ? lin_launch<MxRestArgs>(&mx_rest<true>, a, dim3(grid), 256, s)
                 : lin_launch<MxRestArgs>(&mx_rest<false>, a, dim3(grid), 256, s);
}
template <class C>
hipError_t launch_mx_tile(const MxArgs& a, int grid, hipStream_t s) {
    return lin_launch<MxArgs>(&mx_tile<C>, a, dim3(grid), C::NT, s);
}
template <class C>
hipError_t launch_mx_large(const MxArgs& a, int grid, hipStream_t s) {
    return lin_launch<MxArgs>(&mx_large<C>, a, dim3(grid), C::NT, s);
}
template <class C>
hipError_t launch_mx_few(const MxArgs& a, int grid, hipStream_t s) {
    return lin_launch<MxArgs>(&mx_few<C>, a, dim3(grid), C::NT, s);
}

#define NORM_VARIANT(D, TPR, CH) NormVariant<NormArgs>{TPR, CH, &launch_norm<D, TPR, CH>}
#define NORM_VARIANTS(D)                                                                                  \
    NORM_VARIANT(D, 64, 1), NORM_VARIANT(D, 64, 2), NORM_VARIANT(D, 256, 1), NORM_VARIANT(D, 512, 1),     \
        NORM_VARIANT(D, 512, 2), NORM_VARIANT(D, 1024, 2), NormVariant<NormArgs>{1024, 0, &launch_norm_long<D>}
#define NORM_GRAD_VARIANT(D, TPR, CH) NormVariant<NormGradArgs>{TPR, CH, &launch_norm_grad<D, TPR, CH>}
#define NORM_GRAD_VARIANTS(D)                                                                             \
    NORM_GRAD_VARIANT(D, 64, 1), NORM_GRAD_VARIANT(D, 128, 1), NORM_GRAD_VARIANT(D, 256, 1),              \
        NORM_GRAD_VARIANT(D, 512, 1), NORM_GRAD_VARIANT(D, 1024, 1), NORM_GRAD_VARIANT(D, 1024, 2),       \
        NormVariant<NormGradArgs>{1024, 0, &launch_norm_grad_long<D>}
#define MX_TILE_CFG(D, F, GATED, BM, BN, S, WGM, WGN) MxCfg<D, F, BM, BN, S, WGM, WGN, GATED != 0>
#define MX_TILE(D, F, GATED, BM, BN, S, WGM, WGN)                                                               \
    MxVariant {                                                                                                 \
        F, GATED, BM, GATED ? BN / 2 : BN, 128, 64 * WGM * WGN, 0,                                              \
            163840 / MX_TILE_CFG(D, F, GATED, BM, BN, S, WGM, WGN)::LDS,                                        \
            &launch_mx_tile<MX_TILE_CFG(D, F, GATED, BM, BN, S, WGM, WGN)>                                      \
    }
#define MX_LARGE(D, F, GATED)                                                                                   \
    MxVariant {                                                                                                 \
        F, GATED, 256, GATED ? 128 : 256, F == MX8 ? 128 : 256, 256, 0, 1, &launch_mx_large<MxLargeCfg<D, F, GATED != 0>> \
    }
#define MX_FEW_CFG(D, F, GATED, FM, FN, NW, S) MxFewCfg<D, F, FM, FN, NW, S, GATED != 0>
#define MX_FEW(D, F, GATED, FM, FN, NW, S)                                                                      \
    MxVariant {                                                                                                 \
        F, GATED, 16 * FM, 16 * FN, 256, 64 * NW, NW, 163840 / MX_FEW_CFG(D, F, GATED, FM, FN, NW, S)::LDS,     \
            &launch_mx_few<MX_FEW_CFG(D, F, GATED, FM, FN, NW, S)>                                              \
    }
// (fp32 outputs of MX8 are bound by making the values, and have no tiles of more rows:
// 256 rows of 4096 x 4096 34 us with tiles of 32 x 32 in two waves, 51 with 64 x 32)
#define MX_FEWS_WIDE(D, F, GATED)                                                                               \
    MX_FEW(D, F, GATED, 1, 1, 4, 3), MX_FEW(D, F, GATED, 1, 2, 4, 3), MX_FEW(D, F, GATED, 2, 2, 2, 3)
#define MX_FEWS(D, F, GATED)                                                                                    \
    MX_FEWS_WIDE(D, F, GATED), MX_FEW(D, F, GATED, 1, 4, 2, 3), MX_FEW(D, F, GATED, 3, 2, 2, 3),                 \
        MX_FEW(D, F, GATED, 4, 2, 2, 2)
#define MX_CLASS(D, F, GATED, DEEP)                                                                             \
    MX_LARGE(D, F, GATED), MX_TILE(D, F, GATED, 128, 128, DEEP, 2, 2), MX_FEWS(D, F, GATED)
// (fp32 outputs of MX8 activations: few rows alone, see MxFewCfg::WIDE; more rows go through linear_kernel)
#define MX_VARIANTS_MX4(D) MX_CLASS(D, MX4, 0, 4), MX_CLASS(D, MX4, 1, 4)
#define MX_VARIANTS(D) MX_CLASS(D, MX8, 0, 3), MX_CLASS(D, MX8, 1, 3), MX_VARIANTS_MX4(D)
#define MX_VARIANTS_F32 MX_FEWS_WIDE(DT_F32, MX8, 0), MX_FEWS_WIDE(DT_F32, MX8, 1), MX_VARIANTS_MX4(DT_F32)
#define MX_KERNELS(D, norms, grads, table)                                                                      \
    MxKernels {                                                                                                 \
        {norms, (int)(sizeof(norms) / sizeof(norms[0]))}, {grads, (int)(sizeof(grads) / sizeof(grads[0]))},     \
            &launch_norm_join<D>, &launch_quantize_any<D>, &launch_dequantize<D>, table,  \
            (int)(sizeof(table) / sizeof(table[0])), &lin_launch_join<D, false>, &lin_launch_join<D, true>, &launch_mx_rest \
    }

// Per type of the values, each in its own translation unit.
MxKernels mx_kernels_f32();
MxKernels mx_kernels_f16();
MxKernels mx_kernels_bf16();

}  // namespace pgemm
