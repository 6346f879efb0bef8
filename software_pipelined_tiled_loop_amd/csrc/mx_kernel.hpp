// mx_kernel.hpp -- products of weights in 4-bit blocks (MX4) with activations in
// 8- or 4-bit blocks (MX8, MX4), with the feed-forward operators' epilogue.
//
//     linear   Y = act(X W + b) + R          gated   H = act(X Wg + bg) * (X Wu + bu)
//
// Both operands lie with the contraction contiguous: X[M][K] and W[N][K], 32
// entries to a scale.  v_mfma_scale_f32_32x32x64_f8f6f4 multiplies blocks of
// either format, scales included; the weights go first, so that a lane's results
// are four consecutive columns of a row.  Its operands, of lane l: row l % 32;
// e2m1: the 16 bytes of block l / 32 of the step's two; e4m3: the 16-byte pieces
// l / 32 and 2 + l / 32 of the step's 64 bytes; and the scale of block l / 32.
#pragma once

#include "mx_format.hpp"

namespace pgemm {

typedef __attribute__((ext_vector_type(8))) int i32x8;
typedef __attribute__((ext_vector_type(16))) float f32x16;

struct MxArgs {
    const void* A;      // activations' codes and scales
    const void* SA;
    const void* B[2];   // weights' (gated: Wg, Wu)
    const void* SB[2];
    int64_t lda, lsa, ldb, lsb;  // bytes
    int filled;         // entries of a stored row: whole groups
    EpiArgs e;
};

// e2m1 by F, 32 x 32 x 64.
template <int F>
__device__ __forceinline__ void mx_mfma32(f32x16& acc, const i32x8& x, const i32x8& w, int sx, int sw) {
    acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, x, acc, 4, F == MX8 ? 0 : 4, 0, sw, 0, sx);
}
__device__ __forceinline__ i32x8 two_chunks(i32x4 a, i32x4 b) { return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7); }

// A wave's 32 x 32 outputs, operands straight from memory.
template <int D, int F, bool GATED>
__global__ void __launch_bounds__(64) mx_simple(MxArgs g) {
    const int tiles_n = (g.e.N + 31) / 32;
    const int m0 = (int)blockIdx.x / tiles_n * 32, n0 = (int)blockIdx.x % tiles_n * 32;
    const int lane = (int)threadIdx.x, r = lane & 31, half = lane >> 5;
    const int64_t m = min(m0 + r, g.e.M - 1), n = min(n0 + r, g.e.N - 1);  // rows beyond the edge feed nothing that is stored
    constexpr int NP = GATED ? 2 : 1;
    f32x16 acc[NP];
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[p][i] = 0.0f;
    const char* a = (const char*)g.A + m * g.lda;
    const uint8_t* sa = (const uint8_t*)g.SA + m * g.lsa;
    for (int s = 0; s < g.filled / 64; ++s) {
        i32x8 x;
        if constexpr (F == MX8) {
            x = two_chunks(*(const i32x4*)(a + s * 64 + half * 16), *(const i32x4*)(a + s * 64 + 32 + half * 16));
        } else {
            x = two_chunks(*(const i32x4*)(a + s * 32 + half * 16), i32x4{0, 0, 0, 0});
        }
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const i32x8 w = two_chunks(*(const i32x4*)((const char*)g.B[p] + n * g.ldb + s * 32 + half * 16), i32x4{0, 0, 0, 0});
            mx_mfma32<F>(acc[p], x, w, sa[2 * s + half], ((const uint8_t*)g.SB[p])[n * g.lsb + 2 * s + half]);
        }
    }
    const Epi<D, GATED> ep(g.e, m0, n0, 0, r, 0);
    with_act(g.e.act.kind, [&](auto kind) {
        constexpr int KIND = decltype(kind)::value;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int c = 8 * (i / 4) + 4 * half + i % 4;
            if (c < ep.valid(0)) ep.template put1<KIND>(0, c, acc[0][i], acc[NP - 1][i]);
        }
    });
}

}  // namespace pgemm
