// norm_kernel.hpp -- the root-mean-square norm with the residual's addition, and
// its backward pass, on gfx950.
//
//     h = x + r,  s = 1 / sqrt(mean(h^2) + eps),  y = h s w
//     backward, with g = dy w:  dx = dh + s g - h s^3 mean(g h),  dw = sum over rows of dy h s
//
// Both are bound by memory: a row's values are read once, held in registers over
// the sums, and written once.
#pragma once

#include "mx_format.hpp"

namespace pgemm {

struct NormArgs {
    const void* X;
    const void* R;   // residual; null: none
    const void* w;   // gain; null: one
    void* H;         // x + r; null: not kept
    void* Y;         // null: none
    void* Q;         // MX codes and scales; null: none
    void* S;
    int64_t ldx, ldr, ldh, ldy, ldq, lds;
    float eps;
    int M, N;
    int filled;      // entries of a row that are written: stored MX entries, or N
    int y_f32;       // Y is fp32 (else X's type)
    int format;      // MxFormat of Q
};

// Sum over the wave, in every lane.
__device__ __forceinline__ float wave_sum(float x) {
    const auto dpp = [](float v, auto ctrl) {
        return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v),
                                                                    decltype(ctrl)::value, 0xf, 0xf, true));
    };
    x += dpp(x, KindC<0xB1>{});   // lane ^ 1
    x += dpp(x, KindC<0x4E>{});   // lane ^ 2
    x += dpp(x, KindC<0x141>{});  // the other four of eight
    x += dpp(x, KindC<0x140>{});  // the other eight of sixteen
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
}
// Sums of P values over the TPR threads of a row; `red` has P x 16 floats, free to be written.
template <int TPR, int P>
__device__ __forceinline__ void row_sums(float (&x)[P], float* red) {
#pragma unroll
    for (int p = 0; p < P; ++p) x[p] = wave_sum(x[p]);
    if constexpr (TPR > 64) {
        const int wave = (int)threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int p = 0; p < P; ++p) red[p * 16 + wave] = x[p];
        }
        __syncthreads();
#pragma unroll
        for (int p = 0; p < P; ++p) {
            x[p] = red[p * 16];
#pragma unroll
            for (int i = 1; i < TPR / 64; ++i) x[p] += red[p * 16 + i];
        }
    }
}
__device__ __forceinline__ float inverse_rms(float squares, int N, float eps) {
    return 1.0f / __builtin_sqrtf(squares / (float)N + eps);
}

// Rows of a workgroup: one for each TPR threads, at least one wave's.
template <int TPR>
constexpr int norm_threads = TPR < 256 ? 256 : TPR;

// TPR threads a row, CH groups of eight columns a thread.
template <int D, int TPR, int CH>
__global__ void __launch_bounds__(norm_threads<TPR>) rms_norm_rows(NormArgs g) {
    typedef typename Elem<D>::type T;
    constexpr int RPW = norm_threads<TPR> / TPR;
    __shared__ float red[2][16];
    const int t = (int)threadIdx.x % TPR;
    int turn = 0;
    for (int64_t row = (int64_t)blockIdx.x * RPW + threadIdx.x / TPR; row < g.M; row += (int64_t)gridDim.x * RPW) {
        f32x8 v[CH];
        float sum[1] = {0.0f};
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int n = (c * TPR + t) * 8;
            v[c] = load8_at((const T*)g.X + row * g.ldx + n, g.N - n);
        }
        if (g.R) {
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int n = (c * TPR + t) * 8;
                v[c] += load8_at((const T*)g.R + row * g.ldr + n, g.N - n);
            }
        }
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[0] = fmaf(v[c][i], v[c][i], sum[0]);
        row_sums<TPR, 1>(sum, red[turn]);
        turn ^= 1;
        const float s = inverse_rms(sum[0], g.N, g.eps);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int n = (c * TPR + t) * 8;
            if (n >= g.filled) continue;
            const int valid = g.N - n;
            if (g.H) store8_at((T*)g.H + row * g.ldh + n, v[c], valid);
            f32x8 y = v[c] * s;
            if (g.w) y *= load8_at((const T*)g.w + n, valid);
            if (g.Y) {
                if (g.y_f32) store8_at((float*)g.Y + row * g.ldy + n, y, valid);
                else store8_at((T*)g.Y + row * g.ldy + n, y, valid);
            }
            if (g.Q) {
                char* q = (char*)g.Q + row * g.ldq;
                uint8_t* sc = (uint8_t*)g.S + row * g.lds;
                if (g.format == MX8) mx_put8<MX8>(q, sc, n, y);
                else mx_put8<MX4>(q, sc, n, y);
            }
        }
    }
}

// Rows too long for the registers: read twice.
template <int D>
__global__ void __launch_bounds__(1024) rms_norm_long(NormArgs g) {
    typedef typename Elem<D>::type T;
    __shared__ float red[2][16];
    int turn = 0;
    for (int64_t row = blockIdx.x; row < g.M; row += gridDim.x) {
        const auto h8 = [&](int n) {
            f32x8 v = load8_at((const T*)g.X + row * g.ldx + n, g.N - n);
            if (g.R) v += load8_at((const T*)g.R + row * g.ldr + n, g.N - n);
            return v;
        };
        float sum[1] = {0.0f};
        for (int n = (int)threadIdx.x * 8; n < g.N; n += 8192) {
            const f32x8 v = h8(n);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[0] = fmaf(v[i], v[i], sum[0]);
        }
        row_sums<1024, 1>(sum, red[turn]);
        turn ^= 1;
        const float s = inverse_rms(sum[0], g.N, g.eps);
        for (int n = (int)threadIdx.x * 8; n < g.filled; n += 8192) {
            const int valid = g.N - n;
            const f32x8 v = h8(n);
            if (g.H) store8_at((T*)g.H + row * g.ldh + n, v, valid);
            f32x8 y = v * s;
            if (g.w) y *= load8_at((const T*)g.w + n, valid);
            if (g.Y) {
                if (g.y_f32) store8_at((float*)g.Y + row * g.ldy + n, y, valid);
                else store8_at((T*)g.Y + row * g.ldy + n, y, valid);
            }
            if (g.Q) {
                char* q = (char*)g.Q + row * g.ldq;
                uint8_t* sc = (uint8_t*)g.S + row * g.lds;
                if (g.format == MX8) mx_put8<MX8>(q, sc, n, y);
                else mx_put8<MX4>(q, sc, n, y);
            }
        }
    }
}

struct NormGradArgs {
    const void* dY;
    const void* H;
    const void* w;   // null: one
    const void* dH;  // the gradient that arrives at h; null: none
    void* dX;        // null: not computed
    float* sums;     // [blocks][np8]: sums of dy h s over a block's rows; null: none
    int64_t lddy, ldh, lddh, lddx;
    float eps;
    int M, N, np8;
    int rows;        // of a block
};

// A block of `rows` rows; its columns' sums of dy h s stay in registers.
template <int D, int TPR, int CH>
__global__ void __launch_bounds__(norm_threads<TPR>) rms_norm_grad(NormGradArgs g) {
    typedef typename Elem<D>::type T;
    constexpr int RPW = norm_threads<TPR> / TPR;
    __shared__ float red[2][32];
    __shared__ f32x8 join[RPW > 1 ? norm_threads<TPR> : 1];
    const int t = (int)threadIdx.x % TPR, first = (int)blockIdx.x * g.rows;
    const int end = first + g.rows < g.M ? first + g.rows : g.M;
    f32x8 w[CH], dw[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int n = (c * TPR + t) * 8;
        dw[c] = zero8();
        w[c] = zero8() + 1.0f;
        if (g.w) w[c] = load8_at((const T*)g.w + n, g.N - n);
    }
    int turn = 0;
    for (int64_t row = first + (int)threadIdx.x / TPR; row < end; row += RPW) {
        f32x8 h[CH], dy[CH];
        float sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int n = (c * TPR + t) * 8;
            h[c] = load8_at((const T*)g.H + row * g.ldh + n, g.N - n);
            dy[c] = load8_at((const T*)g.dY + row * g.lddy + n, g.N - n);
        }
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                sum[0] = fmaf(h[c][i], h[c][i], sum[0]);
                sum[1] = fmaf(dy[c][i] * w[c][i], h[c][i], sum[1]);
            }
        row_sums<TPR, 2>(sum, red[turn]);
        turn ^= 1;
        const float s = inverse_rms(sum[0], g.N, g.eps), m = s * (s * (sum[1] / (float)g.N));
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int n = (c * TPR + t) * 8;
            if (n >= g.N) continue;
            const f32x8 hs = h[c] * s;
            dw[c] += dy[c] * hs;
            if (g.dX) {
                f32x8 d = dy[c] * w[c] * s - hs * m;
                if (g.dH) d += load8_at((const T*)g.dH + row * g.lddh + n, g.N - n);
                store8_at((T*)g.dX + row * g.lddx + n, d, g.N - n);
            }
        }
    }
    if (!g.sums) return;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int n = (c * TPR + t) * 8;
        if constexpr (RPW > 1) {
            __syncthreads();
            join[threadIdx.x] = dw[c];
            __syncthreads();
            if (threadIdx.x >= TPR) continue;
#pragma unroll
            for (int i = 1; i < RPW; ++i) dw[c] += join[i * TPR + t];
        }
        if (n < g.np8) *(f32x8*)(g.sums + (int64_t)blockIdx.x * g.np8 + n) = dw[c];
    }
}

// Rows too long for the registers: read twice, and the block's sums kept in memory,
// where each thread finds its own columns again.
template <int D>
__global__ void __launch_bounds__(1024) rms_norm_grad_long(NormGradArgs g) {
    typedef typename Elem<D>::type T;
    __shared__ float red[2][32];
    const int first = (int)blockIdx.x * g.rows;
    const int end = first + g.rows < g.M ? first + g.rows : g.M;
    int turn = 0;
    for (int64_t row = first; row < end; ++row) {
        const auto at = [&](const void* p, int64_t ld, int n) { return load8_at((const T*)p + row * ld + n, g.N - n); };
        const auto gain = [&](int n) { return g.w ? load8_at((const T*)g.w + n, g.N - n) : zero8() + 1.0f; };
        float sum[2] = {0.0f, 0.0f};
        for (int n = (int)threadIdx.x * 8; n < g.N; n += 8192) {
            const f32x8 h = at(g.H, g.ldh, n), dy = at(g.dY, g.lddy, n), w = gain(n);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                sum[0] = fmaf(h[i], h[i], sum[0]);
                sum[1] = fmaf(dy[i] * w[i], h[i], sum[1]);
            }
        }
        row_sums<1024, 2>(sum, red[turn]);
        turn ^= 1;
        const float s = inverse_rms(sum[0], g.N, g.eps), m = s * (s * (sum[1] / (float)g.N));
        for (int n = (int)threadIdx.x * 8; n < g.N; n += 8192) {
            const f32x8 hs = at(g.H, g.ldh, n) * s, dy = at(g.dY, g.lddy, n);
            if (g.sums) {
                f32x8* o = (f32x8*)(g.sums + (int64_t)blockIdx.x * g.np8 + n);
                *o = row == first ? dy * hs : *o + dy * hs;
            }
            if (g.dX) {
                f32x8 d = dy * gain(n) * s - hs * m;
                if (g.dH) d += at(g.dH, g.lddh, n);
                store8_at((T*)g.dX + row * g.lddx + n, d, g.N - n);
            }
        }
    }
}

}  // namespace pgemm
