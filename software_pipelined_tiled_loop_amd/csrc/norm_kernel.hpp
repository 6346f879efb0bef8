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
// Sums of P values over the TPR threads of a row; `red`, the row's, has P x 16 floats, free to be written.
template <int TPR, int P>
__device__ __forceinline__ void row_sums(float (&x)[P], float* red) {
#pragma unroll
    for (int p = 0; p < P; ++p) x[p] = wave_sum(x[p]);
    if constexpr (TPR > 64) {
        const int wave = (int)threadIdx.x % TPR >> 6;
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

// Eight elements as they lie in memory.
template <class T>
__device__ __forceinline__ Packed8<T> raw8(const T* p, int valid) {
    Packed8<T> x;
    if (valid >= 8) {
        x = *(const Packed8<T>*)p;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x.v[i] = i < valid ? p[i] : (T)0.0f;
    }
    return x;
}
template <class T>
__device__ __forceinline__ f32x8 wide8(const Packed8<T>& x) {
    f32x8 v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)x.v[i];
    return v;
}
template <class T>
__device__ __forceinline__ Packed8<T> ones8() {
    Packed8<T> x;
#pragma unroll
    for (int i = 0; i < 8; ++i) x.v[i] = (T)1.0f;
    return x;
}

// Rows of a workgroup: one for each TPR threads, at least one wave's.
template <int TPR>
constexpr int norm_threads = TPR < 256 ? 256 : TPR;

// TPR threads a row, CH groups of eight columns a thread.  Bound by memory, so as many threads a row
// as leave each one load of a tensor: 4096 rows of bf16 with a residual, both outputs written, take
// with 4096 columns 22.5 us by 512 threads (6.0 TB/s, in the shared cache partly), 24.4 by 256 with two
// groups, 30 by 128 with four; with 8192 columns 44 by 512 with two, 47 by 1024; with 2048
// 13.7 by 256, 13.5 by 128 with two; with 1024 6.9 by a wave with two, 8.8 by 256.
template <int D, int TPR, int CH>
__global__ void __launch_bounds__(norm_threads<TPR>) rms_norm_rows(NormArgs g) {
    typedef typename Elem<D>::type T;
    constexpr int RPW = norm_threads<TPR> / TPR;
    __shared__ float red[2][16];
    const int t = (int)threadIdx.x % TPR;
    int turn = 0;
    for (int64_t row = (int64_t)blockIdx.x * RPW + threadIdx.x / TPR; row < g.M; row += (int64_t)gridDim.x * RPW) {
        f32x8 v[CH];
        Packed8<T> r[CH], w[CH];
        float sum[1] = {0.0f};
        // everything that is read is under way before the sum is formed
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int n = (c * TPR + t) * 8;
            v[c] = load8_at((const T*)g.X + row * g.ldx + n, g.N - n);
            if (g.R) r[c] = raw8((const T*)g.R + row * g.ldr + n, g.N - n);
            w[c] = g.w ? raw8((const T*)g.w + n, g.N - n) : ones8<T>();
        }
        if (g.R) {
#pragma unroll
            for (int c = 0; c < CH; ++c) v[c] += wide8(r[c]);
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
            const f32x8 y = v[c] * s * wide8(w[c]);
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
    void* dw;        // their sum itself, where there is one block
    int dw_f32;      // (fp32, else H's type)
    int64_t lddy, ldh, lddh, lddx;
    float eps;
    int M, N, np8;
    int rows;        // of a block
};

// A block of `rows` rows, as many at once as its threads hold; its columns' sums of
// dy h s stay in registers.  The next rows are under way while one is summed.  Two
// workgroups of 512 threads a CU cover each other's barriers: 4096 x 4096 in bf16 with dh takes
// 25.8 us (134 MB, 5.2 TB/s, in the shared cache partly), 30.2 by one of 1024 threads, 35.9 by
// one of 512, 28.7 by four; 49 without the next rows under way, in blocks of eight rows.
template <int TPR>
constexpr int norm_grad_threads = TPR < 512 ? 512 : TPR;

template <int D, int TPR, int CH>
__global__ void __launch_bounds__(norm_grad_threads<TPR>) rms_norm_grad(NormGradArgs g) {
    typedef typename Elem<D>::type T;
    constexpr int NT = norm_grad_threads<TPR>, RPW = NT / TPR;
    __shared__ float red[2][RPW][32];
    __shared__ f32x8 join[RPW > 1 ? NT : 1];
    const int t = (int)threadIdx.x % TPR, mine = (int)threadIdx.x / TPR;
    const int64_t first = (int64_t)blockIdx.x * g.rows, end = first + g.rows < g.M ? first + g.rows : g.M;
    Packed8<T> w[CH], h[CH], dy[CH], dh[CH];
    f32x8 dw[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int n = (c * TPR + t) * 8;
        dw[c] = zero8();
        w[c] = g.w ? raw8((const T*)g.w + n, g.N - n) : ones8<T>();
    }
    const auto fetch = [&](int64_t row) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int n = (c * TPR + t) * 8, valid = row < end ? g.N - n : 0;
            h[c] = raw8((const T*)g.H + row * g.ldh + n, valid);
            dy[c] = raw8((const T*)g.dY + row * g.lddy + n, valid);
            if (g.dH) dh[c] = raw8((const T*)g.dH + row * g.lddh + n, valid);
        }
    };
    constexpr bool AHEAD = CH == 1;  // the next rows' values beside this one's: what the registers hold
    if constexpr (AHEAD) fetch(first + mine);
    int turn = 0;
    for (int64_t base = first; base < end; base += RPW) {
        const int64_t row = base + mine;
        if constexpr (!AHEAD) fetch(row);
        f32x8 hs[CH], d[CH];
        float sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            hs[c] = wide8(h[c]);
            d[c] = wide8(dy[c]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                sum[0] = fmaf(hs[c][i], hs[c][i], sum[0]);
                sum[1] = fmaf(d[c][i] * (float)w[c].v[i], hs[c][i], sum[1]);
            }
        }
        Packed8<T> e[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) e[c] = dh[c];
        if constexpr (AHEAD) fetch(row + RPW);
        row_sums<TPR, 2>(sum, red[turn][mine]);
        turn ^= 1;
        const float s = inverse_rms(sum[0], g.N, g.eps), m = s * (s * (sum[1] / (float)g.N));
        if (row >= end) continue;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int n = (c * TPR + t) * 8;
            if (n >= g.N) continue;
            hs[c] *= s;
            dw[c] += d[c] * hs[c];
            if (g.dX) {
                f32x8 x = d[c] * wide8(w[c]) * s - hs[c] * m;
                if (g.dH) x += wide8(e[c]);
                store8_at((T*)g.dX + row * g.lddx + n, x, g.N - n);
            }
        }
    }
    if (!g.sums && !g.dw) return;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int n = (c * TPR + t) * 8;
        if constexpr (RPW > 1) {
            __syncthreads();
            join[threadIdx.x] = dw[c];
            __syncthreads();
            if (threadIdx.x >= TPR) continue;
#pragma unroll 4
            for (int i = 1; i < RPW; ++i) dw[c] += join[i * TPR + t];
        }
        if (g.sums) {
            if (n < g.np8) *(f32x8*)(g.sums + (int64_t)blockIdx.x * g.np8 + n) = dw[c];
        } else if (g.dw_f32) {
            store8_at((float*)g.dw + n, dw[c], g.N - n);
        } else {
            store8_at((T*)g.dw + n, dw[c], g.N - n);
        }
    }
}

// Rows too long for the registers: read twice, and the block's sums kept in memory,
// where each thread finds its own columns again.
template <int D>
__global__ void __launch_bounds__(1024) rms_norm_grad_long(NormGradArgs g) {
    typedef typename Elem<D>::type T;
    __shared__ float red[2][32];
    const int64_t first = (int64_t)blockIdx.x * g.rows, end = first + g.rows < g.M ? first + g.rows : g.M;
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

// The blocks' sums in a fixed order: 64 interleaved runs of blocks, then the
// runs.  512 blocks of 4096 columns take 4.9 us, most of it the launch.  Sixteen columns a workgroup, so that few columns spread over the CUs too.
struct NormSumArgs {
    const float* sums;  // [blocks][np8]
    void* out;
    int blocks, np8, N, out_f32;
};
template <int D>
__global__ void __launch_bounds__(1024) rms_norm_join(NormSumArgs g) {
    typedef typename Elem<D>::type T;
    __shared__ float red[64][16];
    const int c = (int)threadIdx.x & 15, run = (int)threadIdx.x >> 4;
    for (int64_t n0 = (int64_t)blockIdx.x * 16; n0 < g.N; n0 += (int64_t)gridDim.x * 16) {
        const int64_t n = n0 + c;
        float x = 0.0f;
        if (n < g.N) {
#pragma unroll 8
            for (int b = run; b < g.blocks; b += 64) x += g.sums[(int64_t)b * g.np8 + n];
        }
        red[run][c] = x;
        __syncthreads();
        if (run == 0 && n < g.N) {
            for (int k = 1; k < 64; ++k) x += red[k][c];
            if (g.out_f32) ((float*)g.out)[n] = x;
            else ((T*)g.out)[n] = (T)x;
        }
        __syncthreads();
    }
}

}  // namespace pgemm
