// mx_format.hpp -- blocks of 32 entries that share a power of two as scale, in
// 8 bits (e4m3) and 4 bits (e2m1), on gfx950.
//
// A block's entries stand for q 2^e.  e is the smallest (not under -127) for
// which no entry rounds beyond the format's largest value: entries are rounded to
// nearest even, so the largest one, a, has to stay under half way to the value
// that would follow (e2m1: 6, then 8, which is even: a < 7 2^e; e4m3: 448, then
// 480, which is odd: a <= 464 2^e).  A scale two steps under the largest entry's
// exponent, as is also common, clips up to a quarter off that entry.
// The scale is stored as the byte e + 127.  A block with an infinity or a NaN has
// the byte 255, which stands for NaN in every entry, and zero codes.
//
// Rows are stored in whole groups of 256 entries, with zeros behind the last
// one: a K tile of the product is never cut, and a row's codes are whole 16-byte
// chunks.
#pragma once

#include "linear_kernel.hpp"

namespace pgemm {

enum MxFormat : int { MX8 = 0, MX4 = 1 };

constexpr int kMxBlock = 32, kMxGroup = 256;
PGEMM_HD constexpr int64_t mx_filled(int64_t K) { return (K + kMxGroup - 1) / kMxGroup * kMxGroup; }
PGEMM_HD constexpr int64_t mx_code_bytes(int64_t K, int format) { return mx_filled(K) >> (format == MX4 ? 1 : 0); }

// The scale's byte for the bits of a block's largest |entry|.
template <int F>
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t bits) {
    // adding carries into the exponent where the significand rounds beyond the largest value
    constexpr uint32_t up = F == MX8 ? 0x17ffffu : 0x200000u, down = F == MX8 ? 8u : 2u;
    const uint32_t e = (bits + up) >> 23;
    return bits >= 0x7f800000u ? 255u : e > down ? e - down : 0u;
}
// 2^-e, exactly: e + 127 is at most 252 where the entries are finite.
__device__ __forceinline__ float mx_inverse(uint32_t byte) {
    return byte == 255u ? 0.0f : __builtin_bit_cast(float, (254u - byte) << 23);
}
__device__ __forceinline__ float mx_scale(uint32_t byte) {
    return __builtin_bit_cast(float, byte == 0 ? 0x400000u : byte == 255u ? 0x7fc00000u : byte << 23);
}
__device__ __forceinline__ uint32_t abs_bits(float x) { return __builtin_bit_cast(uint32_t, x) & 0x7fffffffu; }
// The largest |entry| of eight, as bits: a NaN is larger than everything.
__device__ __forceinline__ uint32_t largest8(const f32x8& v) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i]));
    return m;
}
// The largest of four neighbouring lanes.
__device__ __forceinline__ uint32_t largest_of_quad(uint32_t m) {
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xf, 0xf, true));  // lane ^ 1
    return max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xf, 0xf, true));  // lane ^ 2
}
// Codes of eight entries, two dwords (e2m1: the first one only).
template <int F>
__device__ __forceinline__ i32x2 mx_codes(const f32x8& v, uint32_t byte) {
    const float s = mx_inverse(byte);
    f32x8 a;
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = byte == 255u ? 0.0f : v[i] * s;
    i32x2 q = {0, 0};
    if constexpr (F == MX8) {
#pragma unroll
        for (int d = 0; d < 2; ++d) {
            q[d] = __builtin_amdgcn_cvt_pk_fp8_f32(a[4 * d], a[4 * d + 1], 0, false);
            q[d] = __builtin_amdgcn_cvt_pk_fp8_f32(a[4 * d + 2], a[4 * d + 3], q[d], true);
        }
    } else {
        uint32_t c = 0;
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, a[0], a[1], 1.0f, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, a[2], a[3], 1.0f, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, a[4], a[5], 1.0f, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, a[6], a[7], 1.0f, 3);
        q[0] = (int)c;
    }
    return q;
}
// What eight codes stand for.
template <int F>
__device__ __forceinline__ f32x8 mx_values(const i32x2& q, uint32_t byte) {
    typedef __attribute__((ext_vector_type(2))) float f32x2;
    const float s = mx_scale(byte);
    f32x2 p[4];
    if constexpr (F == MX8) {
#pragma unroll
        for (int d = 0; d < 2; ++d) {
            p[2 * d] = __builtin_amdgcn_cvt_pk_f32_fp8(q[d], false);
            p[2 * d + 1] = __builtin_amdgcn_cvt_pk_f32_fp8(q[d], true);
        }
    } else {
        p[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4((uint32_t)q[0], 1.0f, 0);
        p[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4((uint32_t)q[0], 1.0f, 1);
        p[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4((uint32_t)q[0], 1.0f, 2);
        p[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4((uint32_t)q[0], 1.0f, 3);
    }
    f32x8 v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = p[i / 2][i % 2] * s;
    return v;
}

// ---- quantisation and its inverse -----------------------------------------------------------

struct MxCopyArgs {
    void* X;        // values
    void* Q;        // codes
    void* S;        // scales
    int64_t ldx, ldq, lds;  // elements; bytes
    int rows, K;
    int filled;     // entries of a stored row
};

template <class T>
struct __attribute__((packed, aligned(sizeof(T)))) Packed8 {
    T v[8];
};
// Eight elements at any element's address, the first `valid` of them, zeros for the rest.
template <class T>
__device__ __forceinline__ f32x8 load8_at(const T* p, int valid) {
    f32x8 v = zero8();
    if (valid >= 8) {
        const Packed8<T> x = *(const Packed8<T>*)p;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (float)x.v[i];
    } else {
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (i < valid) v[i] = (float)p[i];
    }
    return v;
}
template <class T>
__device__ __forceinline__ void store8_at(T* p, const f32x8& v, int valid) {
    if (valid >= 8) {
        Packed8<T> x;
#pragma unroll
        for (int i = 0; i < 8; ++i) x.v[i] = (T)v[i];
        *(Packed8<T>*)p = x;
    } else {
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (i < valid) p[i] = (T)v[i];
    }
}
// Codes of the eight entries from k on, and every fourth lane the block's scale.
template <int F>
__device__ __forceinline__ void mx_put8(char* q, uint8_t* s, int k, const f32x8& v) {
    const uint32_t byte = mx_scale_byte<F>(largest_of_quad(largest8(v)));
    const i32x2 c = mx_codes<F>(v, byte);
    if constexpr (F == MX8) *(i32x2*)(q + k) = c;
    else *(int*)(q + k / 2) = c[0];
    if ((k & 31) == 0) s[k >> 5] = (uint8_t)byte;
}

// Rows whose entries lie side by side: a lane has eight of them, four lanes a block.
template <int D, int F>
__global__ void __launch_bounds__(256) mx_quantize_rows(MxCopyArgs g) {
    typedef typename Elem<D>::type T;
    const int per_row = g.filled / 8;
    const int64_t total = (int64_t)g.rows * per_row;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / per_row;
        const int k = (int)(i - row * per_row) * 8;
        const f32x8 v = load8_at((const T*)g.X + row * g.ldx + k, g.K - k);
        mx_put8<F>((char*)g.Q + row * g.ldq, (uint8_t*)g.S + row * g.lds, k, v);
    }
}

// Rows that are columns in memory (a weight stored K x N): a thread has one row's block.
template <int D, int F>
__global__ void __launch_bounds__(256) mx_quantize_columns(MxCopyArgs g) {
    typedef typename Elem<D>::type T;
    const int blocks = g.filled / 32;
    const int64_t strips = ((int64_t)g.rows + 63) / 64, total = strips * (blocks / 4);
    for (int64_t i = blockIdx.x; i < total; i += gridDim.x) {
        const int64_t row = i % strips * 64 + (threadIdx.x & 63);
        const int b = (int)(i / strips) * 4 + (int)(threadIdx.x >> 6);
        if (row >= g.rows) continue;
        const T* x = (const T*)g.X + (int64_t)b * 32 * g.ldx + row;
        f32x8 v[4];
        uint32_t most = 0;
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j / 8][j % 8] = b * 32 + j < g.K ? (float)x[j * g.ldx] : 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) most = max(most, largest8(v[j]));
        const uint32_t byte = mx_scale_byte<F>(most);
        i32x2 c[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) c[j] = mx_codes<F>(v[j], byte);
        char* q = (char*)g.Q + row * g.ldq + b * (F == MX8 ? 32 : 16);
        if constexpr (F == MX8) {
            *(i32x4*)q = i32x4{c[0][0], c[0][1], c[1][0], c[1][1]};
            *(i32x4*)(q + 16) = i32x4{c[2][0], c[2][1], c[3][0], c[3][1]};
        } else {
            *(i32x4*)q = i32x4{c[0][0], c[1][0], c[2][0], c[3][0]};
        }
        ((uint8_t*)g.S)[row * g.lds + b] = (uint8_t)byte;
    }
}

template <int D, int F>
__global__ void __launch_bounds__(256) mx_dequantize_rows(MxCopyArgs g) {
    typedef typename Elem<D>::type T;
    const int per_row = (g.K + 7) / 8;
    const int64_t total = (int64_t)g.rows * per_row;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / per_row;
        const int k = (int)(i - row * per_row) * 8;
        const char* q = (const char*)g.Q + row * g.ldq;
        i32x2 c = {0, 0};
        if constexpr (F == MX8) c = *(const i32x2*)(q + k);
        else c[0] = *(const int*)(q + k / 2);
        const f32x8 v = mx_values<F>(c, ((const uint8_t*)g.S)[row * g.lds + (k >> 5)]);
        store8_at((T*)g.X + row * g.ldx + k, v, g.K - k);
    }
}

}  // namespace pgemm
