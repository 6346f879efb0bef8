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
// 2^-e, exactly: where the entries are finite e + 127 is at most 247 (e4m3) and 253 (e2m1).
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
    int shift;      // log2 of the threads that share a row's stretch
    int stretches;  // of a row
};

// Rows of eight entries a thread: a workgroup has 256 >> shift rows (a row's stretch
// of 256 kRun groups of eight where rows are longer).
constexpr int kRun = 2;

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

// Where a thread of a workgroup stands: its row, and its first entry; the following ones are `step` further on.
struct MxPlace {
    int64_t row;
    int k, step;
};
__device__ __forceinline__ MxPlace mx_place(const MxCopyArgs& g, int64_t b) {
    const int64_t lot = g.stretches == 1 ? b : b / g.stretches;
    const int stretch = (int)(b - lot * g.stretches), t = (int)threadIdx.x & ((1 << g.shift) - 1);
    return MxPlace{(lot << (8 - g.shift)) + ((int)threadIdx.x >> g.shift), (stretch * (kRun << g.shift) + t) * 8, 8 << g.shift};
}

// Rows whose entries lie side by side: a lane has eight of them, four lanes a block, and two
// such groups under way.  Bound by memory: 16384 x 4096 of bf16 to 4 bits takes 27 us
// (6.3 TB/s, in the shared cache partly), to 8 bits 30, of fp32 to 4 bits 48.
template <int D, int F>
__global__ void __launch_bounds__(256) mx_quantize_rows(MxCopyArgs g) {
    typedef typename Elem<D>::type T;
    const int64_t lots = ((int64_t)g.rows + (256 >> g.shift) - 1) >> (8 - g.shift);
    for (int64_t b = blockIdx.x; b < lots * g.stretches; b += gridDim.x) {
        const MxPlace p = mx_place(g, b);
        if (p.row >= g.rows) continue;
        f32x8 v[kRun];
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            const int k = p.k + i * p.step;
            v[i] = load8_at((const T*)g.X + p.row * g.ldx + k, g.K - k);
        }
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            const int k = p.k + i * p.step;
            if (k < g.filled) mx_put8<F>((char*)g.Q + p.row * g.ldq, (uint8_t*)g.S + p.row * g.lds, k, v[i]);
        }
    }
}

// The same way back.  16384 x 4096 to bf16 takes 36 us from 4 bits (4.7 TB/s) and from 8: the writes bound it.
template <int D, int F>
__global__ void __launch_bounds__(256) mx_dequantize_rows(MxCopyArgs g) {
    typedef typename Elem<D>::type T;
    const int64_t lots = ((int64_t)g.rows + (256 >> g.shift) - 1) >> (8 - g.shift);
    for (int64_t b = blockIdx.x; b < lots * g.stretches; b += gridDim.x) {
        const MxPlace p = mx_place(g, b);
        if (p.row >= g.rows) continue;
        const char* q = (const char*)g.Q + p.row * g.ldq;
        i32x2 c[kRun];
        uint32_t s[kRun];
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            const int k = p.k + i * p.step;
            c[i] = i32x2{0, 0};
            s[i] = 0;
            if (k >= g.K) continue;
            if constexpr (F == MX8) c[i] = *(const i32x2*)(q + k);
            else c[i][0] = *(const int*)(q + k / 2);
            s[i] = ((const uint8_t*)g.S)[p.row * g.lds + (k >> 5)];
        }
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            const int k = p.k + i * p.step;
            store8_at((T*)g.X + p.row * g.ldx + k, mx_values<F>(c[i], s[i]), g.K - k);
        }
    }
}

constexpr int kEach = 2, kColumnRows = 64 * kEach;  // rows of a thread, of a workgroup
template <class T>
struct __attribute__((packed, aligned(sizeof(T)))) PackedRows {
    T v[kEach];
};
// Rows that are columns in memory (a weight stored K x N).  A workgroup has 128
// rows by 256 entries: a wave the rows' blocks of 32, a thread two rows' block,
// loaded in 32 stretches of two elements that lie side by side over the lanes.
// Codes and scales go through LDS, so that rows are written in whole lines.  Bound by
// memory: 16384 x 4096 of bf16 to 4 bits takes 31.8 us (5.3 TB/s, in the shared cache
// partly), to 8 bits 35.6; four rows a thread, whose registers leave a CU one
// workgroup, which loads and computes in turns, 53.
template <int D, int F>
__global__ void __launch_bounds__(512) mx_quantize_columns(MxCopyArgs g) {
    typedef typename Elem<D>::type T;
    constexpr int CB = F == MX8 ? 32 : 16, RB = 8 * CB, CHUNKS = RB / 16;  // bytes of a block's codes, of a row's; its chunks
    __shared__ __attribute__((aligned(16))) char codes[kColumnRows * RB];
    __shared__ __attribute__((aligned(8))) uint8_t scales[kColumnRows * 8];
    const int lane = (int)threadIdx.x & 63, blk = (int)threadIdx.x >> 6;
    const int64_t strips = ((int64_t)g.rows + kColumnRows - 1) / kColumnRows, total = strips * (g.filled / 256);
    for (int64_t b = blockIdx.x; b < total; b += gridDim.x) {
        const int64_t row0 = b % strips * kColumnRows;
        const int k0 = (int)(b / strips) * 256, kb = k0 + 32 * blk;
        const int64_t row = row0 + kEach * lane;
        const int valid = (int)(g.rows - row < kEach ? g.rows - row : kEach);
        const T* x = (const T*)g.X + (int64_t)kb * g.ldx + row;
        PackedRows<T> raw[32];
        if (row0 + kColumnRows <= g.rows && kb + 32 <= g.K) {  // all of the workgroup's rows: no branch between the loads
#pragma unroll
            for (int j = 0; j < 32; ++j) raw[j] = *(const PackedRows<T>*)(x + j * g.ldx);
        } else {
#pragma unroll
            for (int j = 0; j < 32; ++j)
#pragma unroll
                for (int e = 0; e < kEach; ++e) raw[j].v[e] = kb + j < g.K && e < valid ? x[j * g.ldx + e] : (T)0.0f;
        }
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            f32x8 v[4];
            uint32_t most = 0;
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j / 8][j % 8] = (float)raw[j].v[e];
#pragma unroll
            for (int j = 0; j < 4; ++j) most = max(most, largest8(v[j]));
            const uint32_t byte = mx_scale_byte<F>(most);
            i32x2 c[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) c[j] = mx_codes<F>(v[j], byte);
            const int r = kEach * lane + e;
            // chunks of a row XOR-swizzled by the lane against bank conflicts
            const auto put = [&](int chunk, i32x4 q) { *(i32x4*)(codes + r * RB + ((chunk ^ (lane & 7)) << 4)) = q; };
            if constexpr (F == MX8) {
                put(2 * blk, i32x4{c[0][0], c[0][1], c[1][0], c[1][1]});
                put(2 * blk + 1, i32x4{c[2][0], c[2][1], c[3][0], c[3][1]});
            } else {
                put(blk, i32x4{c[0][0], c[1][0], c[2][0], c[3][0]});
            }
            scales[r * 8 + blk] = (uint8_t)byte;
        }
        __syncthreads();
        const int64_t left = g.rows - row0;
        for (int i = (int)threadIdx.x; i < kColumnRows * CHUNKS; i += 512) {
            const int r = i / CHUNKS, chunk = i % CHUNKS;
            if (r < left)
                *(i32x4*)((char*)g.Q + (row0 + r) * g.ldq + (int64_t)k0 * CB / 32 + chunk * 16) =
                    *(const i32x4*)(codes + r * RB + ((chunk ^ ((r / kEach) & 7)) << 4));
        }
        if (threadIdx.x < kColumnRows && (int)threadIdx.x < left) {
            // (rows of scales are 4-byte aligned)
            int* s = (int*)((uint8_t*)g.S + (row0 + threadIdx.x) * g.lds + k0 / 32);
            s[0] = *(const int*)(scales + threadIdx.x * 8);
            s[1] = *(const int*)(scales + threadIdx.x * 8 + 4);
        }
        __syncthreads();
    }
}

}  // namespace pgemm
