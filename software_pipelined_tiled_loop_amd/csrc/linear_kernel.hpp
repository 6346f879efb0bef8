// linear_kernel.hpp -- the feed-forward operators' kernels for gfx950: a
// matrix product with a fused epilogue (bias, activation, residual, the kept
// pre-activations), the gated block (two products, activation and product in
// one kernel), and the products of both backward passes.
//
// Mathematics.  With A the activations (rows m, contraction index k) and B
// the weights (columns n):
//     acc[m][n] = sum_k A(m, k) B(k, n)
//     linear   Z = acc + b,  Y = act(Z) + R
//     gated    G = acc_g + bg,  U = acc_u + bu,  H = act(G) U
// The backward pass is made of the same products with other operands:
//     dX = dZ W^T (gated: dG Wg^T + dU Wu^T, one contraction over both
//     halves), dW = X^T dZ (gated: two outputs of one launch sharing X).
//
// Operand layouts.  Each operand is stored either with the contraction index
// contiguous (LAY_K: X, dZ as left operand, W stored [N][K], W as operand of
// dX) or with its row / column index contiguous (LAY_X: W stored [K][N], X and
// dZ as operands of dW).  Both are copied to LDS as they lie in memory, by
// LDS-DMA (buffer_load_dwordx4 ... lds), in 16-byte chunks XOR-swizzled as in
// pgemm_kernel.hpp; LAY_K fragments are read with ds_read_b128, LAY_X ones
// with the transposing reads (fp32: ds_read_b32).  So no operand is ever
// transposed in memory, forward or backward.
//
// The MFMAs are issued with the operands exchanged (B fragment first): the
// result block then holds, in each lane, four consecutive columns n of one
// row m, one 16-byte piece of the output tile that the epilogue lays out in LDS.
//
// K loop: a ring of S LDS stages with one barrier per K tile, as in
// pgemm_kernel.hpp.  Only whole K tiles of the contraction go through the
// ring.  The last one, when it is cut by the end of K, or when an operand's
// contiguous extent is not whole 16-byte chunks (a chunk of its last rows
// could then end past the allocation), is loaded after the ring has drained,
// through registers, with element loads where a chunk straddles an edge and
// zeros beyond the edge.  Rows and columns beyond the output's edge load
// zeros, or values that feed only outputs which are never stored.
#pragma once

#include "pgemm_kernel.hpp"

namespace pgemm {

enum Lay : int { LAY_K = 0, LAY_X = 1 };
enum ActKind : int { ACTK_NONE = 0, ACTK_RELU = 1, ACTK_SILU = 2, ACTK_GELU = 3, ACTK_GELU_TANH = 4 };

// Activations silu and gelu_tanh share one form,
//     act(x) = x * sigmoid(x * P(x^2)):
//   silu       P = 1
//   gelu_tanh  P = sqrt(8/pi) (1 + 0.044715 t): (1 + tanh a)/2 = sigmoid(2a)
// and the slopes
//     act'(x) = p + x p (1 - p) (P + 2 t P'),  p = sigmoid(x P).
// gelu is x Phi(x), its slope Phi + x phi with phi(x) = exp(-x^2/2) / sqrt(2 pi);
//     Phi(-y) = exp(-y^2/2) Q(y) for y >= 0,  Phi(y) = 1 - Phi(-y),
// where Q falls from 1/2 as slowly as 1/y: gelu_q.  Each takes one exponential and
// one reciprocal, for value and slope together, and stays accurate relative to
// itself far below zero, down to fp32's smallest normal number.
struct ActArgs {
    int kind;      // ActKind
    float c[2];    // coefficients of -log2(e) * P: sigmoid(x P) = 1 / (1 + exp2(x c(t)))
};

struct EpiArgs {
    void* Y[2];           // output (gated: H); two for a launch with two outputs side by side (dWg, dWu)
    int64_t ldy;
    const void* R;        // residual, Y's type
    int64_t ldr;
    void* Z;              // kept pre-activation (gated: G), operand type; may be null
    void* U;              // gated: kept U
    int64_t ldz, ldu;
    const void* bias[2];  // operand type; may be null (gated: bg, bu)
    const float* rows[2]; // fp16 gradients: factor of each row, or column, of output `out`
    const float* cols[2]; // (see linear_slope); null: none
    ActArgs act;
    int M, N;
    int out_f32;          // Y and R are fp32 (else the operand type)
};

struct LinArgs {
    const void* A[2];     // of contraction half h, or of output `out` where there are two
    const void* B[2];     // likewise; gated: Wg, Wu
    int64_t lda, ldb;
    int K;                // contraction length of one half
    int nfull;            // K tiles of a half that go through the ring
    int halves;           // contraction halves (1, or 2 for the gated dX)
    int outs;             // outputs side by side (1, or 2 for the gated dW)
    int tiles_m, tiles_n, group_m;
    int splits;           // workgroups that share one output tile's K tiles
    float* part;          // fp32 sums of each split: [split][plane][M][np8] (planes: outs, or 2 for gated)
    int np8;
    EpiArgs e;
};

// ---- one operand's LDS tile: EXT rows (or columns) by BK of the contraction --------------

template <int D, int LAY, int EXT, int BK>
struct Opnd {
    static constexpr int ES = Traits<D>::ES, EPC = Traits<D>::EPC, KSTEP = Traits<D>::KSTEP;
    static constexpr int KC = BK * ES / 16, NCH = EXT * ES / 16;
    static constexpr int BYTES = EXT * BK * ES;
    static constexpr bool along_k = LAY == LAY_K;  // rows in memory run along the contraction
    // LDS reads of one fragment
    static constexpr int READS = LAY == LAY_K ? 1 : (ES == 4 ? 4 : 2);
    static_assert(BYTES % 1024 == 0, "tile must be whole 1-KiB blocks");
    static_assert(LAY != LAY_K || KC == 4 || KC == 8, "rows must be 64 or 128 bytes");
    static_assert(LAY != LAY_X || ((NCH & (NCH - 1)) == 0 && NCH >= 4 && EXT * ES <= 1024), "bad row of the tile");

    // Memory chunk that sits at LDS byte `off` of the tile: extent index e
    // and contraction index k of its first element.
    static PGEMM_HD void chunk(int off, int& e, int& k) {
        if constexpr (LAY == LAY_K) {
            int kc;
            a_inv<KC>(off, e, kc);
            k = kc * EPC;
        } else {
            k = off / (EXT * ES);
            e = (((off % (EXT * ES)) >> 4) ^ b_swz<D, NCH>(k)) * EPC;
        }
    }
    // LDS byte that `lane` addresses for read h of the fragment of extent
    // block e0 .. e0+15 at K step ks (lane semantics of the transposing reads:
    // b_frag_off in pgemm_kernel.hpp).
    static PGEMM_HD int frag(int ks, int e0, int lane, int h) {
        const int li = lane & 15, lg = lane >> 4;
        if constexpr (LAY == LAY_K) {
            return a_off<KC>(e0 + li, ks * 4 + lg);
        } else {
            int k, e;
            if constexpr (ES == 2) {
                k = ks * KSTEP + 8 * lg + 4 * h + (li >> 2);
                e = e0 + 4 * (li & 3);
            } else {
                k = ks * KSTEP + 4 * lg + h;
                e = e0 + li;
            }
            return k * EXT * ES + (((e / EPC) ^ b_swz<D, NCH>(k)) << 4) + (e % EPC) * ES;
        }
    }
    static __device__ __forceinline__ void read(const char PGEMM_LDS* tile, int ks, int e0, int lane, i32x4& out) {
        if constexpr (LAY == LAY_K) {
            out = *(const i32x4 PGEMM_LDS*)(tile + frag(ks, e0, lane, 0));
        } else if constexpr (ES == 2) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const i16x4 v =
                    __builtin_amdgcn_ds_read_tr16_b64_v4i16((i16x4 PGEMM_LDS*)(tile + frag(ks, e0, lane, h)));
                const i32x2 w = __builtin_bit_cast(i32x2, v);
                out[2 * h] = w[0];
                out[2 * h + 1] = w[1];
            }
        } else {
#pragma unroll
            for (int h = 0; h < 4; ++h) out[h] = *(const int PGEMM_LDS*)(tile + frag(ks, e0, lane, h));
        }
    }
    // Byte offset in memory of the chunk (e, k) from the tile's origin.
    static PGEMM_HD uint32_t mem_off(int e, int k, int64_t ld) {
        return LAY == LAY_K ? (uint32_t)(e * (int)ld + k) * ES : (uint32_t)(k * (int)ld + e) * ES;
    }
    // Bytes from the matrix's origin to the tile at extent e0, K tile kt.
    static PGEMM_HD int64_t origin(int64_t e0, int64_t kt, int64_t ld) {
        return (LAY == LAY_K ? e0 * ld + kt * BK : kt * BK * ld + e0) * ES;
    }
    static PGEMM_HD int64_t step(int64_t ld) { return (LAY == LAY_K ? (int64_t)BK : (int64_t)BK * ld) * ES; }

    // Elements of chunk (e, k) inside a matrix that ends at (e_left, k_left).
    static PGEMM_HD int cut_valid(int e, int k, int e_left, int k_left) {
        const int in_row = LAY == LAY_K ? k_left - k : e_left - e;
        const bool row_ok = LAY == LAY_K ? e < e_left : k < k_left;
        return !row_ok || in_row <= 0 ? 0 : in_row < EPC ? in_row : EPC;
    }
    // How many of K's K tiles may go through the ring, whose 16-byte loads
    // check an extent index against the operand's edge only where the chunk
    // starts: whole tiles, and for LAY_X rows that are not whole chunks only
    // as many that a chunk straddling the edge in the last row loaded ends
    // inside the rows behind it.
    static PGEMM_HD int ring_tiles(int64_t K, int64_t extent, int64_t ld) {
        int64_t n = K / BK;
        if (LAY == LAY_X && extent % EPC != 0)
            while (n > 0 && (K - n * BK) * ld < EPC - 1) --n;
        return (int)n;
    }

    // The cut K tile, through registers: N blocks of 1 KiB from block p0, zeros
    // beyond the edges.  Where rows hold a chunk or more, a chunk that the edge
    // cuts is loaded as the 16 bytes that end there and moved down by as many
    // bytes as lie beyond (`beyond`: the same for every chunk cut, as the edge
    // is); shorter rows go element by element.  All loads are under way at once:
    // one after the other the K tile took 16 us.
    template <int N>
    static __device__ __forceinline__ void load_cut(const char* mem, int64_t ld, int e_left, int k_left, int row_length,
                                                    char PGEMM_LDS* tile, int p0, int lane) {
        if (row_length < EPC) {
            const __amdgpu_buffer_rsrc_t r = make_rsrc(mem);
            for (int p = p0; p < p0 + N; ++p) {
                int e, k;
                chunk(p * 1024 + lane * 16, e, k);
                const int valid = cut_valid(e, k, e_left, k_left);
                *(i32x4 PGEMM_LDS*)(tile + p * 1024 + lane * 16) =
                    load_chunk_any<ES>(r, mem_off(e, k, ld), valid, valid == EPC);
            }
            return;
        }
        const int beyond = cut_shift(row_length);  // bytes
        // offsets from 16 bytes before the tile: the chunk cut may begin before it
        const __amdgpu_buffer_rsrc_t r = make_rsrc(mem - 16);
        i32x4 v[N];
        bool cut[N];
#pragma unroll
        for (int q = 0; q < N; ++q) {
            int e, k;
            chunk((p0 + q) * 1024 + lane * 16, e, k);
            const int valid = cut_valid(e, k, e_left, k_left);
            cut[q] = valid < EPC;
            const uint32_t off = mem_off(e, k, ld) + 16 - (cut[q] ? beyond : 0);
            v[q] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(r, valid > 0 ? off : OOB, 0, 0));
        }
#pragma unroll
        for (int q = 0; q < N; ++q) {
            if (beyond) {
                const i32x4 s = move_down(v[q], beyond);
#pragma unroll
                for (int d = 0; d < 4; ++d) v[q][d] = cut[q] ? s[d] : v[q][d];
            }
            *(i32x4 PGEMM_LDS*)(tile + (p0 + q) * 1024 + lane * 16) = v[q];
        }
    }
    // Bytes of a row's last chunk beyond the row's end.
    static PGEMM_HD int cut_shift(int row_length) { return (EPC - row_length % EPC) % EPC * ES; }
    // The 16 bytes of v from byte `by` (0 < by < 16, uniform) on, then zeros.
    static __device__ __forceinline__ i32x4 move_down(i32x4 v, int by) {
        const int w = by >> 2, sh = 8 * (by & 3);
        uint32_t x[5];
#pragma unroll
        for (int d = 0; d < 4; ++d)
            x[d] = w == 0 ? (uint32_t)v[d]
                   : w == 1 ? (d < 3 ? (uint32_t)v[d < 3 ? d + 1 : 3] : 0u)
                   : w == 2 ? (d < 2 ? (uint32_t)v[d < 2 ? d + 2 : 3] : 0u)
                            : (d < 1 ? (uint32_t)v[3] : 0u);
        x[4] = 0;
#pragma unroll
        for (int d = 0; d < 4; ++d) v[d] = (int)(uint32_t)((((uint64_t)x[d + 1] << 32) | x[d]) >> sh);
        return v;
    }
};

// One MFMA block with the operands exchanged: lane l of the result holds
// columns 4*(l/16) .. +3 (of the B block) of row l%16 (of the A block).
template <int D>
__device__ __forceinline__ void mfma_swapped(f32x4& acc, const i32x4& a, const i32x4& b) {
    if constexpr (D == DT_BF16) {
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b), __builtin_bit_cast(bf16x8, a),
                                                      acc, 0, 0, 0);
    } else if constexpr (D == DT_F16) {
        acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, b), __builtin_bit_cast(f16x8, a), acc,
                                                     0, 0, 0);
    } else {
        const f32x4 af = __builtin_bit_cast(f32x4, a);  // whole vectors: see mfma_block
        const f32x4 bf = __builtin_bit_cast(f32x4, b);
#pragma unroll
        for (int jm = 0; jm < 4; ++jm) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(bf[jm], af[jm], acc, 0, 0, 0);
    }
}

// ---- values: eight consecutive columns of a row ----------------------------------------------

template <int D> struct Elem { typedef __bf16 type; };
template <> struct Elem<DT_F16> { typedef _Float16 type; };
template <> struct Elem<DT_F32> { typedef float type; };

typedef __attribute__((ext_vector_type(8))) float f32x8;
template <class T> struct Vec8 { typedef f32x8 type; };
template <> struct Vec8<__bf16> { typedef bf16x8 type; };
template <> struct Vec8<_Float16> { typedef f16x8 type; };

__device__ __forceinline__ f32x8 zero8() { return f32x8{0, 0, 0, 0, 0, 0, 0, 0}; }
__device__ __forceinline__ f32x8 join8(f32x4 a, f32x4 b) { return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7); }

template <class T>
__device__ __forceinline__ f32x8 load8(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    if constexpr (sizeof(T) == 4) {
        return join8(__builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0)),
                     __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off + 16, 0, 0)));
    } else {
        const typename Vec8<T>::type h =
            __builtin_bit_cast(typename Vec8<T>::type, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
        f32x8 v;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = (float)h[e];
        return v;
    }
}
// Stores round to the output's type, to nearest even, once.  The uniform part
// of the offset is added in the lanes, not passed as the instruction's scalar
// offset: with one the compiler lets the very next instruction overwrite the
// registers of a 16-byte store, and here that changed what was stored (first
// dword of a group, seen in the kept pre-activations of a large tile).
template <class T>
__device__ __forceinline__ void store8(__amdgpu_buffer_rsrc_t r, uint32_t at, f32x8 v) {
    if constexpr (sizeof(T) == 4) {
        const f32x4 a = __builtin_shufflevector(v, v, 0, 1, 2, 3), b = __builtin_shufflevector(v, v, 4, 5, 6, 7);
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(i32x4, a), r, at, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(i32x4, b), r, at + 16, 0, 0);
    } else {
        typename Vec8<T>::type h;
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = (T)v[e];
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(i32x4, h), r, at, 0, 0);
    }
}
template <class T>
__device__ __forceinline__ float load1(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    if constexpr (sizeof(T) == 4)
        return __builtin_bit_cast(float, (int)__builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0));
    else
        return (float)__builtin_bit_cast(T, (short)__builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0));
}
template <class T>
__device__ __forceinline__ void store1(__amdgpu_buffer_rsrc_t r, uint32_t off, float v) {
    if constexpr (sizeof(T) == 4)
        __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(int, v), r, off, 0, 0);
    else
        __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(short, (T)v), r, off, 0, 0);
}

// Whether some group of eight columns is cut by the output's edge.
__device__ __forceinline__ bool cols_cut(int n) { return (n & 7) != 0; }

// -log2(e) * P(t), so that sigmoid(x P) = 1 / (1 + exp2(x c(t))).
template <int DEG>
__device__ __forceinline__ float act_poly(const ActArgs& a, float t) {
    float p = a.c[DEG];
#pragma unroll
    for (int d = DEG - 1; d >= 0; --d) p = fmaf(p, t, a.c[d]);
    return p;
}

template <int DEG>
__device__ __forceinline__ float act_smooth(const ActArgs& a, float x) {
    const float p = DEG == 0 ? a.c[0] : act_poly<DEG>(a, x * x);
    return x * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * p));
}

// Q(y) = Phi(-y) exp(y^2 / 2), y >= 0, as a polynomial without constant term in
// s = 1 / (1 + 0.3046 y) (both fall as 1/y): least squares of the relative error,
// iterated towards its minimax on 0 <= y <= 14, beyond which exp(-y^2 / 2) is zero.
// 9e-8 relative, 3.7e-7 evaluated in fp32.
__device__ __forceinline__ float gelu_q(float y) {
    const float s = __builtin_amdgcn_rcpf(fmaf(0.3046f, y, 1.0f));
    float q = 0.03676469251513481f;
    q = fmaf(q, s, -0.15391618013381958f);
    q = fmaf(q, s, 0.18829947710037231f);
    q = fmaf(q, s, -0.04002207890152931f);
    q = fmaf(q, s, 0.12202255427837372f);
    q = fmaf(q, s, 0.10302632302045822f);
    q = fmaf(q, s, 0.12234748154878616f);
    q = fmaf(q, s, 0.12147778272628784f);
    return q * s;
}
// Phi(x); e receives exp(-x^2 / 2).
__device__ __forceinline__ float gelu_phi(float x, float& e) {
    e = __builtin_amdgcn_exp2f(-0.7213475204f * (x * x));  // NaN where x is
    const float w = e * gelu_q(__builtin_fabsf(x));
    return x > 0.0f ? 1.0f - w : w;
}

template <int KIND>
__device__ __forceinline__ float act1(const ActArgs& a, float x) {
    if constexpr (KIND == ACTK_NONE) return x;
    else if constexpr (KIND == ACTK_RELU) return x < 0.0f ? 0.0f : x;  // NaN stays NaN
    else if constexpr (KIND == ACTK_SILU) return act_smooth<0>(a, x);
    else if constexpr (KIND == ACTK_GELU_TANH) return act_smooth<1>(a, x);
    else {
        float e;
        return x * gelu_phi(x, e);
    }
}
template <int KIND>
__device__ __forceinline__ f32x8 act8(const ActArgs& a, f32x8 x) {
    if constexpr (KIND != ACTK_NONE) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = act1<KIND>(a, x[e]);
    }
    return x;
}
// Calls f with the activation as a constant: one branch, not one a group.
template <int K>
struct KindC {
    static constexpr int value = K;
};
template <class F>
__device__ __forceinline__ void with_act(int kind, F&& f) {
    switch (kind) {
        case ACTK_NONE: f(KindC<ACTK_NONE>{}); break;
        case ACTK_RELU: f(KindC<ACTK_RELU>{}); break;
        case ACTK_SILU: f(KindC<ACTK_SILU>{}); break;
        case ACTK_GELU_TANH: f(KindC<ACTK_GELU_TANH>{}); break;
        default: f(KindC<ACTK_GELU>{}); break;
    }
}

// act(x) and act'(x) of a smooth activation.  Beyond |x| = 128 exponential and
// sigmoid are 0 or 1 (gelu_tanh: beyond 12), so x and t held there leave the slope
// as it is and keep it finite (x^3 does not overflow, no infinity meets a zero); e is
// held too, so that e p = 1 - p where p vanishes.
template <int DEG>
__device__ __forceinline__ void act_slope(const ActArgs& a, float x, float& y, float& d) {
    const float t = fminf(x * x, 4096.0f);
    const float c = DEG == 0 ? a.c[0] : act_poly<DEG>(a, t);
    const float e = __builtin_amdgcn_exp2f(x * c);
    const float p = __builtin_amdgcn_rcpf(1.0f + e);  // NaN where x is
    const float h = __builtin_amdgcn_fmed3f(x, -128.0f, 128.0f);
    y = x * p;
    // d(x P)/dx = P + 2 t P', from the coefficients of -log2(e) P
    const float s = -0.6931471806f * (DEG == 1 ? fmaf(2.0f * t, a.c[1], c) : c);
    d = fmaf(h * p * s, fminf(e, 0x1p126f) * p, p);
}
__device__ __forceinline__ void gelu_slope(float x, float& y, float& d) {
    float e;
    const float p = gelu_phi(x, e);
    y = x * p;
    d = fmaf(__builtin_amdgcn_fmed3f(x, -128.0f, 128.0f), 0.3989422804f * e, p);
}

template <int KIND>
__device__ __forceinline__ void act_slope8(const ActArgs& a, f32x8 x, f32x8& y, f32x8& d) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float yi = x[i], di = 1.0f;
        if constexpr (KIND == ACTK_RELU) {
            yi = x[i] < 0.0f ? 0.0f : x[i];
            di = x[i] > 0.0f ? 1.0f : 0.0f;
        } else if constexpr (KIND == ACTK_GELU) {
            gelu_slope(x[i], yi, di);
        } else if constexpr (KIND != ACTK_NONE) {
            act_slope<KIND == ACTK_SILU ? 0 : 1>(a, x[i], yi, di);
        }
        y[i] = yi;
        d[i] = di;
    }
}

// The fused epilogue of one tile, eight columns of a row at a time (16-byte
// accesses of 16-bit types).  Rows and columns are relative to (m0, n0); a lane
// holds the offsets of its first group (row, col) and moves from there by rows
// that are the same for all lanes.  A group that the edge of the output cuts
// goes element by element.
template <int D, bool GATED>
struct Epi {
    typedef typename Elem<D>::type T;
    static constexpr uint32_t TS = sizeof(T);
    // the operands of fp16 gradients' products are scaled (linear_slope)
    static constexpr bool SCALED = D == DT_F16 && !GATED;
    const EpiArgs& e;
    __amdgpu_buffer_rsrc_t y, r, z, u;
    const float *srow, *scol;
    int n0, row, col, rows, cols;
    uint32_t ys, oy, orr, oz, ou;  // bytes of an element of Y; the lane's offsets

    __device__ __forceinline__ Epi(const EpiArgs& a, int m0, int n0_, int out, int row_, int col_)
        : e(a), n0(n0_), row(row_), col(col_) {
        ys = sizeof(T) == 4 || e.out_f32 ? 4u : TS;
        y = make_rsrc((char*)(out ? e.Y[1] : e.Y[0]) + (m0 * e.ldy + n0) * (int64_t)ys);
        r = make_rsrc(e.R ? (const char*)e.R + (m0 * e.ldr + n0) * (int64_t)ys : nullptr);
        z = make_rsrc(e.Z ? (char*)e.Z + (m0 * e.ldz + n0) * (int64_t)TS : nullptr);
        u = make_rsrc(e.U ? (char*)e.U + (m0 * e.ldu + n0) * (int64_t)TS : nullptr);
        srow = scol = nullptr;
        if constexpr (SCALED) {
            if (const float* s = out ? e.rows[1] : e.rows[0]) srow = s + m0;
            if (const float* s = out ? e.cols[1] : e.cols[0]) scol = s + n0;
        }
        rows = e.M - m0;
        cols = e.N - n0;
        oy = (uint32_t)(row * (int)e.ldy + col) * ys;
        orr = (uint32_t)(row * (int)e.ldr + col) * ys;
        oz = (uint32_t)(row * (int)e.ldz + col) * TS;
        ou = (uint32_t)(row * (int)e.ldu + col) * TS;
    }
    // Columns of the group `by` rows on inside the output (8 or more: all).
    __device__ __forceinline__ int valid(int by) const { return row + by < rows ? cols - col : 0; }
    __device__ __forceinline__ bool same() const { return ys == TS; }  // Y has the operand type
    // A gradient has no bias: its columns' factors take that place.
    __device__ __forceinline__ f32x8 bias(int which) const {
        if (SCALED && scol)
            return cols - col < 8 ? zero8() : load8<float>(make_rsrc(scol), (uint32_t)col * 4u);
        if (!e.bias[which] || cols - col < 8) return zero8();
        return load8<T>(make_rsrc((const T*)e.bias[which] + n0), (uint32_t)col * TS);
    }
    // Whether the group `by` rows on is whole; its offset, or one out of range,
    // where loads give zeros and stores do nothing: no branch, so the groups of
    // a batch are scheduled together.
    __device__ __forceinline__ bool whole(int by) const { return row + by < rows && cols - col >= 8; }
    static __device__ __forceinline__ uint32_t at(bool ok, uint32_t o) { return ok ? o : OOB; }
    // The residual of a group as it lies in memory, where Y has the operand type.
    struct Raw {
        i32x4 a[sizeof(T) / 2];
    };
    __device__ __forceinline__ Raw residual(int by) const {
        const uint32_t o = at(whole(by), orr + (uint32_t)(by * (int)e.ldr) * TS);
        Raw x;
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i)
            x.a[i] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(r, o + 16 * i, 0, 0));
        return x;
    }
    static __device__ __forceinline__ f32x8 value(const Raw& x) {
        if constexpr (sizeof(T) == 4) {
            return join8(__builtin_bit_cast(f32x4, x.a[0]), __builtin_bit_cast(f32x4, x.a[1]));
        } else {
            const typename Vec8<T>::type h = __builtin_bit_cast(typename Vec8<T>::type, x.a[0]);
            f32x8 v;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = (float)h[i];
            return v;
        }
    }
    // U whole groups, `step` rows apart: v (gated: and w) the product's sums, b0
    // and b1 the biases, res the residual.  What is uniform is decided once for
    // all of them: a branch for each group and option took longer than the
    // arithmetic (325 clocks a group of eight columns with nothing to add).
    template <int KIND, int U>
    __device__ __forceinline__ void put(int by, int step, f32x8 (&v)[U], f32x8 (&w)[GATED ? U : 1], const f32x8& b0,
                                        const f32x8& b1, const Raw (&res)[U]) const {
        uint32_t o[U];
#pragma unroll
        for (int q = 0; q < U; ++q) o[q] = whole(by + q * step) ? 0u : OOB;
        const auto to = [&](int q, uint32_t lane, int64_t ld, uint32_t size) {
            return (lane + (uint32_t)((by + q * step) * (int)ld) * size) | o[q];
        };
        if (SCALED && srow) {
            const __amdgpu_buffer_rsrc_t s = make_rsrc(srow);
#pragma unroll
            for (int q = 0; q < U; ++q) v[q] *= load1<float>(s, (uint32_t)(row + by + q * step) * 4u | o[q]);
        }
        if (SCALED && scol) {
#pragma unroll
            for (int q = 0; q < U; ++q) v[q] *= b0;
        } else if (e.bias[0]) {
#pragma unroll
            for (int q = 0; q < U; ++q) v[q] += b0;
        }
        if (e.Z) {
#pragma unroll
            for (int q = 0; q < U; ++q) store8<T>(z, to(q, oz, e.ldz, TS), v[q]);
        }
#pragma unroll
        for (int q = 0; q < U; ++q) v[q] = act8<KIND>(e.act, v[q]);
        if constexpr (GATED) {
            if (e.bias[1]) {
#pragma unroll
                for (int q = 0; q < U; ++q) w[q] += b1;
            }
            if (e.U) {
#pragma unroll
                for (int q = 0; q < U; ++q) store8<T>(u, to(q, ou, e.ldu, TS), w[q]);
            }
#pragma unroll
            for (int q = 0; q < U; ++q) v[q] *= w[q];
        }
        if (same()) {
            if (e.R) {
#pragma unroll
                for (int q = 0; q < U; ++q) v[q] += value(res[q]);
            }
#pragma unroll
            for (int q = 0; q < U; ++q) store8<T>(y, to(q, oy, e.ldy, TS), v[q]);
        } else {
            if (e.R) {
#pragma unroll
                for (int q = 0; q < U; ++q) v[q] += load8<float>(r, to(q, orr, e.ldr, 4u));
            }
#pragma unroll
            for (int q = 0; q < U; ++q) store8<float>(y, to(q, oy, e.ldy, 4u), v[q]);
        }
    }
    // Element x of a group.
    template <int KIND>
    __device__ __forceinline__ void put1(int by, int x, float v, float w) const {
        const uint32_t bo = (uint32_t)(col + x) * TS, at = (uint32_t)x * ys;
        if (SCALED && (srow || scol))  // one of them
            v *= load1<float>(make_rsrc(srow ? srow : scol), (uint32_t)(srow ? row + by : col + x) * 4u);
        if (e.bias[0]) v += load1<T>(make_rsrc((const T*)e.bias[0] + n0), bo);
        if (e.Z) store1<T>(z, oz + (uint32_t)(by * (int)e.ldz + x) * TS, v);
        v = act1<KIND>(e.act, v);
        if constexpr (GATED) {
            if (e.bias[1]) w += load1<T>(make_rsrc((const T*)e.bias[1] + n0), bo);
            if (e.U) store1<T>(u, ou + (uint32_t)(by * (int)e.ldu + x) * TS, w);
            v *= w;
        }
        const uint32_t ro = orr + (uint32_t)(by * (int)e.ldr) * ys + at, o = oy + (uint32_t)(by * (int)e.ldy) * ys + at;
        if (same()) {
            if (e.R) v += load1<T>(r, ro);
            store1<T>(y, o, v);
        } else {
            if (e.R) v += load1<float>(r, ro);
            store1<float>(y, o, v);
        }
    }
};

// ---- the tile kernel ---------------------------------------------------------------------------

// Bound by the matrix cores, and by the clock they leave the part at.  What a
// wave reads from LDS per multiply-add falls with its share of the tile: one
// element for 64 where it is 128 x 128, for 43 where it is 128 x 64, for 32
// where it is 64 x 64; so the 256 x 256 tile has four waves, not eight.
// Measured, calls back to back on the same inputs:
//   256 x 256, bf16 4096^3           96.7 us W [N][K], 97.5 W [K][N], dW 97.7
//                                    (1421 TFLOP/s; eight waves of 128 x 64 101.8)
//   the same, inputs in no cache     99 to 104 us; bias, gelu_tanh, residual 111
//   gated, 4096 x 8192 x 4096        402 to 413 us with G and U kept (1350 TFLOP/s)
//   128 x 128 four stages, bf16      1024 x 4096 x 4096 33 us (1040 TFLOP/s)
//   128 x 128 two stages, bf16       2048 x 4096 x 4096 57 us (1200 TFLOP/s)
// A tile's fixed cost (first loads, epilogue) is 17 us of a 256 x 256 tile of
// K = 64; a second workgroup on the CU would hide it, but the accumulators and
// the ring fill the CU.
template <int D, int LA_, int LB_, int BM_, int BN_, int BK_, int S_, int WGM_, int WGN_, bool GATED_>
struct LinCfg {
    static constexpr int Dt = D, BM = BM_, BN = BN_, BK = BK_, S = S_, WGM = WGM_, WGN = WGN_;
    static constexpr bool GATED = GATED_;
    typedef Traits<D> T;
    static constexpr int ES = T::ES;
    static constexpr int NP = GATED ? 2 : 1;   // B panels side by side in LDS (gated: Wg, Wu)
    static constexpr int BNP = BN / NP;        // output columns of the tile
    typedef Opnd<D, LA_, BM, BK> OA;
    typedef Opnd<D, LB_, BNP, BK> OB;
    static constexpr int NW = WGM * WGN, NT = 64 * NW;
    // 16-bit types: one wave per SIMD and workgroup, its MFMAs placed by hand
    // (lone_step), its accumulators in AGPRs: all 256 for a wave of 128 x 128.
    // (fp32: the four MFMAs of a block depend on each other; left to the compiler.)
    static constexpr bool LONE = ES == 2 && NW == 4;
    static constexpr int WM = BM / WGM, WNP = BNP / WGN;
    static constexpr int FM = WM / 16, FNP = WNP / 16, FN = FNP * NP;
    static constexpr int A_BYTES = OA::BYTES, B_BYTES = OB::BYTES * NP;
    static constexpr int STAGE = A_BYTES + B_BYTES, LDS = S * STAGE;
    static constexpr int MINW = 163840 / LDS * NW / 4;  // waves per SIMD, by the CU's LDS
    static constexpr int A_INSTR = A_BYTES / 1024 / NW, B_INSTR = B_BYTES / 1024 / NW, LPS = A_INSTR + B_INSTR;
    static constexpr int NKS = BK / T::KSTEP;
    static_assert(NKS == 2, "the loop body is written for two K steps per K tile");
    static_assert(A_BYTES % (1024 * NW) == 0 && OB::BYTES % (1024 * (NW / NP)) == 0, "1-KiB blocks per wave");
    static_assert(LDS <= 163840 && S >= 2 && S <= 4 && LPS * (S - 2) <= 63, "ring");
};

template <class C>
struct LinFrags {
    i32x4 a[C::FM];
    i32x4 b[C::FN];
};

// The wave's side of the producer: descriptors of the next K tile of A and of
// the wave's B panel, and this wave's 1-KiB blocks of it.
template <class C>
struct LinSrc {
    i32x4 ra, rb;
    const char* ha;        // first K tile of the second contraction half
    const char* hb;
    int64_t sa, sb;        // bytes from one K tile to the next
    int turn;              // K tiles until the second half begins
    int left;              // K tiles still to load
    uint32_t va[C::A_INSTR], vb[C::B_INSTR];  // each lane's offset from the K tile's origin

    static __device__ __forceinline__ void move(i32x4& r, int64_t by) {
        const uint64_t p = (((uint64_t)(uint32_t)r[1] << 32) | (uint32_t)r[0]) + (uint64_t)by;
        r[0] = (int)(uint32_t)p;
        r[1] = (int)(uint32_t)(p >> 32);  // the address stays below 2^48: the stride field stays zero
    }
    // On to the next K tile, in four short parts that a lone wave spreads
    // between its MFMAs.  Slots past the last one get an empty range, so every
    // lane reads zeros.
    template <int PART>
    __device__ __forceinline__ void advance() {
        if constexpr (PART == 0) {
            --left;
            ra[2] = rb[2] = left > 0 ? (int)0x80000000u : 0;
        } else if constexpr (PART == 1) {
            move(ra, sa);
        } else if constexpr (PART == 2) {
            move(rb, sb);
        } else if (--turn == 0) {
            ra[0] = (int)(uint32_t)(uint64_t)ha;
            ra[1] = (int)(uint32_t)((uint64_t)ha >> 32);
            rb[0] = (int)(uint32_t)(uint64_t)hb;
            rb[1] = (int)(uint32_t)((uint64_t)hb >> 32);
        }
    }
    __device__ __forceinline__ void advance_all() {
        advance<0>();
        advance<1>();
        advance<2>();
        advance<3>();
    }
    // Block Q of the K tile, to LDS: its place (M0), and the load, which needs
    // an instruction between them.
    template <int Q>
    __device__ __forceinline__ void place(uint32_t a_lds, uint32_t b_lds) const {
        constexpr uint32_t off = (Q < C::A_INSTR ? Q : Q - C::A_INSTR) * 1024u;
        asm volatile("s_add_u32 m0, %0, %1" : : "s"(Q < C::A_INSTR ? a_lds : b_lds), "n"(off) : "m0", "scc");
    }
    template <int Q>
    __device__ __forceinline__ void load() const {
        asm volatile("buffer_load_dwordx4 %0, %1, 0 offen lds"
                     :
                     : "v"(Q < C::A_INSTR ? va[Q < C::A_INSTR ? Q : 0] : vb[Q < C::A_INSTR ? 0 : Q - C::A_INSTR]),
                       "s"(Q < C::A_INSTR ? ra : rb)
                     : "memory");
    }
};

template <class C, int Q0, int Q1>
__device__ __forceinline__ void lin_pieces(const LinSrc<C>& s, uint32_t a, uint32_t b) {
    if constexpr (Q0 < Q1) {
        s.template place<Q0>(a, b);
        asm volatile("s_nop 0");
        s.template load<Q0>();
        lin_pieces<C, Q0 + 1, Q1>(s, a, b);
    }
}

template <class C>
__device__ __forceinline__ void lin_read(const char PGEMM_LDS* stage, int ks, int r, int wm0, int wnp, int lane,
                                         LinFrags<C>& f) {
    // order b0, a0, b1 .. , a1 ..: the order in which the MFMAs need them
    if (r == 1 || r > C::FN) {
        const int i = r == 1 ? 0 : r - C::FN;
        C::OA::read(stage, ks, wm0 + 16 * i, lane, f.a[i]);
    } else {
        const int j = r == 0 ? 0 : r - 1;
        const int panel = j / C::FNP;
        C::OB::read(stage + C::A_BYTES + panel * C::OB::BYTES, ks, wnp + 16 * (j % C::FNP), lane, f.b[j]);
    }
}

// The MFMA of a lone wave, from inline asm with the accumulator held in AGPRs:
// left to the compiler, some accumulators land in VGPRs and 17 to 109
// registers spill.  The hazards the compiler cannot see are the caller's:
// acc_settle() between any other access to the accumulators and these.
template <int D>
__device__ __forceinline__ void mfma_lone(f32x4& acc, const i32x4& a, const i32x4& b) {
    if constexpr (D == DT_BF16)
        asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(b), "v"(a));
    else
        asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(acc) : "v"(b), "v"(a));
}
__device__ __forceinline__ void acc_settle() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// One K step of a lone wave.  No other wave of its workgroup issues on its SIMD,
// so what stands between two MFMAs has to fit the 16 clocks that the matrix core
// is busy with the first: one instruction in each place, or two where a step has
// only 16.  (With the sixteen LDS-DMA blocks' three instructions in a row in
// every second place the core was busy 57 % of the time.)  64 MFMAs a step: reads
// of the next fragments in places 0, 4, 8 ..; with DMA, each block's M0 and load
// in the two places behind them; without, the producer's way to the next K tile.
// (Every third place instead, which leaves the last quarter of the step free, is
// 2 % slower, 4 % with inputs in no cache.)  16 MFMAs: a read and an M0, then a
// load, in turns.
template <class C, bool READS, bool DMA, int M = 0>
__device__ __forceinline__ void lone_step(f32x4 (&acc)[C::FM][C::FN], const LinFrags<C>& use, LinFrags<C>& nxt,
                                          const char PGEMM_LDS* rstage, int rks, LinSrc<C>& src, uint32_t sa,
                                          uint32_t sb, int wm0, int wnp, int lane) {
    constexpr int NMF = C::FM * C::FN, NR = C::FM + C::FN;
    constexpr int EVERY = NMF >= 64 ? 4 : 2, Q = M / EVERY, SET = EVERY == 4 ? 1 : 0;
    static_assert(C::LPS <= NMF / EVERY && NR <= NMF / EVERY, "places");
    if constexpr (M < NMF) {
        mfma_lone<C::Dt>(acc[M / C::FN][M % C::FN], use.a[M / C::FN], use.b[M % C::FN]);
        if constexpr (READS && M % EVERY == 0 && Q < NR) lin_read<C>(rstage, rks, Q, wm0, wnp, lane, nxt);
        if constexpr (DMA && M % EVERY == SET && Q < C::LPS) src.template place<Q>(sa, sb);
        if constexpr (DMA && M % EVERY == SET + 1 && Q < C::LPS) src.template load<Q>();
        if constexpr (!DMA && M % EVERY == 1 && Q < 4) src.template advance<Q>();
        __builtin_amdgcn_sched_barrier(0);
        lone_step<C, READS, DMA, M + 1>(acc, use, nxt, rstage, rks, src, sa, sb, wm0, wnp, lane);
    }
}

// The MFMAs of one K step in eight groups; after each, a share of the next
// K tile's LDS-DMA blocks (DMA) and of the next step's fragment reads.
template <class C, bool READS, bool DMA, int G = 0>
__device__ __forceinline__ void lin_step(f32x4 (&acc)[C::FM][C::FN], const LinFrags<C>& use, LinFrags<C>& nxt,
                                         const char PGEMM_LDS* rstage, int rks, LinSrc<C>& src, uint32_t sa,
                                         uint32_t sb, int wm0, int wnp, int lane) {
    constexpr int NMF = C::FM * C::FN, NG = NMF < 8 ? NMF : 8, GS = NMF / NG;
    constexpr int NR = C::FM + C::FN, RPG = (NR + NG - 1) / NG, PPG = (C::LPS + NG - 1) / NG;
    if constexpr (C::LONE) {
        lone_step<C, READS, DMA>(acc, use, nxt, rstage, rks, src, sa, sb, wm0, wnp, lane);
    } else if constexpr (G < NG) {
#pragma unroll
        for (int m = G * GS; m < (G + 1) * GS; ++m)
            mfma_swapped<C::Dt>(acc[m / C::FN][m % C::FN], use.a[m / C::FN], use.b[m % C::FN]);
        if constexpr (DMA) {
            constexpr int P0 = G * PPG < C::LPS ? G * PPG : C::LPS;
            constexpr int P1 = (G + 1) * PPG < C::LPS ? (G + 1) * PPG : C::LPS;
            lin_pieces<C, P0, P1>(src, sa, sb);
        }
        if constexpr (READS) {
#pragma unroll
            for (int r = G * RPG; r < (G + 1) * RPG; ++r)
                if (r < NR) lin_read<C>(rstage, rks, r, wm0, wnp, lane, nxt);
        }
        __builtin_amdgcn_sched_barrier(0);
        lin_step<C, READS, DMA, G + 1>(acc, use, nxt, rstage, rks, src, sa, sb, wm0, wnp, lane);
    }
}

// Full wait of this wave's loads and LDS operations, then the barrier.
__device__ __forceinline__ void drain_barrier() { wait_barrier<0>(); }

// The epilogue goes through LDS: the accumulators' lanes hold four columns of
// sixteen rows, and indexing them needs straight-line code, which for a whole
// tile (128 groups a lane, several activations) is far larger than the
// instruction cache and was fetched at 13 to 36 us a tile.  Each wave writes
// its sums to its own part of the ring's memory (16-byte chunks, XOR-swizzled
// by the row against bank conflicts), in as many passes as fit, and a short
// loop reads them back eight columns a lane, a row's lanes side by side.
template <class C>
struct LinOut {
    static constexpr int WN = C::FN * 16, NCHK = WN / 4;    // sums of a row; in 16-byte chunks
    static constexpr int AREA = C::LDS / C::NW;              // bytes of a wave
    static constexpr int FIT = AREA / (WN * 4) / 16;         // 16-row blocks that fit
    static constexpr int BLOCKS = FIT < C::FM ? FIT : C::FM;  // of a pass
    static constexpr int PASSES = C::FM / BLOCKS;
    static constexpr int LPR = C::WNP / 8;                   // lanes of a row
    static constexpr int RPI = 64 / LPR;                     // rows at a time
    static constexpr int STEPS = BLOCKS * 16 / RPI;
    // Groups of a lane in flight (with the next batch's residual): what the
    // registers beside the accumulators hold.
    static constexpr int WANT = C::ES == 4 ? (C::GATED ? 1 : 2) : C::GATED ? 2 : 4;
    static constexpr int UNROLL = STEPS < WANT ? STEPS : WANT;
    static_assert(PASSES * BLOCKS == C::FM && STEPS % UNROLL == 0 && (NCHK & (NCHK - 1)) == 0, "passes");
    // Even chunks in the first half of a row, odd ones in the second: the lanes
    // of a row read every second chunk at a time.
    static PGEMM_HD int at(int row, int chunk) {
        return (row * NCHK + (chunk & 1) * (NCHK / 2) + ((chunk >> 1) ^ (row & (NCHK / 2 - 1)))) * 16;
    }
};

template <class C>
__device__ __forceinline__ void lin_epilogue(const EpiArgs& e, int m0, int n0, int out, char PGEMM_LDS* smem,
                                             f32x4 (&acc)[C::FM][C::FN], int wave, int lane, int wm0, int wnp) {
    typedef LinOut<C> O;
    const int li = lane & 15, lg = lane >> 4, r0 = lane / O::LPR, c8 = lane % O::LPR;
    const Epi<C::Dt, C::GATED> ep(e, m0, n0, out, wm0 + r0, wnp + 8 * c8);
    char PGEMM_LDS* area = smem + wave * O::AREA;
    const f32x8 b0 = ep.bias(0), b1 = C::GATED ? ep.bias(1) : b0;
    // The residual of the next batch of groups is under way while one is
    // computed, across the passes too: what a CU has in flight bounds how fast
    // the tile's residual arrives.
    typename Epi<C::Dt, C::GATED>::Raw next[O::UNROLL];
    const auto fetch = [&](int by) {
        if (!e.R || !ep.same()) return;
#pragma unroll
        for (int q = 0; q < O::UNROLL; ++q) next[q] = ep.residual(by + q * O::RPI);
    };
    fetch(0);
    drain_barrier();  // the ring's memory is free
#pragma unroll 1
    for (int pass = 0; pass < O::PASSES; ++pass) {
#pragma unroll
        for (int p = 0; p < O::PASSES; ++p) {
            if (p != pass) continue;
#pragma unroll
            for (int i = 0; i < O::BLOCKS; ++i)
#pragma unroll
                for (int j = 0; j < C::FN; ++j)
                    *(f32x4 PGEMM_LDS*)(area + O::at(16 * i + li, 4 * j + lg)) = acc[p * O::BLOCKS + i][j];
        }
        asm volatile("" ::: "memory");  // a wave's LDS operations stay in order
        const int down = pass * O::BLOCKS * 16;
        with_act(e.act.kind, [&](auto kind) {
            constexpr int KIND = decltype(kind)::value;
#pragma unroll 1
            for (int s = 0; s < O::STEPS; s += O::UNROLL) {
                typename Epi<C::Dt, C::GATED>::Raw res[O::UNROLL];
                f32x8 v[O::UNROLL], w[C::GATED ? O::UNROLL : 1];
#pragma unroll
                for (int q = 0; q < O::UNROLL; ++q) res[q] = next[q];
                fetch(down + (s + O::UNROLL) * O::RPI);
#pragma unroll
                for (int q = 0; q < O::UNROLL; ++q) {
                    const int row = r0 + (s + q) * O::RPI;
                    const auto sums = [&](int c) {
                        return join8(*(const f32x4 PGEMM_LDS*)(area + O::at(row, c)),
                                     *(const f32x4 PGEMM_LDS*)(area + O::at(row, c + 1)));
                    };
                    v[q] = sums(2 * c8);
                    if constexpr (C::GATED) w[q] = sums(C::WNP / 4 + 2 * c8);
                }
                ep.template put<KIND>(down + s * O::RPI, O::RPI, v, w, b0, b1, res);
            }
            if (cols_cut(e.N)) {
#pragma unroll 1
                for (int s = 0; s < O::STEPS; ++s) {
                    const int n = ep.valid(down + s * O::RPI);
#pragma unroll 1
                    for (int x = 0; x < (n < 8 ? n : 0); ++x) {
                        const auto one = [&](int c) {
                            return *(const float PGEMM_LDS*)(area + O::at(r0 + s * O::RPI, c >> 2) + 4 * (c & 3));
                        };
                        ep.template put1<KIND>(down + s * O::RPI, x, one(8 * c8 + x),
                                               C::GATED ? one(C::WNP + 8 * c8 + x) : 0.0f);
                    }
                }
            }
        });
        asm volatile("" ::: "memory");
    }
}

template <class C>
__global__ void __launch_bounds__(C::NT, C::MINW) linear_kernel(LinArgs g) {
    __shared__ __attribute__((aligned(1024))) char smem_raw[C::LDS];
    char PGEMM_LDS* smem = (char PGEMM_LDS*)smem_raw;
    typedef typename C::OA OA;
    typedef typename C::OB OB;

    // Logical tiles: output tiles in a grouped raster, split-major, one
    // contiguous range per XCD (wg_tiles_of).
    const int tiles_n = g.tiles_n * g.outs, per_split = g.tiles_m * tiles_n;
    const WgTiles w = wg_tiles_of(per_split * g.splits, (int)blockIdx.x, (int)gridDim.x);
    if (w.count == 0) return;
    int L = w.start + w.lb, split = 0;
    if (g.splits > 1) {
        split = __builtin_amdgcn_readfirstlane(L / per_split);
        L -= split * per_split;
    }
    int tm, tn;
    raster(L, g.tiles_m, tiles_n, g.group_m, tm, tn);
    tm = __builtin_amdgcn_readfirstlane(tm);
    tn = __builtin_amdgcn_readfirstlane(tn);
    const int out = tn >= g.tiles_n ? 1 : 0;
    tn -= out * g.tiles_n;
    const int m0 = tm * C::BM, n0 = tn * C::BNP;

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm0 = (wave / C::WGN) * C::WM;
    const int wnp = (wave % C::WGN) * C::WNP;
    const int rows_left = g.e.M - m0, cols_left = g.e.N - n0;

    f32x4 acc[C::FM][C::FN];
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if constexpr (C::LONE) acc_settle();

    // This split's K tiles of the ring: [t0, t1) of both halves' nfull.
    const int64_t total = (int64_t)g.nfull * g.halves;
    const int t0 = (int)(total * split / g.splits), t1 = (int)(total * (split + 1) / g.splits);
    const int panel = C::NP == 2 ? wave / (C::NW / 2) : 0;  // the wave's blocks of B lie in one panel
    const int b_block = wave * C::B_INSTR - panel * (OB::BYTES / 1024);
    const int b_base = C::A_BYTES + wave * C::B_INSTR * 1024, a_base = wave * C::A_INSTR * 1024;
    const char* a_half[2];
    const char* b_half[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int i = g.outs == 2 ? out : h < g.halves ? h : 0;
        a_half[h] = (const char*)g.A[i] + OA::origin(m0, 0, g.lda);
        b_half[h] = (const char*)g.B[C::NP == 2 ? panel : i] + OB::origin(n0, 0, g.ldb);
    }

    if (t1 > t0) {
        LinSrc<C> src;
        const int half = t0 >= g.nfull ? 1 : 0;
        int first = t0 - half * g.nfull;
        // With the whole contraction in one go, the XCDs begin at different
        // places of it and come round to their start: what several read, one
        // then fetches from memory and the others find in the shared cache,
        // in turns.  Neighbours (x, x ^ 1), which mostly share rows, start half
        // of K apart, and those of one parity, which share columns, a quarter.
        // 4096^3 with inputs in no cache: 109 us in step, 107 us with XCD x at
        // x / 8 (where one of two neighbours fetches 7/8 of their rows).
        const bool round = g.halves == 1 && g.splits == 1;
        const int x = blockIdx.x & 7;
        if (round) first = (int)((int64_t)g.nfull * (((x & 6) + 4 * (x & 1)) & 7) >> 3);
        src.turn = half ? 0x7fffffff : g.nfull - first;
        src.left = t1 - t0;
        src.sa = OA::step(g.lda);
        src.sb = OB::step(g.ldb);
        src.ra = make_rsrc_sgpr((half ? a_half[1] : a_half[0]) + src.sa * first);
        src.rb = make_rsrc_sgpr((half ? b_half[1] : b_half[0]) + src.sb * first);
        src.ha = round ? a_half[0] : a_half[1];
        src.hb = round ? b_half[0] : b_half[1];
#pragma unroll
        for (int q = 0; q < C::A_INSTR; ++q) {
            int e, k;
            OA::chunk(a_base + q * 1024 + lane * 16, e, k);
            src.va[q] = e < rows_left ? OA::mem_off(e, k, g.lda) : OOB;
        }
#pragma unroll
        for (int q = 0; q < C::B_INSTR; ++q) {
            int e, k;
            OB::chunk((b_block + q) * 1024 + lane * 16, e, k);
            src.vb[q] = e < cols_left ? OB::mem_off(e, k, g.ldb) : OOB;
        }

        const uint32_t lds0 = (uint32_t)(size_t)smem;
        // Prologue: slots 0 .. S-2.
#pragma unroll
        for (int p = 0; p < C::S - 1; ++p) {
            lin_pieces<C, 0, C::LPS>(src, lds0 + p * C::STAGE + a_base, lds0 + p * C::STAGE + b_base);
            src.advance_all();
        }
        wait_barrier<C::LPS*(C::S - 2)>();
        lin_pieces<C, 0, C::LPS>(src, lds0 + (C::S - 1) * C::STAGE + a_base, lds0 + (C::S - 1) * C::STAGE + b_base);
        LinFrags<C> f[2];
#pragma unroll
        for (int r = 0; r < C::FM + C::FN; ++r) lin_read<C>(smem, 0, r, wm0, wnp, lane, f[0]);
        int cur = 0;
        for (int t = t0; t < t1; ++t) {
            const int nst = cur + 1 == C::S ? 0 : cur + 1;
            lin_step<C, true, false>(acc, f[0], f[1], smem + cur * C::STAGE, 1, src, 0, 0, wm0, wnp, lane);
            wait_barrier<C::LPS*(C::S - 2)>();  // K tile t+1 is in LDS, stage `cur` is free
            if constexpr (!C::LONE) src.advance_all();
            const uint32_t freed = lds0 + cur * C::STAGE;
            lin_step<C, true, true>(acc, f[1], f[0], smem + nst * C::STAGE, 0, src, freed + a_base, freed + b_base,
                                    wm0, wnp, lane);
            cur = nst;
        }
        __builtin_amdgcn_s_waitcnt(0);  // no load may still be writing LDS
    }

    // What is left of each half after the ring's K tiles, by the last split.
    if (split == g.splits - 1) {
        const int ncut = (g.K + C::BK - 1) / C::BK - g.nfull;
        for (int c = 0; c < ncut * g.halves; ++c) {
            const int h = c >= ncut ? 1 : 0, kt = g.nfull + c - h * ncut, k_left = g.K - kt * C::BK;
            drain_barrier();  // every wave has read the stage
            OA::template load_cut<C::A_INSTR>((h ? a_half[1] : a_half[0]) + OA::step(g.lda) * kt, g.lda, rows_left,
                                              k_left, OA::along_k ? g.K : g.e.M, smem, wave * C::A_INSTR, lane);
            OB::template load_cut<C::B_INSTR>((h ? b_half[1] : b_half[0]) + OB::step(g.ldb) * kt, g.ldb, cols_left,
                                              k_left, OB::along_k ? g.K : g.e.N,
                                              smem + C::A_BYTES + panel * OB::BYTES, b_block, lane);
            drain_barrier();
            LinFrags<C> f;
#pragma unroll
            for (int ks = 0; ks < C::NKS; ++ks) {
#pragma unroll
                for (int r = 0; r < C::FM + C::FN; ++r) lin_read<C>(smem, ks, r, wm0, wnp, lane, f);
#pragma unroll
                for (int m = 0; m < C::FM * C::FN; ++m) {
                    if constexpr (C::LONE)
                        mfma_lone<C::Dt>(acc[m / C::FN][m % C::FN], f.a[m / C::FN], f.b[m % C::FN]);
                    else
                        mfma_swapped<C::Dt>(acc[m / C::FN][m % C::FN], f.a[m / C::FN], f.b[m % C::FN]);
                }
            }
        }
    }
    if constexpr (C::LONE) acc_settle();

    const int li = lane & 15, lg4 = 4 * (lane >> 4);
    if (g.part) {
        // fp32 sums of this split, joined by linear_join in the order of the splits
        const int planes = C::GATED ? 2 : g.outs;
        float* base = g.part + ((int64_t)split * planes + out) * g.e.M * g.np8;
#pragma unroll
        for (int i = 0; i < C::FM; ++i) {
            const int row = m0 + wm0 + 16 * i + li;
#pragma unroll
            for (int j = 0; j < C::FN; ++j) {
                const int col = n0 + wnp + 16 * (j % C::FNP) + lg4;
                if (row < g.e.M && col < g.np8)
                    *(f32x4*)(base + ((int64_t)(j / C::FNP) * g.e.M + row) * g.np8 + col) = acc[i][j];
            }
        }
        return;
    }
    lin_epilogue<C>(g.e, m0, n0, out, smem, acc, wave, lane, wm0, wnp);
}

// ---- few rows -----------------------------------------------------------------------------------

// One token to a few dozen: the weights' bytes bound the time, so what counts is
// how many of them each CU has under way.  The waves of a workgroup share its
// output tile (16 FM rows, NCOL columns) and deal out its K tiles in turn; each
// has a ring of its own, which only it fills and reads, so nothing in the loop
// waits for another wave: a wave waits for its own oldest K tile (vmcnt) while
// S - 1 more are in flight.  At the end the waves' sums are added in LDS, in the
// order of the waves.
// Measured, bf16 weights from memory: one token by 4096 x 4096 8.2 us (4.1 TB/s,
// of which 2 us are the launch and the first loads), 16 by 4096 x 16384 28.6 us
// (4.7 TB/s) and 4.6 for the join, one token gated to 16384 x 4096 50.5 us (5.3
// TB/s); a kernel that only reads takes 6.3 us for the first (5.3 TB/s), 20.9 and
// 40.7 for the others (6.4, 6.6).
template <int D, int LA_, int LB_, int FM_, int NCOL_, int NW_, int S_, bool GATED_>
struct FewCfg {
    static constexpr int Dt = D, FM = FM_, NCOL = NCOL_, NW = NW_, S = S_;
    static constexpr bool GATED = GATED_;
    static constexpr int NP = GATED ? 2 : 1, NCOLP = NCOL / NP;  // output columns of the tile
    static constexpr int ES = Traits<D>::ES, BK = 128 / ES, NKS = BK / Traits<D>::KSTEP;
    static constexpr int BM = 16 * FM, NT = 64 * NW;
    typedef Opnd<D, LA_, BM, BK> OA;
    typedef Opnd<D, LB_, NCOLP, BK> OB;
    static constexpr int FNP = NCOLP / 16, FN = FNP * NP;
    static constexpr int STAGE = OA::BYTES + NP * OB::BYTES, RING = S * STAGE, LDS = NW * RING;
    static constexpr int LPA = OA::BYTES / 1024, LPB = OB::BYTES / 1024, LPS = LPA + NP * LPB;
    static_assert(LDS <= 163840 && S >= 2 && LPS * (S - 2) <= 63, "ring");
    static_assert(FM * FN * 1024 <= RING, "the sums fit the wave's ring");
    static_assert(NKS == 2, "K steps");
};

template <class C>
__device__ __forceinline__ void few_multiply(f32x4 (&acc)[C::FM][C::FN], const char PGEMM_LDS* stage, int lane) {
#pragma unroll
    for (int ks = 0; ks < C::NKS; ++ks) {
        i32x4 a[C::FM], b[C::FN];
#pragma unroll
        for (int i = 0; i < C::FM; ++i) C::OA::read(stage, ks, 16 * i, lane, a[i]);
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
            C::OB::read(stage + C::OA::BYTES + (j / C::FNP) * C::OB::BYTES, ks, 16 * (j % C::FNP), lane, b[j]);
#pragma unroll
        for (int i = 0; i < C::FM; ++i)
#pragma unroll
            for (int j = 0; j < C::FN; ++j) mfma_swapped<C::Dt>(acc[i][j], a[i], b[j]);
    }
}

template <class C>
__global__ void __launch_bounds__(C::NT) linear_few(LinArgs g) {
    __shared__ __attribute__((aligned(1024))) char smem_raw[C::LDS];
    typedef typename C::OA OA;
    typedef typename C::OB OB;
    const int tiles_n = g.tiles_n * g.outs, per_split = g.tiles_m * tiles_n;
    const WgTiles w = wg_tiles_of(per_split * g.splits, (int)blockIdx.x, (int)gridDim.x);
    if (w.count == 0) return;
    int L = w.start + w.lb, split = 0;
    if (g.splits > 1) {
        split = __builtin_amdgcn_readfirstlane(L / per_split);
        L -= split * per_split;
    }
    // row tiles of the same columns side by side: they share the weights in L2
    int tn = __builtin_amdgcn_readfirstlane(L / g.tiles_m);
    const int tm = L - tn * g.tiles_m, out = tn >= g.tiles_n ? 1 : 0;
    tn -= out * g.tiles_n;
    const int m0 = tm * C::BM, n0 = tn * C::NCOLP;
    const int rows_left = g.e.M - m0, cols_left = g.e.N - n0;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    char PGEMM_LDS* ring = (char PGEMM_LDS*)smem_raw + wave * C::RING;
    const uint32_t lds0 = (uint32_t)(size_t)ring;

    const char* a_half[2];
    const char* b_half[2];  // gated: the two panels
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int i = g.outs == 2 ? out : h < g.halves ? h : 0;
        a_half[h] = (const char*)g.A[i] + OA::origin(m0, 0, g.lda);
        b_half[h] = (const char*)g.B[C::NP == 2 ? h : i] + OB::origin(n0, 0, g.ldb);
    }
    const int64_t sa = OA::step(g.lda), sb = OB::step(g.ldb);
    uint32_t va[C::LPA], vb[C::LPB];
#pragma unroll
    for (int q = 0; q < C::LPA; ++q) {
        int e, k;
        OA::chunk(q * 1024 + lane * 16, e, k);
        va[q] = e < rows_left ? OA::mem_off(e, k, g.lda) : OOB;
    }
#pragma unroll
    for (int q = 0; q < C::LPB; ++q) {
        int e, k;
        OB::chunk(q * 1024 + lane * 16, e, k);
        vb[q] = e < cols_left ? OB::mem_off(e, k, g.ldb) : OOB;
    }

    f32x4 acc[C::FM][C::FN];
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    // This split's K tiles [t0, t1); the wave's are t0 + wave, + NW, ...
    const int64_t total = (int64_t)g.nfull * g.halves;
    const int t0 = (int)(total * split / g.splits), t1 = (int)(total * (split + 1) / g.splits);
    // Tiles of 64 rows of W [N][K] with the whole contraction begin at one of
    // eight places of it, and come round: workgroups in step read rows a power of
    // two apart at the same offset (one token to 16384 x 4096 31.3 -> 28.2 us, gated
    // 60 -> 52, to 32768 x 8192 110 -> 100; gated to 14336 x 4096 48.3 -> 48.5).  Not
    // narrower tiles (gated to 8192 x 4096 28 -> 32, 4096 x 4096 8.9 -> 9.3) or
    // W [K][N] (9460 x 6427 gated 62 -> 74).
    const int turn = C::NCOLP == 64 && C::OB::along_k && g.splits == 1 && g.halves == 1
                         ? (int)((int64_t)(t1 - t0) * (tn & 7) >> 3) : 0;
    // Loads K tile t into stage st; past the last one every lane reads zeros.
    const auto issue = [&](int t, int st) {
        const int range = t < t1 ? (int)0x80000000u : 0;
        t += turn;  // comes round
        if (t >= t1) t -= t1 - t0;
        const int h = t >= g.nfull ? 1 : 0, kt = t - h * g.nfull;
        const uint32_t at = lds0 + (uint32_t)(st * C::STAGE);
        i32x4 r = make_rsrc_sgpr((h ? a_half[1] : a_half[0]) + sa * kt);
        r[2] = range;
#pragma unroll
        for (int q = 0; q < C::LPA; ++q) dma16(r, va[q], at + q * 1024u);
#pragma unroll
        for (int p = 0; p < C::NP; ++p) {
            r = make_rsrc_sgpr((C::NP == 2 ? b_half[p] : h ? b_half[1] : b_half[0]) + sb * kt);
            r[2] = range;
#pragma unroll
            for (int q = 0; q < C::LPB; ++q) dma16(r, vb[q], at + OA::BYTES + p * OB::BYTES + q * 1024u);
        }
    };
    int t = t0 + wave;
    if (t < t1) {
#pragma unroll
        for (int p = 0; p < C::S - 1; ++p) issue(t + p * C::NW, p);
        int st = 0;
        for (; t < t1; t += C::NW) {
            // the oldest K tile has landed, and the stage before it has been read
            lgkm_drain();
            asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" : : "n"(C::LPS * (C::S - 2)) : "memory");
            issue(t + (C::S - 1) * C::NW, st == 0 ? C::S - 1 : st - 1);
            few_multiply<C>(acc, ring + st * C::STAGE, lane);
            st = st + 1 == C::S ? 0 : st + 1;
        }
    }
    __builtin_amdgcn_s_waitcnt(0);  // no load may still be writing LDS
    asm volatile("" ::: "memory");
    // What is left of each half after the ring's K tiles, one cut tile a wave.
    if (split == g.splits - 1) {
        const int ncut = (g.K + C::BK - 1) / C::BK - g.nfull;
        for (int c = wave; c < ncut * g.halves; c += C::NW) {
            const int h = c >= ncut ? 1 : 0, kt = g.nfull + c - h * ncut, k_left = g.K - kt * C::BK;
            OA::template load_cut<C::LPA>((h ? a_half[1] : a_half[0]) + sa * kt, g.lda, rows_left, k_left,
                                          OA::along_k ? g.K : g.e.M, ring, 0, lane);
#pragma unroll
            for (int p = 0; p < C::NP; ++p)
                OB::template load_cut<C::LPB>((C::NP == 2 ? b_half[p] : h ? b_half[1] : b_half[0]) + sb * kt, g.ldb,
                                              cols_left, k_left, OB::along_k ? g.K : g.e.N,
                                              ring + OA::BYTES + p * OB::BYTES, 0, lane);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            few_multiply<C>(acc, ring, lane);
            lgkm_drain();
            asm volatile("" ::: "memory");
        }
    }

    // The waves' sums, each in its own ring.
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; ++j) *(f32x4 PGEMM_LDS*)(ring + ((i * C::FN + j) * 64 + lane) * 16) = acc[i][j];
    lgkm_barrier();
    constexpr int GPR = C::NCOLP / 8, GROUPS = C::BM * GPR;  // groups of eight columns
    for (int q = (int)threadIdx.x; q < GROUPS; q += C::NT) {
        const int row = q / GPR, c8 = q % GPR;
        if (row >= rows_left || 8 * c8 >= cols_left) continue;
        f32x8 s[C::NP];
#pragma unroll
        for (int p = 0; p < C::NP; ++p) {
            s[p] = zero8();
            const int block = (row >> 4) * C::FN + p * C::FNP + (c8 >> 1);
            const char PGEMM_LDS* at =
                (const char PGEMM_LDS*)smem_raw + (block * 64 + (row & 15) + 32 * (c8 & 1)) * 16;
#pragma unroll
            for (int v = 0; v < C::NW; ++v)
                s[p] += join8(*(const f32x4 PGEMM_LDS*)(at + v * C::RING), *(const f32x4 PGEMM_LDS*)(at + v * C::RING + 256));
        }
        if (g.part) {
            const int planes = C::GATED ? 2 : g.outs;
            float* o = g.part + (((int64_t)split * planes + out) * g.e.M + m0 + row) * g.np8 + n0 + 8 * c8;
#pragma unroll
            for (int p = 0; p < C::NP; ++p) *(f32x8*)(o + (int64_t)p * g.e.M * g.np8) = s[p];
            continue;
        }
        const Epi<C::Dt, C::GATED> ep(g.e, m0, n0, out, row, 8 * c8);
        const f32x8 b0 = ep.bias(0), b1 = C::GATED ? ep.bias(1) : b0;
        typename Epi<C::Dt, C::GATED>::Raw res[1] = {};
        if (g.e.R && ep.same()) res[0] = ep.residual(0);
        f32x8 v[1] = {s[0]}, u[1] = {s[C::NP - 1]};
        with_act(g.e.act.kind, [&](auto kind) {
            constexpr int KIND = decltype(kind)::value;
            ep.template put<KIND>(0, 0, v, u, b0, b1, res);
            if (!ep.whole(0)) {
#pragma unroll
                for (int x = 0; x < 7; ++x)
                    if (x < ep.valid(0)) ep.template put1<KIND>(0, x, s[0][x], s[C::NP - 1][x]);
            }
        });
    }
}

// ---- join of the splits ---------------------------------------------------------------------------

// One thread per eight columns of a row: the splits' sums in the order of the
// splits, then the epilogue.  A workgroup covers one row's stretch of
// kJoinCols columns.  Bound by the launch (4 us) for few rows, by memory for
// many: two splits of 2048 x 4096, 84 MB, 15.6 us (5.4 TB/s, part of it from the
// shared cache).
constexpr int kJoinCols = 512;

template <int D, bool GATED>
__global__ void __launch_bounds__(kJoinCols / 8) linear_join(LinArgs g) {
    const int strips = (g.e.N + kJoinCols - 1) / kJoinCols;
    int b = (int)blockIdx.x;
    const int strip = b % strips;
    b /= strips;
    const int m = b % g.e.M, out = b / g.e.M;
    const int n0 = strip * kJoinCols, col = 8 * (int)threadIdx.x;
    if (n0 + col >= g.e.N) return;
    const int planes = GATED ? 2 : g.outs;
    const int64_t plane = (int64_t)g.e.M * g.np8;
    const float* p = g.part + out * plane + (int64_t)m * g.np8 + n0 + col;
    const Epi<D, GATED> ep(g.e, m, n0, out, 0, col);
    const f32x8 b0 = ep.bias(0), b1 = GATED ? ep.bias(1) : b0;
    typename Epi<D, GATED>::Raw res[1] = {};
    if (g.e.R && ep.same()) res[0] = ep.residual(0);
    f32x8 v[1] = {zero8()}, w[1] = {zero8()};
#pragma unroll 4
    for (int s = 0; s < g.splits; ++s) {
        v[0] += *(const f32x8*)p;
        if constexpr (GATED) w[0] += *(const f32x8*)(p + plane);
        p += planes * plane;
    }
    with_act(g.e.act.kind, [&](auto kind) {
        constexpr int KIND = decltype(kind)::value;
        if (!ep.whole(0)) {
#pragma unroll
            for (int x = 0; x < 7; ++x)
                if (x < ep.valid(0)) ep.template put1<KIND>(0, x, v[0][x], w[0][x]);
        }
        ep.template put<KIND>(0, 0, v, w, b0, b1, res);
    });
}

// ---- gradients at the pre-activations -----------------------------------------------------------

// linear: dZ = dY act'(Z).  gated: dG = dH U act'(G), dU = dH act(G).
// They are rounded to the operand type (the matrix cores take no wider one):
// each factor of the products that follow then carries half a step of that
// type, as X and W do, and the sums over them stay in fp32.  The column sums
// (bias gradients) add the unrounded values.
//
// bf16 has fp32's range.  fp16 has not: dG of fp16 tensors lies anywhere between
// 2^-48 and 2^33, with dH = U = 300 already beyond its largest value.  So fp16
// gradients are held divided by powers of two, which the products' epilogues
// multiply back in fp32: one factor for each row in the copy that dX contracts,
// one for each column in the copy that dW contracts (a factor has to stand outside
// the sum).  Each brings the row's (column's) largest finite entry into [2^14,
// 2^15), so an entry is rounded to fp16's 11 bits down to 2^-29 of that, and off by
// at most 2^-39 of it below.  That takes two passes, over inputs that the second
// finds in the shared cache: SLOPE_RANGE (largest entries, and the column sums),
// linear_colsum (factors), SLOPE_SCALED (the copies).  Where only bias gradients are
// asked for, fp16 runs SLOPE_RANGE too, so that they have the same bits.
//
// Bound by memory: bf16 reads and writes of 2048 x 8192 gated (168 MB) take
// 33.5 us, 5.0 TB/s; of 4096 x 4096 (101 MB) 21.5 to 25.7 us, 4.3 TB/s.  256-byte
// stretches of a row and two rows under way a thread: stretches of 512 bytes
// take 22.7 us for the latter but 37 for the former, four rows under way 52.
// fp16, 2048 x 8192 gated: 39 and 41 us in the two passes, 5 for the factors (one
// pass without factors 37); 1000 x 2003 12, 10 and 5 (one pass 12).
enum SlopePass : int { SLOPE_PLAIN = 0, SLOPE_RANGE = 1, SLOPE_SCALED = 2 };

struct SlopeArgs {
    const void* dY;
    const void* Z;      // linear: Z; gated: G
    const void* U;      // gated
    void* dZ[2];        // linear: dZ; gated: dG, dU (scaled: by rows); null: not stored
    void* dZc[2];       // scaled: by columns
    int64_t ldy, ldz, ldu, ldd;
    float* sums;        // [row block][planes][np8] column sums; null: none
    float* row_max;     // range: [strip][M] largest entries of the planes; null: none
    float* col_max;     // range: [row block][planes][np8]; null: none
    const float* rows;  // scaled: factors [M]
    const float* cols;  // scaled: factors [planes][np8]
    int np8;
    int steps;          // of kSlopeRows rows a workgroup
    int M, N;
    ActArgs act;
};

constexpr int kSlopeRows = 32;   // rows per step: two for each of 16 row groups, both under way at once
constexpr int kSlopeCols = 128;  // columns per workgroup: 16 threads of eight columns

// The first `valid` of eight elements at byte offset `off`, zeros for the rest.
template <class T>
__device__ __forceinline__ f32x8 load_cut8(__amdgpu_buffer_rsrc_t r, uint32_t off, int valid) {
    if (valid >= 8) return load8<T>(r, off);
    f32x8 v = zero8();
#pragma unroll
    for (int x = 0; x < 7; ++x)
        if (x < valid) v[x] = load1<T>(r, off + (uint32_t)(x * sizeof(T)));
    return v;
}

// The factor of a row or column whose largest entry is m >= 0: 2^(floor(log2 m) - 14),
// from the exponent's bits, and 1 where there is nothing but zeros.  Entries below
// 2^-95 need no more (the clamp keeps factor and inverse normal).
__device__ __forceinline__ float scale_of(float m) {
    const uint32_t ex = __builtin_bit_cast(uint32_t, m) >> 23;
    return m == 0.0f ? 1.0f : __builtin_bit_cast(float, (ex < 32u ? 18u : ex - 14u) << 23);
}
// 1 / s of a power of two.
__device__ __forceinline__ float inverse(float s) {
    return __builtin_bit_cast(float, 0x7f000000u - __builtin_bit_cast(uint32_t, s));
}
// |x|, or 0 where x is infinite or NaN (those stay what they are under any factor).
__device__ __forceinline__ float finite_abs(float x) {
    const float a = __builtin_fabsf(x);
    return a < __builtin_huge_valf() ? a : 0.0f;
}

template <int D, bool GATED, int PASS>
__global__ void __launch_bounds__(256) linear_slope(SlopeArgs g) {
    typedef typename Elem<D>::type T;
    constexpr int planes = GATED ? 2 : 1;
    __shared__ f32x8 red[planes][256];
    const int strips = (g.N + kSlopeCols - 1) / kSlopeCols;
    const int strip = (int)blockIdx.x % strips, block = (int)blockIdx.x / strips;
    const int n0 = strip * kSlopeCols, m0 = block * g.steps * kSlopeRows;
    const int col = 8 * ((int)threadIdx.x & 15), r0 = (int)threadIdx.x >> 4;
    const int rows = g.M - m0 < g.steps * kSlopeRows ? g.M - m0 : g.steps * kSlopeRows;
    const int valid = g.N - n0 - col;
    const auto at = [&](const void* p, int64_t ld) {
        return make_rsrc(p ? (const char*)p + (m0 * ld + n0) * (int64_t)sizeof(T) : nullptr);
    };
    const __amdgpu_buffer_rsrc_t ry = at(g.dY, g.ldy), rz = at(g.Z, g.ldz), ru = at(g.U, g.ldu);
    f32x8 s[planes], most[planes], down[planes];  // column sums, largest entries; 1 / the columns' factors
#pragma unroll
    for (int p = 0; p < planes; ++p) {
        s[p] = most[p] = zero8();
        if constexpr (PASS == SLOPE_SCALED) {
            if (valid <= 0) continue;
#pragma unroll
            for (int x = 0; x < 8; ++x) down[p][x] = inverse(g.cols[(int64_t)p * g.np8 + n0 + col + x]);
        }
    }
    // the lanes of a row find its largest entry together: all of them take part
    if (valid > 0 || PASS == SLOPE_RANGE) {
        with_act(g.act.kind, [&](auto kind) {
            constexpr int KIND = decltype(kind)::value;
#pragma unroll 1
            for (int base = r0; base < rows; base += kSlopeRows) {
                f32x8 dy[2], z[2], u[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int row = base + 16 * i;
                    const int n = row < rows ? valid : 0;
                    dy[i] = load_cut8<T>(ry, (uint32_t)(row * (int)g.ldy + col) * sizeof(T), n);
                    if constexpr (GATED || KIND != ACTK_NONE)
                        z[i] = load_cut8<T>(rz, (uint32_t)(row * (int)g.ldz + col) * sizeof(T), n);
                    if constexpr (GATED) u[i] = load_cut8<T>(ru, (uint32_t)(row * (int)g.ldu + col) * sizeof(T), n);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int row = base + 16 * i;
                    f32x8 d[2] = {dy[i], dy[i]};
                    if constexpr (GATED || KIND != ACTK_NONE) {
                        f32x8 y;
                        act_slope8<KIND>(g.act, z[i], y, d[0]);
                        d[0] *= dy[i];
                        if constexpr (GATED) {
                            d[0] *= u[i];
                            d[1] = dy[i] * y;
                        }
                    }
                    if (row >= rows) continue;
                    if constexpr (PASS == SLOPE_RANGE) {
                        float largest = 0.0f;
#pragma unroll
                        for (int p = 0; p < planes; ++p)
#pragma unroll
                            for (int x = 0; x < 8; ++x) {
                                const float a = finite_abs(d[p][x]);
                                most[p][x] = fmaxf(most[p][x], a);
                                largest = fmaxf(largest, a);
                            }
#pragma unroll
                        for (int by = 1; by < 16; by *= 2) largest = fmaxf(largest, __shfl_xor(largest, by, 16));
                        if (col == 0 && g.row_max) g.row_max[(int64_t)strip * g.M + m0 + row] = largest;
                    }
                    const uint32_t o = (uint32_t)(row * (int)g.ldd + col) * sizeof(T);
#pragma unroll
                    for (int p = 0; p < planes; ++p) {
                        if constexpr (PASS != SLOPE_SCALED) s[p] += d[p];
                        // the workspace's rows are whole groups
                        if constexpr (PASS == SLOPE_PLAIN) {
                            if (g.dZ[p]) store8<T>(at(g.dZ[p], g.ldd), o, d[p]);
                        } else if constexpr (PASS == SLOPE_SCALED) {
                            if (g.dZ[p]) store8<T>(at(g.dZ[p], g.ldd), o, d[p] * inverse(g.rows[m0 + row]));
                            if (g.dZc[p]) store8<T>(at(g.dZc[p], g.ldd), o, d[p] * down[p]);
                        }
                    }
                }
            }
        });
    }
    // columns of the sixteen row groups, in their order: a thread a column
    const int c = (int)threadIdx.x % kSlopeCols, p = (int)threadIdx.x / kSlopeCols;
    const bool mine = p < planes && n0 + c < g.np8;
    const int64_t to = ((int64_t)block * planes + p) * g.np8 + n0 + c;
    const auto gather = [&](const f32x8 (&v)[planes], float* out, auto join) {
#pragma unroll
        for (int q = 0; q < planes; ++q) red[q][threadIdx.x] = v[q];
        __syncthreads();
        if (mine) {
            const float* r = (const float*)red[p] + c;
            float x = r[0];
#pragma unroll
            for (int k = 1; k < 16; ++k) x = join(x, r[k * kSlopeCols]);
            out[to] = x;
        }
    };
    if (PASS == SLOPE_RANGE && g.col_max) {
        gather(most, g.col_max, [](float a, float b) { return fmaxf(a, b); });
        if (g.sums) __syncthreads();
    }
    if (PASS != SLOPE_SCALED && g.sums) gather(s, g.sums, [](float a, float b) { return a + b; });
}

// Bias gradients: the row blocks' column sums, in a fixed order: sixteen
// interleaved runs of blocks, then the runs.  The factors of fp16 gradients
// likewise, of the columns (from the row blocks) and, in one plane more, of the
// rows (from the strips).  Bound by the launch: 64 blocks of 4096 columns (1 MB)
// 5.2 us, 16 of 1025 3.9.
struct SumArgs {
    const float* sums;  // [blocks][planes][np8]
    void* out[2];       // planes; null: none
    const float* row_max;
    const float* col_max;
    float* rows;        // factors [M]; null: none are asked for
    float* cols;        // factors [planes][np8]
    int blocks, planes, np8, N;
    int M, strips;
    int out_f32;
};

template <int D>
__global__ void __launch_bounds__(1024) linear_colsum(SumArgs g) {
    typedef typename Elem<D>::type T;
    __shared__ float red[16][64];
    const int c = (int)threadIdx.x & 63, run = (int)threadIdx.x >> 6, p = (int)blockIdx.y;
    // f(x, next) over the blocks of one column, x of the first run's threads at the end
    const auto over = [&](const float* from, int64_t step, int count, bool ok, auto f) {
        float x = 0.0f;
        if (ok) {
#pragma unroll 4
            for (int b = run; b < count; b += 16) x = f(x, from[b * step]);
        }
        red[run][c] = x;
        __syncthreads();
        if (run == 0)
            for (int k = 1; k < 16; ++k) x = f(x, red[k][c]);
        __syncthreads();
        return x;
    };
    if constexpr (D == DT_F16) {
        const bool of_rows = p == g.planes;
        const int end = of_rows ? g.M : g.np8;
        for (int64_t n0 = (int64_t)blockIdx.x * 64; g.rows && n0 < end; n0 += (int64_t)gridDim.x * 64) {
            const int64_t n = n0 + c;
            const float m =
                over(of_rows ? g.row_max + n : g.col_max + (int64_t)p * g.np8 + n,
                     of_rows ? (int64_t)g.M : (int64_t)g.planes * g.np8, of_rows ? g.strips : g.blocks, n < end,
                     [](float a, float b) { return fmaxf(a, b); });
            if (run == 0 && n < end) (of_rows ? g.rows : g.cols + (int64_t)p * g.np8)[n] = scale_of(m);
        }
        if (of_rows) return;
    }
    if (!g.out[p]) return;
    for (int64_t n0 = (int64_t)blockIdx.x * 64; n0 < g.N; n0 += (int64_t)gridDim.x * 64) {
        const int64_t n = n0 + c;
        const float s = over(g.sums + (int64_t)p * g.np8 + n, (int64_t)g.planes * g.np8, g.blocks, n < g.N,
                             [](float a, float b) { return a + b; });
        if (run != 0 || n >= g.N) continue;
        if (g.out_f32)
            ((float*)g.out[p])[n] = s;
        else
            ((T*)g.out[p])[n] = (T)s;
    }
}

}  // namespace pgemm
