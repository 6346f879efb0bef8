// linear_abi.cpp -- the feed-forward operators' C entry points: argument
// checks, the choice of tile and splits, workspaces and launches.
//
// Every operator is a few products of one of three operand layouts
// (linear_variants.hpp); the backward passes begin with one elementwise kernel
// that forms the gradients at the pre-activations and their column sums.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstdio>
#include <cstring>

#include "linear_variants.hpp"
#include "pgemm.h"

using namespace pgemm;

namespace {

constexpr int64_t kMaxDim = 0x7fffff00;
constexpr int64_t kMaxLd = (int64_t)1 << 21;  // 256 rows of 4-byte elements stay below 2^31 bytes
constexpr int kNumCU = 256;
constexpr int64_t kMaxItems = (int64_t)1 << 32;  // a launch has fewer threads than this
constexpr int64_t kMaxSumGroups = 16384;  // workgroups of linear_colsum, which goes on from there by itself

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }
int64_t elem_size(int dtype) { return dtype == PGEMM_F32 ? 4 : 2; }
bool float_type(int dtype) { return dtype == PGEMM_F32 || dtype == PGEMM_F16 || dtype == PGEMM_BF16; }

LinKernels kernels_for(int dtype) {
    return dtype == PGEMM_F32 ? linear_kernels_f32() : dtype == PGEMM_F16 ? linear_kernels_f16()
                                                                        : linear_kernels_bf16();
}

ActArgs act_args(int act) {
    // -log2(e) * P(t); see ActArgs
    constexpr double kLog2e = 1.4426950408889634;
    ActArgs a;
    std::memset(&a, 0, sizeof(a));
    a.kind = act;
    if (act == PGEMM_ACT_SILU) {
        a.c[0] = (float)-kLog2e;
    } else if (act == PGEMM_ACT_GELU_TANH) {
        const double c = 1.5957691216057308;  // sqrt(8 / pi)
        a.c[0] = (float)(-kLog2e * c);
        a.c[1] = (float)(-kLog2e * c * 0.044715);
    }
    return a;
}

// A rows x cols product over K (per contraction half), with `outs` outputs
// side by side.
struct Shape {
    int64_t rows, cols, K;
    int lay, gated, halves, outs;
};

struct Plan {
    const LinVariant* v;
    int64_t tiles_m, tiles_n, splits, part_bytes;
    int np8;
};

// Estimated microseconds of a product with its K tiles split in `splits`.  The
// rates and fixed costs are fitted to choose well, on 2000 products of 1 to 8192
// rows in all layouts and types, each timed on every variant in 1 to 32 splits.
// On 1360 others the choice takes 1.8 % longer than the best (geometric mean of 900
// random sizes; nine in ten within 7 %, the worst 72 %), 1.8 % for 300 multiples of
// 1024 and 3.9 % for 160 weights beyond the shared cache.
//
// Tiles: the workgroups run in rounds, one or two (128 x 128 with two stages) a
// CU at a time.  Rates of the whole part in TFLOP/s and us a round, 16-bit
// types: 256 x 256 1560, 17; 128 x 128 with four stages 820, 6.5, with two 450
// alone and 763 where two share a CU, 3.4 (1024 x 4096 x 4096, 256 workgroups:
// 35 us with four stages, 44 with two; 2048 x 4096 x 4096: 70 and 61).
double est_tiles(const LinVariant& v, const Shape& p, bool f32, int64_t wgs, double kt) {
    const bool large = v.bm == 256, one = v.per_cu == 1;
    const double alone = (large ? (f32 ? 159e6 : 1560e6) : f32 ? 138e6 : one ? 820e6 : 450e6) / kNumCU;
    const double shared = one ? alone : (f32 ? 147e6 : 763e6) / kNumCU;
    const double flop = 2.0 * v.bm * v.bn * v.bk * kt * (p.gated ? 2 : 1);
    const int64_t slots = one ? kNumCU : 2 * kNumCU;
    const int64_t rounds = wgs / slots, rest = wgs % slots;
    const double round_us = (one ? 1 : 2) * flop / shared, fixed = large ? 17.0 : one ? 6.5 : 3.4;
    double us = rounds * (round_us + fixed);
    if (rest > kNumCU) us += round_us + fixed;
    else if (rest > 0) us += flop / alone + fixed;
    return us;
}
// Few rows: the CU with the most workgroups streams 44 bytes/ns or multiplies at
// 0.87 (fp32: 0.42) TFLOP/s, and each round of workgroups costs 3 us.  W [K][N]
// in less than 128 bytes of a row at a time streams slower (one token gated to
// 6144 x 6144, 51.7 us on 32 columns of each weight, 39.1 on 64 in two splits).
double est_few(const LinVariant& v, const Shape& p, bool f32, int64_t wgs, double kt) {
    const double cols = v.bn * (p.gated ? 2 : 1), es = f32 ? 4 : 2;
    const double kb = kt * v.bk * ((p.rows < v.bm ? p.rows : v.bm) + cols) * es / 1e3;
    const double load = (double)ceil_div(wgs, kNumCU);
    const double thin = v.lay == LIN_KX && v.bn * es < 128 ? 1.3 : 1.0;
    const double stream = thin * load * kb / 44.0, mfma = load * 2.0 * v.bm * cols * v.bk * kt / (f32 ? 0.42e6 : 0.87e6);
    return 3.0 * ceil_div(wgs, (int64_t)kNumCU * v.per_cu) + (stream > mfma ? stream : mfma);
}
double est_us(const LinVariant& v, const Shape& p, int dtype, int64_t splits) {
    const bool f32 = dtype == PGEMM_F32;
    const int64_t wgs = ceil_div(p.rows, v.bm) * ceil_div(p.cols, v.bn) * p.outs * splits;
    const double kt = (double)ceil_div(ceil_div(p.K, v.bk) * p.halves, splits);
    double us = v.few ? est_few(v, p, f32, wgs, kt) : est_tiles(v, p, f32, wgs, kt);
    // inputs from the caches and memory: no variant is faster
    const double mem = (double)p.K * p.halves * (f32 ? 4 : 2) * (p.rows + p.cols * (p.gated ? 2.0 : 1.0)) / 16e6;
    if (us < mem) us = mem;
    // the join: a launch, and the partial sums written and read
    if (splits > 1) us += 5.0 + 0.29 * splits + 2.0 * splits * p.rows * p.cols * (p.gated ? 2 : p.outs) * 4.0 / 4.4e6;
    return us;
}

// The tile and the splits of a product, from its sizes and type alone (so the
// workspace functions and the calls agree).  No variant where every one has more
// threads than a launch holds.
Plan search_plan(const Shape& p, int dtype) {
    const LinKernels k = kernels_for(dtype);
    Plan best{};
    double best_us = 0.0;
    for (int i = 0; i < k.n; ++i) {
        const LinVariant& v = k.v[i];
        if (v.lay != p.lay || v.gated != p.gated) continue;
        const int64_t kt = ceil_div(p.K, v.bk) * p.halves;
        const int64_t tiles = ceil_div(p.rows, v.bm) * ceil_div(p.cols, v.bn) * p.outs;
        if (v.bm == 256 && (p.rows <= 64 || p.cols <= 64)) continue;
        if (round_up(tiles, 8) * v.threads >= kMaxItems) continue;  // (split, there are no more than 2048)
        for (int64_t s = 1; s <= 32; ++s) {
            // K tiles for each wave, and not more workgroups than splitting is for
            if (s > 1 && (s * (v.few ? v.few : 4) > kt || tiles * s > (v.few ? 8 : 2) * kNumCU)) break;
            const double us = est_us(v, p, dtype, s);
            if (best.v && us >= best_us) continue;
            best_us = us;
            best.v = &v;
            best.splits = s;
        }
    }
    if (!best.v) return best;
    const LinVariant& v = *best.v;
    best.tiles_m = ceil_div(p.rows, v.bm);
    best.tiles_n = ceil_div(p.cols, v.bn);
    best.np8 = (int)round_up(p.cols, 8);
    best.part_bytes = best.splits > 1 ? best.splits * (p.gated ? 2 : p.outs) * p.rows * best.np8 * 4 : 0;
    return best;
}

// The search takes some microseconds, as long as a small product runs: each
// thread keeps the plans of the last shapes it met (a plan depends on nothing
// but its key).
Plan plan_product(const Shape& p, int dtype) {
    struct Slot {
        Shape key;
        int dtype;
        Plan plan;
    };
    static thread_local Slot slots[64];
    uint64_t h = (uint64_t)p.rows * 0x9e3779b97f4a7c15ull + (uint64_t)p.cols * 0xc2b2ae3d27d4eb4full +
                 (uint64_t)p.K * 0x165667b19e3779f9ull +
                 (uint64_t)(p.lay + 3 * p.gated + 6 * p.halves + 18 * p.outs + 54 * dtype) * 0xd6e8feb86659fd93ull;
    Slot& s = slots[(h ^ (h >> 29)) >> 32 & 63];
    const Shape& k = s.key;
    if (!s.plan.v || s.dtype != dtype || k.rows != p.rows || k.cols != p.cols || k.K != p.K || k.lay != p.lay ||
        k.gated != p.gated || k.halves != p.halves || k.outs != p.outs) {
        s.plan = search_plan(p, dtype);
        s.key = p;
        s.dtype = dtype;
    }
    return s.plan;
}

// Bytes of the splits' sums, or PGEMM_ERR_TOO_LARGE.
int64_t part_bytes(const Shape& p, int dtype) {
    if (p.rows == 0 || p.cols == 0) return 0;
    const Plan pl = plan_product(p, dtype);
    return pl.v ? round_up(pl.part_bytes, 256) : PGEMM_ERR_TOO_LARGE;
}

int hip_failed(const char* what, hipError_t e) {
    std::fprintf(stderr, "pgemm: launch of %s failed: %s (%d)\n", what, hipGetErrorString(e), (int)e);
    return PGEMM_ERR_HIP;
}

// Runs a product whose operands, outputs and epilogue `a` already holds.
int run_product(const Shape& p, LinArgs& a, int dtype, void* part, hipStream_t stream) {
    if (p.rows == 0 || p.cols == 0) return PGEMM_OK;
    const LinKernels k = kernels_for(dtype);
    const Plan pl = plan_product(p, dtype);
    if (!pl.v) return PGEMM_ERR_TOO_LARGE;  // found out before, with the workspace
    const LinVariant& v = *pl.v;
    a.K = (int)p.K;
    a.halves = p.halves;
    a.outs = p.outs;
    a.tiles_m = (int)pl.tiles_m;
    a.tiles_n = (int)pl.tiles_n;
    a.group_m = 4;
    a.splits = (int)pl.splits;
    a.part = pl.splits > 1 ? (float*)part : nullptr;
    a.np8 = pl.np8;
    a.e.M = (int)p.rows;
    a.e.N = (int)p.cols;
    a.nfull = v.ring_tiles(p.K, p.rows, a.lda, p.cols, a.ldb);
    const int64_t grid = round_up(pl.tiles_m * pl.tiles_n * p.outs * pl.splits, 8);
    hipError_t e = v.launch(a, (int)grid, stream);
    if (e != hipSuccess) return hip_failed("linear_kernel", e);
    if (pl.splits > 1) {
        const int64_t g2 = ceil_div(p.cols, kJoinCols) * p.rows * p.outs;
        e = (p.gated ? k.join_gated : k.join)(a, (int)g2, stream);
        if (e != hipSuccess) return hip_failed("linear_join", e);
    }
    return PGEMM_OK;
}

bool in_range(int64_t M, int64_t N, int64_t K) { return M <= kMaxDim && N <= kMaxDim && K <= kMaxDim; }
// Work items of the largest grids (tiles, rows x strips) fit an int.
bool grids_fit(int64_t a, int64_t b) { return ceil_div(a, 64) * ceil_div(b, 64) < 0x3fffff00 && a * ceil_div(b, kJoinCols) < 0x3fffff00; }

int check_sizes(int64_t M, int64_t N, int64_t K, int dtype) {
    if (!float_type(dtype)) return PGEMM_ERR_UNSUPPORTED_DTYPE;
    if (M < 0 || N < 0 || K < 0) return PGEMM_ERR_INVALID_ARG;
    if (M > 0 && N >= kMaxLd) return PGEMM_ERR_TOO_LARGE;  // every call has a matrix of M rows of N
    if (!in_range(M, N, K) || !grids_fit(M, N) || !grids_fit(M, K) || !grids_fit(K, N) || !grids_fit(N, K))
        return PGEMM_ERR_TOO_LARGE;
    return PGEMM_OK;
}

// A matrix of `rows` rows of `cols` elements: 0, or the error.
int check_matrix(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t es, bool needed) {
    if (!p) return needed && rows > 0 && cols > 0 ? PGEMM_ERR_INVALID_ARG : PGEMM_OK;
    if (ld < (cols > 1 ? cols : 1) || (uintptr_t)p % es) return PGEMM_ERR_INVALID_ARG;
    return ld >= kMaxLd ? PGEMM_ERR_TOO_LARGE : PGEMM_OK;
}
int check_vector(const void* p, int64_t es) { return (uintptr_t)p % es ? PGEMM_ERR_INVALID_ARG : PGEMM_OK; }
int check_workspace(const void* p, int64_t bytes, int64_t need) {
    if (need < 0) return (int)need;
    return need > 0 && (!p || (uintptr_t)p % 16 || bytes < need) ? PGEMM_ERR_INVALID_ARG : PGEMM_OK;
}
bool known(int order, int act, int out, int dtype) {
    return (order == PGEMM_KN || order == PGEMM_NK) && act >= PGEMM_ACT_NONE && act <= PGEMM_ACT_GELU_TANH &&
           (out == dtype || out == PGEMM_F32);
}
#define PGEMM_TRY(x)                     \
    do {                                 \
        const int r_ = (x);              \
        if (r_ != PGEMM_OK) return r_;   \
    } while (0)

Shape forward_shape(int64_t M, int64_t N, int64_t K, int order, int gated) {
    return Shape{M, N, K, order == PGEMM_KN ? LIN_KX : LIN_KK, gated, 1, 1};
}
// dX: the contraction runs over N, along W[K][N]'s rows or W[N][K]'s columns.
Shape dx_shape(int64_t M, int64_t N, int64_t K, int order, int halves) {
    return Shape{M, K, N, order == PGEMM_KN ? LIN_KK : LIN_KX, 0, halves, 1};
}
// dW in its own storage order: K x N, or N x K.
Shape dw_shape(int64_t M, int64_t N, int64_t K, int order, int outs) {
    return order == PGEMM_KN ? Shape{K, N, M, LIN_XX, 0, 1, outs} : Shape{N, K, M, LIN_XX, 0, 1, outs};
}
int64_t larger(int64_t a, int64_t b) { return a > b ? a : b; }
// The larger of two counts of bytes, or an error among them.
int64_t both(int64_t a, int64_t b) { return a < 0 ? a : b < 0 ? b : larger(a, b); }

// Workspace of a backward pass: gradients at the pre-activations (fp16: in two
// copies, with the largest entries and factors of rows and columns), the row
// blocks' column sums, the splits' sums (of dX, then of dW).
struct Backward {
    int64_t ldd, np8, steps, blocks, strips;
    int64_t dz_bytes;                // of one plane of one copy
    int64_t copies;
    int64_t row_max, col_max, rows, cols, scale_bytes;  // fp16: offsets behind the copies, and the bytes of all
    int64_t sum_bytes, split_bytes;
    int64_t kept(int planes) const { return planes * copies * dz_bytes + scale_bytes; }
    int64_t total(int planes, bool keeps) const { return (keeps ? kept(planes) : 0) + sum_bytes + split_bytes; }
};
Backward backward_layout(int64_t M, int64_t N, int64_t K, int dtype, int planes) {
    Backward b;
    b.ldd = round_up(N, 64);
    b.np8 = round_up(N, 8);
    // Two steps of rows a workgroup where that leaves four workgroups a CU
    // (2048 x 8192 gated: 41 us in one step, 34 in two, 34 in four; 1000 x 2003,
    // 256 workgroups in two steps: 12 us in one, 17 in two).
    b.steps = ceil_div(M, 2 * kSlopeRows) * ceil_div(N, kSlopeCols) >= 4 * kNumCU ? 2 : 1;
    b.blocks = ceil_div(M, b.steps * kSlopeRows);
    b.strips = ceil_div(N, kSlopeCols);
    b.dz_bytes = M * b.ldd * elem_size(dtype);  // a multiple of 128
    b.copies = dtype == PGEMM_F16 ? 2 : 1;
    b.scale_bytes = 0;
    if (dtype == PGEMM_F16) {
        const auto take = [&](int64_t floats) {
            const int64_t at = b.scale_bytes;
            b.scale_bytes += round_up(floats * 4, 256);
            return at;
        };
        b.row_max = take(b.strips * M);
        b.col_max = take(b.blocks * planes * b.np8);
        b.rows = take(M);
        b.cols = take(planes * b.np8);
    }
    b.sum_bytes = round_up(b.blocks * planes * b.np8 * 4, 256);
    b.split_bytes = 0;
    for (int order = 0; order < 2; ++order) {
        b.split_bytes = both(b.split_bytes, part_bytes(dx_shape(M, N, K, order, planes), dtype));
        b.split_bytes = both(b.split_bytes, part_bytes(dw_shape(M, N, K, order, planes), dtype));
    }
    return b;
}

struct Grad {
    const void *dY, *X, *W[2], *Z, *U;
    int64_t lddy, ldx, ldw, ldz, ldu;
    void *dX, *dW[2], *db[2];
    int64_t lddx, lddw;
};

// The backward pass of both operators (planes: 1, or 2 for gated).
int run_backward(int64_t M, int64_t N, int64_t K, const Grad& q, int w_order, int dw_order, int act, int grad_dtype,
                 int dtype, int planes, void* workspace, hipStream_t stream) {
    const LinKernels k = kernels_for(dtype);
    const Backward b = backward_layout(M, N, K, dtype, planes);
    const bool gated = planes == 2, keeps = gated || act != PGEMM_ACT_NONE;
    const bool products = q.dX || q.dW[0], bias = q.db[0] || q.db[1];
    // What stands in the workspace for dZ (dG, dU) as operand of dX and of dW.
    const bool stored = keeps && products && M > 0 && N > 0, scaled = stored && dtype == PGEMM_F16;
    char* ws = (char*)workspace;
    const auto plane = [&](int64_t i) -> void* { return ws ? ws + i * b.dz_bytes : nullptr; };
    char* scales = ws ? ws + planes * b.copies * b.dz_bytes : nullptr;
    char* rest = ws ? ws + (keeps ? b.kept(planes) : 0) : nullptr;
    float* sums = (float*)rest;
    void* part = rest ? rest + b.sum_bytes : nullptr;
    const float* row_factors = scaled ? (const float*)(scales + b.rows) : nullptr;
    const float* col_factors = scaled ? (const float*)(scales + b.cols) : nullptr;
    SlopeArgs s;
    std::memset(&s, 0, sizeof(s));
    s.dY = q.dY;
    s.ldy = q.lddy;
    s.Z = q.Z;
    s.ldz = q.ldz;
    s.U = q.U;
    s.ldu = q.ldu;
    s.ldd = b.ldd;
    s.sums = bias ? sums : nullptr;
    s.np8 = (int)b.np8;
    s.steps = (int)b.steps;
    s.M = (int)M;
    s.N = (int)N;
    s.act = act_args(act);
    if (scaled) {
        s.row_max = (float*)(scales + b.row_max);
        s.col_max = (float*)(scales + b.col_max);
    } else if (stored) {
        for (int p = 0; p < planes; ++p) s.dZ[p] = plane(p);
    }
    const auto slope = [&](int pass) {
        const hipError_t e = k.slope(s, gated, pass, (int)(b.strips * b.blocks), stream);
        return e == hipSuccess ? (int)PGEMM_OK : hip_failed("linear_slope", e);
    };
    // no column: dX is all zeros (a product over nothing), the rest is empty
    if (M > 0 && N > 0 && (stored || bias)) PGEMM_TRY(slope(dtype == PGEMM_F16 ? SLOPE_RANGE : SLOPE_PLAIN));
    if (N > 0 && (bias || scaled)) {
        SumArgs t;
        std::memset(&t, 0, sizeof(t));
        t.sums = sums;
        t.out[0] = q.db[0];
        t.out[1] = q.db[1];
        t.blocks = (int)b.blocks;
        t.planes = planes;
        t.np8 = (int)b.np8;
        t.N = (int)N;
        t.out_f32 = grad_dtype == PGEMM_F32;
        if (scaled) {
            t.row_max = s.row_max;
            t.col_max = s.col_max;
            t.rows = (float*)(scales + b.rows);
            t.cols = (float*)(scales + b.cols);
            t.M = (int)M;
            t.strips = (int)b.strips;
        }
        const int64_t longest = scaled ? larger(M, b.np8) : N;
        const int64_t groups = ceil_div(longest, 64);
        const hipError_t e = k.colsum(t, (int)(groups < kMaxSumGroups ? groups : kMaxSumGroups), stream);
        if (e != hipSuccess) return hip_failed("linear_colsum", e);
    }
    if (scaled) {
        s.rows = row_factors;
        s.cols = col_factors;
        for (int p = 0; p < planes; ++p) {
            s.dZ[p] = q.dX ? plane(p) : nullptr;
            s.dZc[p] = q.dW[0] ? plane(planes + p) : nullptr;
        }
        PGEMM_TRY(slope(SLOPE_SCALED));
    }
    const void* dx[2] = {keeps ? plane(0) : q.dY, gated ? plane(1) : keeps ? plane(0) : q.dY};
    const void* dw[2] = {scaled ? plane(planes) : dx[0], scaled ? plane(2 * planes - 1) : dx[1]};
    const int64_t ldd = keeps ? b.ldd : q.lddy;
    if (q.dX) {
        LinArgs a;
        std::memset(&a, 0, sizeof(a));
        for (int h = 0; h < 2; ++h) {
            a.A[h] = dx[h];
            a.B[h] = q.W[h];
        }
        a.lda = ldd;
        a.ldb = q.ldw;
        a.e.Y[0] = a.e.Y[1] = q.dX;
        a.e.ldy = q.lddx;
        a.e.rows[0] = a.e.rows[1] = row_factors;
        a.e.out_f32 = dtype == PGEMM_F32;
        PGEMM_TRY(run_product(dx_shape(M, N, K, w_order, planes), a, dtype, part, stream));
    }
    if (q.dW[0]) {
        LinArgs a;
        std::memset(&a, 0, sizeof(a));
        for (int h = 0; h < 2; ++h) {
            a.A[h] = dw_order == PGEMM_KN ? q.X : dw[h];
            a.B[h] = dw_order == PGEMM_KN ? dw[h] : q.X;
            a.e.Y[h] = q.dW[h];
            // dZ's columns are dW's columns, or its rows where it lies N x K
            if (scaled) (dw_order == PGEMM_KN ? a.e.cols : a.e.rows)[h] = col_factors + (gated ? h : 0) * b.np8;
        }
        a.lda = dw_order == PGEMM_KN ? q.ldx : ldd;
        a.ldb = dw_order == PGEMM_KN ? ldd : q.ldx;
        a.e.ldy = q.lddw;
        a.e.out_f32 = grad_dtype == PGEMM_F32;
        PGEMM_TRY(run_product(dw_shape(M, N, K, dw_order, planes), a, dtype, part, stream));
    }
    return PGEMM_OK;
}

int check_weight(const void* W, int64_t N, int64_t K, int64_t ldw, int order, int64_t es, bool needed) {
    return order == PGEMM_KN ? check_matrix(W, K, N, ldw, es, needed) : check_matrix(W, N, K, ldw, es, needed);
}

int64_t forward_workspace(int64_t M, int64_t N, int64_t K, int dtype, int gated) {
    PGEMM_TRY(check_sizes(M, N, K, dtype));
    return both(part_bytes(forward_shape(M, N, K, PGEMM_KN, gated), dtype),
                part_bytes(forward_shape(M, N, K, PGEMM_NK, gated), dtype));
}

int64_t backward_workspace(int64_t M, int64_t N, int64_t K, int act, int dtype, int planes) {
    PGEMM_TRY(check_sizes(M, N, K, dtype));
    if (act < PGEMM_ACT_NONE || act > PGEMM_ACT_GELU_TANH) return PGEMM_ERR_INVALID_ARG;
    const Backward b = backward_layout(M, N, K, dtype, planes);
    if (b.split_bytes < 0 || b.strips * b.blocks * 256 >= kMaxItems) return PGEMM_ERR_TOO_LARGE;
    return b.total(planes, planes == 2 || act != PGEMM_ACT_NONE);
}

}  // namespace

extern "C" {

int64_t pgemm_linear_workspace(int64_t M, int64_t N, int64_t K, int dtype) {
    return forward_workspace(M, N, K, dtype, 0);
}
int64_t pgemm_gated_workspace(int64_t M, int64_t N, int64_t K, int dtype) {
    return forward_workspace(M, N, K, dtype, 1);
}
int64_t pgemm_linear_backward_workspace(int64_t M, int64_t N, int64_t K, int act, int dtype) {
    return backward_workspace(M, N, K, act, dtype, 1);
}
int64_t pgemm_gated_backward_workspace(int64_t M, int64_t N, int64_t K, int dtype) {
    return backward_workspace(M, N, K, PGEMM_ACT_SILU, dtype, 2);
}

int pgemm_linear(int64_t M, int64_t N, int64_t K, const void* X, int64_t ldx, const void* W, int64_t ldw,
                 int w_order, const void* bias, const void* R, int64_t ldr, int act, void* Z, int64_t ldz, void* Y,
                 int64_t ldy, int out_dtype, int dtype, void* workspace, int64_t workspace_bytes, void* stream) {
    PGEMM_TRY(check_sizes(M, N, K, dtype));
    if (!known(w_order, act, out_dtype, dtype)) return PGEMM_ERR_INVALID_ARG;
    const int64_t es = elem_size(dtype), os = elem_size(out_dtype);
    PGEMM_TRY(check_matrix(X, M, K, ldx, es, N > 0));
    PGEMM_TRY(check_weight(W, N, K, ldw, w_order, es, M > 0));
    PGEMM_TRY(check_vector(bias, es));
    PGEMM_TRY(check_matrix(R, M, N, ldr, os, false));
    PGEMM_TRY(check_matrix(Z, M, N, ldz, es, false));
    PGEMM_TRY(check_matrix(Y, M, N, ldy, os, true));
    if (M == 0 || N == 0) return PGEMM_OK;
    const Shape p = forward_shape(M, N, K, w_order, 0);
    PGEMM_TRY(check_workspace(workspace, workspace_bytes, forward_workspace(M, N, K, dtype, 0)));
    LinArgs a;
    std::memset(&a, 0, sizeof(a));
    a.A[0] = a.A[1] = X;
    a.B[0] = a.B[1] = W;
    a.lda = ldx;
    a.ldb = ldw;
    a.e.Y[0] = a.e.Y[1] = Y;
    a.e.ldy = ldy;
    a.e.R = R;
    a.e.ldr = ldr;
    a.e.Z = Z;
    a.e.ldz = ldz;
    a.e.bias[0] = bias;
    a.e.act = act_args(act);
    a.e.out_f32 = out_dtype == PGEMM_F32;
    return run_product(p, a, dtype, workspace, (hipStream_t)stream);
}

int pgemm_gated(int64_t M, int64_t N, int64_t K, const void* X, int64_t ldx, const void* Wg, const void* Wu,
                int64_t ldw, int w_order, const void* bias_g, const void* bias_u, int act, void* G, int64_t ldg,
                void* U, int64_t ldu, void* H, int64_t ldh, int out_dtype, int dtype, void* workspace,
                int64_t workspace_bytes, void* stream) {
    PGEMM_TRY(check_sizes(M, N, K, dtype));
    if (!known(w_order, act, out_dtype, dtype)) return PGEMM_ERR_INVALID_ARG;
    const int64_t es = elem_size(dtype), os = elem_size(out_dtype);
    PGEMM_TRY(check_matrix(X, M, K, ldx, es, N > 0));
    PGEMM_TRY(check_weight(Wg, N, K, ldw, w_order, es, M > 0));
    PGEMM_TRY(check_weight(Wu, N, K, ldw, w_order, es, M > 0));
    PGEMM_TRY(check_vector(bias_g, es));
    PGEMM_TRY(check_vector(bias_u, es));
    PGEMM_TRY(check_matrix(G, M, N, ldg, es, false));
    PGEMM_TRY(check_matrix(U, M, N, ldu, es, false));
    PGEMM_TRY(check_matrix(H, M, N, ldh, os, true));
    if (M == 0 || N == 0) return PGEMM_OK;
    const Shape p = forward_shape(M, N, K, w_order, 1);
    PGEMM_TRY(check_workspace(workspace, workspace_bytes, forward_workspace(M, N, K, dtype, 1)));
    LinArgs a;
    std::memset(&a, 0, sizeof(a));
    a.A[0] = a.A[1] = X;
    a.B[0] = Wg;
    a.B[1] = Wu;
    a.lda = ldx;
    a.ldb = ldw;
    a.e.Y[0] = a.e.Y[1] = H;
    a.e.ldy = ldh;
    a.e.Z = G;
    a.e.ldz = ldg;
    a.e.U = U;
    a.e.ldu = ldu;
    a.e.bias[0] = bias_g;
    a.e.bias[1] = bias_u;
    a.e.act = act_args(act);
    a.e.out_f32 = out_dtype == PGEMM_F32;
    return run_product(p, a, dtype, workspace, (hipStream_t)stream);
}

int pgemm_linear_backward(int64_t M, int64_t N, int64_t K, const void* dY, int64_t lddy, const void* X, int64_t ldx,
                          const void* W, int64_t ldw, int w_order, const void* Z, int64_t ldz, int act, void* dX,
                          int64_t lddx, void* dW, int64_t lddw, int dw_order, void* dbias, int grad_dtype, int dtype,
                          void* workspace, int64_t workspace_bytes, void* stream) {
    PGEMM_TRY(check_sizes(M, N, K, dtype));
    if (!known(w_order, act, grad_dtype, dtype) || !known(dw_order, act, grad_dtype, dtype))
        return PGEMM_ERR_INVALID_ARG;
    const int64_t es = elem_size(dtype), gs = elem_size(grad_dtype);
    PGEMM_TRY(check_matrix(dY, M, N, lddy, es, dX || dW || dbias));
    PGEMM_TRY(check_matrix(X, M, K, ldx, es, dW && N > 0));
    PGEMM_TRY(check_weight(W, N, K, ldw, w_order, es, dX && M > 0));
    PGEMM_TRY(check_matrix(Z, M, N, ldz, es, act != PGEMM_ACT_NONE));
    PGEMM_TRY(check_matrix(dX, M, K, lddx, es, false));
    PGEMM_TRY(check_weight(dW, N, K, lddw, dw_order, gs, false));
    PGEMM_TRY(check_vector(dbias, gs));
    PGEMM_TRY(check_workspace(workspace, workspace_bytes, backward_workspace(M, N, K, act, dtype, 1)));
    Grad q;
    std::memset(&q, 0, sizeof(q));
    q.dY = dY;
    q.lddy = lddy;
    q.X = X;
    q.ldx = ldx;
    q.W[0] = q.W[1] = W;
    q.ldw = ldw;
    q.Z = Z;
    q.ldz = ldz;
    q.dX = dX;
    q.lddx = lddx;
    q.dW[0] = q.dW[1] = dW;
    q.lddw = lddw;
    q.db[0] = dbias;
    return run_backward(M, N, K, q, w_order, dw_order, act, grad_dtype, dtype, 1, workspace, (hipStream_t)stream);
}

int pgemm_gated_backward(int64_t M, int64_t N, int64_t K, const void* dH, int64_t lddh, const void* X, int64_t ldx,
                         const void* Wg, const void* Wu, int64_t ldw, int w_order, const void* G, int64_t ldg,
                         const void* U, int64_t ldu, int act, void* dX, int64_t lddx, void* dWg, void* dWu,
                         int64_t lddw, int dw_order, void* dbias_g, void* dbias_u, int grad_dtype, int dtype,
                         void* workspace, int64_t workspace_bytes, void* stream) {
    PGEMM_TRY(check_sizes(M, N, K, dtype));
    if (!known(w_order, act, grad_dtype, dtype) || !known(dw_order, act, grad_dtype, dtype) || !dWg != !dWu)
        return PGEMM_ERR_INVALID_ARG;
    const int64_t es = elem_size(dtype), gs = elem_size(grad_dtype);
    const bool any = dX || dWg || dbias_g || dbias_u;
    PGEMM_TRY(check_matrix(dH, M, N, lddh, es, any));
    PGEMM_TRY(check_matrix(G, M, N, ldg, es, any));
    PGEMM_TRY(check_matrix(U, M, N, ldu, es, any));
    PGEMM_TRY(check_matrix(X, M, K, ldx, es, dWg && N > 0));
    PGEMM_TRY(check_weight(Wg, N, K, ldw, w_order, es, dX && M > 0));
    PGEMM_TRY(check_weight(Wu, N, K, ldw, w_order, es, dX && M > 0));
    PGEMM_TRY(check_matrix(dX, M, K, lddx, es, false));
    PGEMM_TRY(check_weight(dWg, N, K, lddw, dw_order, gs, false));
    PGEMM_TRY(check_weight(dWu, N, K, lddw, dw_order, gs, false));
    PGEMM_TRY(check_vector(dbias_g, gs));
    PGEMM_TRY(check_vector(dbias_u, gs));
    PGEMM_TRY(check_workspace(workspace, workspace_bytes, backward_workspace(M, N, K, act, dtype, 2)));
    Grad q;
    std::memset(&q, 0, sizeof(q));
    q.dY = dH;
    q.lddy = lddh;
    q.X = X;
    q.ldx = ldx;
    q.W[0] = Wg;
    q.W[1] = Wu;
    q.ldw = ldw;
    q.Z = G;
    q.ldz = ldg;
    q.U = U;
    q.ldu = ldu;
    q.dX = dX;
    q.lddx = lddx;
    q.dW[0] = dWg;
    q.dW[1] = dWu;
    q.lddw = lddw;
    q.db[0] = dbias_g;
    q.db[1] = dbias_u;
    return run_backward(M, N, K, q, w_order, dw_order, act, grad_dtype, dtype, 2, workspace, (hipStream_t)stream);
}

}  // extern "C"
