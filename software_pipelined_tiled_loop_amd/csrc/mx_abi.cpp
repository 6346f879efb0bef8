// mx_abi.cpp -- C entry points of the norm and of the microscaled operators:
// argument checks, the choice of kernels, workspaces and launches.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstdio>
#include <cstring>

#include "mx_variants.hpp"
#include "pgemm.h"

using namespace pgemm;

namespace {

constexpr int64_t kMaxDim = 0x7fffff00;
constexpr int64_t kMaxLd = (int64_t)1 << 21;  // elements; bytes of codes and scales
constexpr int kNumCU = 256;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }
int64_t smaller(int64_t a, int64_t b) { return a < b ? a : b; }
double larger(double a, double b) { return a > b ? a : b; }
int64_t elem_size(int dtype) { return dtype == PGEMM_F32 ? 4 : 2; }
bool float_type(int dtype) { return dtype == PGEMM_F32 || dtype == PGEMM_F16 || dtype == PGEMM_BF16; }

MxKernels kernels_for(int dtype) {
    return dtype == PGEMM_F32 ? mx_kernels_f32() : dtype == PGEMM_F16 ? mx_kernels_f16() : mx_kernels_bf16();
}

#define PGEMM_TRY(x)                     \
    do {                                 \
        const int r_ = (x);              \
        if (r_ != PGEMM_OK) return r_;   \
    } while (0)

int launched(const char* what, hipError_t e) {
    if (e == hipSuccess) return PGEMM_OK;
    std::fprintf(stderr, "pgemm: launch of %s failed: %s (%d)\n", what, hipGetErrorString(e), (int)e);
    return PGEMM_ERR_HIP;
}

// Types and sizes that every operator checks.
int check_sizes(int64_t rows, int64_t cols, int dtype) {
    if (!float_type(dtype)) return PGEMM_ERR_UNSUPPORTED_DTYPE;
    if (rows < 0 || cols < 0) return PGEMM_ERR_INVALID_ARG;
    return rows > kMaxDim || cols >= kMaxLd ? PGEMM_ERR_TOO_LARGE : PGEMM_OK;
}
// A matrix of `rows` rows of `cols` elements: 0, or the error.
int check_matrix(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t es, bool needed) {
    if (!p) return needed && rows > 0 && cols > 0 ? PGEMM_ERR_INVALID_ARG : PGEMM_OK;
    if (ld < (cols > 1 ? cols : 1) || (uintptr_t)p % es) return PGEMM_ERR_INVALID_ARG;
    return ld >= kMaxLd ? PGEMM_ERR_TOO_LARGE : PGEMM_OK;
}
int check_vector(const void* p, int64_t es) { return (uintptr_t)p % es ? PGEMM_ERR_INVALID_ARG : PGEMM_OK; }
// Codes and scales of `rows` rows of K entries.
int check_blocks(const void* Q, int64_t ldq, const void* S, int64_t lds, int64_t rows, int64_t K, int format) {
    if (format != PGEMM_MX8 && format != PGEMM_MX4) return PGEMM_ERR_INVALID_ARG;
    if (rows == 0 || K == 0) return PGEMM_OK;
    if (!Q || !S || (uintptr_t)Q % 16 || (uintptr_t)S % 4 || ldq % 16 || lds % 4) return PGEMM_ERR_INVALID_ARG;
    if (ldq < mx_code_bytes(K, format) || lds < mx_filled(K) / kMxBlock) return PGEMM_ERR_INVALID_ARG;
    return ldq >= kMaxLd || lds >= kMaxLd ? PGEMM_ERR_TOO_LARGE : PGEMM_OK;
}
int check_workspace(const void* p, int64_t bytes, int64_t need) {
    if (need < 0) return (int)need;
    return need > 0 && (!p || (uintptr_t)p % 16 || bytes < need) ? PGEMM_ERR_INVALID_ARG : PGEMM_OK;
}

// Workgroups for `items`, `per` at a time; kernels go on from there by themselves.
int grid_for(int64_t items, int64_t per) { return (int)smaller(ceil_div(items, per), 1 << 20); }

// How the threads of mx_quantize_rows and mx_dequantize_rows share rows of `groups` groups of eight; returns the grid.
int share_rows(MxCopyArgs& a, int64_t groups) {
    a.shift = 5;
    while (a.shift < 8 && ((int64_t)kRun << a.shift) < groups) ++a.shift;
    a.stretches = (int)ceil_div(groups, (int64_t)kRun << a.shift);
    return grid_for(ceil_div(a.rows, 256 >> a.shift) * a.stretches, 1);
}

// ---- the norm ----------------------------------------------------------------------------------

// The first kernel whose row holds `filled` columns.
template <class Args>
const NormVariant<Args>& norm_variant(const NormTable<Args>& t, int64_t filled) {
    int i = 0;
    while (i + 1 < t.n && (int64_t)t.v[i].threads * t.v[i].groups * 8 < filled) ++i;
    return t.v[i];
}

// Blocks of rows of the backward pass, two a CU (one where a row takes all of a workgroup's 1024 threads);
// their sums are joined afterwards.
struct NormBlocks {
    int64_t rows, blocks, np8;
};
NormBlocks norm_blocks(int64_t M, int64_t N, const NormVariant<NormGradArgs>& v) {
    NormBlocks b;
    const bool wide = v.threads == 1024;
    const int64_t at_once = wide ? 1 : 512 / v.threads, steps = ceil_div(M, at_once), most = wide ? kNumCU : 2 * kNumCU;
    // up to four steps stay in one block, which writes the sums itself
    b.rows = (steps <= 4 ? steps : ceil_div(steps, most)) * at_once;
    if (b.rows == 0) b.rows = at_once;
    b.blocks = ceil_div(M, b.rows);
    b.np8 = round_up(N, 8);
    return b;
}

// ---- the products -------------------------------------------------------------------------------

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

// A product's kernel and the splits of its contraction.
struct Plan {
    const MxVariant* v;
    int64_t tiles_m, tiles_n, splits, np8, part_bytes;
};

// Estimated microseconds: a launch's fixed part, what each further round of workgroups
// adds, and the contraction in steps of 256 entries.  A step takes its loads' latency
// in each round, or the time in which a CU takes its workgroups' bytes (mx_few) or
// multiplies (mx_tile; mx_large, alone on its CU).  Fitted to these kernels' times, with weights that
// come from memory, at 580 shapes of 1 to 4096 rows, 128 to 28672 columns and 128 to 16384
// entries, each with 1 to 8 splits: the choice is within 1.5 % of the best one on average
// for each format and product, and within 40 % at the worst.  The sides
// of it, in us, at 4096 columns of 4096 entries in 4 bits, weights in the cache: 64 rows 6.2 by mx_few's
// tiles of 32 x 32, 13 by mx_tile; 256 rows 14.1 and 13.2; 2048 rows 31.5 by mx_tile,
// 32.5 by mx_large; 4096 rows 57 and 38.  A split's join costs more than it gives
// unless there are few workgroups: 512 rows 13.9 in one go, 23 in two splits.
double est_us(const MxVariant& v, int64_t M, int64_t N, int64_t filled, int64_t splits) {
    const double wgs = (double)(ceil_div(M, v.bm) * ceil_div(N, v.bn) * splits);
    const auto whole = [](double x) { return (double)(int64_t)(x + 0.999999); };
    const double per_cu = whole(wgs / kNumCU), rounds = whole(wgs / (kNumCU * v.per_cu));
    const int planes = v.gated ? 2 : 1;
    const bool mx8 = v.format == MX8;
    double us;
    if (v.few) {
        const double steps = (double)ceil_div(ceil_div(filled / 256, splits), v.few);
        const double bytes = (double)v.few * (v.bm * (mx8 ? 256 : 128) + planes * v.bn * 128);
        us = 3.2 + 0.00075 * v.bm * v.bn * planes + 2.7 * (rounds - 1) + steps * larger(0.115 * rounds, per_cu * bytes / 42.8e3);
    } else if (v.bm == 128) {
        const double steps = (double)smaller(2 * ceil_div(ceil_div(filled, 512), splits), filled / 256);
        us = 6.6 + 3.1 * (rounds - 1) + (mx8 ? 0.91 : 0.73) * per_cu * steps;
    } else {
        const double steps = (double)smaller(4 * ceil_div(ceil_div(filled, 1024), splits), filled / 256);
        us = 3.6 + 8.0 * per_cu + (mx8 ? 2.26 : 1.29) * per_cu * steps;
    }
    if (splits > 1) us += 5.2 + 0.08 * splits + 0.32 * splits * M * N * planes * 4e-6;
    return us;
}

// From sizes, format and type alone, so that the workspace functions and the calls agree.
Plan plan_product(int64_t M, int64_t N, int64_t K, int format, int gated, int dtype) {
    const MxKernels k = kernels_for(dtype);
    const int64_t filled = mx_filled(K);
    Plan best;
    std::memset(&best, 0, sizeof(best));
    double best_us = 0.0;
    for (int i = 0; i < k.n; ++i) {
        const MxVariant& v = k.v[i];
        if (v.format != format || v.gated != gated) continue;
        const int64_t tiles = ceil_div(M, v.bm) * ceil_div(N, v.bn);
        if (round_up(tiles, 8) * v.threads >= (int64_t)1 << 32) continue;
        for (int64_t s : {1, 2, 3, 4, 6, 8}) {
            if (s > 1 && (s * (v.few ? v.few : 2) * v.bk > filled || tiles * s > 4 * kNumCU)) break;
            const double us = est_us(v, M, N, filled, s);
            if (best.v && us >= best_us) continue;
            best_us = us;
            best.v = &v;
            best.splits = s;
        }
    }
    if (!best.v) return best;
    best.tiles_m = ceil_div(M, best.v->bm);
    best.tiles_n = ceil_div(N, best.v->bn);
    best.np8 = round_up(N, 8);
    best.part_bytes = best.splits > 1 ? best.splits * (gated ? 2 : 1) * M * best.np8 * 4 : 0;
    return best;
}

// fp32 outputs of MX8 activations: the scaled MFMAs' sums are not fp32's there, so mx_few
// multiplies the entries' values (MxFewCfg::WIDE).  With more rows the values are
// written out once, in bf16, which holds them, and linear_kernel multiplies them: by
// 4096 x 4096 128 rows take 18 us in mx_few, 38 that way; 256 rows 34 and 36; 512 rows 65 and 42.  Of those 42 the values
// take 15, the product 22 and its join 6; of 4096 rows' 114 the values 25.
constexpr int64_t kFewRows = 256;
bool through_values(int64_t M, int64_t K, int format, int dtype) {
    return format == MX8 && dtype == PGEMM_F32 && M > kFewRows && K > 0;
}
// Its workspace: the values, the products' sums (where an epilogue follows), the product's own.
struct Values {
    int64_t x, w, z, ldz, own, total;
};
int64_t values_layout(int64_t M, int64_t N, int64_t K, int planes, Values& l) {
    const int64_t filled = mx_filled(K);
    l.own = pgemm_linear_workspace(M, N, filled, PGEMM_BF16);
    if (l.own < 0) return l.own;
    l.ldz = round_up(N, 8);
    if (l.ldz >= kMaxLd) return PGEMM_ERR_TOO_LARGE;
    l.x = round_up(M * filled * 2, 256);
    l.w = round_up(N * filled * 2, 256);
    l.z = round_up(M * l.ldz * 4, 256);
    return l.total = l.x + l.w + planes * l.z + l.own;
}

// `plan`: the choice, where there is one.
int64_t product_workspace(int64_t M, int64_t N, int64_t K, int format, int dtype, int planes, Plan& plan) {
    if (!float_type(dtype)) return PGEMM_ERR_UNSUPPORTED_DTYPE;
    if (format != PGEMM_MX8 && format != PGEMM_MX4) return PGEMM_ERR_INVALID_ARG;
    if (M < 0 || N < 0 || K < 0) return PGEMM_ERR_INVALID_ARG;
    if (M > kMaxDim || N >= kMaxLd || mx_filled(K) >= kMaxLd || ceil_div(M, 64) * ceil_div(N, 64) >= (int64_t)1 << 24)
        return PGEMM_ERR_TOO_LARGE;
    if (M == 0 || N == 0) return 0;
    if (through_values(M, K, format, dtype)) {
        Values l;
        return values_layout(M, N, K, planes, l);
    }
    plan = plan_product(M, N, K, format, planes == 2, dtype);
    return plan.v ? round_up(plan.part_bytes, 256) : PGEMM_ERR_TOO_LARGE;
}

struct Product {
    const void *XQ, *XS, *WQ[2], *WS[2];
    int64_t ldxq, ldxs, ldwq, ldws;
    const void *bias[2], *R;
    int64_t ldr;
    void* Y;
    int64_t ldy;
};

int run_values(int64_t M, int64_t N, int64_t K, const Product& q, const EpiArgs& e, int planes, void* workspace,
               hipStream_t stream) {
    Values l;
    if (values_layout(M, N, K, planes, l) < 0) return PGEMM_ERR_TOO_LARGE;  // found out before, with the workspace
    const int64_t filled = mx_filled(K);
    char* ws = (char*)workspace;
    char *x = ws, *w = ws + l.x, *z = w + l.w, *own = z + planes * l.z;
    const bool bare = planes == 1 && !e.bias[0] && !e.R && e.act.kind == ACTK_NONE;  // the sums are the output
    PGEMM_TRY(pgemm_mx_dequantize(M, filled, q.XQ, q.ldxq, q.XS, q.ldxs, PGEMM_MX8, x, filled, PGEMM_BF16, stream));
    for (int p = 0; p < planes; ++p) {  // one weight after the other, in the same place
        PGEMM_TRY(pgemm_mx_dequantize(N, filled, q.WQ[p], q.ldwq, q.WS[p], q.ldws, PGEMM_MX4, w, filled, PGEMM_BF16, stream));
        PGEMM_TRY(pgemm_linear(M, N, filled, x, filled > 0 ? filled : 1, w, filled > 0 ? filled : 1, PGEMM_NK, nullptr, nullptr, 0,
                               PGEMM_ACT_NONE, nullptr, 0, bare ? q.Y : (void*)(z + p * l.z), bare ? q.ldy : l.ldz, PGEMM_F32,
                               PGEMM_BF16, own, l.own, stream));
    }
    if (bare) return PGEMM_OK;
    MxRestArgs a;
    a.Z = (const float*)z;
    a.plane = l.z / 4;
    a.ldz = l.ldz;
    a.e = e;
    return launched("mx_rest", kernels_for(PGEMM_F32).rest(a, planes == 2, grid_for(ceil_div(N, 1024) * M, 1), stream));
}

int run_product(int64_t M, int64_t N, int64_t K, const Product& q, int format, int act, int dtype, int planes,
                void* workspace, int64_t workspace_bytes, hipStream_t stream) {
    Plan p;
    const int64_t need = product_workspace(M, N, K, format, dtype, planes, p), es = elem_size(dtype);
    if (need < 0) return (int)need;
    if (act < PGEMM_ACT_NONE || act > PGEMM_ACT_GELU_TANH) return PGEMM_ERR_INVALID_ARG;
    PGEMM_TRY(check_blocks(q.XQ, q.ldxq, q.XS, q.ldxs, N > 0 ? M : 0, K, format));
    for (int p = 0; p < planes; ++p) {
        PGEMM_TRY(check_blocks(q.WQ[p], q.ldwq, q.WS[p], q.ldws, M > 0 ? N : 0, K, PGEMM_MX4));
        PGEMM_TRY(check_vector(q.bias[p], es));
    }
    PGEMM_TRY(check_matrix(q.R, M, N, q.ldr, es, false));
    PGEMM_TRY(check_matrix(q.Y, M, N, q.ldy, es, true));
    if (M == 0 || N == 0) return PGEMM_OK;
    PGEMM_TRY(check_workspace(workspace, workspace_bytes, need));
    MxArgs a;
    std::memset(&a, 0, sizeof(a));
    a.A = q.XQ;
    a.SA = q.XS;
    for (int p = 0; p < 2; ++p) {
        a.B[p] = q.WQ[p];
        a.SB[p] = q.WS[p];
        a.e.bias[p] = q.bias[p];
    }
    a.lda = q.ldxq;
    a.lsa = q.ldxs;
    a.ldb = q.ldwq;
    a.lsb = q.ldws;
    a.filled = (int)mx_filled(K);
    a.e.Y[0] = a.e.Y[1] = q.Y;
    a.e.ldy = q.ldy;
    a.e.R = q.R;
    a.e.ldr = q.ldr;
    a.e.act = act_args(act);
    a.e.M = (int)M;
    a.e.N = (int)N;
    a.e.out_f32 = dtype == PGEMM_F32;
    if (through_values(M, K, format, dtype)) return run_values(M, N, K, q, a.e, planes, workspace, stream);
    a.tiles_m = (int)p.tiles_m;
    a.tiles_n = (int)p.tiles_n;
    a.group_m = 4;
    a.splits = (int)p.splits;
    a.part = p.splits > 1 ? (float*)workspace : nullptr;
    a.np8 = (int)p.np8;
    PGEMM_TRY(launched("mx_product", p.v->launch(a, (int)round_up(p.tiles_m * p.tiles_n * p.splits, 8), stream)));
    if (p.splits == 1) return PGEMM_OK;
    LinArgs j;
    std::memset(&j, 0, sizeof(j));
    j.outs = 1;
    j.splits = a.splits;
    j.part = a.part;
    j.np8 = a.np8;
    j.e = a.e;
    const MxKernels k = kernels_for(dtype);
    return launched("linear_join", (planes == 2 ? k.join_gated : k.join)(j, (int)(ceil_div(N, kJoinCols) * M), stream));
}

}  // namespace

extern "C" {

int64_t pgemm_rms_norm_backward_workspace(int64_t M, int64_t N, int dtype) {
    PGEMM_TRY(check_sizes(M, N, dtype));
    const NormVariant<NormGradArgs>& v = norm_variant(kernels_for(dtype).norm_grad, N);
    const NormBlocks b = norm_blocks(M, N, v);
    return b.blocks > 1 || (v.groups == 0 && M > 0) ? round_up(b.blocks * b.np8 * 4, 256) : 0;
}

int pgemm_rms_norm(int64_t M, int64_t N, const void* X, int64_t ldx, const void* R, int64_t ldr, const void* weight,
                   double eps, void* H, int64_t ldh, void* Y, int64_t ldy, int out_dtype, void* Q, int64_t ldq, void* S,
                   int64_t lds, int format, int dtype, void* stream) {
    PGEMM_TRY(check_sizes(M, N, dtype));
    if ((out_dtype != dtype && out_dtype != PGEMM_F32) || !(eps >= 0.0 && eps <= 3e38) || !Q != !S) return PGEMM_ERR_INVALID_ARG;
    const int64_t es = elem_size(dtype);
    PGEMM_TRY(check_matrix(X, M, N, ldx, es, true));
    PGEMM_TRY(check_matrix(R, M, N, ldr, es, false));
    PGEMM_TRY(check_vector(weight, es));
    PGEMM_TRY(check_matrix(H, M, N, ldh, es, false));
    PGEMM_TRY(check_matrix(Y, M, N, ldy, elem_size(out_dtype), false));
    if (Q) PGEMM_TRY(check_blocks(Q, ldq, S, lds, M, N, format));
    if (M == 0 || N == 0 || (!H && !Y && !Q)) return PGEMM_OK;
    NormArgs a;
    std::memset(&a, 0, sizeof(a));
    a.X = X;
    a.R = R;
    a.w = weight;
    a.H = H;
    a.Y = Y;
    a.Q = Q;
    a.S = S;
    a.ldx = ldx;
    a.ldr = ldr;
    a.ldh = ldh;
    a.ldy = ldy;
    a.ldq = ldq;
    a.lds = lds;
    a.eps = (float)eps;
    a.M = (int)M;
    a.N = (int)N;
    a.filled = (int)(Q ? mx_filled(N) : N);
    a.y_f32 = out_dtype == PGEMM_F32;
    a.format = format;
    const NormVariant<NormArgs>& v = norm_variant(kernels_for(dtype).norm, a.filled);
    // at most eight workgroups a CU, which go on to further rows: 4096 x 4096 in bf16 takes 22.5 us with 2048
    // workgroups, 24.2 with one a row
    const int64_t grid = smaller(grid_for(M, v.threads < 256 ? 256 / v.threads : 1), 8 * kNumCU);
    return launched("rms_norm", v.launch(a, (int)grid, (hipStream_t)stream));
}

int pgemm_rms_norm_backward(int64_t M, int64_t N, const void* dY, int64_t lddy, const void* H, int64_t ldh,
                            const void* weight, double eps, const void* dH, int64_t lddh, void* dX, int64_t lddx,
                            void* dweight, int grad_dtype, int dtype, void* workspace, int64_t workspace_bytes,
                            void* stream) {
    PGEMM_TRY(check_sizes(M, N, dtype));
    if ((grad_dtype != dtype && grad_dtype != PGEMM_F32) || !(eps >= 0.0 && eps <= 3e38)) return PGEMM_ERR_INVALID_ARG;
    const int64_t es = elem_size(dtype);
    PGEMM_TRY(check_matrix(dY, M, N, lddy, es, dX || dweight));
    PGEMM_TRY(check_matrix(H, M, N, ldh, es, dX || dweight));
    PGEMM_TRY(check_vector(weight, es));
    PGEMM_TRY(check_matrix(dH, M, N, lddh, es, false));
    PGEMM_TRY(check_matrix(dX, M, N, lddx, es, false));
    PGEMM_TRY(check_vector(dweight, elem_size(grad_dtype)));
    if (N == 0 || (!dX && !dweight)) return PGEMM_OK;
    if (dweight) PGEMM_TRY(check_workspace(workspace, workspace_bytes, pgemm_rms_norm_backward_workspace(M, N, dtype)));
    const MxKernels k = kernels_for(dtype);
    const NormVariant<NormGradArgs>& v = norm_variant(k.norm_grad, N);
    const NormBlocks b = norm_blocks(M, N, v);
    const bool joined = b.blocks != 1 || v.groups == 0;
    if (M > 0) {
        NormGradArgs a;
        std::memset(&a, 0, sizeof(a));
        a.dY = dY;
        a.H = H;
        a.w = weight;
        a.dH = dH;
        a.dX = dX;
        if (joined) a.sums = dweight ? (float*)workspace : nullptr;
        else a.dw = dweight;
        a.dw_f32 = grad_dtype == PGEMM_F32;
        a.lddy = lddy;
        a.ldh = ldh;
        a.lddh = lddh;
        a.lddx = lddx;
        a.eps = (float)eps;
        a.M = (int)M;
        a.N = (int)N;
        a.np8 = (int)b.np8;
        a.rows = (int)b.rows;
        PGEMM_TRY(launched("rms_norm_grad", v.launch(a, (int)b.blocks, (hipStream_t)stream)));
    }
    if (!dweight || !joined) return PGEMM_OK;
    NormSumArgs t;
    std::memset(&t, 0, sizeof(t));
    t.sums = (const float*)workspace;
    t.out = dweight;
    t.blocks = (int)b.blocks;
    t.np8 = (int)b.np8;
    t.N = (int)N;
    t.out_f32 = grad_dtype == PGEMM_F32;
    return launched("rms_norm_join", k.norm_join(t, grid_for(N, 16), (hipStream_t)stream));
}

int pgemm_mx_quantize(int64_t rows, int64_t K, const void* X, int64_t ldx, int x_order, int dtype, void* Q, int64_t ldq,
                      void* S, int64_t lds, int format, void* stream) {
    if (!float_type(dtype)) return PGEMM_ERR_UNSUPPORTED_DTYPE;
    if (rows < 0 || K < 0 || (x_order != PGEMM_KN && x_order != PGEMM_NK)) return PGEMM_ERR_INVALID_ARG;
    if (rows > kMaxDim || K > kMaxDim) return PGEMM_ERR_TOO_LARGE;
    if (x_order == PGEMM_KN) PGEMM_TRY(check_matrix(X, K, rows, ldx, elem_size(dtype), true));
    else PGEMM_TRY(check_matrix(X, rows, K, ldx, elem_size(dtype), true));
    PGEMM_TRY(check_blocks(Q, ldq, S, lds, rows, K, format));
    if (rows == 0 || K == 0) return PGEMM_OK;
    MxCopyArgs a;
    std::memset(&a, 0, sizeof(a));
    a.X = const_cast<void*>(X);
    a.Q = Q;
    a.S = S;
    a.ldx = ldx;
    a.ldq = ldq;
    a.lds = lds;
    a.rows = (int)rows;
    a.K = (int)K;
    a.filled = (int)mx_filled(K);
    const bool columns = x_order == PGEMM_KN;
    const int grid = columns ? grid_for(ceil_div(rows, kColumnRows) * (a.filled / 256), 1) : share_rows(a, a.filled / 8);
    return launched("mx_quantize", kernels_for(dtype).quantize(a, format, columns, grid, (hipStream_t)stream));
}

int pgemm_mx_dequantize(int64_t rows, int64_t K, const void* Q, int64_t ldq, const void* S, int64_t lds, int format,
                        void* X, int64_t ldx, int dtype, void* stream) {
    PGEMM_TRY(check_sizes(rows, K, dtype));
    PGEMM_TRY(check_blocks(Q, ldq, S, lds, rows, K, format));
    PGEMM_TRY(check_matrix(X, rows, K, ldx, elem_size(dtype), true));
    if (rows == 0 || K == 0) return PGEMM_OK;
    MxCopyArgs a;
    std::memset(&a, 0, sizeof(a));
    a.X = X;
    a.Q = const_cast<void*>(Q);
    a.S = const_cast<void*>(S);
    a.ldx = ldx;
    a.ldq = ldq;
    a.lds = lds;
    a.rows = (int)rows;
    a.K = (int)K;
    a.filled = (int)mx_filled(K);
    const int grid = share_rows(a, ceil_div(K, 8));
    return launched("mx_dequantize", kernels_for(dtype).dequantize(a, format, grid, (hipStream_t)stream));
}

int64_t pgemm_mx_linear_workspace(int64_t M, int64_t N, int64_t K, int x_format, int dtype) {
    Plan p;
    return product_workspace(M, N, K, x_format, dtype, 1, p);
}
int64_t pgemm_mx_gated_workspace(int64_t M, int64_t N, int64_t K, int x_format, int dtype) {
    Plan p;
    return product_workspace(M, N, K, x_format, dtype, 2, p);
}

int pgemm_mx_linear(int64_t M, int64_t N, int64_t K, const void* XQ, int64_t ldxq, const void* XS, int64_t ldxs,
                    int x_format, const void* WQ, int64_t ldwq, const void* WS, int64_t ldws, const void* bias,
                    const void* R, int64_t ldr, int act, void* Y, int64_t ldy, int dtype, void* workspace,
                    int64_t workspace_bytes, void* stream) {
    Product q;
    std::memset(&q, 0, sizeof(q));
    q.XQ = XQ;
    q.XS = XS;
    q.ldxq = ldxq;
    q.ldxs = ldxs;
    q.WQ[0] = q.WQ[1] = WQ;
    q.WS[0] = q.WS[1] = WS;
    q.ldwq = ldwq;
    q.ldws = ldws;
    q.bias[0] = bias;
    q.R = R;
    q.ldr = ldr;
    q.Y = Y;
    q.ldy = ldy;
    return run_product(M, N, K, q, x_format, act, dtype, 1, workspace, workspace_bytes, (hipStream_t)stream);
}

int pgemm_mx_gated(int64_t M, int64_t N, int64_t K, const void* XQ, int64_t ldxq, const void* XS, int64_t ldxs,
                   int x_format, const void* WgQ, const void* WuQ, int64_t ldwq, const void* WgS, const void* WuS,
                   int64_t ldws, const void* bias_g, const void* bias_u, int act, void* H, int64_t ldh, int dtype,
                   void* workspace, int64_t workspace_bytes, void* stream) {
    Product q;
    std::memset(&q, 0, sizeof(q));
    q.XQ = XQ;
    q.XS = XS;
    q.ldxq = ldxq;
    q.ldxs = ldxs;
    q.WQ[0] = WgQ;
    q.WQ[1] = WuQ;
    q.WS[0] = WgS;
    q.WS[1] = WuS;
    q.ldwq = ldwq;
    q.ldws = ldws;
    q.bias[0] = bias_g;
    q.bias[1] = bias_u;
    q.Y = H;
    q.ldy = ldh;
    return run_product(M, N, K, q, x_format, act, dtype, 2, workspace, workspace_bytes, (hipStream_t)stream);
}

}  // extern "C"
