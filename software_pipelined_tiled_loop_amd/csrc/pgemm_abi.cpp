// pgemm_abi.cpp -- the C ABI: argument validation, the planner and the launch.
//
// The planner picks (tile, stages, producer) for a problem:
//   * producer: DIRECT whenever both operands meet the 16-byte vector rules;
//     otherwise the register-staged variants the alignment admits (GENERIC,
//     and STAGED_A / STAGED_B when B / A alone keeps the rules), chosen with
//     tile and depth by their measured efficiencies (REGISTER only on
//     request);
//   * tile and stages (DIRECT): the compiled variant -- tile class and ring
//     depth -- with the smallest estimated time of the busiest CU (its tiles
//     in rounds of co-resident workgroups at that depth's residency, a
//     partial last round at its measured cost, the class's fixed cost per
//     round, and that depth's measured K-tile efficiency, which holds what
//     the ring's lookahead leaves of the load latency); for fp16, bf16 and
//     int8 near-equal estimates go to the larger tile (tie_margin).  Page
//     "Software pipelines and asynchronous copies", section "Selecting the
//     number of stages", asks for stage counts compared on the kernel
//     itself; its uncovered-latency estimate max(0, L - (S-1)*C) (section
//     "Worked example: Choosing between two and four stages") is reported
//     with the plan, with C the time one K tile takes on a SIMD shared by
//     the workgroups resident on the CU (its MFMA cycles over the measured
//     efficiency).  No depth beyond the number of K tiles is considered
//     (section "Prologue, steady state, and epilogue": fewer K tiles than
//     stages).
//   * register-staged producers take tile and depth together from measured
//     per-variant efficiencies (register pressure decides their depth).
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdio>
#include <cstdint>
#include <cstring>

#include "pgemm.h"
#include "variants.hpp"

using namespace pgemm;

namespace {

constexpr int kNumCU = 256;
constexpr int kLdsPerCU = 163840;

// Measured constants, regenerated by the re-run tile search (bench.py
// --retune, which times every compiled variant against the kernel as it now
// is; page "Double Buffering: Software Pipelining the K-Loop", section "What
// Could Be Improved") into planner_tables.json, from which build.py writes
// planner_tables.inc:
//   kLoadLatencyCycles   effective global->LDS latency a ring has to cover,
//                        SIMD clocks: the vmcnt wait per K tile of the
//                        single-buffer kernel (whole latency exposed), from
//                        the wait-profile build;
//   kPrologueCycles      fixed cost of a round for a class the table lacks;
//   kTieMargin[dtype]    estimates within this factor count as equal and the
//                        larger tile wins (for the dtypes whose clock falls
//                        with data movement; 1.0 = cheapest estimate);
//   kClassTable          per DIRECT variant (tile class, ring depth): eff
//                        (fraction of dense peak of the K loop at that
//                        depth, from its 4096^3 time), first and round (the
//                        class's fixed cycles of the first round of
//                        workgroups -- prologue with cold loads, epilogue and
//                        C store -- and of each later one, whose start
//                        overlaps the previous round's tail, fitted at the
//                        class's fastest depth to 4096 x 4096 outputs at
//                        K = 4096 and K = 256 and 8192 x 8192 at K = 128);
//                        and lam (cost of a partial last round: r < occ
//                        co-resident workgroups take r + lam*(occ - r)
//                        workgroup-times, from the time of one workgroup per
//                        CU against occ, at that depth);
//   kStagedTable         per register-staged variant (tile, depth, producer):
//                        eff on the ragged problem (misaligned A; misaligned
//                        B for STAGED_B) or, for REGISTER, at 4096^3.
struct ClassEntry {
    int dt, bm, bn, bk, s;
    double eff, lam, first, round;
};
struct StagedEntry {
    int dt, bm, bn, bk, s, p;
    double eff;
};
#include "planner_tables.inc"

double tie_margin(int dtype) { return kTieMargin[dtype]; }

struct Table {
    const VariantDesc* v;
    int n;
};

Table table_for(int dtype) {
    Table t{nullptr, 0};
    switch (dtype) {
        case PGEMM_F32: t.v = variants_f32(&t.n); break;
        case PGEMM_F16: t.v = variants_f16(&t.n); break;
        case PGEMM_BF16: t.v = variants_bf16(&t.n); break;
        case PGEMM_I8: t.v = variants_i8(&t.n); break;
        default: break;
    }
    return t;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

int elem_bytes(int dtype) { return dtype == PGEMM_F32 ? 4 : dtype == PGEMM_I8 ? 1 : 2; }

// Dense MFMA rate per SIMD per clock for the dtype (MI355X: 256 CUs x 4 SIMDs at 2.4 GHz).
double flops_per_simd_clk(int dtype) {
    switch (dtype) {
        case PGEMM_F32: return 64.0;
        case PGEMM_I8: return 2048.0;
        default: return 1024.0;
    }
}

// Register estimate of a variant (accumulators + two fragment sets + staging
// + addressing) -> waves per SIMD.  Used only to estimate residency.
int est_vgprs(const VariantDesc& d) {
    const int nw = d.wgm * d.wgn;
    const int wm = d.bm / d.wgm, wn = d.bn / d.wgn;
    const int fm = wm / 16, fn = wn / 16;
    const int es = elem_bytes(d.dtype);
    const int acc = fm * fn * 4;
    const int frags = 2 * (fm + fn) * 4;
    const int staging = d.producer == PROD_DIRECT ? 0 : (d.bm * d.bk + d.bk * d.bn) * es / (64 * nw) / 4;
    return acc + frags + staging + 40;
}

int wg_per_cu(const VariantDesc& d) {
    const int nw = d.wgm * d.wgn;
    int v = est_vgprs(d);
    v = (v + 7) / 8 * 8;
    int waves_per_simd = 512 / (v < 512 ? v : 512);
    if (waves_per_simd > 8) waves_per_simd = 8;
    int by_regs = waves_per_simd * 4 / nw;
    int by_lds = kLdsPerCU / d.lds_bytes;
    int r = by_regs < by_lds ? by_regs : by_lds;
    return r < 1 ? 1 : r;
}

// MFMA cycles of one K tile on one SIMD, with `share` workgroups per CU.
double tile_compute_cycles(const VariantDesc& d, int share) {
    const double flops = 2.0 * d.bm * d.bn * d.bk;
    return flops / (4.0 * flops_per_simd_clk(d.dtype)) * share;
}

// Measured behaviour of a tile class (kClassTable).  A class missing from
// the table (a tests checks none is) falls back to an operand-traffic
// estimate.
struct ClassModel {
    double eff, lam, first, round;
};

ClassModel class_model(const VariantDesc& d) {
    // the row of this tile class at this ring depth; else (register-staged
    // variants, whose own efficiency comes from kStagedTable) the class's
    // row at the nearest depth
    const ClassEntry* hit = nullptr;
    for (const ClassEntry& x : kClassTable)
        if (x.dt == d.dtype && x.bm == d.bm && x.bn == d.bn && x.bk == d.bk &&
            (!hit || std::abs(x.s - d.stages) < std::abs(hit->s - d.stages)))
            hit = &x;
    if (hit)
        return {hit->eff, hit->lam, hit->first >= 0.0 ? hit->first : kPrologueCycles,
                hit->round >= 0.0 ? hit->round : kPrologueCycles};
    const double per = (double)(d.bm + d.bn) / (2.0 * d.bm * d.bn);
    const double ref = 512.0 / (2.0 * 256 * 256);
    const double e = ref / per;
    return {0.4 * (e > 1.0 ? 1.0 : std::pow(e, 0.5)), 0.3, kPrologueCycles, kPrologueCycles};
}

double tile_efficiency(const VariantDesc& d) { return class_model(d).eff; }

// Output tiles on the busiest CU: the dispatcher spreads workgroups over all
// CUs before it stacks them.
int64_t tiles_per_cu(const VariantDesc& d, int64_t M, int64_t N) {
    return ceil_div(ceil_div(M, d.bm) * ceil_div(N, d.bn), kNumCU);
}

// Estimated SIMD clocks of the busiest CU for variant d at efficiency eff:
// its tiles run in rounds of up to wg_per_cu co-resident workgroups, a
// partial last round costs as the class model says, and the rounds pay the
// class's fixed costs: prologue, epilogue and C store, which weigh most on
// short problems (page "Software pipelines and asynchronous copies", section
// "Common errors": forgetting startup and drain).
double est_cycles(const VariantDesc& d, int64_t M, int64_t N, int64_t K, double eff) {
    const ClassModel cm = class_model(d);
    const int64_t occ = wg_per_cu(d);
    const int64_t n = tiles_per_cu(d, M, N);
    const int64_t full = n / occ, r = n % occ;
    const double units = (double)(full * occ) + (r ? (double)r + cm.lam * (double)(occ - r) : 0.0);
    const double kp = (double)(ceil_div(K, d.bk) * d.bk);
    const double per_tile = 2.0 * d.bm * d.bn * kp / (eff * 4.0 * flops_per_simd_clk(d.dtype));
    const int64_t rounds = ceil_div(n, occ);
    return units * per_tile + (rounds > 0 ? cm.first + (double)(rounds - 1) * cm.round : 0.0);
}

// MFMA cycles of one K tile on one SIMD with the workgroups that actually
// share the CU: at most wg_per_cu, and no more than the CU has tiles.
double shared_tile_cycles(const VariantDesc& d, int64_t M, int64_t N) {
    const int64_t n = tiles_per_cu(d, M, N);
    const int occ = wg_per_cu(d);
    return tile_compute_cycles(d, (int)(n < occ ? (n < 1 ? 1 : n) : occ));
}

// Cycles one K tile takes on a SIMD with the workgroups that share the CU:
// its MFMA cycles over the class's measured efficiency.  The load latency of
// the depth model is covered by this time.
double covering_cycles(const VariantDesc& d, int64_t M, int64_t N) {
    const double e = tile_efficiency(d);
    return shared_tile_cycles(d, M, N) / (e > 0.05 ? e : 0.05);
}

// Register-staged producers (REGISTER, GENERIC, STAGED_A/B): measured
// efficiency of each (tile class, ring depth) pair (kStagedTable).  For these
// producers the best depth depends on register pressure as much as on
// latency (staging registers next to the doubled fragment set, at the 256
// registers a wave of a two-waves-per-SIMD workgroup may hold), so the
// planner picks the (tile, depth) pair directly from the table.
double staged_efficiency(const VariantDesc& d) {
    for (const StagedEntry& x : kStagedTable)
        if (x.dt == d.dtype && x.bm == d.bm && x.bn == d.bn && x.bk == d.bk && x.s == d.stages && x.p == d.producer)
            return x.eff;
    return 0.5 * tile_efficiency(d);
}


// Workgroups to launch: one per output tile (default), or, on request
// (pgemm_opts.workgroups), fewer persistent ones that loop over the tiles
// with one K-tile ring across tile boundaries.  Always a multiple of 8 (the
// kernel splits the tiles into one contiguous range per XCD); surplus
// workgroups find no tile and exit.
//
// Persistence is not the default.  Measured on MI355X (bf16): 2-7 % faster
// on 128 x 128 tiles at 4096^2 with K <= 1024 and 4 % at 8192^2 x 1024, but
// 9 % slower at 8192^2 x 4096.  The C stores count in the same vmcnt as the
// ring's loads, so a persistent workgroup's next ready barrier also waits for
// its own stores; with one workgroup per tile a retiring workgroup's stores
// drain while a fresh one (with its own counters) starts on the CU.  A
// persistent grid must also match residency exactly: the dispatcher packs
// workgroups onto CUs, so a smaller grid leaves CUs idle.
int launch_grid(int64_t M, int64_t N, const VariantDesc& d, const pgemm_opts* opts) {
    const int64_t tiles = ceil_div(M, d.bm) * ceil_div(N, d.bn);
    int64_t grid = ceil_div(tiles, 8) * 8;
    if (opts && opts->workgroups > 0) {
        const int64_t want = ceil_div(opts->workgroups, 8) * 8;
        if (want < grid) grid = want;
    }
    return grid < 8 ? 8 : (int)grid;
}

bool producer_matches(const VariantDesc& d, int want) { return d.producer == want; }

// Whether a producer can run on operands of the given pgemm_aligned class
// (which operands hold whole 16-byte chunks per row): the REGISTER
// producer's unchecked 16-byte loads need it for both operands; LDS-DMA needs
// it for B, while for A the DIRECT producer completes a K tail that is not
// whole chunks by element loads (dma_patch).
bool admissible(int producer, int aligned) {
    const bool a = aligned == PGEMM_ALIGNED_BOTH || aligned == PGEMM_ALIGNED_A;
    const bool b = aligned == PGEMM_ALIGNED_BOTH || aligned == PGEMM_ALIGNED_B;
    switch (producer) {
        case PROD_DIRECT: return b;
        case PROD_REGISTER: return a && b;
        case PROD_STAGED_A: return b;
        case PROD_STAGED_B: return a;
        case PROD_GENERIC: return true;
        default: return false;
    }
}

struct Choice {
    int index = -1;
    int stages_req = 0;
    double uncovered = 0.0;
};

int plan_impl(int64_t M, int64_t N, int64_t K, int dtype, int stages, int aligned, const pgemm_opts* opts,
              Choice& out) {
    Table t = table_for(dtype);
    if (!t.v) return PGEMM_ERR_UNSUPPORTED_DTYPE;
    if (stages < 0 || stages > 4) return PGEMM_ERR_BAD_STAGES;
    if (aligned < PGEMM_ALIGNED_NONE || aligned > PGEMM_ALIGNED_B) return PGEMM_ERR_INVALID_ARG;
    // 0: the planner chooses among the producers the alignment admits
    int want_prod = aligned == PGEMM_ALIGNED_BOTH || aligned == PGEMM_ALIGNED_B ? PROD_DIRECT : 0;
    if (opts && opts->producer != PGEMM_PRODUCER_AUTO) {
        if (opts->producer < PGEMM_PRODUCER_DIRECT || opts->producer > PGEMM_PRODUCER_STAGED_B)
            return PGEMM_ERR_INVALID_ARG;
        if (!admissible(opts->producer, aligned)) return PGEMM_ERR_INFEASIBLE_PLAN;
        want_prod = opts->producer;
    }
    const bool force_tile = opts && (opts->tile_m || opts->tile_n || opts->tile_k);
    if (opts && (opts->skew < 0 || opts->skew > 64 || opts->workgroups < 0 || opts->waves < 0 ||
                 opts->reserved[0] != 0))
        return PGEMM_ERR_INVALID_ARG;
    const int force_waves = opts ? opts->waves : 0;

    // Register-staged producers: the (producer, tile, depth) with the best
    // estimated time at its measured efficiency, among the forced producer or
    // every one the alignment admits; an explicit depth restricts the choice
    // to variants of that depth.
    if (want_prod != PROD_DIRECT) {
        double best_time = 0.0;
        int best = -1;
        for (int i = 0; i < t.n; ++i) {
            const VariantDesc& d = t.v[i];
            if (want_prod ? !producer_matches(d, want_prod)
                          : (d.producer == PROD_DIRECT || d.producer == PROD_REGISTER || !admissible(d.producer, aligned)))
                continue;
            if (force_tile && (d.bm != opts->tile_m || d.bn != opts->tile_n || d.bk != opts->tile_k)) continue;
            if (force_waves && d.wgm * d.wgn != force_waves) continue;
            if (stages != 0 && d.stages != stages) continue;
            const double time = est_cycles(d, M, N, K, staged_efficiency(d));
            if (best < 0 || time < best_time * 0.999) {
                best = i;
                best_time = time;
            }
        }
        if (best < 0) return PGEMM_ERR_INFEASIBLE_PLAN;
        const VariantDesc& d = t.v[best];
        out.index = best;
        out.stages_req = d.stages;
        out.uncovered = pgemm_model_uncovered_cycles(kLoadLatencyCycles, covering_cycles(d, M, N), d.stages);
        return PGEMM_OK;
    }

    // DIRECT: every compiled variant -- each tile class at each ring depth,
    // no deeper than the problem has K tiles -- is estimated with its own
    // measured row (page "Software pipelines and asynchronous copies",
    // section "Selecting the number of stages": compare the stage counts on
    // the kernel itself), and the cheapest wins; for fp16, bf16 and int8 the
    // larger tile among near-equal ones.  An explicit depth keeps only that
    // depth.
    struct Cand {
        int index;
        double time;
    };
    Cand cands[128];
    int nc = 0;
    for (int i = 0; i < t.n && nc < 128; ++i) {
        const VariantDesc& d = t.v[i];
        if (!producer_matches(d, want_prod)) continue;
        if (force_tile && (d.bm != opts->tile_m || d.bn != opts->tile_n || d.bk != opts->tile_k)) continue;
        if (force_waves && d.wgm * d.wgn != force_waves) continue;
        if (stages != 0) {
            if (d.stages != stages) continue;
        } else {
            // a ring deeper than the K tiles loads nothing more and costs LDS
            const int64_t kt = ceil_div(K, (int64_t)d.bk);
            if (d.stages > 1 && d.stages > kt) continue;
        }
        cands[nc++] = {i, est_cycles(d, M, N, K, tile_efficiency(d))};
    }
    if (nc == 0) return PGEMM_ERR_INFEASIBLE_PLAN;
    double best_time = cands[0].time;
    for (int j = 1; j < nc; ++j) best_time = cands[j].time < best_time ? cands[j].time : best_time;
    int pick = -1;
    for (int j = 0; j < nc; ++j) {
        if (cands[j].time > best_time * tie_margin(dtype)) continue;
        const VariantDesc& d = t.v[cands[j].index];
        if (pick < 0) {
            pick = cands[j].index;
            continue;
        }
        const VariantDesc& p = t.v[pick];
        const int64_t area = (int64_t)d.bm * d.bn, parea = (int64_t)p.bm * p.bn;
        if (area > parea || (area == parea && cands[j].time < est_cycles(p, M, N, K, tile_efficiency(p))))
            pick = cands[j].index;
    }
    out.index = pick;
    out.stages_req = t.v[pick].stages;
    out.uncovered = pgemm_model_uncovered_cycles(kLoadLatencyCycles, covering_cycles(t.v[pick], M, N),
                                                 t.v[pick].stages);
    return PGEMM_OK;
}

void fill_info(int dtype, const VariantDesc& d, int idx, int64_t M, int64_t N, int64_t K, double uncovered,
               const pgemm_opts* opts, pgemm_plan_info* info) {
    std::memset(info, 0, sizeof(*info));
    info->tile_m = d.bm;
    info->tile_n = d.bn;
    info->tile_k = d.bk;
    info->stages = d.stages;
    info->num_k_tiles = (int)ceil_div(K, d.bk);
    const int nk1 = info->num_k_tiles < 1 ? 1 : info->num_k_tiles;
    info->stages_eff = d.stages < nk1 ? d.stages : nk1;
    info->producer = d.producer;
    info->threads = d.threads;
    info->waves_m = d.wgm;
    info->waves_n = d.wgn;
    info->lds_bytes = d.lds_bytes;
    info->wg_per_cu = wg_per_cu(d);
    info->grid = launch_grid(M, N, d, opts);
    int base = 0;  // global index: variants of lower dtypes come first
    for (int t = 0; t < dtype; ++t) base += table_for(t).n;
    info->variant = base + idx;
    info->est_uncovered_cycles = uncovered;
}

}  // namespace

extern "C" {

double pgemm_model_uncovered_cycles(double latency, double compute_per_tile, int stages) {
    if (stages <= 1) return latency;
    const double u = latency - (stages - 1) * compute_per_tile;
    return u > 0.0 ? u : 0.0;
}

int64_t pgemm_model_lds_bytes(int bm, int bn, int bk, int stages, int elem_bytes, int a_pad_elems_per_k) {
    // stages * (A tile + B tile) elements, plus any padding of the A rows
    return (int64_t)stages * ((int64_t)bm * bk + (int64_t)bk * bn + (int64_t)bk * a_pad_elems_per_k) * elem_bytes;
}

double pgemm_model_global_loads_per_output(int bm, int bn, int64_t K) {
    // A workgroup loads BM*K elements of A and K*BN of B for BM*BN outputs:
    // K/BN + K/BM global loads per output element.
    return (double)K / bn + (double)K / bm;
}

double pgemm_model_compute_load_ratio(int bm, int bn, int bk, int elem_bytes) {
    if (bm <= 0 || bn <= 0 || bk <= 0 || elem_bytes <= 0) return 0.0;
    // two flops per multiply-add of the K tile, over the A and B bytes it loads
    const double flops = 2.0 * bm * bn * bk;
    const double bytes = ((double)bm * bk + (double)bk * bn) * elem_bytes;
    return flops / bytes;
}

const char* pgemm_strerror(int status) {
    switch (status) {
        case PGEMM_OK: return "ok";
        case PGEMM_ERR_INVALID_ARG: return "invalid argument (size, leading dimension or null pointer)";
        case PGEMM_ERR_UNSUPPORTED_DTYPE: return "unsupported dtype";
        case PGEMM_ERR_BAD_STAGES: return "stages must be 0 (auto) or 1..4";
        case PGEMM_ERR_INFEASIBLE_PLAN: return "no compiled variant satisfies the requested options";
        case PGEMM_ERR_NONINTEGRAL_SCALAR: return "int8 GEMM needs integer alpha and beta in int32 range";
        case PGEMM_ERR_HIP: return "HIP runtime error at launch";
        case PGEMM_ERR_TOO_LARGE: return "problem exceeds 32-bit tile addressing";
        default: return "unknown status";
    }
}

int pgemm_version(void) { return 10100; }  // 1.1: the feed-forward operators; those behind them did not raise it

int pgemm_num_variants(void) {
    int n = 0;
    for (int d = 0; d < 4; ++d) n += table_for(d).n;
    return n;
}

int pgemm_variant_info(int index, pgemm_plan_info* out, int* dtype) {
    if (!out || index < 0) return PGEMM_ERR_INVALID_ARG;
    for (int d = 0; d < 4; ++d) {
        Table t = table_for(d);
        if (index < t.n) {
            fill_info(d, t.v[index], index, t.v[index].bm, t.v[index].bn, t.v[index].bk, 0.0, nullptr, out);
            if (dtype) *dtype = d;
            return PGEMM_OK;
        }
        index -= t.n;
    }
    return PGEMM_ERR_INVALID_ARG;
}

int pgemm_plan(int64_t M, int64_t N, int64_t K, int dtype, int stages, int aligned, const pgemm_opts* opts,
               pgemm_plan_info* out) {
    if (!out) return PGEMM_ERR_INVALID_ARG;
    if (dtype < 0 || dtype > 3) return PGEMM_ERR_UNSUPPORTED_DTYPE;
    if (M < 0 || N < 0 || K < 0) return PGEMM_ERR_INVALID_ARG;
    Choice c;
    int r = plan_impl(M, N, K, dtype, stages, aligned, opts, c);
    if (r != PGEMM_OK) return r;
    Table t = table_for(dtype);
    fill_info(dtype, t.v[c.index], c.index, M, N, K, c.uncovered, opts, out);
    return PGEMM_OK;
}

int pgemm_gemm_ex(int64_t M, int64_t N, int64_t K, double alpha, const void* A, int64_t lda, const void* B,
                  int64_t ldb, double beta, void* C, int64_t ldc, int dtype, int stages, const pgemm_opts* opts,
                  void* stream) {
    // ---- argument checks: all before anything touches the GPU ----
    if (dtype < 0 || dtype > 3) return PGEMM_ERR_UNSUPPORTED_DTYPE;
    if (stages < 0 || stages > 4) return PGEMM_ERR_BAD_STAGES;
    if (M < 0 || N < 0 || K < 0) return PGEMM_ERR_INVALID_ARG;
    if (lda < (K > 1 ? K : 1) || ldb < (N > 1 ? N : 1) || ldc < (N > 1 ? N : 1)) return PGEMM_ERR_INVALID_ARG;
    if (dtype == PGEMM_I8) {
        // integers in int32 range, -2^31 .. 2^31 - 1
        const auto int32_valued = [](double x) {
            return std::isfinite(x) && x == std::floor(x) && x >= -2147483648.0 && x <= 2147483647.0;
        };
        if (!int32_valued(alpha) || !int32_valued(beta)) return PGEMM_ERR_NONINTEGRAL_SCALAR;
    }
    if (M == 0 || N == 0) return PGEMM_OK;
    if (!C) return PGEMM_ERR_INVALID_ARG;
    if (K > 0 && (!A || !B)) return PGEMM_ERR_INVALID_ARG;
    const int es = elem_bytes(dtype);
    const int epc = 16 / es;
    // 32-bit tile addressing: byte offsets inside one tile must stay below 2^31,
    // and a tile origin plus one tile extent (at most 256) must fit a 32-bit int.
    if (M > 0x7fffff00 || N > 0x7fffff00 || K > 0x7fffff00) return PGEMM_ERR_TOO_LARGE;
    if ((double)lda * es * 256.0 >= 2147483648.0 || (double)ldb * es * 128.0 >= 2147483648.0 ||
        (double)ldc * 4.0 * 256.0 >= 2147483648.0)
        return PGEMM_ERR_TOO_LARGE;
    if (ceil_div(M, 128) * ceil_div(N, 64) > 0x7ffffff0) return PGEMM_ERR_TOO_LARGE;
    // Element alignment is required.  Rows may start at any element: LDS-DMA
    // and 16-byte loads take element-aligned addresses (measured on gfx950).
    // The chunk rule per operand selects the producers: no 16-byte chunk
    // straddles the end of A's K columns (A) or of B's N columns (B).
    if (((uintptr_t)A % es) || ((uintptr_t)B % es) || ((uintptr_t)C % 4)) return PGEMM_ERR_INVALID_ARG;
    const bool a_ok = K == 0 || K % epc == 0;
    const bool b_ok = K == 0 || N % epc == 0;
    const int aligned = a_ok && b_ok ? PGEMM_ALIGNED_BOTH
                        : a_ok       ? PGEMM_ALIGNED_A
                        : b_ok       ? PGEMM_ALIGNED_B
                                     : PGEMM_ALIGNED_NONE;

    Choice c;
    int r = plan_impl(M, N, K, dtype, stages, aligned, opts, c);
    if (r != PGEMM_OK) return r;
    const VariantDesc& d = table_for(dtype).v[c.index];

    KernelArgs a;
    std::memset(&a, 0, sizeof(a));
    a.A = A;
    a.B = B;
    a.C = C;
    a.lda = lda;
    a.ldb = ldb;
    a.ldc = ldc;
    a.M = (int)M;
    a.N = (int)N;
    a.K = (int)K;
    a.tiles_m = (int)ceil_div(M, d.bm);
    a.tiles_n = (int)ceil_div(N, d.bn);
    a.group_m = 4;
    a.alpha = (float)alpha;
    a.beta = (float)beta;
    a.ialpha = dtype == PGEMM_I8 ? (int)(int64_t)alpha : 0;
    a.ibeta = dtype == PGEMM_I8 ? (int)(int64_t)beta : 0;
    a.beta_nonzero = beta != 0.0;
    a.dbg_sleep = opts ? opts->skew : 0;
    const int grid = launch_grid(M, N, d, opts);
    const bool persistent = grid < ceil_div((int64_t)a.tiles_m * a.tiles_n, 8) * 8;
    hipError_t e = (persistent ? d.launch_persistent : d.launch)(a, grid, (hipStream_t)stream);
    if (e != hipSuccess) {
        // The status code alone cannot say which runtime error it was.
        std::fprintf(stderr, "pgemm: launch of %s %dx%dx%d S=%d (grid %d) failed: %s (%d)\n",
                     dtype == PGEMM_F32 ? "f32" : dtype == PGEMM_F16 ? "f16" : dtype == PGEMM_BF16 ? "bf16" : "i8",
                     d.bm, d.bn, d.bk, d.stages, grid, hipGetErrorString(e), (int)e);
        return PGEMM_ERR_HIP;
    }
    return PGEMM_OK;
}

int pgemm_gemm(int64_t M, int64_t N, int64_t K, double alpha, const void* A, int64_t lda, const void* B, int64_t ldb,
               double beta, void* C, int64_t ldc, int dtype, int stages, void* stream) {
    return pgemm_gemm_ex(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, dtype, stages, nullptr, stream);
}

}  // extern "C"
