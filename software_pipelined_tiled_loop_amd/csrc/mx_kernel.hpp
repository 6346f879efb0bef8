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
// (The 32 x 32 ones need half as many reads of LDS for a product as the 16 x 16 ones, of
// which mx_large has its own way.)
//
// mx_tile has 128 x 128 outputs, two workgroups a CU, and is for grids too small for
// mx_large's tiles.  Of 4096 columns and entries it takes in 4 bits 11.7 us for 256 rows, 15.3 for
// 512, 17.6 for 1024 and 31.9 for 2048 (2157 TFLOP/s); with MX8 activations 17.4 for
// 512, 20.4 and 34.8 for the last two.  Up to one round of the CUs the time is the K loop's
// latency, 0.3 us for 128 entries with weights from the cache, 0.4 with weights from memory.
#pragma once

#include "mx_format.hpp"

namespace pgemm {

typedef __attribute__((ext_vector_type(8))) int i32x8;
typedef __attribute__((ext_vector_type(16))) float f32x16;

__device__ __forceinline__ i32x8 two_chunks(i32x4 a, i32x4 b) { return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7); }

struct MxArgs {
    const void* A;      // activations' codes and scales
    const void* SA;
    const void* B[2];   // weights' (gated: Wg, Wu)
    const void* SB[2];
    int64_t lda, lsa, ldb, lsb;  // bytes
    int filled;         // entries of a stored row: whole groups
    int tiles_m, tiles_n, group_m;
    int splits;         // workgroups that share one output tile's K tiles
    float* part;        // fp32 sums of each split: [split][plane][M][np8]
    int np8;
    EpiArgs e;
};

// LDS tile of codes: rows of KC 16-byte chunks.  A fragment is 32 rows at one chunk
// (two chunks, for the two halves of the wave): the LDS serves the sixteen lanes of
// a half that have the same parity at a time, so those rows' chunks are spread over
// all sixteen places of their 256-byte lines.
template <int KC>
PGEMM_HD constexpr int mx_off(int row, int kc) {
    if constexpr (KC == 8) return ((row >> 1) << 8) + ((((row & 1) * 8 + kc) ^ ((row >> 1) & 15)) << 4);
    else return ((row >> 2) << 8) + ((((row & 3) * 4 + kc) ^ ((row >> 2) & 7)) << 4);
}
template <int KC>
PGEMM_HD void mx_inv(int off, int& row, int& kc) {
    const int line = off >> 8;
    if constexpr (KC == 8) {
        const int u = ((off >> 4) & 15) ^ (line & 15);
        row = 2 * line + (u >> 3);
        kc = u & 7;
    } else {
        const int u = ((off >> 4) & 15) ^ (line & 7);
        row = 4 * line + (u >> 2);
        kc = u & 3;
    }
}

// Scales go to LDS for 512 entries at a time, 16 bytes of a row, in a ring of their
// own: four bytes a row with every 128 entries made as many requests to the cache as
// the codes.
constexpr int kScaleGroup = 512;

// F: the activations' format.  Tiles of BM rows by BN weights' rows (gated: half of
// them of each weight), K tiles of 128 entries.
template <int D, int F, int BM_, int BN_, int S_, int WGM_, int WGN_, bool GATED_>
struct MxCfg {
    static constexpr int Dt = D, Fmt = F, BM = BM_, BN = BN_, S = S_, WGM = WGM_, WGN = WGN_;
    static constexpr bool GATED = GATED_;
    static constexpr int ES = D == DT_F32 ? 4 : 2;  // of a value
    static constexpr int BK = 128, NKS = 2, G = kScaleGroup / BK;  // entries; K steps; K tiles of a group of scales
    static constexpr int KCA = F == MX8 ? 8 : 4, KCB = 4;          // 16-byte chunks of a row
    static constexpr int NP = GATED ? 2 : 1, BNP = BN / NP;
    static constexpr int NW = WGM * WGN, NT = 64 * NW;
    static constexpr int WM = BM / WGM, WNP = BNP / WGN;
    static constexpr int FM = WM / 32, FNP = WNP / 32, FN = FNP * NP;
    static constexpr int A_BYTES = BM * KCA * 16, B_BYTES = BN * KCB * 16;
    static constexpr int SA_BYTES = BM * 16, S_STAGE = (BM + BN) * 16;  // scales: two stages behind the ring
    static constexpr int STAGE = A_BYTES + B_BYTES, AT_S = S * STAGE, LDS = AT_S + 2 * S_STAGE;
    static constexpr int MINW = 163840 / LDS * NW / 4;  // waves per SIMD, by the CU's LDS
    // LDS-DMA pieces of a wave, 1 KiB each
    static constexpr int A_INSTR = A_BYTES / 1024 / NW, B_INSTR = B_BYTES / 1024 / NW;
    static constexpr int LPS = A_INSTR + B_INSTR, S_INSTR = S_STAGE / 1024 / NW;
    static constexpr int XCH = F == MX8 ? 2 : 1;  // chunks of an activations' fragment
    static_assert(A_BYTES % (1024 * NW) == 0 && B_BYTES % (1024 * NW) == 0 && NW % 4 == 0, "a wave's pieces lie in one operand");
    static_assert(S_INSTR * NW * 64 == BM + BN && BM % (64 * S_INSTR) == 0 && BNP % (64 * S_INSTR) == 0, "scale pieces");
    static_assert(LDS <= 163840 && S >= 2 && LPS * (S - 2) <= 63, "ring");
    // Behind the ready edge of a group's last K tile the group after next is issued, and first read behind that of the
    // next group's last one: two edges later or more (a row's last group may be two K tiles), by when 2 LPS pieces have followed.
    static_assert(LPS * (S - 2) <= 2 * LPS, "scales are covered by the edge before their first read");
};

// Where the scales lie, as a wave goes along its K tiles, two of them at a time: half a
// group of scales, and a row ends with a pair.
template <class C>
struct MxTileWalk {
    uint32_t scale = C::AT_S;  // of the next pair's first K tile, in LDS (places in a group are 0 and 8)
    uint32_t stage = C::AT_S;  // the pair's scales' stage
    int row_left;              // pairs to the row's end
    bool half = false, ends = false;  // the next pair is its group's second; the pair is its group's last one
    PGEMM_HD explicit MxTileWalk(int pairs) : row_left(pairs) {}
    // Behind the pair's first K tile; where `ends`, the stage is free behind the second one's ready edge.
    PGEMM_HD void pair() {
        stage = scale & ~15u;
        ends = --row_left == 0 || half;
        half = !ends;
        scale = ends ? (uint32_t)(2 * C::AT_S + C::S_STAGE) - stage : stage + 8;
    }
};

template <class C>
struct MxFrags {
    i32x4 a[C::FM][C::XCH];
    i32x4 b[C::FN];
};
template <class C>
struct MxScales {
    int a[C::FM], b[C::FN];
};

// A scaled MFMA with the accumulators in AGPRs, from inline asm (as mfma_lone):
// weights times activations, byte KS (0 or 1) of each side's scales.  The compiler may
// put the scales' filling up to 32 bits right before it, so it brings its own two wait
// states, which pass while the MFMA before it runs.
template <class C, int KS>
__device__ __forceinline__ void mx_mfma(f32x16& acc, const i32x4 (&x)[C::XCH], const i32x4& w, int sx, int sw) {
    if constexpr (C::Fmt == MX8) {
        const i32x8 xx = two_chunks(x[0], x[1]);
        asm volatile("s_nop 1\n\tv_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[%5,%5,0] op_sel_hi:[0,0,0] cbsz:4"
                     : "+a"(acc)
                     : "v"(w), "v"(xx), "v"(sw), "v"(sx), "n"(KS));
    } else {
        asm volatile(
            "s_nop 1\n\tv_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[%5,%5,0] op_sel_hi:[0,0,0] cbsz:4 blgp:4"
            : "+a"(acc)
            : "v"(w), "v"(x[0]), "v"(sw), "v"(sx), "n"(KS));
    }
}

// Of a K tile's four blocks, K step ks takes ks and 2 + ks, so that a lane's scales
// of both steps lie side by side.  A lane of half g reads block 2 g + ks of e2m1,
// piece g of each of the two blocks of e4m3.
template <class C>
PGEMM_HD int mx_chunk_a(int ks, int g, int c) { return C::Fmt == MX8 ? 4 * c + 2 * ks + g : 2 * g + ks; }
template <class C>
PGEMM_HD int mx_chunk_b(int ks, int g) { return 2 * g + ks; }

// Reads of a K step's fragments in the order in which its MFMAs need them.
template <class C, int R>
__device__ __forceinline__ void mx_read(const char PGEMM_LDS* st, int ks, int wm0, int wn0, int lane, MxFrags<C>& f) {
    constexpr int XA = C::FM * C::XCH;
    const int r = lane & 31, g = lane >> 5;
    // b0, a0 (its chunks), the other b, the other a
    if constexpr (R == 0 || (R > C::XCH && R < C::XCH + C::FN)) {
        constexpr int j = R == 0 ? 0 : R - C::XCH;
        constexpr int panel = j / C::FNP;
        const int row = panel * C::BNP + wn0 + 32 * (j % C::FNP) + r;
        f.b[j] = *(const i32x4 PGEMM_LDS*)(st + C::A_BYTES + mx_off<C::KCB>(row, mx_chunk_b<C>(ks, g)));
    } else {
        constexpr int x = R <= C::XCH ? R - 1 : R - C::FN;
        static_assert(x >= 0 && x < XA, "reads");
        constexpr int i = x / C::XCH, c = x % C::XCH;
        f.a[i][c] = *(const i32x4 PGEMM_LDS*)(st + mx_off<C::KCA>(wm0 + 32 * i + r, mx_chunk_a<C>(ks, g, c)));
    }
}
// Scales of a K tile, from its place in the group on: the two bytes of blocks 2 g and 2 g + 1.
template <class C, int R>
__device__ __forceinline__ void mx_read_scale(const char PGEMM_LDS* st, int wm0, int wn0, int lane, MxScales<C>& s) {
    const int r = lane & 31, g = lane >> 5;
    const auto get = [&](int row) -> int { return *(const unsigned short PGEMM_LDS*)(st + row * 16 + 2 * g); };
    if constexpr (R < C::FN) s.b[R] = get(C::BM + R / C::FNP * C::BNP + wn0 + 32 * (R % C::FNP) + r);
    else s.a[R - C::FN] = get(wm0 + 32 * (R - C::FN) + r);
}

// Fragments and scales of the first K tile's first step.
template <class C, int R = 0>
__device__ __forceinline__ void mx_first(const char PGEMM_LDS* st, const char PGEMM_LDS* ss, int wm0, int wn0, int lane,
                                         MxFrags<C>& f, MxScales<C>& s) {
    constexpr int NR = C::FM * C::XCH + C::FN;
    if constexpr (R < NR) mx_read<C, R>(st, 0, wm0, wn0, lane, f);
    if constexpr (R < C::FM + C::FN) mx_read_scale<C, R>(ss, wm0, wn0, lane, s);
    if constexpr (R < NR) mx_first<C, R + 1>(st, ss, wm0, wn0, lane, f, s);
}

// The wave's side of the producer.  A K tile's place in the rows goes into the loads
// as their scalar offset; behind the rows' end it comes round to their beginning,
// also for the slots past the last K tile, which nobody reads.
template <class C>
struct MxSrc {
    i32x4 ra, rb, rs;            // the codes' rows; the next group of the scales that the wave loads
    uint32_t k, k_end;           // bytes in the weights' rows: the next K tile, the rows' end
    int s_turn, s_left;          // groups until the row's end, groups still to load
    int s_bytes, s_groups;       // bytes from rs's address to the end of the last row; groups of a row
    uint32_t va[C::A_INSTR], vb[C::B_INSTR], vs[C::S_INSTR];

    template <int PART>
    __device__ __forceinline__ void advance() {
        if constexpr (PART == 0) k += 16 * C::KCB;
        else k = k == k_end ? 0 : k;
    }
    // The next group of scales, to LDS.  The last one of a row may be half a group: its
    // other half is the next row's first bytes, or beyond the range, and not read.
    __device__ __forceinline__ void scales(uint32_t at) {
        rs[2] = s_left > 0 ? s_bytes : 0;
        i32x4 r;
#pragma unroll
        for (int d = 0; d < 4; ++d) r[d] = __builtin_amdgcn_readfirstlane(rs[d]);
#pragma unroll
        for (int q = 0; q < C::S_INSTR; ++q) dma16(r, vs[q], at + q * 1024u);
        --s_left;
        int by = 16;
        if (--s_turn == 0) by -= 16 * s_groups;
        const uint64_t p = (((uint64_t)(uint32_t)rs[1] << 32) | (uint32_t)rs[0]) + (int64_t)by;
        rs[0] = (int)(uint32_t)p;
        rs[1] = (int)(uint32_t)(p >> 32);  // the address stays below 2^48: the stride field stays zero
        s_bytes -= by;
    }
    // Piece I of the K tile, to LDS: its place (M0), and the load, which needs an instruction between them.
    template <int I>
    __device__ __forceinline__ void place(uint32_t a, uint32_t b) const {
        constexpr uint32_t off = (I < C::A_INSTR ? I : I - C::A_INSTR) * 1024u;
        asm volatile("s_add_u32 m0, %0, %1" : : "s"(I < C::A_INSTR ? a : b), "n"(off) : "m0", "scc");
    }
    template <int I>
    __device__ __forceinline__ void load() const {
        asm volatile("buffer_load_dwordx4 %0, %1, %2 offen lds"
                     :
                     : "v"(I < C::A_INSTR ? va[I < C::A_INSTR ? I : 0] : vb[I < C::A_INSTR ? 0 : I - C::A_INSTR]),
                       "s"(I < C::A_INSTR ? ra : rb), "s"(I < C::A_INSTR ? k * (C::KCA / C::KCB) : k)
                     : "memory");
    }
};
template <class C, int END, int I = 0>
__device__ __forceinline__ void mx_pieces(const MxSrc<C>& s, uint32_t a, uint32_t b) {
    if constexpr (I < END) {
        s.template place<I>(a, b);
        asm volatile("s_nop 0");
        s.template load<I>();
        mx_pieces<C, END, I + 1>(s, a, b);
    }
}

// Where a step reads and loads.
struct MxAt {
    const char PGEMM_LDS* codes;   // the stage of the fragments that it reads
    const char PGEMM_LDS* scales;  // the next K tile's scales in their group
    uint32_t a, b;                 // where the wave's pieces of the free stage go
    int wm0, wn0, lane;
};

// One K step, with what else is to be done spread between its MFMAs: reads of the
// next step's fragments (behind the ready edge the next K tile's, its scales first)
// and, in turns with them, half of a K tile's pieces, M0 first and the load an
// instruction later.  A K tile's pieces begin in the step behind the ready edge that
// frees their stage and end in the one that follows, so that they come at an even
// pace: the address path takes 16 clocks a piece and CU.
template <class C, bool LAST>
struct MxStep {
    static constexpr int NMF = C::FM * C::FN, NR = C::FM * C::XCH + C::FN, NS = LAST ? C::FM + C::FN : 0;
    static constexpr int HALF = C::LPS / 2, P0 = LAST ? 0 : HALF, NP = LAST ? HALF : C::LPS - HALF;
    static constexpr int READS = NS + NR, PIECES = 2 * NP, ADV = LAST ? 0 : 2;
    static constexpr int PAIRS = READS < PIECES ? READS : PIECES, JOBS = READS + PIECES + ADV;
    template <int J>
    static __device__ __forceinline__ void read(const MxAt& at, MxFrags<C>& nxt, MxScales<C>& sc) {
        if constexpr (J < NS) mx_read_scale<C, J>(at.scales, at.wm0, at.wn0, at.lane, sc);
        else mx_read<C, J - NS>(at.codes, LAST ? 0 : 1, at.wm0, at.wn0, at.lane, nxt);
    }
    template <int J, bool NOP>
    static __device__ __forceinline__ void piece(const MxAt& at, const MxSrc<C>& src) {
        if constexpr (J % 2 == 0) {
            src.template place<P0 + J / 2>(at.a, at.b);
            if constexpr (NOP) asm volatile("s_nop 0");
        } else {
            src.template load<P0 + J / 2>();
        }
    }
    template <int J>
    static __device__ __forceinline__ void job(const MxAt& at, MxFrags<C>& nxt, MxScales<C>& sc, MxSrc<C>& src) {
        if constexpr (J < 2 * PAIRS) {
            if constexpr (J % 2 == 0) read<J / 2>(at, nxt, sc);
            else piece<J / 2, false>(at, src);
        } else if constexpr (J < READS + PIECES) {
            if constexpr (READS > PIECES) read<J - PIECES>(at, nxt, sc);
            else piece<J - READS, true>(at, src);
        } else {
            src.template advance<J - READS - PIECES>();
        }
    }
    template <int J, int END>
    static __device__ __forceinline__ void jobs(const MxAt& at, MxFrags<C>& nxt, MxScales<C>& sc, MxSrc<C>& src) {
        if constexpr (J < END) {
            job<J>(at, nxt, sc, src);
            jobs<J + 1, END>(at, nxt, sc, src);
        }
    }
    template <int M = 0>
    static __device__ __forceinline__ void run(f32x16 (&acc)[C::FM][C::FN], const MxFrags<C>& use, const MxScales<C>& us,
                                               MxFrags<C>& nxt, MxScales<C>& sc, MxSrc<C>& src, const MxAt& at) {
        if constexpr (M < NMF) {
            constexpr int i = M / C::FN, j = M % C::FN;
            mx_mfma<C, LAST ? 1 : 0>(acc[i][j], use.a[i], use.b[j], us.a[i], us.b[j]);
            jobs<M * JOBS / NMF, (M + 1) * JOBS / NMF>(at, nxt, sc, src);
            __builtin_amdgcn_sched_barrier(0);
            run<M + 1>(acc, use, us, nxt, sc, src, at);
        }
    }
};

// The epilogue through LDS: as LinOut and lin_epilogue, on blocks of 32 x 32.
template <class C>
struct MxOut {
    static constexpr int WN = C::FN * 32, NCHK = WN / 4;     // sums of a row; in 16-byte chunks
    static constexpr int AREA = C::LDS / C::NW / 16 * 16;    // bytes of a wave
    static constexpr int FIT = AREA / (WN * 4) / 32;         // 32-row blocks that fit
    static constexpr int BLOCKS = FIT < C::FM ? FIT : C::FM;  // of a pass
    static constexpr int PASSES = C::FM / BLOCKS;
    static constexpr int LPR = C::WNP / 8;                   // lanes of a row
    static constexpr int RPI = 64 / LPR;                     // rows at a time
    static constexpr int STEPS = BLOCKS * 32 / RPI;
    static constexpr int WANT = C::ES == 4 ? (C::GATED ? 1 : 2) : C::GATED ? 2 : 4;
    static constexpr int UNROLL = STEPS < WANT ? STEPS : WANT;
    static_assert(BLOCKS > 0 && PASSES * BLOCKS == C::FM && STEPS % UNROLL == 0 && (NCHK & (NCHK - 1)) == 0, "passes");
    static PGEMM_HD int at(int row, int chunk) {
        return (row * NCHK + (chunk & 1) * (NCHK / 2) + ((chunk >> 1) ^ (row & (NCHK / 2 - 1)))) * 16;
    }
};

template <class C>
__device__ __forceinline__ void mx_epilogue(const EpiArgs& e, int m0, int n0, char PGEMM_LDS* smem,
                                            f32x16 (&acc)[C::FM][C::FN], int wave, int lane, int wm0, int wn0) {
    typedef MxOut<C> O;
    typedef Epi<C::Dt, C::GATED> E;
    const int r0 = lane / O::LPR, c8 = lane % O::LPR;
    const E ep(e, m0, n0, 0, wm0 + r0, wn0 + 8 * c8);
    char PGEMM_LDS* area = smem + wave * O::AREA;
    const f32x8 b0 = ep.bias(0), b1 = C::GATED ? ep.bias(1) : b0;
    typename E::Raw next[O::UNROLL];
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
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const f32x16& a = acc[p * O::BLOCKS + i][j];
                        *(f32x4 PGEMM_LDS*)(area + O::at(32 * i + (lane & 31), 8 * j + 2 * q + (lane >> 5))) =
                            f32x4{a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]};
                    }
        }
        asm volatile("" ::: "memory");  // a wave's LDS operations stay in order
        const int down = pass * O::BLOCKS * 32;
        with_act(e.act.kind, [&](auto kind) {
            constexpr int KIND = decltype(kind)::value;
#pragma unroll 1
            for (int s = 0; s < O::STEPS; s += O::UNROLL) {
                typename E::Raw res[O::UNROLL];
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
__global__ void __launch_bounds__(C::NT, C::MINW) mx_tile(MxArgs g) {
    __shared__ __attribute__((aligned(1024))) char smem_raw[C::LDS];
    char PGEMM_LDS* smem = (char PGEMM_LDS*)smem_raw;

    const int per_split = g.tiles_m * g.tiles_n;
    const WgTiles w = wg_tiles_of(per_split * g.splits, (int)blockIdx.x, (int)gridDim.x);
    if (w.count == 0) return;
    int L = w.start + w.lb, split = 0;
    if (g.splits > 1) {
        split = __builtin_amdgcn_readfirstlane(L / per_split);
        L -= split * per_split;
    }
    int tm, tn;
    raster(L, g.tiles_m, g.tiles_n, g.group_m, tm, tn);
    tm = __builtin_amdgcn_readfirstlane(tm);
    tn = __builtin_amdgcn_readfirstlane(tn);
    const int m0 = tm * C::BM, n0 = tn * C::BNP;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm0 = (wave / C::WGN) * C::WM, wn0 = (wave % C::WGN) * C::WNP;
    const int rows_left = g.e.M - m0, cols_left = g.e.N - n0;

    f32x16 acc[C::FM][C::FN];
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
#pragma unroll
            for (int x = 0; x < 16; ++x) acc[i][j][x] = 0.0f;
    acc_settle();

    // This split's K tiles [t0, t1): whole groups of scales.
    const int total = g.filled / C::BK, groups = (total + C::G - 1) / C::G;
    const int g0 = (int)((int64_t)groups * split / g.splits), g1 = (int)((int64_t)groups * (split + 1) / g.splits);
    const int t0 = g0 * C::G, t1 = min(g1 * C::G, total);
    if (t1 > t0) {
        MxSrc<C> src;
        // With the whole contraction in one go the XCDs begin at different places of it (see linear_kernel).
        const int x = blockIdx.x & 7;
        const int begin = g.splits == 1 ? (int)((int64_t)groups * (((x & 6) + 4 * (x & 1)) & 7) >> 3) : g0;
        const int first = begin * C::G;
        src.k = first * (16 * C::KCB);
        src.k_end = total * (16 * C::KCB);
        src.s_turn = groups - begin;
        src.s_left = g1 - g0;
        src.s_groups = groups;
        const int panel = C::NP == 2 ? wave / (C::NW / 2) : 0;  // the wave's pieces of B lie in one panel
        const int b_block = wave * C::B_INSTR - panel * (C::B_BYTES / C::NP / 1024);
        src.ra = make_rsrc_sgpr((const char*)g.A + m0 * g.lda);
        src.rb = make_rsrc_sgpr((const char*)(panel ? g.B[1] : g.B[0]) + n0 * g.ldb);
#pragma unroll
        for (int q = 0; q < C::A_INSTR; ++q) {
            int row, kc;
            mx_inv<C::KCA>((wave * C::A_INSTR + q) * 1024 + lane * 16, row, kc);
            src.va[q] = row < rows_left ? (uint32_t)(row * (int)g.lda + kc * 16) : OOB;
        }
#pragma unroll
        for (int q = 0; q < C::B_INSTR; ++q) {
            int row, kc;
            mx_inv<C::KCB>((b_block + q) * 1024 + lane * 16, row, kc);
            src.vb[q] = row < cols_left ? (uint32_t)(row * (int)g.ldb + kc * 16) : OOB;
        }
        // scales: rows of the activations, then of each panel of the weights
        const int s_row = wave * C::S_INSTR * 64;
        const bool of_a = s_row < C::BM;
        const int s_panel = of_a ? 0 : (s_row - C::BM) / C::BNP, s_first = of_a ? s_row : s_row - C::BM - s_panel * C::BNP;
        const int s_rows = of_a ? min(rows_left, C::BM) : min(cols_left, C::BNP);
        const int64_t ls = of_a ? g.lsa : g.lsb;
        src.rs = make_rsrc_sgpr((of_a ? (const char*)g.SA + m0 * ls : (const char*)(s_panel ? g.SB[1] : g.SB[0]) + n0 * ls) +
                                begin * 16);
        src.s_bytes = __builtin_amdgcn_readfirstlane((s_rows - 1) * (int)ls + g.filled / 32 - begin * 16);
#pragma unroll
        for (int q = 0; q < C::S_INSTR; ++q) {
            const int row = s_first + q * 64 + lane;
            src.vs[q] = row < s_rows ? (uint32_t)(row * (int)ls) : OOB;
        }

        const uint32_t lds0 = (uint32_t)(size_t)smem;
        const uint32_t at_a = wave * C::A_INSTR * 1024, at_b = C::A_BYTES + wave * C::B_INSTR * 1024;
        const uint32_t at_s = lds0 + C::AT_S + s_row * 16;
        // Prologue: two groups of scales, slots 0 .. S-2.
        src.scales(at_s);
        src.scales(at_s + C::S_STAGE);
#pragma unroll
        for (int p = 0; p < C::S - 1; ++p) {
            mx_pieces<C, C::LPS>(src, lds0 + p * C::STAGE + at_a, lds0 + p * C::STAGE + at_b);
            src.template advance<0>();
            src.template advance<1>();
        }
        wait_barrier<C::LPS*(C::S - 2)>();
        constexpr uint32_t LASTST = (C::S - 1) * C::STAGE;
        mx_pieces<C, C::LPS / 2>(src, lds0 + LASTST + at_a, lds0 + LASTST + at_b);
        MxFrags<C> f[2];
        MxScales<C> sc[2];
        mx_first<C>(smem, smem + C::AT_S, wm0, wn0, lane, f[0], sc[0]);
        // Stages as bytes from the ring's beginning.
        uint32_t cur = 0, prev = LASTST;
        MxTileWalk<C> walk((total - first) / 2);
        const auto tile = [&](const MxScales<C>& us, MxScales<C>& next, uint32_t next_scale, uint32_t free_scales) {
            const uint32_t nxt = cur == LASTST ? 0 : cur + C::STAGE;
            MxAt at;
            at.wm0 = wm0;
            at.wn0 = wn0;
            at.lane = lane;
            at.scales = smem + next_scale;
            at.codes = smem + cur;
            at.a = lds0 + prev + at_a;
            at.b = lds0 + prev + at_b;
            MxStep<C, false>::run(acc, f[0], us, f[1], next, src, at);
            // The next K tile is in LDS (and the scales, which are older than the codes
            // that may be under way), this one's stage is free.
            wait_barrier<C::LPS*(C::S - 2)>();
            if (free_scales) src.scales(free_scales);
            at.codes = smem + nxt;
            at.a = lds0 + cur + at_a;
            at.b = lds0 + cur + at_b;
            MxStep<C, true>::run(acc, f[1], us, f[0], next, src, at);
            prev = cur;
            cur = nxt;
        };
        for (int t = t0; t < t1; t += 2) {
            tile(sc[0], sc[1], walk.scale + 4, 0);
            walk.pair();
            tile(sc[1], sc[0], walk.scale, walk.ends ? at_s + (walk.stage - C::AT_S) : 0);
        }
        __builtin_amdgcn_s_waitcnt(0);  // no load may still be writing LDS
    }
    acc_settle();

    if (g.part) {
        // fp32 sums of this split, joined by linear_join in the order of the splits
        float* base = g.part + (int64_t)split * C::NP * g.e.M * g.np8;
#pragma unroll
        for (int i = 0; i < C::FM; ++i) {
            const int row = m0 + wm0 + 32 * i + (lane & 31);
#pragma unroll
            for (int j = 0; j < C::FN; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int col = n0 + wn0 + 32 * (j % C::FNP) + 8 * q + 4 * (lane >> 5);
                    const f32x16& a = acc[i][j];
                    if (row < g.e.M && col < g.np8)
                        *(f32x4*)(base + ((int64_t)(j / C::FNP) * g.e.M + row) * g.np8 + col) =
                            f32x4{a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]};
                }
        }
        return;
    }
    mx_epilogue<C>(g.e, m0, n0, smem, acc, wave, lane, wm0, wn0);
}

// ---- few rows -----------------------------------------------------------------------------------

// One token to a few dozen: bound by the weights' bytes.  As linear_few: the waves of
// a workgroup share its outputs (16 FM rows, 16 FNP columns) and deal out the rows'
// units of 256 entries in turn; each has a ring of its own in LDS, which only it fills
// and reads, so nothing in the loop waits for another wave.  16 rows by 4096 x 16384 in 4 bits take
// 9.2 us with weights from the shared cache (36 MB: 3.9 TB/s) and 11.7 from memory, 33 by a pair of 8190 x 4001
// 13.4 and 15.4; one token by 4096 x 4096 5.6 (the launch 2.5 of it), by a pair of 8192 x 4096 8.1 and 10.5.  Three stages, since with weights from memory two take up to 1.4 times as long (one row by
// 4096 x 16384 10.8 and 15.4); a fourth gives nothing.  (Straight from memory to
// registers, neighbouring lanes hold different rows: four times the accesses to the
// cache, 14 us for 16 by 4096 x 16384 in 4 bits however much was under way.)
// The 16 x 16 x 128 instruction's lane 16 q + r takes of a unit's step (128 entries) block q of
// row r, of MX8 activations the 16-byte pieces q and 4 + q, and the scale of block q.
template <int D, int F, int FM_, int FN_, int NW_, int S_, bool GATED_>
struct MxFewCfg {
    static constexpr int Dt = D, Fmt = F, FM = FM_, FNP = FN_, NW = NW_, S = S_;
    static constexpr bool GATED = GATED_;
    // Of MX8 operands the scaled MFMAs keep 13 bits below a group's largest product: under a
    // 16-bit output's rounding, but not an fp32 one's, which takes bf16 MFMAs of the entries' values.
    static constexpr bool WIDE = F == MX8 && D == DT_F32;
    static constexpr int NP = GATED ? 2 : 1, FN = FNP * NP, NCOLP = 16 * FNP;
    static constexpr int BM = 16 * FM, NT = 64 * NW, XT = F == MX8 ? 2 : 1;  // XT: tiles of 128-byte rows of the activations
    static constexpr int A_TILE = BM * 128, B_TILE = NCOLP * 128;
    static constexpr int LPA = A_TILE / 1024, LPB = B_TILE / 1024;           // pieces
    static constexpr int SPA = (BM + 31) / 32, SPB = (NCOLP + 31) / 32;      // pieces of scales, 32 rows each
    static constexpr int AT_B = XT * A_TILE, AT_S = AT_B + NP * B_TILE;
    static constexpr int STAGE = AT_S + (SPA + NP * SPB) * 256, RING = S * STAGE, LDS = NW * RING;
    static constexpr int LPS = XT * LPA + NP * LPB + SPA + NP * SPB;
    static_assert(LDS <= 163840 && S >= 2 && LPS * (S - 2) <= 63 && FM * FN * 1024 <= RING, "ring");
};

// As dma16, of four bytes a lane.
__device__ __forceinline__ void dma4(const i32x4& rsrc, uint32_t voff, uint32_t lds_base) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds"
                 :
                 : "v"(voff), "s"(rsrc), "s"(lds_base)
                 : "memory", "m0");
}

// Eight entries' values in bf16, exactly where they are 2^-133 or more.
template <int F>
__device__ __forceinline__ bf16x8 mx_bf16(int lo, int hi, uint32_t byte) {
    const f32x8 v = mx_values<F>(i32x2{lo, hi}, byte);
    bf16x8 h;
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = (__bf16)v[i];
    return h;
}
// The same on bf16 MFMAs: of four blocks each lane takes its own one, eight entries a step.
template <class C>
__device__ __forceinline__ void mx_few_multiply_wide(f32x4 (&acc)[C::FM][C::FN], const char PGEMM_LDS* st, int lane) {
    const int r = lane & 15, q = lane >> 4;
    const auto scale = [&](int piece, int row, int ks) -> uint32_t {
        return *(const uint8_t PGEMM_LDS*)(st + C::AT_S + piece * 256 + row * 8 + ks * 4 + q);
    };
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
        bf16x8 b[C::FN][4];
#pragma unroll
        for (int j = 0; j < C::FN; ++j) {
            const int p = j / C::FNP, row = 16 * (j % C::FNP) + r;
            const i32x4 c = *(const i32x4 PGEMM_LDS*)(st + C::AT_B + p * C::B_TILE + a_off<8>(row, ks * 4 + q));
            const uint32_t byte = scale(C::SPA + p * C::SPB, row, ks);
#pragma unroll
            for (int t = 0; t < 4; ++t) b[j][t] = mx_bf16<MX4>(c[t], 0, byte);
        }
#pragma unroll
        for (int i = 0; i < C::FM; ++i) {
            const int row = 16 * i + r;
            const uint32_t byte = scale(0, row, ks);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const i32x4 c = *(const i32x4 PGEMM_LDS*)(st + ks * C::A_TILE + a_off<8>(row, 2 * q + h));
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const bf16x8 x = mx_bf16<MX8>(c[2 * t], c[2 * t + 1], byte);
#pragma unroll
                    for (int j = 0; j < C::FN; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[j][2 * h + t], x, acc[i][j], 0, 0, 0);
                }
            }
        }
    }
}

template <class C>
__device__ __forceinline__ void mx_few_multiply(f32x4 (&acc)[C::FM][C::FN], const char PGEMM_LDS* st, int lane) {
    const int r = lane & 15, q = lane >> 4;
    const auto scale = [&](int piece, int row, int ks) -> int {
        return *(const uint8_t PGEMM_LDS*)(st + C::AT_S + piece * 256 + row * 8 + ks * 4 + q);
    };
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
        i32x4 b[C::FN];
        int sb[C::FN];
#pragma unroll
        for (int j = 0; j < C::FN; ++j) {
            const int p = j / C::FNP, row = 16 * (j % C::FNP) + r;
            b[j] = *(const i32x4 PGEMM_LDS*)(st + C::AT_B + p * C::B_TILE + a_off<8>(row, ks * 4 + q));
            sb[j] = scale(C::SPA + p * C::SPB, row, ks);
        }
#pragma unroll
        for (int i = 0; i < C::FM; ++i) {
            const int row = 16 * i + r;
            i32x8 x;
            if constexpr (C::Fmt == MX8) {
                const char PGEMM_LDS* t = st + ks * C::A_TILE;
                x = two_chunks(*(const i32x4 PGEMM_LDS*)(t + a_off<8>(row, q)), *(const i32x4 PGEMM_LDS*)(t + a_off<8>(row, 4 + q)));
            } else {
                x = two_chunks(*(const i32x4 PGEMM_LDS*)(st + a_off<8>(row, ks * 4 + q)), i32x4{0, 0, 0, 0});
            }
            const int sx = scale(0, row, ks);
#pragma unroll
            for (int j = 0; j < C::FN; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    two_chunks(b[j], i32x4{0, 0, 0, 0}), x, acc[i][j], 4, C::Fmt == MX8 ? 0 : 4, 0, sb[j], 0, sx);
        }
    }
}

template <class C>
__global__ void __launch_bounds__(C::NT) mx_few(MxArgs g) {
    __shared__ __attribute__((aligned(1024))) char smem_raw[C::LDS];
    const int per_split = g.tiles_m * g.tiles_n;
    const WgTiles w = wg_tiles_of(per_split * g.splits, (int)blockIdx.x, (int)gridDim.x);
    if (w.count == 0) return;
    int L = w.start + w.lb, split = 0;
    if (g.splits > 1) {
        split = __builtin_amdgcn_readfirstlane(L / per_split);
        L -= split * per_split;
    }
    // row tiles of the same columns side by side: they share the weights in L2
    const int tn = __builtin_amdgcn_readfirstlane(L / g.tiles_m), tm = __builtin_amdgcn_readfirstlane(L - tn * g.tiles_m);
    const int m0 = tm * C::BM, n0 = tn * C::NCOLP;
    const int rows_left = g.e.M - m0, cols_left = g.e.N - n0;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    char PGEMM_LDS* ring = (char PGEMM_LDS*)smem_raw + wave * C::RING;
    const uint32_t lds0 = (uint32_t)(size_t)ring;

    // Each lane's offsets in a unit: 16 bytes of a row of codes, four of a row of scales.
    uint32_t va[C::LPA], vb[C::LPB], vsa[C::SPA], vsb[C::SPB];
#pragma unroll
    for (int p = 0; p < C::LPA; ++p) {
        int row, kc;
        a_inv<8>(p * 1024 + lane * 16, row, kc);
        va[p] = row < rows_left ? (uint32_t)(row * (int)g.lda + kc * 16) : OOB;
    }
#pragma unroll
    for (int p = 0; p < C::LPB; ++p) {
        int row, kc;
        a_inv<8>(p * 1024 + lane * 16, row, kc);
        vb[p] = row < cols_left ? (uint32_t)(row * (int)g.ldb + kc * 16) : OOB;
    }
#pragma unroll
    for (int p = 0; p < C::SPA; ++p) {
        const int row = p * 32 + (lane >> 1);
        vsa[p] = row < C::BM && row < rows_left ? (uint32_t)(row * (int)g.lsa + (lane & 1) * 4) : OOB;
    }
#pragma unroll
    for (int p = 0; p < C::SPB; ++p) {
        const int row = p * 32 + (lane >> 1);
        vsb[p] = row < C::NCOLP && row < cols_left ? (uint32_t)(row * (int)g.lsb + (lane & 1) * 4) : OOB;
    }
    f32x4 acc[C::FM][C::FN];
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    const int total = g.filled / 256;
    const int t0 = (int)((int64_t)total * split / g.splits), t1 = (int)((int64_t)total * (split + 1) / g.splits);
    // Loads unit t into stage st; past the last one every lane reads zeros.
    const auto issue = [&](int t, int st) {
        const int range = t < t1 ? (int)0x80000000u : 0;
        const uint32_t at = lds0 + (uint32_t)(st * C::STAGE);
        const auto rows = [&](const char* base, int64_t by) {
            i32x4 r = make_rsrc_sgpr(base + by * t);
            r[2] = range;
            return r;
        };
#pragma unroll
        for (int p = 0; p < C::NP; ++p) {
            const i32x4 rb = rows((const char*)g.B[p] + n0 * g.ldb, 128);
#pragma unroll
            for (int x = 0; x < C::LPB; ++x) dma16(rb, vb[x], at + C::AT_B + p * C::B_TILE + x * 1024u);
            const i32x4 rs = rows((const char*)g.SB[p] + n0 * g.lsb, 8);
#pragma unroll
            for (int x = 0; x < C::SPB; ++x) dma4(rs, vsb[x], at + C::AT_S + (C::SPA + p * C::SPB + x) * 256u);
        }
#pragma unroll
        for (int h = 0; h < C::XT; ++h) {
            const i32x4 ra = rows((const char*)g.A + m0 * g.lda + h * 128, C::XT * 128);
#pragma unroll
            for (int x = 0; x < C::LPA; ++x) dma16(ra, va[x], at + h * C::A_TILE + x * 1024u);
        }
        const i32x4 rs = rows((const char*)g.SA + m0 * g.lsa, 8);
#pragma unroll
        for (int x = 0; x < C::SPA; ++x) dma4(rs, vsa[x], at + C::AT_S + x * 256u);
    };
    int t = t0 + wave;
    if (t < t1) {
#pragma unroll
        for (int p = 0; p < C::S - 1; ++p) issue(t + p * C::NW, p);
        int st = 0;
        for (; t < t1; t += C::NW) {
            // the oldest unit has landed, and the stage before it has been read
            lgkm_drain();
            asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" : : "n"(C::LPS * (C::S - 2)) : "memory");
            issue(t + (C::S - 1) * C::NW, st == 0 ? C::S - 1 : st - 1);
            if constexpr (C::WIDE) mx_few_multiply_wide<C>(acc, ring + st * C::STAGE, lane);
            else mx_few_multiply<C>(acc, ring + st * C::STAGE, lane);
            st = st + 1 == C::S ? 0 : st + 1;
        }
    }
    __builtin_amdgcn_s_waitcnt(0);  // no load may still be writing LDS
    asm volatile("" ::: "memory");

    // The waves' sums, each in its own ring.
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; ++j) *(f32x4 PGEMM_LDS*)(ring + ((i * C::FN + j) * 64 + lane) * 16) = acc[i][j];
    lgkm_barrier();
    constexpr int GPR = C::NCOLP / 8, GROUPS = C::BM * GPR;  // groups of eight columns
    for (int x = (int)threadIdx.x; x < GROUPS; x += C::NT) {
        const int row = x / GPR, c8 = x % GPR;
        if (row >= rows_left || 8 * c8 >= cols_left) continue;
        f32x8 s[C::NP];
#pragma unroll
        for (int p = 0; p < C::NP; ++p) {
            s[p] = zero8();
            const int block = (row >> 4) * C::FN + p * C::FNP + (c8 >> 1);
            const char PGEMM_LDS* at = (const char PGEMM_LDS*)smem_raw + (block * 64 + (row & 15) + 32 * (c8 & 1)) * 16;
#pragma unroll
            for (int v = 0; v < C::NW; ++v)
                s[p] += join8(*(const f32x4 PGEMM_LDS*)(at + v * C::RING), *(const f32x4 PGEMM_LDS*)(at + v * C::RING + 256));
        }
        if (g.part) {
            float* o = g.part + ((int64_t)split * C::NP * g.e.M + m0 + row) * g.np8 + n0 + 8 * c8;
#pragma unroll
            for (int p = 0; p < C::NP; ++p) *(f32x8*)(o + (int64_t)p * g.e.M * g.np8) = s[p];
            continue;
        }
        const Epi<C::Dt, C::GATED> ep(g.e, m0, n0, 0, row, 8 * c8);
        const f32x8 b0 = ep.bias(0), b1 = C::GATED ? ep.bias(1) : b0;
        typename Epi<C::Dt, C::GATED>::Raw res[1] = {};
        if (g.e.R && ep.same()) res[0] = ep.residual(0);
        f32x8 v[1] = {s[0]}, y[1] = {s[C::NP - 1]};
        with_act(g.e.act.kind, [&](auto kind) {
            constexpr int KIND = decltype(kind)::value;
            ep.template put<KIND>(0, 0, v, y, b0, b1, res);
            if (!ep.whole(0)) {
#pragma unroll
                for (int z = 0; z < 7; ++z)
                    if (z < ep.valid(0)) ep.template put1<KIND>(0, z, s[0][z], s[C::NP - 1][z]);
            }
        });
    }
}

// ---- fp32 outputs of many rows of MX8 ----------------------------------------------------------------

// The epilogue of products that linear_kernel has formed of the entries' values in bf16
// (fp32, [plane][M][ldz]): four columns a thread.  Bound by memory.
struct MxRestArgs {
    const float* Z;
    int64_t plane, ldz;
    EpiArgs e;
};
template <bool GATED>
__global__ void __launch_bounds__(256) mx_rest(MxRestArgs g) {
    const int strips = (g.e.N + 1023) / 1024;
    for (int64_t b = blockIdx.x; b < (int64_t)strips * g.e.M; b += gridDim.x) {
        const int64_t m = b / strips;
        const int n0 = (int)(b - m * strips) * 1024 + 4 * (int)threadIdx.x;
        with_act(g.e.act.kind, [&](auto kind) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int n = n0 + i;
                if (n >= g.e.N) break;
                float z = g.Z[m * g.ldz + n];
                if (g.e.bias[0]) z += ((const float*)g.e.bias[0])[n];
                z = act1<decltype(kind)::value>(g.e.act, z);
                if constexpr (GATED) {
                    float u = g.Z[g.plane + m * g.ldz + n];
                    if (g.e.bias[1]) u += ((const float*)g.e.bias[1])[n];
                    z *= u;
                }
                if (g.e.R) z += ((const float*)g.e.R)[m * g.e.ldr + n];
                ((float*)g.e.Y[0])[m * g.e.ldy + n] = z;
            }
        });
    }
}

}  // namespace pgemm
