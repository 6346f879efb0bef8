// mx_large.hpp -- the microscaled products' kernel for large outputs: tiles of
// 256 x 256, four waves of 128 x 128, one workgroup a CU.
//
// What bounds it is power: scaled MFMAs on 4-bit operands are so cheap that moving
// the operands costs the part as much, and its clock falls to 1.4 to 1.9 GHz.  So
//   * 16 x 16 x 128 MFMAs: alone, on random data, 8370 TFLOP/s in 4 bits where
//     32 x 32 x 64 ones leave the clock lower and reach 7690 (8-bit activations: 4830
//     and 4570);
//   * codes come in whole 128-byte lines of a row (64 bytes of a row fetch the line
//     twice), scales 32 bytes of a row at a time, in a ring of their own;
//   * each code is read once from LDS by each wave that multiplies it.
//
// A period is 128 bytes of an activations' row: 256 entries in 4 bits, 128 in 8.  Its
// weights' fragments stay in registers while the wave goes through its rows in four
// blocks of 32.  A block's LDS rows are free when the block before it has been
// multiplied, the weights' when the period begins: so two periods' worth of LDS
// takes loads that are issued up to 1.75 periods before they are read, at an even pace:
//   edge X, blocks 0 and 1: load rows of block 3 of the next period, of block 0 of the
//                           one after, and half of that one's weights
//   edge Y, blocks 2 and 3: the other half, and rows of blocks 1 and 2
// Block b reads block b + 1's fragments, block 3 those of the next period's block 0 and
// its weights, each behind the last MFMA that needs what was in its registers.  (In 8
// bits the weights' 128 bytes of a row last two periods, a quarter at a time.)
#pragma once

#include "mx_kernel.hpp"

namespace pgemm {

template <int D, int F, bool GATED_>
struct MxLargeCfg {
    static constexpr int Dt = D, Fmt = F, BM = 256, BN = 256, WGM = 2, WGN = 2;
    static constexpr bool GATED = GATED_;
    static constexpr int ES = D == DT_F32 ? 4 : 2;
    static constexpr int NP = GATED ? 2 : 1, BNP = BN / NP, NW = 4, NT = 256;
    static constexpr int BK = F == MX8 ? 128 : 256;       // entries of a period
    static constexpr int KS = F == MX8 ? 1 : 2;           // MFMA steps of it
    static constexpr int TURNS = F == MX8 ? 2 : 1;        // periods that a unit of the weights lasts
    static constexpr int WM = 128, WNP = BNP / WGN, FM = 8, FNP = WNP / 16, FN = FNP * NP;
    static constexpr int UNIT = 256 * 128;                // bytes of a unit: 128 bytes of each row
    static constexpr int AT_B = 2 * UNIT, AT_S = 4 * UNIT;
    static constexpr int SB = 32, G = SB * 32 / BK;       // bytes of a row in a group of scales; its periods
    static constexpr int S_STAGE = 512 * SB, TOTAL = AT_S + 2 * S_STAGE;
    static constexpr int LDS = AT_S;                      // what the epilogue uses
    static constexpr int PB = 8 / TURNS;                  // the wave's pieces of the weights a period
    static constexpr int PIECES = 8 + PB;                 // of codes a period
    static constexpr int WAIT_X = PIECES, WAIT_Y = PIECES / 2 + 4;
    static_assert(TOTAL == 163840 && FN == 8, "all of a CU's LDS");
};

// Codes of a unit: chunk kc of a row.  MX4 fragments read chunks 2 q + ks (lanes that
// are served together differ by two chunks), MX8 ones q and 4 + q.
template <int F>
PGEMM_HD constexpr int mx_swz16(int line) { return F == MX8 ? (line & 7) << 1 : (line & 1) | (line & 6) << 1; }
template <int F>
PGEMM_HD constexpr int mx_off16(int row, int kc) {
    return (row >> 1 << 8) + ((((row & 1) * 8 + kc) ^ mx_swz16<F>(row >> 1)) << 4);
}
template <int F>
PGEMM_HD void mx_inv16(int off, int& row, int& kc) {
    const int line = off >> 8, u = ((off >> 4) & 15) ^ mx_swz16<F>(line);
    row = 2 * line + (u >> 3);
    kc = u & 7;
}

template <class C>
struct MxLargeState {
    i32x4 a[2][2][2];   // [buffer][row block][MX4: step, MX8: piece]
    int sa[2][2];
    i32x4 b[C::FN][C::KS];
    int sb[C::FN];
};

template <class C, int KSTEP>
__device__ __forceinline__ void mx_mfma16(f32x4& acc, const i32x4 (&x)[2], const i32x4& w, int sx, int sw) {
    if constexpr (C::Fmt == MX8) {
        const i32x8 xx = two_chunks(x[0], x[1]);
        asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[0,0,0] op_sel_hi:[0,0,0] cbsz:4"
                     : "+a"(acc)
                     : "v"(w), "v"(xx), "v"(sw), "v"(sx));
    } else {
        asm volatile(
            "v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[%5,%5,0] op_sel_hi:[0,0,0] cbsz:4 blgp:4"
            : "+a"(acc)
            : "v"(w), "v"(x[KSTEP]), "v"(sw), "v"(sx), "n"(KSTEP));
    }
}

// What a period's loads and reads go by.
struct MxLargeAt {
    const char PGEMM_LDS* a;        // units of the period's rows, and of the next period's
    const char PGEMM_LDS* a_next;
    const char PGEMM_LDS* b_next;   // the next period's weights
    const char PGEMM_LDS* s;        // scales of the period and of the next one, at their places in the group
    const char PGEMM_LDS* s_next;
    uint32_t la1, la2, lb;          // LDS places of the wave's pieces: next period's rows, the one after, and its weights
    uint32_t k1, k2, kb;            // bytes in the rows
};

template <class C>
struct MxLarge {
    i32x4 ra, rb;
    uint32_t va[8], vb[8];
    int lane, wm0, wn0;
    MxLargeState<C> f;

    // Fragment reads.  Lane 16 q + r: row r.
    template <int BUF, int I>
    __device__ __forceinline__ void read_a(const char PGEMM_LDS* unit, int block) {  // I: row block * 2 + step or piece
        const int r = lane & 15, q = lane >> 4, row = wm0 + 32 * block + 16 * (I / 2) + r;
        f.a[BUF][I / 2][I % 2] = *(const i32x4 PGEMM_LDS*)(unit + mx_off16<C::Fmt>(row, C::Fmt == MX8 ? 4 * (I % 2) + q : 2 * q + I % 2));
    }
    __device__ __forceinline__ int scale(const char PGEMM_LDS* s, int row) const {
        const int q = lane >> 4;
        if constexpr (C::Fmt == MX8) return *(const uint8_t PGEMM_LDS*)(s + row * C::SB + q);
        else return *(const unsigned short PGEMM_LDS*)(s + row * C::SB + 2 * q);
    }
    template <int BUF, int I>
    __device__ __forceinline__ void read_sa(const char PGEMM_LDS* s, int block) {
        f.sa[BUF][I] = scale(s, wm0 + 32 * block + 16 * I + (lane & 15));
    }
    template <int J>
    __device__ __forceinline__ int row_b() const { return J / C::FNP * C::BNP + wn0 + 16 * (J % C::FNP) + (lane & 15); }
    // TURN: which half of the unit's line (MX8)
    template <int J, int KSTEP, int TURN>
    __device__ __forceinline__ void read_b(const char PGEMM_LDS* unit) {
        const int q = lane >> 4;
        f.b[J][KSTEP] = *(const i32x4 PGEMM_LDS*)(unit + mx_off16<C::Fmt>(row_b<J>(), C::Fmt == MX8 ? 4 * TURN + q : 2 * q + KSTEP));
    }
    template <int J>
    __device__ __forceinline__ void read_sb(const char PGEMM_LDS* s) { f.sb[J] = scale(s, 256 + row_b<J>()); }

    // Pieces: of rows, X of the 2 of a block; of the weights.  M0 first, the load an instruction later.
    template <int BLOCK, int X>
    __device__ __forceinline__ void place_a(uint32_t at) const {
        asm volatile("s_add_u32 m0, %0, %1" : : "s"(at), "n"(BLOCK * 4096 + X * 1024) : "m0", "scc");
    }
    template <int BLOCK, int X>
    __device__ __forceinline__ void load_a(uint32_t k) const {
        asm volatile("buffer_load_dwordx4 %0, %1, %2 offen lds" : : "v"(va[2 * BLOCK + X]), "s"(ra), "s"(k) : "memory");
    }
    template <int Q>
    __device__ __forceinline__ void place_b(uint32_t at) const {
        asm volatile("s_add_u32 m0, %0, %1" : : "s"(at), "n"(Q * 1024) : "m0", "scc");
    }
    template <int Q>
    __device__ __forceinline__ void load_b(uint32_t k) const {
        asm volatile("buffer_load_dwordx4 %0, %1, %2 offen lds" : : "v"(vb[Q]), "s"(rb), "s"(k) : "memory");
    }

    // Piece P of the PIECES of a period, in their order (TURN: the period's place among those of a unit of weights).
    //   0, 1 rows of block 3 (next period)   2, 3 of block 0 (the one after)   weights, first half
    //   weights, second half                 rows of blocks 1 and 2 (the one after)
    template <int P, int TURN, bool PLACE>
    __device__ __forceinline__ void piece(const MxLargeAt& at) const {
        constexpr int B0 = C::TURNS == 2 && TURN == 0 ? 4 : 0;
        if constexpr (P < 2) {
            if constexpr (PLACE) place_a<3, P>(at.la1);
            else load_a<3, P>(at.k1);
        } else if constexpr (P < 4) {
            if constexpr (PLACE) place_a<0, P - 2>(at.la2);
            else load_a<0, P - 2>(at.k2);
        } else if constexpr (P < 4 + C::PB) {
            if constexpr (PLACE) place_b<B0 + P - 4>(at.lb);
            else load_b<B0 + P - 4>(at.kb);
        } else {
            constexpr int X = P - 4 - C::PB;
            if constexpr (PLACE) place_a<1 + X / 2, X % 2>(at.la2);
            else load_a<1 + X / 2, X % 2>(at.k2);
        }
    }
    template <int FIRST, int END, int TURN>
    __device__ __forceinline__ void pieces(const MxLargeAt& at) const {
        if constexpr (FIRST < END) {
            piece<FIRST, TURN, true>(at);
            asm volatile("s_nop 0");
            piece<FIRST, TURN, false>(at);
            pieces<FIRST + 1, END, TURN>(at);
        }
    }

    // All of a unit of weights; rows of the blocks from FIRST on.
    template <int Q>
    __device__ __forceinline__ void all_b(uint32_t at, uint32_t k) const {
        if constexpr (Q < 8) {
            place_b<Q>(at);
            asm volatile("s_nop 0");
            load_b<Q>(k);
            all_b<Q + 1>(at, k);
        }
    }
    template <int FIRST, int END, int X = 0>
    __device__ __forceinline__ void rows_a(uint32_t at, uint32_t k) const {
        if constexpr (FIRST < END) {
            place_a<FIRST, X>(at);
            asm volatile("s_nop 0");
            load_a<FIRST, X>(k);
            rows_a<FIRST + X, END, (X + 1) % 2>(at, k);
        }
    }

    // What stands between the MFMAs of block BLOCK: E, evenly, the next block's rows in
    // turns with the block's pieces; in block 3, behind each pair of MFMAs, the next
    // period's weights into the registers that have become free.
    template <int BLOCK, int TURN>
    struct Block {
        static constexpr int NM = 2 * C::KS * C::FN, NPC = C::PIECES / 4, P0 = BLOCK * NPC;
        static constexpr int READS = 6, E = READS + 2 * NPC, BUF = BLOCK & 1, NXT = BUF ^ 1;
        template <int I>
        static __device__ __forceinline__ void read(MxLarge& m, const MxLargeAt& at) {
            const char PGEMM_LDS* unit = BLOCK == 3 ? at.a_next : at.a;
            if constexpr (I < 4) m.template read_a<NXT, I>(unit, (BLOCK + 1) & 3);
            else m.template read_sa<NXT, I - 4>(BLOCK == 3 ? at.s_next : at.s, (BLOCK + 1) & 3);
        }
        // scales first: the next block's first MFMA waits for them
        template <int J>
        static __device__ __forceinline__ void item(MxLarge& m, const MxLargeAt& at) {
            if constexpr (J < 2 * READS && J < 4 * NPC) {
                if constexpr (J % 2 == 0) read<(J / 2 + 4) % READS>(m, at);
                else m.template piece<P0 + J / 4, TURN, (J / 2) % 2 == 0>(at);
            } else {
                constexpr int X = J - READS;  // no reads left: pieces alone, an MFMA between M0 and the load
                if constexpr (J < E) m.template piece<P0 + X / 2, TURN, X % 2 == 0>(at);
            }
        }
        template <int J, int END>
        static __device__ __forceinline__ void items(MxLarge& m, const MxLargeAt& at) {
            if constexpr (J < END) {
                item<J>(m, at);
                items<J + 1, END>(m, at);
            }
        }
        template <int M = 0>
        static __device__ __forceinline__ void run(MxLarge& m, f32x4 (&acc)[C::FM][C::FN], const MxLargeAt& at) {
            if constexpr (M < NM) {
                constexpr int T = M / 2, I = M % 2, KSTEP = T / C::FN, J = T % C::FN;
                mx_mfma16<C, KSTEP>(acc[2 * BLOCK + I][J], m.f.a[BUF][I], m.f.b[J][KSTEP], m.f.sa[BUF][I], m.f.sb[J]);
                if constexpr (BLOCK == 3) {
                    if constexpr (I == 1) {
                        m.template read_b<J, KSTEP, (TURN + 1) % C::TURNS>(at.b_next);
                        if constexpr (KSTEP == C::KS - 1) m.template read_sb<J>(at.s_next);
                    } else {
                        items<T * E / (NM / 2), (T + 1) * E / (NM / 2)>(m, at);
                    }
                } else {
                    items<M * E / NM, (M + 1) * E / NM>(m, at);
                }
                __builtin_amdgcn_sched_barrier(0);
                run<M + 1>(m, acc, at);
            }
        }
    };
    template <int J = 0>
    __device__ __forceinline__ void first_b(const char PGEMM_LDS* unit, const char PGEMM_LDS* s) {
        if constexpr (J < C::FN) {
            read_b<J, 0, 0>(unit);
            if constexpr (C::KS == 2) read_b<J, C::KS - 1, 0>(unit);
            read_sb<J>(s);
            first_b<J + 1>(unit, s);
        }
    }
};

template <class C>
__global__ void __launch_bounds__(C::NT, 1) mx_large(MxArgs g) {
    __shared__ __attribute__((aligned(1024))) char smem_raw[C::TOTAL];
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

    f32x4 acc[C::FM][C::FN];
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    acc_settle();

    // This split's periods: whole groups of scales.
    const int total = g.filled / C::BK, groups = (total + C::G - 1) / C::G;
    const int g0 = (int)((int64_t)groups * split / g.splits), g1 = (int)((int64_t)groups * (split + 1) / g.splits);
    const int t0 = g0 * C::G, t1 = min(g1 * C::G, total);
    if (t1 > t0) {
        MxLarge<C> m;
        m.lane = lane;
        m.wm0 = wm0;
        m.wn0 = wn0;
        // With the whole contraction in one go the XCDs begin at different places of it (see linear_kernel).
        const int x = blockIdx.x & 7;
        const int begin = g.splits == 1 ? (int)((int64_t)groups * (((x & 6) + 4 * (x & 1)) & 7) >> 3) : g0;
        const int first = begin * C::G;
        const int panel = C::NP == 2 ? wave / 2 : 0;
        m.ra = make_rsrc_sgpr((const char*)g.A + m0 * g.lda);
        m.rb = make_rsrc_sgpr((const char*)(panel ? g.B[1] : g.B[0]) + n0 * g.ldb);
        // Rows: of block b the sixteen from a_row + 32 b on; weights: 64 rows from 64 * wave on.
        const int a_row = (wave >> 1) * 128 + (wave & 1) * 16;
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            int row, kc;
            mx_inv16<C::Fmt>((a_row + 32 * (p / 2) + 8 * (p % 2)) * 128 + lane * 16, row, kc);
            m.va[p] = row < rows_left ? (uint32_t)(row * (int)g.lda + kc * 16) : OOB;
            mx_inv16<C::Fmt>((64 * wave + 8 * p) * 128 + lane * 16, row, kc);
            row -= panel * C::BNP;
            m.vb[p] = row < cols_left ? (uint32_t)(row * (int)g.ldb + kc * 16) : OOB;
        }
        // Scales: 128 rows a wave, of the activations or of a panel of the weights, two lanes a row.
        const int s_row = wave * 128;
        const bool of_a = s_row < 256;
        const int s_panel = of_a ? 0 : (s_row - 256) / C::BNP, s_first = of_a ? s_row : s_row - 256 - s_panel * C::BNP;
        const int s_rows = of_a ? min(rows_left, 256) : min(cols_left, C::BNP);
        const int64_t ls = of_a ? g.lsa : g.lsb;
        uint32_t vs[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int row = s_first + 32 * q + (lane >> 1);
            vs[q] = row < s_rows ? (uint32_t)(row * (int)ls + (lane & 1) * 16) : OOB;
        }
        const char* s_base = (of_a ? (const char*)g.SA + m0 * ls : (const char*)(s_panel ? g.SB[1] : g.SB[0]) + n0 * ls);
        const int s_end = (s_rows - 1) * (int)ls + g.filled / 32;  // bytes from there to the end of the last row
        int s_group = begin, s_left = g1 - g0;
        const uint32_t lds0 = (uint32_t)(size_t)smem;
        // The next group of scales, to LDS.  The last one of a row may be cut: what lies
        // behind it is the next row's, or beyond the range, and not read.
        const auto scales = [&](uint32_t stage) {
            i32x4 r = make_rsrc_sgpr(s_base + s_group * C::SB);
            r[2] = __builtin_amdgcn_readfirstlane(s_left > 0 ? s_end - s_group * C::SB : 0);
#pragma unroll
            for (int q = 0; q < 4; ++q) dma16(r, vs[q], lds0 + C::AT_S + stage + wave * 4096 + q * 1024u);
            --s_left;
            if (++s_group == groups) s_group = 0;
        };
        // Bytes in the rows of the next periods' codes: of one, two periods on.
        const uint32_t a_end = total * 128u;
        const auto round = [&](uint32_t k) { return k >= a_end ? k - a_end : k; };
        const uint32_t at_a = lds0 + a_row * 128, at_b = lds0 + C::AT_B + wave * 8192;
        const uint32_t b_end = total * (128u / C::TURNS);
        uint32_t ka = first * 128u, kw = first * (128u / C::TURNS);  // this period's, this unit of weights'
        const auto round_b = [&](uint32_t k) { return k >= b_end ? k - b_end : k; };

        // Prologue: two groups of scales; the first period, and what the two before it would have loaded.
        scales(0);
        scales(C::S_STAGE);
        const uint32_t k_1 = round(ka + 128), kw_1 = round_b(kw + 128);
        {
            MxLargeAt at;
            m.template all_b<0>(at_b, kw);
            m.template rows_a<0, 3>(at_a, ka);
            at.la1 = at_a;
            at.k1 = ka;
            at.la2 = at_a + C::UNIT;
            at.k2 = k_1;
            at.lb = at_b + C::UNIT;
            at.kb = kw_1;
            m.template pieces<0, C::PIECES, C::TURNS - 1>(at);
        }
        wait_barrier<C::WAIT_X>();
        m.template read_a<0, 0>(smem, 0);
        m.template read_a<0, 1>(smem, 0);
        m.template read_a<0, 2>(smem, 0);
        m.template read_a<0, 3>(smem, 0);
        m.template read_sa<0, 0>(smem + C::AT_S, 0);
        m.template read_sa<0, 1>(smem + C::AT_S, 0);
        m.first_b(smem + C::AT_B, smem + C::AT_S);

        uint32_t ua = 0, ub = 0;     // unit of the period's rows, of its weights
        uint32_t s_at = C::AT_S;     // its scales
        int place = 0, row_left = total - first, n = t1 - t0;
        uint32_t free_scales = ~0u;  // a stage of scales that is free from this period on
        const auto period = [&](auto turn) {
            constexpr int TURN = decltype(turn)::value;
            // TURN 1 of a unit of weights loads the first half of the unit two on, its own place; TURN 0 the second of the next.
            MxLargeAt at;
            const uint32_t s_stage = (s_at - C::AT_S) / C::S_STAGE * C::S_STAGE;
            --row_left;
            const bool ends = ++place == C::G || row_left == 0;
            const uint32_t s_next = ends ? C::AT_S + C::S_STAGE - s_stage : s_at + C::BK / 32;
            at.a = smem + ua;
            at.a_next = smem + (C::UNIT - ua);
            at.s = smem + s_at;
            at.s_next = smem + s_next;
            at.la1 = at_a + C::UNIT - ua;
            at.la2 = at_a + ua;
            at.k1 = round(ka + 128);
            at.k2 = round(at.k1 + 128);
            if constexpr (C::TURNS == 1) {
                at.b_next = smem + C::AT_B + C::UNIT - ub;
                at.lb = at_b + ub;
                at.kb = round_b(round_b(kw + 128) + 128);
            } else if constexpr (TURN == 0) {
                at.b_next = smem + C::AT_B + ub;
                at.lb = at_b + C::UNIT - ub;
                at.kb = round_b(kw + 128);
            } else {
                at.b_next = smem + C::AT_B + C::UNIT - ub;
                at.lb = at_b + ub;
                at.kb = round_b(round_b(kw + 128) + 128);
            }
            wait_barrier<C::WAIT_X>();
            if (free_scales != ~0u) scales(free_scales);
            MxLarge<C>::template Block<0, TURN>::run(m, acc, at);
            MxLarge<C>::template Block<1, TURN>::run(m, acc, at);
            wait_barrier<C::WAIT_Y>();
            MxLarge<C>::template Block<2, TURN>::run(m, acc, at);
            MxLarge<C>::template Block<3, TURN>::run(m, acc, at);
            free_scales = ends ? s_stage : ~0u;
            if (ends) place = 0;
            s_at = s_next;
            ua = C::UNIT - ua;
            ka = at.k1;
            if constexpr (TURN == C::TURNS - 1) {
                ub = C::UNIT - ub;
                kw = round_b(kw + 128);
            }
        };
        for (int t = 0; t < n; t += C::TURNS) {
            period(KindC<0>{});
            if constexpr (C::TURNS == 2) period(KindC<1>{});
        }
        __builtin_amdgcn_s_waitcnt(0);  // no load may still be writing LDS
    }
    acc_settle();

    const int li = lane & 15, lg4 = 4 * (lane >> 4);
    if (g.part) {
        // fp32 sums of this split, joined by linear_join in the order of the splits
        float* base = g.part + (int64_t)split * C::NP * g.e.M * g.np8;
#pragma unroll
        for (int i = 0; i < C::FM; ++i) {
            const int row = m0 + wm0 + 16 * i + li;
#pragma unroll
            for (int j = 0; j < C::FN; ++j) {
                const int col = n0 + wn0 + 16 * (j % C::FNP) + lg4;
                if (row < g.e.M && col < g.np8)
                    *(f32x4*)(base + ((int64_t)(j / C::FNP) * g.e.M + row) * g.np8 + col) = acc[i][j];
            }
        }
        return;
    }
    lin_epilogue<C>(g.e, m0, n0, 0, smem, acc, wave, lane, wm0, wn0);
}

}  // namespace pgemm
