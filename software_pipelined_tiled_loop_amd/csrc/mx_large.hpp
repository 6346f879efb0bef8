// mx_large.hpp -- the microscaled products' kernel for large outputs: tiles of
// 256 x 256, four waves of 128 x 128, one workgroup a CU.
//
// Scaled MFMAs on 4-bit operands are so cheap that feeding them costs as much, in clocks and
// in power.  A tile of 4096 entries takes 69400 clocks in 4 bits, 58200 of them in the K loop,
// where its MFMAs alone take 36400 (8-bit activations: 101500, 90300 and 67100); and on random data the clock
// is 1.9 to 2.2 GHz (by the card) where zeros, in as many clocks, run at 2.39.  So
//   * 16 x 16 x 128 MFMAs: alone, on random data, 8290 TFLOP/s in 4 bits at 2.27 GHz where
//     32 x 32 x 64 ones lower the clock to 1.91 and reach 7490 (8-bit activations:
//     4860 and 4490);
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
//
// Loads arrive in the order in which they were issued, so an edge's vmcnt says which of
// them it leaves under way: X the pieces of the period before it (WAIT_X), Y this period's and the
// last four of the one before (WAIT_Y).  A group of scales is loaded behind edge X of the first period
// of the group before it and read from block 3 of that group's last period on.  Edge X of
// any later period covers it; where that group is a single period, which in 4 bits
// a row's last one may be, edge Y of the same period has to (MxLargeWalk::wait_y).
//
// A call of 4096^3 in 4 bits takes 41 to 42 us (3350 TFLOP/s), 44 with operands that come from memory, of
// 8192^3 238 (4620) and 247; with MX8 activations 51 and 55, 350 (3140) and 360.  Of a tile's
// clocks 11000 are its epilogue.
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
    static constexpr int PB = 8 / TURNS;                  // the wave's pieces of the weights a period
    static constexpr int PIECES = 8 + PB;                 // of codes a period
    // Loads that the edges leave under way: see above.  Y_SCALES covers scales issued behind the edge X before it.
    static constexpr int WAIT_X = PIECES, WAIT_Y = PIECES / 2 + 4, WAIT_Y_SCALES = PIECES / 2;
    static constexpr bool SINGLE = BK == kMxGroup;        // a row's last group of scales may be a single period
    static_assert(TOTAL == 163840 && FN == 8, "all of a CU's LDS");
    static_assert(WAIT_X <= PIECES && WAIT_Y_SCALES <= PIECES / 2, "scales are covered by the edge before their first read");
};

// Where the scales of the periods lie, and when a group of them is loaded: a wave's way
// along its periods, a row's last group perhaps cut.
template <class C>
struct MxLargeWalk {
    uint32_t stage = C::AT_S, place = 0;    // of this period's scales: in LDS, and in their group, in bytes of a row
    uint32_t next_stage = 0, next_place = 0;
    uint32_t free = ~0u;                    // a stage that is free from this period on: the next group is loaded into it
    int row_left;                           // periods to the row's end
    bool ends = false;                      // the period is its group's last one
    PGEMM_HD explicit MxLargeWalk(int left) : row_left(left) {}
    PGEMM_HD void enter() {
        ends = --row_left == 0 || place + C::BK / 32 == C::SB;
        next_stage = ends ? 2 * C::AT_S + C::S_STAGE - stage : stage;
        next_place = ends ? 0 : place + C::BK / 32;
    }
    PGEMM_HD bool loads() const { return free != ~0u; }
    // Block 3 reads the scales that were loaded behind this period's own edge X.
    PGEMM_HD bool reads_at_once() const { return C::SINGLE && ends && loads(); }
    PGEMM_HD int wait_y() const { return reads_at_once() ? C::WAIT_Y_SCALES : C::WAIT_Y; }
    PGEMM_HD void leave() {
        free = ends ? stage - C::AT_S : ~0u;
        stage = next_stage;
        place = next_place;
    }
};

// Of two blocks' 32 weights' rows the even block's are 0 .. 3, 8 .. 11, 16 .., the odd one's four further on: a lane's
// results, four rows of a block, then join to eight columns of the output.
PGEMM_HD constexpr int mx_row_b(int r) { return 8 * (r >> 2) + (r & 3); }

// Codes of a unit: chunk kc of a row.  The LDS serves sixteen lanes at a time, eight rows of one parity at two of the
// chunks: MX4 fragments read chunks 2 q + ks, MX8 ones q and 4 + q.  The eight rows' 256-byte lines, four
// bits of them for the weights' rows as they are dealt, are told apart by three bits.
template <int F, bool B>
PGEMM_HD constexpr int mx_swz16(int line) {
    const int l = B ? (line & 1) | (line >> 2 & 3) << 1 : line & 7;
    return F == MX8 ? l << 1 : (l & 1) | (l & 6) << 1;
}
template <int F, bool B>
PGEMM_HD constexpr int mx_off16(int row, int kc) {
    return (row >> 1 << 8) + ((((row & 1) * 8 + kc) ^ mx_swz16<F, B>(row >> 1)) << 4);
}
template <int F, bool B>
PGEMM_HD void mx_inv16(int off, int& row, int& kc) {
    const int line = off >> 8, u = ((off >> 4) & 15) ^ mx_swz16<F, B>(line);
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
    uint32_t a[2], a_next[2];       // LDS: each lane's first row of the period's unit, and of the next period's (by step or piece)
    uint32_t b_next[2];             // of the next period's weights
    uint32_t sa, sa_next, sb_next;  // of their scales
    uint32_t la1, la2, lb;          // LDS places of the wave's pieces: next period's rows, the one after, and its weights
    uint32_t k1, k2, kb;            // bytes in the rows
};

template <class T>
__device__ __forceinline__ T mx_lds(uint32_t at) { return *(const T PGEMM_LDS*)at; }

template <class C>
struct MxLarge {
    i32x4 ra, rb;                   // rows from kBack bytes before them on (see piece)
    uint32_t va[8], vb[8];
    MxLargeState<C> f;
    static constexpr uint32_t kBack = 4096;

    // Fragment reads: row block I / 2 of a block, step or piece I % 2.
    template <int BUF, int I>
    __device__ __forceinline__ void read_a(const uint32_t (&unit)[2], int block) {
        f.a[BUF][I / 2][I % 2] = mx_lds<i32x4>(unit[I % 2] + (32 * block + 16 * (I / 2)) * 128);
    }
    static __device__ __forceinline__ int scale(uint32_t at) {
        if constexpr (C::Fmt == MX8) return mx_lds<uint8_t>(at);
        else return mx_lds<unsigned short>(at);
    }
    template <int BUF, int I>
    __device__ __forceinline__ void read_sa(uint32_t at, int block) { f.sa[BUF][I] = scale(at + (32 * block + 16 * I) * C::SB); }
    // Row of the weights' block J that lane 0 of a half row reads; lane r is mx_row_b(r) rows on.
    template <int J>
    static constexpr int row_b = J / C::FNP * C::BNP + 32 * (J % C::FNP / 2) + 4 * (J % 2);
    // WHICH: the step, or the half of the unit's line (MX8)
    template <int J, int KSTEP, int WHICH>
    __device__ __forceinline__ void read_b(const uint32_t (&unit)[2]) { f.b[J][KSTEP] = mx_lds<i32x4>(unit[WHICH] + row_b<J> * 128); }
    template <int J>
    __device__ __forceinline__ void read_sb(uint32_t at) { f.sb[J] = scale(at + row_b<J> * C::SB); }

    // Pieces of 1 KiB: LDS at M0 plus the instruction's offset, which the memory's address takes too (so va and vb
    // are that much less, and the rows' address kBack bytes, which they have more).
    // M0 is set for all pieces in a row of 4 KiB, an instruction before the first load.
    template <int OFF>
    static __device__ __forceinline__ void load(uint32_t v, const i32x4& r, uint32_t k) {
        asm volatile("buffer_load_dwordx4 %0, %1, %2 offen offset:%3 lds" : : "v"(v), "s"(r), "s"(k), "n"(OFF) : "memory");
    }
    template <int ADD>
    static __device__ __forceinline__ void place(uint32_t at) {
        asm volatile("s_add_u32 m0, %0, %1" : : "s"(at), "n"(ADD) : "m0", "scc");
    }
    static constexpr int H = C::PB / 2;  // pieces of weights in a row
    // Piece P of the PIECES of a period, in their order (TURN: the period's place among those of a unit of weights).
    //   0, 1 rows of block 3 (next period)   2, 3 of block 0 (the one after)   weights, first half
    //   weights, second half                 rows of blocks 1 and 2 (the one after)
    static constexpr bool placed(int p) { return p < 4 || p >= 4 + C::PB ? p % 2 == 0 : (p - 4) % H == 0; }
    static constexpr int block_of(int p) { return p < 2 ? 3 : p < 4 ? 0 : p < 4 + C::PB ? -1 : 1 + (p - 4 - C::PB) / 2; }
    static constexpr int weights_of(int p, int turn) { return (C::TURNS == 2 && turn == 0 ? 4 : 0) + p - 4; }
    template <int P, int TURN, bool PLACE>
    __device__ __forceinline__ void piece(const MxLargeAt& at) const {
        if constexpr (block_of(P) >= 0) {
            constexpr int BLOCK = block_of(P), X = P % 2;
            if constexpr (PLACE) place<BLOCK * 4096>(P < 2 ? at.la1 : at.la2);
            else load<X * 1024>(va[2 * BLOCK + X], ra, P < 2 ? at.k1 : at.k2);
        } else {
            constexpr int Q = weights_of(P, TURN);
            if constexpr (PLACE) place<Q * 1024>(at.lb);
            else load<Q % H * 1024>(vb[Q], rb, at.kb);
        }
    }
    // Steps of pieces FIRST to END - 1: each group's M0, then its loads.
    static constexpr int steps(int first, int end) {
        int n = 0;
        for (int p = first; p < end; ++p) n += placed(p) ? 2 : 1;
        return n;
    }
    // The piece of step S, twice, plus one where the step sets M0.
    static constexpr int step_of(int first, int s) {
        int p = first;
        while (true) {
            if (placed(p)) {
                if (s == 0) return 2 * p + 1;
                --s;
            }
            if (s == 0) return 2 * p;
            --s;
            ++p;
        }
    }
    template <int FIRST, int END, int TURN>
    __device__ __forceinline__ void pieces(const MxLargeAt& at) const {
        if constexpr (FIRST < END) {
            if constexpr (placed(FIRST)) {
                piece<FIRST, TURN, true>(at);
                asm volatile("s_nop 0");
            }
            piece<FIRST, TURN, false>(at);
            pieces<FIRST + 1, END, TURN>(at);
        }
    }
    // In the prologue: all of a unit of weights; rows of the blocks from FIRST on.
    template <int Q>
    __device__ __forceinline__ void all_b(uint32_t at, uint32_t k) const {
        if constexpr (Q < 8) {
            if constexpr (Q % H == 0) {
                place<Q * 1024>(at);
                asm volatile("s_nop 0");
            }
            load<Q % H * 1024>(vb[Q], rb, k);
            all_b<Q + 1>(at, k);
        }
    }
    template <int FIRST, int END>
    __device__ __forceinline__ void rows_a(uint32_t at, uint32_t k) const {
        if constexpr (FIRST < END) {
            place<FIRST * 4096>(at);
            asm volatile("s_nop 0");
            load<0>(va[2 * FIRST], ra, k);
            load<1024>(va[2 * FIRST + 1], ra, k);
            rows_a<FIRST + 1, END>(at, k);
        }
    }

    // What stands between the MFMAs of block BLOCK: E, evenly, the next block's rows in
    // turns with the block's pieces; in block 3, behind each pair of MFMAs, the next
    // period's weights into the registers that have become free.
    template <int BLOCK, int TURN>
    struct Block {
        static constexpr int NM = 2 * C::KS * C::FN, P0 = BLOCK * (C::PIECES / 4);
        static constexpr int READS = 6, STEPS = steps(P0, P0 + C::PIECES / 4), E = READS + STEPS;
        static constexpr int PAIRS = READS < STEPS ? READS : STEPS, BUF = BLOCK & 1, NXT = BUF ^ 1;
        template <int I>
        static __device__ __forceinline__ void read(MxLarge& m, const MxLargeAt& at) {
            constexpr int R = (I + 4) % READS;  // scales first: the next block's first MFMA waits for them
            if constexpr (R < 4) m.template read_a<NXT, R>(BLOCK == 3 ? at.a_next : at.a, (BLOCK + 1) & 3);
            else m.template read_sa<NXT, R - 4>(BLOCK == 3 ? at.sa_next : at.sa, (BLOCK + 1) & 3);
        }
        template <int S>
        static __device__ __forceinline__ void step(const MxLarge& m, const MxLargeAt& at) {
            constexpr int X = step_of(P0, S);
            m.template piece<X / 2, TURN, X % 2 != 0>(at);
        }
        // (the steps alone, where there are more of them than reads, stand behind different MFMAs)
        template <int J>
        static __device__ __forceinline__ void item(MxLarge& m, const MxLargeAt& at) {
            if constexpr (J < 2 * PAIRS) {
                if constexpr (J % 2 == 0) read<J / 2>(m, at);
                else step<J / 2>(m, at);
            } else if constexpr (READS > PAIRS) {
                read<J - PAIRS>(m, at);
            } else {
                step<J - PAIRS>(m, at);
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
                        m.template read_b<J, KSTEP, C::TURNS == 2 ? 1 - TURN : KSTEP>(at.b_next);
                        if constexpr (KSTEP == C::KS - 1) m.template read_sb<J>(at.sb_next);
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
    __device__ __forceinline__ void first_b(const uint32_t (&unit)[2], uint32_t scales) {
        if constexpr (J < C::FN) {
            read_b<J, 0, 0>(unit);
            if constexpr (C::KS == 2) read_b<J, C::KS - 1, 1>(unit);
            read_sb<J>(scales);
            first_b<J + 1>(unit, scales);
        }
    }
};

// The epilogue.  The weights' rows are dealt to the blocks' rows such that a lane has of
// each pair of blocks eight columns side by side (mx_row_b), 16 bytes of the output.  One
// wave a SIMD has nothing to hide its instructions behind, so they are few: the output's
// range ends with its last row, which drops the stores beyond, and a lane's offsets move
// by rows alone.  (With Epi::put, a general one, it took 6 us a tile besides the stores;
// through LDS, as lin_epilogue goes, 4.5.)  The accumulators have to be named by constants: each
// iteration of the short loop picks its own of them.  A group that the edge of
// the output cuts goes element by element, from LDS, where a loop can index it.
template <class C>
struct MxFinish {
    typedef typename Elem<C::Dt>::type T;
    static constexpr uint32_t TS = sizeof(T);
    static constexpr int PAIRS = C::FNP / 2, U = C::GATED ? 2 : 4, HALVES = C::FM / U;  // U groups at once: what the registers hold
    struct Raw {
        i32x4 a[TS / 2];
    };
    const EpiArgs& e;
    __amdgpu_buffer_rsrc_t y, r;
    uint32_t oy, orr;      // bytes of the lane's first group
    int n0, col, cols, valid_rows;
    f32x8 b0[PAIRS], b1[C::GATED ? PAIRS : 1];
    Raw next[U];

    __device__ __forceinline__ MxFinish(const EpiArgs& a, int m0, int n0_, int row, int col_) : e(a), n0(n0_), col(col_) {
        const int rows = min(e.M - m0, C::BM);
        cols = e.N - n0;
        valid_rows = rows - row;
        const auto whole = [&](const void* p, int64_t ld) {
            const uint32_t range = (uint32_t)((rows - 1) * (int)ld + min(cols, C::BNP)) * TS;
            return __builtin_amdgcn_make_buffer_rsrc(p ? (char*)const_cast<void*>(p) + (m0 * ld + n0) * (int64_t)TS : nullptr, (short)0,
                                                     range, 0x00020000);
        };
        y = whole(e.Y[0], e.ldy);
        r = whole(e.R, e.ldr);
        oy = (uint32_t)(row * (int)e.ldy + col) * TS;
        orr = (uint32_t)(row * (int)e.ldr + col) * TS;
#pragma unroll
        for (int p = 0; p < PAIRS; ++p) {
            b0[p] = bias(0, p);
            if constexpr (C::GATED) b1[p] = bias(1, p);
        }
    }
    __device__ __forceinline__ bool cut(int p) const { return cols - col - 32 * p < 8; }
    __device__ __forceinline__ f32x8 bias(int which, int p) const {
        if (!e.bias[which] || cut(p)) return zero8();
        return load8<T>(make_rsrc((const T*)e.bias[which] + n0), (uint32_t)(col + 32 * p) * TS);
    }
    __device__ __forceinline__ void fetch(int it) {
        if (!e.R) return;
        const int p = it / HALVES;
        const uint32_t o = (orr + (uint32_t)(16 * U * (it % HALVES) * (int)e.ldr + 32 * p) * TS) | (cut(p) ? OOB : 0u);
#pragma unroll
        for (int q = 0; q < U; ++q)
#pragma unroll
            for (int d = 0; d < (int)TS / 2; ++d)
                next[q].a[d] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                             r, o + (uint32_t)(16 * q * (int)e.ldr) * TS + 16 * d, 0, 0));
    }
    static __device__ __forceinline__ f32x8 value(const Raw& x) {
        if constexpr (TS == 4) {
            return join8(__builtin_bit_cast(f32x4, x.a[0]), __builtin_bit_cast(f32x4, x.a[1]));
        } else {
            const typename Vec8<T>::type h = __builtin_bit_cast(typename Vec8<T>::type, x.a[0]);
            f32x8 v;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = (float)h[i];
            return v;
        }
    }
    // Element x of the group of v (w) `by` rows on in pair p, where the output's edge cuts it.
    template <int KIND>
    __device__ __forceinline__ void one(int by, int p, int x, float v, float w) const {
        const int c = col + 32 * p + x;
        if (e.bias[0]) v += (float)((const T*)e.bias[0])[n0 + c];
        v = act1<KIND>(e.act, v);
        if constexpr (C::GATED) {
            if (e.bias[1]) w += (float)((const T*)e.bias[1])[n0 + c];
            v *= w;
        }
        if (e.R) v += load1<T>(r, orr + (uint32_t)(by * (int)e.ldr + 32 * p + x) * TS);
        store1<T>(y, oy + (uint32_t)(by * (int)e.ldy + 32 * p + x) * TS, v);
    }
    static __device__ __forceinline__ f32x8 pair(const f32x4& a, const f32x4& b) {
        // read where they are used: the compiler copies all 256 to VGPRs at once, and spills
        const auto from = [](float x) {
            float v;
            asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(v) : "a"(x));
            return v;
        };
        f32x8 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = from(a[i]);
            v[4 + i] = from(b[i]);
        }
        return v;
    }
    template <int KIND>
    __device__ __forceinline__ void run(f32x4 (&acc)[C::FM][C::FN], char PGEMM_LDS* own) {
        fetch(0);
#pragma unroll 1
        for (int it = 0; it < PAIRS * HALVES; ++it) {
            f32x8 v[U], w[C::GATED ? U : 1], c0, c1;
#pragma unroll
            for (int x = 0; x < PAIRS * HALVES; ++x) {
                if (x != it) continue;
                const int xp = x / HALVES, xh = x % HALVES;
#pragma unroll
                for (int q = 0; q < U; ++q) {
                    v[q] = pair(acc[U * xh + q][2 * xp], acc[U * xh + q][2 * xp + 1]);
                    if constexpr (C::GATED) w[q] = pair(acc[U * xh + q][C::FNP + 2 * xp], acc[U * xh + q][C::FNP + 2 * xp + 1]);
                }
                c0 = b0[xp];
                c1 = b1[C::GATED ? xp : 0];
            }
            const int p = it / HALVES, by = 16 * U * (it % HALVES);
            if (cols_cut(e.N)) {
#pragma unroll
                for (int q = 0; q < U; ++q)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        *(f32x4 PGEMM_LDS*)(own + (2 * q + h) * 4096) =
                            f32x4{v[q][4 * h], v[q][4 * h + 1], v[q][4 * h + 2], v[q][4 * h + 3]};
                        if constexpr (C::GATED)
                            *(f32x4 PGEMM_LDS*)(own + (2 * U + 2 * q + h) * 4096) =
                                f32x4{w[q][4 * h], w[q][4 * h + 1], w[q][4 * h + 2], w[q][4 * h + 3]};
                    }
            }
            if (e.bias[0]) {
#pragma unroll
                for (int q = 0; q < U; ++q) v[q] += c0;
            }
#pragma unroll
            for (int q = 0; q < U; ++q) v[q] = act8<KIND>(e.act, v[q]);
            if constexpr (C::GATED) {
                if (e.bias[1]) {
#pragma unroll
                    for (int q = 0; q < U; ++q) w[q] += c1;
                }
#pragma unroll
                for (int q = 0; q < U; ++q) v[q] *= w[q];
            }
            if (e.R) {
#pragma unroll
                for (int q = 0; q < U; ++q) v[q] += value(next[q]);
                if (it + 1 < PAIRS * HALVES) fetch(it + 1);
            }
            const uint32_t o = (oy + (uint32_t)(by * (int)e.ldy + 32 * p) * TS) | (cut(p) ? OOB : 0u);
#pragma unroll
            for (int q = 0; q < U; ++q) store8<T>(y, o + (uint32_t)(16 * q * (int)e.ldy) * TS, v[q]);
            if (!cols_cut(e.N)) continue;
            const int n = cols - col - 32 * p;
#pragma unroll 1
            for (int q = 0; q < U; ++q) {
#pragma unroll 1
                for (int x = 0; x < (n < 8 && by + 16 * q < valid_rows ? n : 0); ++x) {
                    const char PGEMM_LDS* at = own + (2 * q + (x >> 2)) * 4096 + 4 * (x & 3);
                    one<KIND>(by + 16 * q, p, x, *(const float PGEMM_LDS*)at,
                              C::GATED ? *(const float PGEMM_LDS*)(at + 2 * U * 4096) : 0.0f);
                }
            }
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
        // With the whole contraction in one go the XCDs begin at different places of it (see linear_kernel).
        const int x = blockIdx.x & 7;
        const int begin = g.splits == 1 ? (int)((int64_t)groups * (((x & 6) + 4 * (x & 1)) & 7) >> 3) : g0;
        const int first = begin * C::G;
        const int panel = C::NP == 2 ? wave / 2 : 0;
        m.ra = make_rsrc_sgpr((const char*)g.A + m0 * g.lda - MxLarge<C>::kBack);
        m.rb = make_rsrc_sgpr((const char*)(panel ? g.B[1] : g.B[0]) + n0 * g.ldb - MxLarge<C>::kBack);
        // Rows: of block b the sixteen from a_row + 32 b on; weights: 64 rows from 64 * wave on.
        const int a_row = (wave >> 1) * 128 + (wave & 1) * 16;
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            int row, kc;
            mx_inv16<C::Fmt, false>((a_row + 32 * (p / 2) + 8 * (p % 2)) * 128 + lane * 16, row, kc);
            m.va[p] = row < rows_left ? (uint32_t)(row * (int)g.lda + kc * 16) + MxLarge<C>::kBack - p % 2 * 1024 : OOB;
            mx_inv16<C::Fmt, true>((64 * wave + 8 * p) * 128 + lane * 16, row, kc);
            row -= panel * C::BNP;
            m.vb[p] = row < cols_left ? (uint32_t)(row * (int)g.ldb + kc * 16) + MxLarge<C>::kBack - p % MxLarge<C>::H * 1024 : OOB;
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
            // (a row's halves swapped in every second eight rows: reads of sixteen rows meet no bank twice)
            vs[q] = row < s_rows ? (uint32_t)(row * (int)ls + (((lane & 1) ^ (lane >> 4 & 1)) << 4)) : OOB;
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
        // Each lane's first row in a unit, at the chunk of each step (piece, half of the line); its first scales.
        const int r = lane & 15, q = lane >> 4;
        uint32_t oa[2], ob[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            oa[i] = lds0 + mx_off16<C::Fmt, false>(wm0 + r, C::Fmt == MX8 ? 4 * i + q : 2 * q + i);
            ob[i] = lds0 + C::AT_B + mx_off16<C::Fmt, true>(wn0 + mx_row_b(r), C::Fmt == MX8 ? 4 * i + q : 2 * q + i);
        }
        const uint32_t swap_a = (r >> 3) << 4, swap_b = (r >> 2 & 1) << 4, of_q = C::Fmt == MX8 ? q : 2 * q;
        const uint32_t osa = lds0 + (wm0 + r) * C::SB + of_q, osb = lds0 + (256 + wn0 + mx_row_b(r)) * C::SB + of_q;
        const auto scales_a = [&](uint32_t stage, uint32_t place) { return osa + stage + (place ^ swap_a); };
        const auto scales_b = [&](uint32_t stage, uint32_t place) { return osb + stage + (place ^ swap_b); };
        m.template read_a<0, 0>(oa, 0);
        m.template read_a<0, 1>(oa, 0);
        m.template read_a<0, 2>(oa, 0);
        m.template read_a<0, 3>(oa, 0);
        m.template read_sa<0, 0>(scales_a(C::AT_S, 0), 0);
        m.template read_sa<0, 1>(scales_a(C::AT_S, 0), 0);
        m.first_b(ob, scales_b(C::AT_S, 0));

        uint32_t ua = 0, ub = 0;       // unit of the period's rows, of its weights
        MxLargeWalk<C> walk(total - first);
        const auto period = [&](auto turn) {
            constexpr int TURN = decltype(turn)::value;
            MxLargeAt at;
            walk.enter();
            const uint32_t ub_next = TURN == C::TURNS - 1 ? C::UNIT - ub : ub;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                at.a[i] = oa[i] + ua;
                at.a_next[i] = oa[i] + (C::UNIT - ua);
                at.b_next[i] = ob[i] + ub_next;
            }
            at.sa = scales_a(walk.stage, walk.place);
            at.sa_next = scales_a(walk.next_stage, walk.next_place);
            at.sb_next = scales_b(walk.next_stage, walk.next_place);
            at.la1 = at_a + C::UNIT - ua;
            at.la2 = at_a + ua;
            at.k1 = round(ka + 128);
            at.k2 = round(at.k1 + 128);
            // (of a unit's two periods, MX8, the first loads the rest of the next unit, the second the half of the one after)
            at.lb = at_b + (C::TURNS == 2 && TURN == 0 ? C::UNIT - ub : ub);
            at.kb = round_b(kw + 128);
            if constexpr (TURN == C::TURNS - 1) at.kb = round_b(at.kb + 128);
            wait_barrier<C::WAIT_X>();
            if (walk.loads()) scales(walk.free);
            MxLarge<C>::template Block<0, TURN>::run(m, acc, at);
            MxLarge<C>::template Block<1, TURN>::run(m, acc, at);
            if (walk.wait_y() == C::WAIT_Y) wait_barrier<C::WAIT_Y>();
            else wait_barrier<C::WAIT_Y_SCALES>();
            MxLarge<C>::template Block<2, TURN>::run(m, acc, at);
            MxLarge<C>::template Block<3, TURN>::run(m, acc, at);
            walk.leave();
            ua = C::UNIT - ua;
            ka = at.k1;
            if constexpr (TURN == C::TURNS - 1) {
                ub = ub_next;
                kw = round_b(kw + 128);
            }
        };
        for (int t = t0; t < t1; t += C::TURNS) {
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
                const int col = n0 + wn0 + 32 * (j % C::FNP / 2) + 4 * (j % 2) + 2 * lg4;
                if (row < g.e.M && col < g.np8)
                    *(f32x4*)(base + ((int64_t)(j / C::FNP) * g.e.M + row) * g.np8 + col) = acc[i][j];
            }
        }
        return;
    }
    MxFinish<C> fin(g.e, m0, n0, wm0 + (lane & 15), wn0 + 8 * (lane >> 4));
    if (cols_cut(g.e.N)) drain_barrier();  // the ring's memory is free
    with_act(g.e.act.kind, [&](auto kind) {
        fin.template run<decltype(kind)::value>(acc, smem + (wave * 64 + lane) * 16);  // 16 bytes of each lane, 4 KiB apart
    });
}

}  // namespace pgemm
