// Host emulation of the feed-forward kernels' data path (no GPU), with the
// kernels' own index functions from linear_kernel.hpp.  For every tile class
// it checks that
//   * the producer fills every byte of the stage exactly once, each chunk
//     from the element that belongs there,
//   * every fragment read stays inside its operand's tile, and the emulated
//     MFMAs with exchanged operands give the product in the lanes that the
//     epilogue reads,
// and, by brute force over small and ragged matrices at every tile origin,
//   * every 16-byte load of the ring ends inside its matrix, and every element
//     load of the cut tiles too,
//   * together they cover the whole contraction of every row and column.
// Prints "OK <checks>"; exits non-zero on the first mismatch.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>

#include "../software_pipelined_tiled_loop_amd/csrc/linear_variants.hpp"

using namespace pgemm;

static long checks = 0;
#define EXPECT(c, ...)                                       \
    do {                                                     \
        ++checks;                                            \
        if (!(c)) {                                          \
            std::printf("FAIL %s: %s: ", __func__, #c);      \
            std::printf(__VA_ARGS__);                        \
            std::printf("\n");                               \
            std::exit(1);                                    \
        }                                                    \
    } while (0)

// One operand: fills the tile from value(e, k), reads every fragment back.
template <class O, int EXT, int BK, int NW>
static std::vector<int> fill(int (*value)(int, int)) {
    std::vector<int> lds(O::BYTES / O::ES, -1);
    std::vector<int> hits(O::BYTES / 16, 0);
    constexpr int per = O::BYTES / 1024 / NW;
    static_assert(per * NW * 1024 == O::BYTES, "blocks");
    for (int wave = 0; wave < NW; ++wave)
        for (int q = 0; q < per; ++q)
            for (int lane = 0; lane < 64; ++lane) {
                const int off = (wave * per + q) * 1024 + lane * 16;
                int e, k;
                O::chunk(off, e, k);
                EXPECT(e >= 0 && e < EXT && k >= 0 && k < BK, "off %d", off);
                ++hits[off / 16];
                const bool along_k = O::mem_off(0, 1, 1000) == (uint32_t)O::ES;
                for (int x = 0; x < O::EPC; ++x)
                    lds[off / O::ES + x] = along_k ? value(e, k + x) : value(e + x, k);
            }
    for (int h : hits) EXPECT(h == 1, "chunk filled %d times", h);
    return lds;
}

// The values a lane's fragment holds, [k slot 0..EPC-1], after the reads (the
// transposing reads: element e of lane i comes from lane 4e + i/4 of its
// 16-lane block, element i%4).
template <int D, int LAY, int EXT, int BK>
static void fragment(const std::vector<int>& lds, int ks, int e0, std::vector<int> (&out)[64]) {
    typedef Opnd<D, LAY, EXT, BK> O;
    for (int lane = 0; lane < 64; ++lane) {
        out[lane].clear();
        if (LAY == LAY_K || O::ES == 4) {
            for (int h = 0; h < O::READS; ++h) {
                const int off = O::frag(ks, e0, lane, h), n = LAY == LAY_K ? O::EPC : 1;
                EXPECT(off >= 0 && off + n * O::ES <= O::BYTES, "read at %d", off);
                for (int x = 0; x < n; ++x) out[lane].push_back(lds[off / O::ES + x]);
            }
        } else {
            for (int h = 0; h < 2; ++h)
                for (int e = 0; e < 4; ++e) {
                    const int i = lane & 15, from = (lane & 48) + 4 * e + i / 4;
                    const int off = O::frag(ks, e0, from, h);
                    EXPECT(off >= 0 && off + 8 <= O::BYTES && off % 8 == 0, "read at %d", off);
                    out[lane].push_back(lds[off / O::ES + i % 4]);
                }
        }
    }
}

static int va(int e, int k) { return (e * 7 + k * 3) % 11 - 5; }
static int vb(int e, int k) { return (e * 5 + k * 13 + (e * k) % 7) % 9 - 4; }

// The epilogue's place in LDS: each pass's sums land on chunks of their own
// inside the wave's area, and the lanes that read a row's groups cover it.
template <class C>
static void check_out() {
    typedef LinOut<C> O;
    std::vector<int> hits(O::AREA / 16, 0);
    for (int i = 0; i < O::BLOCKS; ++i)
        for (int j = 0; j < C::FN; ++j)
            for (int lane = 0; lane < 64; ++lane) {
                const int at = O::at(16 * i + (lane & 15), 4 * j + (lane >> 4));
                EXPECT(at >= 0 && at + 16 <= O::AREA && hits[at / 16]++ == 0, "at %d", at);
            }
    std::vector<int> read(O::AREA / 16, 0);
    for (int s = 0; s < O::STEPS; ++s)
        for (int lane = 0; lane < 64; ++lane)
            for (int p = 0; p < C::NP; ++p)
                for (int h = 0; h < 2; ++h)
                    ++read[O::at(lane / O::LPR + s * O::RPI, p * (C::WNP / 4) + 2 * (lane % O::LPR) + h) / 16];
    for (size_t x = 0; x < hits.size(); ++x) EXPECT(read[x] == hits[x], "chunk %zu", x);
}

template <int D, int LA, int LB, int BM, int BN, int BK, int S, int WGM, int WGN, bool GATED>
static void check_class(LinCfg<D, LA, LB, BM, BN, BK, S, WGM, WGN, GATED>) {
    typedef LinCfg<D, LA, LB, BM, BN, BK, S, WGM, WGN, GATED> C;
    const std::vector<int> a = fill<typename C::OA, BM, BK, C::NW>(va);
    const std::vector<int> b = fill<typename C::OB, C::BNP, BK, C::NW / C::NP>(vb);
    check_out<C>();
    // one wave's corner blocks of each operand
    for (int wave = 0; wave < C::NW; wave += C::NW - 1) {
        const int wm0 = (wave / WGN) * C::WM, wnp = (wave % WGN) * C::WNP;
        for (int i = 0; i < C::FM; i += C::FM - 1 > 0 ? C::FM - 1 : 1)
            for (int j = 0; j < C::FNP; ++j) {
                long acc[64][4] = {};
                for (int ks = 0; ks < C::NKS; ++ks) {
                    static std::vector<int> fa[64], fb[64];
                    fragment<D, LA, BM, BK>(a, ks, wm0 + 16 * i, fa);
                    fragment<D, LB, C::BNP, BK>(b, ks, wnp + 16 * j, fb);
                    // result block (exchanged operands): lane l, register r:
                    // column 4*(l/16)+r of B, row l%16 of A
                    for (int l = 0; l < 64; ++l)
                        for (int r = 0; r < 4; ++r)
                            for (int g = 0; g < 4; ++g)
                                for (size_t x = 0; x < fa[0].size(); ++x)
                                    acc[l][r] += (long)fa[16 * g + l % 16][x] * fb[16 * g + 4 * (l / 16) + r][x];
                }
                for (int l = 0; l < 64; ++l)
                    for (int r = 0; r < 4; ++r) {
                        const int m = wm0 + 16 * i + l % 16, n = wnp + 16 * j + 4 * (l / 16) + r;
                        long want = 0;
                        for (int k = 0; k < BK; ++k) want += (long)va(m, k) * vb(n, k);
                        EXPECT(acc[l][r] == want, "m %d n %d: %ld, want %ld", m, n, acc[l][r], want);
                    }
            }
    }
}

// Loads of one operand over a whole (extent x K) matrix: inside it, and every
// element covered once.
template <int D, int LAY, int EXT, int BK>
static void check_bounds(int extent, int64_t K, int64_t ld) {
    typedef Opnd<D, LAY, EXT, BK> O;
    const int64_t rows = LAY == LAY_K ? extent : K, cols = LAY == LAY_K ? K : extent;
    const int64_t end = rows > 0 && cols > 0 ? ((rows - 1) * ld + cols) * O::ES : 0;
    const int ring = O::ring_tiles(K, extent, ld);
    EXPECT((int64_t)ring * BK <= K, "ring");
    std::vector<int> seen((size_t)extent * K, 0);
    for (int e0 = 0; e0 < extent; e0 += EXT)
        for (int64_t kt = 0; kt * BK < K; ++kt) {
            const int64_t org = O::origin(e0, kt, ld);
            const int e_left = extent - e0, k_left = (int)(K - kt * BK);
            for (int off = 0; off < O::BYTES; off += 16) {
                int e, k;
                O::chunk(off, e, k);
                int n;
                if (kt < ring) {
                    if (e >= e_left) continue;
                    n = O::EPC;
                    const int64_t at = org + O::mem_off(e, k, ld);
                    EXPECT(at >= 0 && at + 16 <= end, "ring load at %ld of %ld (extent %d K %ld ld %ld)", (long)at,
                           (long)end, extent, (long)K, (long)ld);
                } else {
                    n = O::cut_valid(e, k, e_left, k_left);
                    const int64_t at = org + O::mem_off(e, k, ld);
                    const int64_t row = LAY == LAY_K ? K : extent;
                    if (n > 0 && row >= O::EPC) {
                        // one 16-byte load, of a chunk cut the one that ends at the edge
                        const int64_t from = at - (n < O::EPC ? O::cut_shift((int)row) : 0);
                        EXPECT(from >= 0 && from + 16 <= end, "cut load at %ld of %ld", (long)from, (long)end);
                        EXPECT(n == O::EPC || (O::EPC - n) * O::ES == O::cut_shift((int)row), "shift");
                    } else if (n > 0) {
                        EXPECT(at >= 0 && at + n * O::ES <= end, "cut load at %ld of %ld", (long)at, (long)end);
                    }
                }
                for (int x = 0; x < n; ++x) {
                    const int ee = e0 + e + (LAY == LAY_X ? x : 0);
                    const int64_t kk = kt * BK + k + (LAY == LAY_K ? x : 0);
                    if (ee < extent && kk < K) ++seen[(size_t)ee * K + kk];
                    else EXPECT(kt < ring && LAY == LAY_X, "a cut load past the edge");
                }
            }
        }
    for (int s : seen) EXPECT(s == 1, "element loaded %d times (extent %d K %ld)", s, extent, (long)K);
}

template <int D, int EXT, int BK>
static void check_bounds_all() {
    // (16 columns: only along K)
    constexpr int LX = EXT * Traits<D>::ES >= 64 ? LAY_X : LAY_K;
    for (int extent : {1, 3, 7, 8, 9, 16, 63, 64, 100, 129, 200, 255, 257})
        for (int K : {1, 2, 7, 8, 15, 31, 32, 33, 63, 64, 65, 96, 127, 128, 130, 200})
            for (int pad : {0, 1, 5}) {
                check_bounds<D, LAY_K, EXT, BK>(extent, K, K + pad);
                check_bounds<D, LX, EXT, BK>(extent, K, (LX == LAY_X ? extent : K) + pad);
            }
}

// A few-rows kernel: each wave fills its own stage.
template <int D, int LA, int LB, int FM, int NCOL, int NW, int S, bool GATED>
static void check_class(FewCfg<D, LA, LB, FM, NCOL, NW, S, GATED>) {
    typedef FewCfg<D, LA, LB, FM, NCOL, NW, S, GATED> C;
    const std::vector<int> a = fill<typename C::OA, C::BM, C::BK, 1>(va);
    const std::vector<int> b = fill<typename C::OB, C::NCOLP, C::BK, 1>(vb);
    for (int i = 0; i < FM; ++i)
        for (int j = 0; j < C::FNP; ++j) {
            long acc[64][4] = {};
            for (int ks = 0; ks < C::NKS; ++ks) {
                static std::vector<int> fa[64], fb[64];
                fragment<D, LA, C::BM, C::BK>(a, ks, 16 * i, fa);
                fragment<D, LB, C::NCOLP, C::BK>(b, ks, 16 * j, fb);
                for (int l = 0; l < 64; ++l)
                    for (int r = 0; r < 4; ++r)
                        for (int g = 0; g < 4; ++g)
                            for (size_t x = 0; x < fa[0].size(); ++x)
                                acc[l][r] += (long)fa[16 * g + l % 16][x] * fb[16 * g + 4 * (l / 16) + r][x];
            }
            for (int l = 0; l < 64; ++l)
                for (int r = 0; r < 4; ++r) {
                    const int m = 16 * i + l % 16, n = 16 * j + 4 * (l / 16) + r;
                    long want = 0;
                    for (int k = 0; k < C::BK; ++k) want += (long)va(m, k) * vb(n, k);
                    EXPECT(acc[l][r] == want, "m %d n %d", m, n);
                }
        }
}

#undef LIN_FEW
#define LIN_FEW(D, LAY, GATED, FM, NCOL, NW, S) \
    LIN_FEW_CFG(D, LAY, GATED, FM, NCOL, NW, S) {}
#undef LIN_VARIANT
#define LIN_VARIANT(D, LAY, GATED, BM, BN, BK, S, WGM, WGN) \
    LIN_CFG(D, LAY, GATED, BM, BN, BK, S, WGM, WGN) {}
template <class... Cs>
static void classes(Cs... cs) {
    (check_class(cs), ...);
}

int main() {
    classes(LIN_CLASS(DT_BF16, 256, 256, 64, 2, 2, 2));
    classes(LIN_CLASS(DT_F32, 256, 256, 32, 2, 2, 4));
    classes(LIN_CLASS(DT_BF16, 128, 128, 64, 2, 2, 2));
    classes(LIN_CLASS(DT_BF16, 128, 128, 64, 4, 2, 2));
    classes(LIN_CLASS(DT_F32, 128, 128, 32, 2, 2, 2));
    classes(LIN_FEW_CLASSES(DT_BF16));
    classes(LIN_FEW_CLASSES(DT_F32));
    check_bounds_all<DT_BF16, 16, 64>();
    check_bounds_all<DT_BF16, 32, 64>();
    check_bounds_all<DT_F32, 64, 32>();
    check_bounds_all<DT_BF16, 256, 64>();
    check_bounds_all<DT_F32, 256, 32>();
    check_bounds_all<DT_BF16, 128, 64>();
    check_bounds_all<DT_BF16, 64, 64>();
    check_bounds_all<DT_F32, 128, 32>();
    std::printf("OK %ld\n", checks);
    return 0;
}
