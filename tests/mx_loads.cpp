// A walk along the K loops of the microscaled products' kernels (no GPU): the order in which a
// wave issues its loads to LDS, what each edge's vmcnt leaves under way, and what is read between
// the edges, by the kernels' own constants and MxLargeWalk, MxTileWalk.  Of every read it checks
//   * that it finds the period (K tile, unit, group of scales) that it is meant to, and
//   * that an edge before it has covered the load, for every wave, as all issue alike;
// and of every load that an edge lies between it and the last read of what it overwrites.
// Loads arrive in the order of their issue.  Prints "OK <checks>".  With an argument, edge Y of mx_large
// waits as if no scales had been issued behind its edge X: prints the stored entries of the rows
// that then read too early.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <set>
#include <vector>

#include "../software_pipelined_tiled_loop_amd/csrc/mx_variants.hpp"

using namespace pgemm;

static long checks = 0;
static bool mistaken = false;
static std::set<int> early;  // stored entries of rows that read too early
static int entries, start, splits, split;

static void expect(bool ok, const char* what, int t) {
    ++checks;
    if (ok) return;
    if (mistaken) {
        early.insert(entries);
        return;
    }
    std::printf("FAIL %s: %d entries, start %d, split %d of %d, at %d\n", what, entries, start, split, splits, t);
    std::exit(1);
}

// LDS regions by number: what each holds, and which load brought it.
struct Lds {
    struct Region {
        int content = -2;
        long load = -1, read = -1;  // its number; the edge behind which it was read last
    };
    std::map<int, Region> at;
    long issued = 0, covered = 0, edge = 0;
    void load(int region, int content) {
        Region& r = at[region];
        expect(r.read < edge, "a load overwrites what is being read", region);
        r.content = content;
        r.load = issued++;
    }
    void wait(int under_way) {
        if (issued - under_way > covered) covered = issued - under_way;
        ++edge;
    }
    void read(int region, int content, const char* what, int t) {
        Region& r = at[region];
        expect(r.content == content, what, t);
        expect(r.load >= 0 && r.load < covered, what, t);
        r.read = edge;
    }
    // A read whose value is not used.
    void touch(int region) { at[region].read = edge; }
};

static int begin_of(int groups, int g0) {
    return splits == 1 ? (int)((int64_t)groups * (((start & 6) + 4 * (start & 1)) & 7) >> 3) : g0;
}

template <class C>
static void walk_large() {
    typedef MxLarge<C> L;
    const auto A = [](int unit, int block, int x) { return unit * 8 + block * 2 + x; };
    const auto B = [](int unit, int piece) { return 100 + unit * 8 + piece; };
    const auto S = [](uint32_t stage, int q) { return 200 + (stage ? 4 : 0) + q; };
    const int total = entries / C::BK, groups = (total + C::G - 1) / C::G;
    const int g0 = (int)((int64_t)groups * split / splits), g1 = (int)((int64_t)groups * (split + 1) / splits);
    const int t0 = g0 * C::G, t1 = g1 * C::G < total ? g1 * C::G : total;
    if (t1 <= t0) return;
    const int begin = begin_of(groups, g0), first = begin * C::G;
    int s_group = begin, s_left = g1 - g0;
    Lds lds;
    const auto scales = [&](uint32_t stage) {
        for (int q = 0; q < 4; ++q) lds.load(S(stage, q), s_left > 0 ? s_group : -1);
        --s_left;
        if (++s_group == groups) s_group = 0;
    };
    const int a_end = total * 128, b_end = total * (128 / C::TURNS);
    const auto round = [&](int k) { return k >= a_end ? k - a_end : k; };
    const auto round_b = [&](int k) { return k >= b_end ? k - b_end : k; };
    int ka = first * 128, kw = first * (128 / C::TURNS);
    struct At {
        int unit1, unit2, unit_b, k1, k2, kb;
    };
    const auto pieces = [&](const At& at, int from, int end, int turn) {
        for (int p = from; p < end; ++p) {
            const int block = L::block_of(p);
            if (block >= 0) lds.load(A(p < 2 ? at.unit1 : at.unit2, block, p % 2), (p < 2 ? at.k1 : at.k2) / 128);
            else lds.load(B(at.unit_b, L::weights_of(p, turn)), at.kb / 128);
        }
    };
    // What is read of period t's rows, scales and weights: `used` is false behind the split's last period.
    const auto period_of = [&](int t) { return (first + t - t0) % total; };
    const auto rows = [&](int unit, int block, uint32_t stage, uint32_t place, int t) {
        const int p = period_of(t);
        for (int x = 0; x < 2; ++x) {
            if (t < t1) lds.read(A(unit, block, x), p, "rows", t);
            else lds.touch(A(unit, block, x));
        }
        if (t < t1) expect((int)place == p % C::G * (C::BK / 32), "place of the scales", t);
        for (int q = 0; q < 4; ++q) {
            if (t < t1) lds.read(S(stage - C::AT_S, q), p / C::G, "scales", t);
            else lds.touch(S(stage - C::AT_S, q));
        }
    };
    const auto weights = [&](int unit, int half, uint32_t stage, uint32_t place, int t) {
        const int p = period_of(t);
        if (t < t1) expect(C::TURNS == 1 || half == p % 2, "half of the weights' lines", t);
        if (t < t1) expect((int)place == p % C::G * (C::BK / 32), "place of the scales", t);
        for (int x = 0; x < 8; ++x) {
            if (t < t1) lds.read(B(unit, x), p / C::TURNS, "weights", t);
            else lds.touch(B(unit, x));
        }
        for (int q = 0; q < 4; ++q) {
            if (t < t1) lds.read(S(stage - C::AT_S, q), p / C::G, "scales of the weights", t);
            else lds.touch(S(stage - C::AT_S, q));
        }
    };
    scales(0);
    scales(C::S_STAGE);
    for (int x = 0; x < 8; ++x) lds.load(B(0, x), kw / 128);
    for (int b = 0; b < 3; ++b)
        for (int x = 0; x < 2; ++x) lds.load(A(0, b, x), ka / 128);
    pieces(At{0, 1, 1, ka, round(ka + 128), round_b(kw + 128)}, 0, C::PIECES, C::TURNS - 1);
    lds.wait(C::WAIT_X);
    rows(0, 0, C::AT_S, 0, t0);
    weights(0, 0, C::AT_S, 0, t0);
    int ua = 0, ub = 0;
    MxLargeWalk<C> walk(total - first);
    for (int t = t0; t < t1; t += C::TURNS)
        for (int turn = 0; turn < C::TURNS; ++turn) {
            const int now = t + turn;
            walk.enter();
            const int ub_next = turn == C::TURNS - 1 ? 1 - ub : ub;
            At at;
            at.unit1 = 1 - ua;
            at.unit2 = ua;
            at.k1 = round(ka + 128);
            at.k2 = round(at.k1 + 128);
            at.unit_b = C::TURNS == 2 && turn == 0 ? 1 - ub : ub;
            at.kb = round_b(kw + 128);
            if (turn == C::TURNS - 1) at.kb = round_b(at.kb + 128);
            lds.wait(C::WAIT_X);
            if (walk.loads()) scales(walk.free);
            for (int b = 0; b < 4; ++b) {
                if (b == 2) lds.wait(mistaken ? C::WAIT_Y : walk.wait_y());
                if (b < 3) {
                    rows(ua, b + 1, walk.stage, walk.place, now);
                } else {
                    rows(1 - ua, 0, walk.next_stage, walk.next_place, now + 1);
                    weights(ub_next, C::TURNS == 2 ? 1 - turn : 0, walk.next_stage, walk.next_place, now + 1);
                }
                pieces(at, b * (C::PIECES / 4), (b + 1) * (C::PIECES / 4), turn);
            }
            walk.leave();
            ua = 1 - ua;
            ka = at.k1;
            if (turn == C::TURNS - 1) {
                ub = ub_next;
                kw = round_b(kw + 128);
            }
        }
}

template <class C>
static void walk_tile() {
    typedef MxStep<C, false> Early;
    typedef MxStep<C, true> Late;
    const auto P = [](int slot, int piece) { return slot * 64 + piece; };
    const auto S = [](uint32_t stage, int q) { return 1000 + (stage ? 64 : 0) + q; };
    const int total = entries / C::BK, groups = (total + C::G - 1) / C::G;
    const int g0 = (int)((int64_t)groups * split / splits), g1 = (int)((int64_t)groups * (split + 1) / splits);
    const int t0 = g0 * C::G, t1 = g1 * C::G < total ? g1 * C::G : total;
    if (t1 <= t0) return;
    const int begin = begin_of(groups, g0), first = begin * C::G;
    int k = first * 16 * C::KCB, s_turn = groups - begin, s_left = g1 - g0, s_group = begin;
    const int k_end = total * 16 * C::KCB;
    Lds lds;
    const auto advance = [&] {
        k += 16 * C::KCB;
        if (k == k_end) k = 0;
    };
    const auto scales = [&](uint32_t stage) {
        for (int q = 0; q < C::S_INSTR; ++q) lds.load(S(stage, q), s_left > 0 ? s_group : -1);
        --s_left;
        ++s_group;
        if (--s_turn == 0) s_group -= groups;
    };
    const auto pieces = [&](int slot, int from, int n) {
        for (int p = from; p < from + n; ++p) lds.load(P(slot, p), k / (16 * C::KCB));
    };
    const auto tile_of = [&](int t) { return (first + t - t0) % total; };
    const auto codes = [&](int slot, int t) {
        for (int p = 0; p < C::LPS; ++p) {
            if (t < t1) lds.read(P(slot, p), tile_of(t), "codes", t);
            else lds.touch(P(slot, p));
        }
    };
    const auto read_scales = [&](uint32_t at, int t) {
        const uint32_t stage = (at & ~15u) - C::AT_S;
        if (t < t1) expect((int)(at & 15) == tile_of(t) % C::G * 4, "place of the scales", t);
        for (int q = 0; q < C::S_INSTR; ++q) {
            if (t < t1) lds.read(S(stage, q), tile_of(t) / C::G, "scales", t);
            else lds.touch(S(stage, q));
        }
    };
    scales(0);
    scales(C::S_STAGE);
    for (int p = 0; p < C::S - 1; ++p) {
        pieces(p, 0, C::LPS);
        advance();
    }
    lds.wait(C::LPS * (C::S - 2));
    pieces(C::S - 1, 0, C::LPS / 2);
    codes(0, t0);
    read_scales(C::AT_S, t0);
    int cur = 0, prev = C::S - 1;
    MxTileWalk<C> walk((total - first) / 2);
    const auto tile = [&](int t, uint32_t next_scale, int64_t free) {
        const int nxt = cur == C::S - 1 ? 0 : cur + 1;
        codes(cur, t);
        pieces(prev, Early::P0, Early::NP);
        advance();
        lds.wait(C::LPS * (C::S - 2));
        if (free >= 0) scales((uint32_t)free);
        codes(nxt, t + 1);
        read_scales(next_scale, t + 1);
        pieces(cur, Late::P0, Late::NP);
        prev = cur;
        cur = nxt;
    };
    for (int t = t0; t < t1; t += 2) {
        tile(t, walk.scale + 4, -1);
        walk.pair();
        tile(t + 1, walk.scale, walk.ends ? (int64_t)walk.stage - C::AT_S : -1);
    }
}

template <class C>
static void walk_few() {
    const int total = entries / 256;
    const int t0 = (int)((int64_t)total * split / splits), t1 = (int)((int64_t)total * (split + 1) / splits);
    for (int wave = 0; wave < C::NW; ++wave) {
        Lds lds;
        const auto issue = [&](int t, int st) {
            for (int p = 0; p < C::LPS; ++p) lds.load(st * 256 + p, t < t1 ? t : -1);
        };
        int t = t0 + wave, st = 0;
        if (t >= t1) continue;
        for (int p = 0; p < C::S - 1; ++p) issue(t + p * C::NW, p);
        for (; t < t1; t += C::NW) {
            lds.wait(C::LPS * (C::S - 2));
            issue(t + (C::S - 1) * C::NW, st == 0 ? C::S - 1 : st - 1);
            for (int p = 0; p < C::LPS; ++p) lds.read(st * 256 + p, t, "unit", t);
            st = st + 1 == C::S ? 0 : st + 1;
        }
    }
}

template <int F, int GATED, int DEEP>
static void walk_class() {
    walk_large<MxLargeCfg<DT_BF16, F, GATED != 0>>();
    walk_tile<MX_TILE_CFG(DT_BF16, F, GATED, 128, 128, DEEP, 2, 2)>();
    walk_few<MX_FEW_CFG(DT_BF16, F, GATED, 1, 1, 4, 3)>();
    walk_few<MX_FEW_CFG(DT_BF16, F, GATED, 3, 2, 2, 3)>();
    walk_few<MX_FEW_CFG(DT_BF16, F, GATED, 4, 2, 2, 2)>();
}

int main(int argc, char**) {
    mistaken = argc > 1;
    for (entries = 256; entries <= 40 * 1024; entries += 256)
        for (int s : {1, 2, 3, 4, 6, 8})
            for (split = 0; split < s; ++split)
                for (start = 0; start < (s == 1 ? 8 : 1); ++start) {
                    splits = s;
                    walk_class<MX8, 0, 3>();
                    walk_class<MX8, 1, 3>();
                    walk_class<MX4, 0, 4>();
                    walk_class<MX4, 1, 4>();
                }
    if (mistaken) {
        for (int e : early) std::printf("%d ", e);
        std::printf("\n");
        return 0;
    }
    std::printf("OK %ld\n", checks);
    return 0;
}
