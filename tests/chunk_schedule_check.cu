// Host-side check of the int8 chunk attention's work split
// (pkv_chunk_schedule.cuh, the code the kernel runs) against brute force over
// random batches: the segments of all CTAs, in order, take every step of every
// unit exactly once; a cut leaves pieces of at least two steps; costs follow
// their definition; no CTA gets far more than its share. Prints "ok <cases>" or
// the first mismatches, and exits non-zero on a mismatch.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "pkv_chunk_schedule.cuh"

using namespace pkv;

namespace {

unsigned long long g_state = 0x9e3779b97f4a7c15ull;
int rnd(int n) {  // splitmix64, then reduced to [0, n)
    g_state += 0x9e3779b97f4a7c15ull;
    unsigned long long z = g_state;
    z = (z ^ (z >> 30)) * 0xbf58476d1ce4e5b9ull;
    z = (z ^ (z >> 27)) * 0x94d049bb133111ebull;
    z ^= z >> 31;
    return static_cast<int>(z % static_cast<unsigned long long>(n));
}

int g_fail = 0;
#define CHECK(cond, ...)                               \
    do {                                               \
        if (!(cond)) {                                 \
            if (g_fail++ < 5) {                        \
                std::printf("mismatch: " __VA_ARGS__); \
                std::printf("\n");                     \
            }                                          \
        }                                              \
    } while (0)

struct Unit {
    int seq, head, tile, ns;
};

void check_case(const std::vector<int>& lens, const std::vector<int>& start, int kvh, int group, int max_blocks,
                int max_q, int grid) {
    const int batch = static_cast<int>(lens.size());
    ChunkShape a{lens.data(), start.data(), batch, kvh, group, max_blocks, max_q};
    std::vector<int64_t> prefix(batch + 1, 0);
    std::vector<Unit> units;
    for (int i = 0; i < batch; ++i) {
        ChunkSeq q;
        const bool ok = chunk_seq(a, i, q);
        const int nq = start[i + 1] - start[i];
        CHECK(ok == (lens[i] >= 0 && lens[i] <= max_blocks * 16 && start[i] >= 0 && nq >= 0 && nq <= lens[i] && nq <= max_q),
              "validity of sequence %d", i);
        const int64_t rows = ok ? static_cast<int64_t>(nq) * group : 0;
        int64_t cost = 0;
        const int64_t base = chunk_cost_base(q, group);
        for (int64_t r0 = 0; r0 < rows; r0 += kChunkRows) {
            const int t = static_cast<int>(r0 / kChunkRows);
            CHECK(chunk_cost_before(base, t) == cost, "cost before tile %d", t);
            cost += ((rows - r0 <= 128) ? 1 : 2) * (base + 4 * t);
            // the last token any row of the tile sees
            int seen = 0;
            for (int64_t r = r0; r < r0 + kChunkRows && r < rows; ++r) {
                const int last = lens[i] - nq + static_cast<int>(r / group);
                if (last + 1 > seen) seen = last + 1;
            }
            CHECK(chunk_steps(q, group, t) == (seen + 127) / 128, "steps of tile %d", t);
        }
        CHECK(chunk_head_cost(q, group) == cost, "head cost of sequence %d", i);
        prefix[i + 1] = prefix[i] + cost * kvh;
        for (int h = 0; h < kvh; ++h)
            for (int t = 0; t < chunk_tiles(q, group); ++t) units.push_back({i, h, t, chunk_steps(q, group, t)});
    }
    const int ctas = chunk_ctas(prefix[batch], group, grid);
    CHECK(ctas >= 1 && ctas <= grid, "%d CTAs of %d", ctas, grid);
    size_t u = 0;
    int done = 0;
    double most = 0, all = 0;
    for (int c = 0; c < ctas; ++c) {
        ChunkPos cur = chunk_cut(a, prefix.data(), c, ctas);
        const ChunkPos end = chunk_cut(a, prefix.data(), c + 1, ctas);
        ChunkSegment g;
        int count = 0;
        double work = 0;
        while (chunk_segment(a, cur, end, g)) {
            if (u >= units.size()) {
                CHECK(false, "segment past the last unit");
                return;
            }
            const Unit& w = units[u];
            CHECK(g.at.seq == w.seq && g.at.head == w.head && g.at.tile == w.tile && g.at.s == done && g.ns == w.ns,
                  "segment (%d %d %d %d) for unit (%d %d %d) step %d", g.at.seq, g.at.head, g.at.tile, g.at.s, w.seq,
                  w.head, w.tile, done);
            CHECK(g.s1 > g.at.s && g.s1 <= g.ns, "steps %d .. %d of %d", g.at.s, g.s1, g.ns);
            if (!g.whole()) CHECK(g.s1 - g.at.s >= kMinPiece, "piece of %d steps", g.s1 - g.at.s);
            CHECK(count == 0 || g.at.s == 0, "a segment in the middle of a range begins inside a unit");
            work += (g.s1 - g.at.s) + 1.0;
            done = g.s1;
            if (done == w.ns) {
                ++u;
                done = 0;
            }
            cur = chunk_after(a, prefix.data(), g);
            ++count;
        }
        CHECK(cur == end || end.seq >= batch, "walk ends off its cut");
        all += work;
        if (work > most) most = work;
    }
    CHECK(u == units.size() && done == 0, "%zu of %zu units taken", u, units.size());
    CHECK(most <= 2.5 * all / ctas + 12, "a CTA takes %.0f of %.0f steps (%d CTAs)", most, all, ctas);
}

}  // namespace

int main() {
    int cases = 0;
    for (int it = 0; it < 4000; ++it, ++cases) {
        const int batch = 1 + rnd(it % 10 == 0 ? 200 : 12);
        const int group = 1 + rnd(it % 7 == 0 ? 130 : 9), kvh = 1 + rnd(9);
        const int max_blocks = 1 + rnd(it % 3 == 0 ? 700 : 40), max_q = 1 + rnd(it % 2 == 0 ? 2000 : 50);
        std::vector<int> lens(batch), start(batch + 1);
        start[0] = rnd(5);
        for (int i = 0; i < batch; ++i) {
            const int kind = rnd(8);
            lens[i] = kind == 0 ? 0 : kind == 1 ? 1 + rnd(3) : 1 + rnd(max_blocks * 16);
            int nq = kind == 2 ? 0 : 1 + rnd(max_q);
            if (nq > lens[i]) nq = rnd(20) == 0 ? nq : lens[i];
            if (rnd(60) == 0) lens[i] = -3;
            if (rnd(60) == 0) lens[i] = max_blocks * 16 + 1;
            start[i + 1] = start[i] + (rnd(80) == 0 ? -1 : nq);
        }
        check_case(lens, start, kvh, group, max_blocks, max_q, 1 + rnd(it % 5 == 0 ? 8 : 200));
    }
    // the largest sizes the call takes: costs and cuts stay inside 64 bits
    {
        std::vector<int> lens{2147483632}, start{0, 65536};
        ChunkShape a{lens.data(), start.data(), 1, 1, 1024, 134217727, 65536};
        ChunkSeq q;
        CHECK(chunk_seq(a, 0, q), "largest sequence");
        std::vector<int64_t> prefix{0, chunk_head_cost(q, 1024)};
        CHECK(prefix[1] > 0, "largest cost");
        ChunkPos last{0, 0, 0, 0};
        for (int c = 1; c < 152; ++c) {
            const ChunkPos p = chunk_cut(a, prefix.data(), c, 152);
            CHECK(p.tile >= 0 && p.tile < chunk_tiles(q, 1024) && p.s >= 0 && p.s < chunk_steps(q, 1024, p.tile), "cut %d", c);
            CHECK(p.tile > last.tile || (p.tile == last.tile && p.s >= last.s), "cuts fall at %d", c);
            last = p;
        }
    }
    if (g_fail) {
        std::printf("%d mismatches\n", g_fail);
        return 1;
    }
    std::printf("ok %d\n", cases);
    return 0;
}
