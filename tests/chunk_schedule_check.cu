// Host-side check of the int8 chunk attention's work split
// (pkv_chunk_schedule.cuh, the code the kernel runs) against brute force over
// random batches: the segments of all CTAs, in order, take every step of every
// unit exactly once; a cut keeps two steps from a unit's ends; costs follow
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
int g_rounds = 0;      // cases with rounds
double g_worst = 0.0;  // largest share a CTA got
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
            cost += base + 4 * t;
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
    const int64_t total = prefix[batch];
    const int ctas = chunk_ctas(total, group, grid);
    CHECK(ctas >= 1 && ctas <= grid, "%d CTAs of %d", ctas, grid);
    int64_t most = 0;
    for (int i = 0; i < batch; ++i) {
        ChunkSeq q;
        chunk_seq(a, i, q);
        int64_t top = 0;
        for (int t = 0; t < chunk_tiles(q, group); ++t) {
            const int64_t c = chunk_tile_cost(chunk_cost_base(q, group), t);
            if (c > top) top = c;
        }
        CHECK(chunk_most(q, group) == top, "costliest unit of sequence %d", i);
        if (top > most) most = top;
    }
    if (total == 0) return;
    const ChunkRounds r = chunk_rounds(total, most, ctas);
    CHECK(r.rounds >= 0 && r.rounds <= kMaxRounds && r.piece >= most, "%d rounds", r.rounds);
    // as the kernel lays them out
    std::vector<int64_t> at(r.rounds * ctas + 1, 0);
    for (size_t i = 0; i < at.size(); ++i) chunk_unit_cut(a, prefix.data(), static_cast<int64_t>(i) * r.piece, at[i]);
    const int64_t from = at.back();
    int64_t all = 0;
    std::vector<int64_t> due(ctas + 1, 0);
    for (int c = 0; c < ctas; ++c) {
        const int64_t left = total / ctas - chunk_dealt(at.data(), r, c, ctas);
        due[c + 1] = due[c] + (left > 0 ? left : 0);
    }
    all = due[ctas];
    const int count = r.rounds + 1;
    std::vector<std::vector<ChunkPos>> ranges(ctas, std::vector<ChunkPos>(2 * count));
    for (int c = 0; c < ctas; ++c) {
        int64_t cost;
        for (int k = 0; k < r.rounds; ++k)
            for (int e = 0; e < 2; ++e)
                ranges[c][2 * k + e] = chunk_unit_cut(a, prefix.data(), (static_cast<int64_t>(k) * ctas + c + e) * r.piece, cost);
        for (int e = 0; e < 2; ++e)
            ranges[c][2 * r.rounds + e] = chunk_rest_cut(a, prefix.data(), from, due[c + e < ctas ? c + e : ctas], all, c + e, ctas);
    }
    // every step of every unit exactly once, in the order (range, CTA)
    size_t u = 0;
    int done = 0;
    std::vector<double> work(ctas, 0.0);
    double sum = 0, biggest = 0;
    for (const Unit& w : units) biggest = w.ns + 3.0 > biggest ? w.ns + 3.0 : biggest;
    for (int k = 0; k < count; ++k)
        for (int c = 0; c < ctas; ++c) {
            ChunkPos cur = ranges[c][2 * k];
            const ChunkPos end = ranges[c][2 * k + 1];
            ChunkSegment g;
            int n = 0;
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
                CHECK(k == r.rounds || g.whole(), "a round cuts a unit");
                if (g.at.s > 0 || g.s1 < g.ns)
                    CHECK((g.at.s == 0 || g.at.s >= kMinPiece) && (g.s1 == g.ns || g.ns - g.s1 >= kMinPiece), "cut at %d or %d of %d",
                          g.at.s, g.s1, g.ns);
                CHECK(n == 0 || g.at.s == 0, "a segment in the middle of a range begins inside a unit");
                work[c] += g.s1 - g.at.s + 3;
                done = g.s1;
                if (done == w.ns) {
                    ++u;
                    done = 0;
                }
                cur = chunk_after(a, g);
                ++n;
            }
            CHECK(cur == end || end.seq >= batch, "walk ends off its cut");
        }
    CHECK(u == units.size() && done == 0, "%zu of %zu units taken", u, units.size());
    // the walker gives the same segments
    for (int c = 0; c < ctas; ++c) {
        ChunkWalk w = chunk_begin(ranges[c].data());
        ChunkSegment g, h;
        for (int k = 0; k < count; ++k) {
            ChunkPos cur = ranges[c][2 * k];
            while (chunk_segment(a, cur, ranges[c][2 * k + 1], g)) {
                CHECK(chunk_walk(a, ranges[c].data(), count, w, h) && h.at == g.at && h.s1 == g.s1, "walker");
                cur = chunk_after(a, g);
            }
        }
        CHECK(!chunk_walk(a, ranges[c].data(), count, w, h), "walker ends");
    }
    for (int c = 0; c < ctas; ++c) sum += work[c];
    for (int c = 0; c < ctas; ++c) {
        CHECK(work[c] <= 1.3 * sum / ctas + 0.75 * biggest + 6, "a CTA takes %.0f of %.0f steps (%d CTAs, %d rounds, biggest %.0f)",
              work[c], sum, ctas, r.rounds, biggest);
        if (work[c] / (sum / ctas + 6) > g_worst) g_worst = work[c] / (sum / ctas + 6);
    }
    if (r.rounds) ++g_rounds;
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
        check_case(lens, start, kvh, group, max_blocks, max_q, 1 + rnd(it % 3 == 0 ? 8 : 200));
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
        const ChunkRounds r = chunk_rounds(prefix[1], chunk_most(q, 1024), 152);
        CHECK(r.rounds == kMaxRounds && r.piece > 0 && r.piece * 152 * kMaxRounds > 0, "largest rounds");
        for (int c = 1; c < 152; ++c) {
            const ChunkPos p = chunk_rest_cut(a, prefix.data(), 0, c, 152, c, 152);
            CHECK(p.tile >= 0 && p.tile < chunk_tiles(q, 1024) && p.s >= 0 && p.s < chunk_steps(q, 1024, p.tile), "cut %d", c);
            CHECK(p.tile > last.tile || (p.tile == last.tile && p.s >= last.s), "cuts fall at %d", c);
            last = p;
        }
    }
    CHECK(g_rounds > 300, "only %d cases with rounds", g_rounds);
    if (g_fail) {
        std::printf("%d mismatches\n", g_fail);
        return 1;
    }
    std::printf("ok %d (%d with rounds, largest share %.2f)\n", cases, g_rounds, g_worst);
    return 0;
}
