// Host-side check of the int8 chunk attention's work split
// (pkv_chunk_schedule.cuh, the code the kernel runs) at the longest contexts a call
// takes, 2^31 - 16 tokens, for few and for many new ones, alone and beside short
// sequences: costs follow their definition in 64 bits, and the segments of all CTAs,
// in order, take every step of every unit exactly once. Prints "ok <cases>" or the
// first mismatches, and exits non-zero on a mismatch.
#include <cstdio>
#include <vector>

#include "pkv_chunk_schedule.cuh"

using namespace pkv;

namespace {

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

void check_case(const std::vector<int>& lens, const std::vector<int>& nqs, int kvh, int group, int grid) {
    const int batch = static_cast<int>(lens.size());
    std::vector<int> start(batch + 1, 0);
    for (int i = 0; i < batch; ++i) start[i + 1] = start[i] + nqs[i];
    ChunkShape a{lens.data(), start.data(), batch, kvh, group, 134217727, 65536};
    std::vector<int64_t> prefix(batch + 1, 0);
    int64_t most = 0;
    for (int i = 0; i < batch; ++i) {
        ChunkSeq q;
        CHECK(chunk_seq(a, i, q), "sequence %d", i);
        const int64_t base = ((static_cast<int64_t>(lens[i]) - nqs[i] + kOverTokens) * group + kChunkRows + 63) / 64;
        CHECK(chunk_cost_base(q, group) == base, "cost of %d tokens, %d new, group %d: %lld", lens[i], nqs[i], group,
              static_cast<long long>(chunk_cost_base(q, group)));
        prefix[i + 1] = prefix[i] + chunk_head_cost(q, group) * kvh;
        CHECK(prefix[i + 1] >= prefix[i], "costs fall at sequence %d", i);
        if (chunk_most(q, group) > most) most = chunk_most(q, group);
    }
    if (g_fail) return;
    const int64_t total = prefix[batch];
    const int ctas = chunk_ctas(total, group, grid);
    const ChunkRounds r = chunk_rounds(total, most, ctas);
    // as the kernel lays them out
    std::vector<int64_t> at(r.rounds * ctas + 1, 0);
    for (size_t i = 0; i < at.size(); ++i) chunk_unit_cut(a, prefix.data(), static_cast<int64_t>(i) * r.piece, at[i]);
    const int64_t from = at.back();
    std::vector<int64_t> due(ctas + 1, 0);
    for (int c = 0; c < ctas; ++c) {
        const int64_t left = total / ctas - chunk_dealt(at.data(), r, c, ctas);
        due[c + 1] = due[c] + (left > 0 ? left : 0);
    }
    int seq = 0, head = 0, tile = 0, done = 0;
    auto skip = [&] {
        while (seq < batch && nqs[seq] == 0) ++seq;
    };
    skip();
    for (int k = 0; k <= r.rounds; ++k)
        for (int c = 0; c < ctas; ++c) {
            int64_t cost;
            ChunkPos cut[2];
            for (int e = 0; e < 2; ++e)
                cut[e] = k < r.rounds ? chunk_unit_cut(a, prefix.data(), (static_cast<int64_t>(k) * ctas + c + e) * r.piece, cost)
                                      : chunk_rest_cut(a, prefix.data(), from, due[c + e], due[ctas], c + e, ctas);
            ChunkPos cur = cut[0];
            ChunkSegment g;
            while (chunk_segment(a, cur, cut[1], g)) {
                if (seq >= batch) {
                    CHECK(false, "segment past the last unit");
                    return;
                }
                const int64_t rows = static_cast<int64_t>(nqs[seq]) * group;
                const int64_t end = (tile + 1) * static_cast<int64_t>(kChunkRows) < rows ? (tile + 1) * static_cast<int64_t>(kChunkRows) : rows;
                const int64_t seen = static_cast<int64_t>(lens[seq]) - nqs[seq] + (end - 1) / group + 1;
                CHECK(g.at.seq == seq && g.at.head == head && g.at.tile == tile && g.at.s == done && g.ns == (seen + 127) / 128,
                      "segment (%d %d %d %d of %d) for unit (%d %d %d) step %d", g.at.seq, g.at.head, g.at.tile, g.at.s, g.ns,
                      seq, head, tile, done);
                CHECK(g.s1 > g.at.s && g.s1 <= g.ns, "steps %d .. %d of %d", g.at.s, g.s1, g.ns);
                if (g_fail) return;
                done = g.s1;
                if (done == g.ns) {
                    done = 0;
                    if ((tile + 1) * static_cast<int64_t>(kChunkRows) < rows)
                        ++tile;
                    else {
                        tile = 0;
                        if (++head == kvh) {
                            head = 0;
                            ++seq;
                            skip();
                        }
                    }
                }
                cur = chunk_after(a, g);
            }
        }
    CHECK(seq == batch && done == 0, "not all units taken: %d of %d sequences", seq, batch);
}

}  // namespace

int main() {
    int cases = 0;
    const int longest = 2147483632;
    for (int nq : {1, 40, 300, 5000, 65536})
        for (int group : {1, 3, 8, 1024})
            for (int kvh : {1, 8})
                for (int grid : {1, 7, 152}) {
                    if (kvh * group > 1024) continue;
                    check_case({longest}, {nq}, kvh, group, grid);
                    check_case({200, longest, 0, 70000, longest - 5, 9}, {200, nq, 0, 300, nq, 0}, kvh, group, grid);
                    cases += 2;
                    if (g_fail) {
                        std::printf("(%d new tokens, %d heads of %d rows, %d CTAs)\n", nq, kvh, group, grid);
                        return 1;
                    }
                }
    std::printf("ok %d\n", cases);
    return 0;
}
