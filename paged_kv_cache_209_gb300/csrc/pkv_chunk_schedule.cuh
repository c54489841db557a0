// Work split of the int8 chunk attention (pkv_chunk_q8.cu).
//
// A unit is a tile of 256 query rows of one (sequence, KV head): rows
// r = t G + g, query t and query head g of the KV head's group of G. It takes
// ns steps of 128 tokens, up to the last token its last row sees. Units are
// ordered sequence-major, then head, then tile.
//
// A launch of C CTAs first deals whole units in `rounds` rounds: in round r, CTA c
// takes the units that begin in piece r C + c of the cost axis, each piece as long
// as the costliest unit. CTAs that run at the same time then work on neighbouring
// units, the tiles of a few (sequence, KV head) pairs, whose K and V stay in L2:
// dealt one contiguous range per CTA instead, the pairs of a large batch are all
// read at once and evict one another (DRAM reads 7 times the cache's bytes on 8
// sequences of 8192 tokens). The rest of the axis, one to two units per CTA, is
// cut by steps so that every CTA's total comes out even; a unit that a cut
// divides leaves pieces, which a second kernel joins. Small launches have no rounds.
//
// Cost of tile t of a sequence with n tokens, nq of them new: about the tokens
// it sees plus a start-up worth kOverTokens, in units of 64 / G tokens, linear in
// t so that a position is found by bisection over closed forms:
//     a + 4 t,   a = ceil(((n - nq + kOverTokens) G + 256) / 64).
// A last tile of few rows costs as much as a full one: converting a step's codes takes
// about as long as its products for both row halves, and the products wait for it.
// (Ragged chunks of 1 to 777 tokens when a tile of one row half counted half: 181 us,
// like this 147. With a start-up of 256 tokens they now take 126 us, of 384 106, 512
// 102, 768 102; 24 new tokens on ragged contexts 45, 37, 39 and 40.)
// The cost only places cuts; a unit's steps are counted exactly.
//
// How even it comes out depends on the sizes. A round's piece is as long as the costliest
// unit, so that pieces drift against the units and some hold two; where that repeats at one
// CTA, what it has too much the rest cannot take back. The slowest CTA's steps (and three
// for each segment) over the even share, 32 query heads on 8, 152 CTAs: 8 sequences of 8192
// tokens with 512 new ones 1.01, 777 1.27, 1000 1.43, 1024 1.33; 4 of 8192 with 1024 1.20;
// 8 of 4096 with 512 1.16; whole prompts, one of 1000 tokens 1.48, one of 2048 1.11, 8 of
// 2048 1.17. (With kOverTokens at 448 the first is 1.18: the sizes at which drift repeats
// move with it.) It shows: 1266 TFLOP/s of the visible pairs with 512 new ones on 8 of
// 8192, 998 with 777, 927 with 1000, 1023 with 1024; 1097 with 1024 on 4 of 8192, 1011
// with 512 on 8 of 4096; 606 for one prompt of 2048, 791 for 8.
//
// Plain integer arithmetic, compiled for the host as well, where a test checks
// it against brute force.
#pragma once

#include <stdint.h>

#ifndef PKV_HD
#define PKV_HD __host__ __device__
#endif

namespace pkv {
namespace {

constexpr int kChunkRows = 256;   // query rows of a unit
constexpr int kChunkStep = 128;   // tokens of a step
constexpr int kOverTokens = 384;  // start-up of a unit (Q, the pipeline's fill, the output) in tokens
constexpr int kMinPiece = 2;      // a cut leaves at least this many steps on either side
constexpr int kMaxRounds = 8;     // rounds of whole units, at most
constexpr int kMinSteps = 3;      // a CTA gets at least about this many steps' cost

// a / b of non-negative numbers (a 64-bit division is a long loop on the GPU, and a
// launch's planning waits for several).
PKV_HD inline int64_t chunk_div(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

struct ChunkShape {
    const int32_t* lens;
    const int32_t* qstart;
    int batch, kv_heads, group, max_blocks, max_query_len;
};

struct ChunkSeq {
    int n, nq, q0;  // tokens, new tokens, first query row
};

// A position between steps: step s of a unit (seq == batch: past the end).
struct ChunkPos {
    int seq, head, tile, s;
    PKV_HD bool same_unit(const ChunkPos& o) const { return seq == o.seq && head == o.head && tile == o.tile; }
    PKV_HD bool operator==(const ChunkPos& o) const { return same_unit(o) && s == o.s; }
};

// Reads sequence i; false (and no queries) when its lengths are malformed.
PKV_HD inline bool chunk_seq(const ChunkShape& a, int i, ChunkSeq& q) {
    q.n = a.lens[i];
    q.q0 = a.qstart[i];
    const int64_t nq = static_cast<int64_t>(a.qstart[i + 1]) - q.q0;
    const bool ok = q.n >= 0 && q.n <= a.max_blocks * 16 && q.q0 >= 0 && nq >= 0 && nq <= q.n && nq <= a.max_query_len;
    q.nq = ok ? static_cast<int>(nq) : 0;
    return ok;
}

PKV_HD inline int chunk_tiles(const ChunkSeq& q, int group) { return (q.nq * group + kChunkRows - 1) / kChunkRows; }

// Steps of tile t.
PKV_HD inline int chunk_steps(const ChunkSeq& q, int group, int t) {
    const int rows = q.nq * group;
    const int end = (t + 1) * kChunkRows < rows ? (t + 1) * kChunkRows : rows;
    return (q.n - q.nq + (end - 1) / group) / kChunkStep + 1;  // (the last token's index: below 2^31)
}

PKV_HD inline int64_t chunk_cost_base(const ChunkSeq& q, int group) {
    return ((static_cast<int64_t>(q.n) - q.nq + kOverTokens) * group + kChunkRows + 63) / 64;  // (n + kOverTokens may pass 2^31)
}
// Cost of the tiles before t (t < tiles), of tile t, and of all tiles of a head.
PKV_HD inline int64_t chunk_cost_before(int64_t base, int64_t t) { return t * base + 2 * t * (t - 1); }
PKV_HD inline int64_t chunk_tile_cost(int64_t base, int t) { return base + 4 * static_cast<int64_t>(t); }
PKV_HD inline int64_t chunk_head_cost(const ChunkSeq& q, int group) {
    return chunk_cost_before(chunk_cost_base(q, group), chunk_tiles(q, group));
}

// The next unit after `p` of `tiles` in its head.
PKV_HD inline ChunkPos chunk_next_unit(const ChunkShape& a, ChunkPos p, int tiles) {
    p.s = 0;
    if (++p.tile < tiles) return p;
    p.tile = 0;
    if (++p.head < a.kv_heads) return p;
    p.head = 0;
    ChunkSeq q;
    do ++p.seq;
    while (p.seq < a.batch && (!chunk_seq(a, p.seq, q) || q.nq == 0));
    return p;
}

// The unit at cost x, 0 <= x < total (prefix: cost before each sequence, [batch + 1]).
struct ChunkPlace {
    ChunkPos unit;
    int64_t rem;         // x less the cost before the unit
    int64_t cost;        // of the unit
    int ns, tiles;       // its steps, the tiles of its head
};
PKV_HD inline ChunkPlace chunk_locate(const ChunkShape& a, const int64_t* prefix, int64_t x) {
    ChunkPlace p;
    int lo = 0, hi = a.batch - 1;  // the last sequence whose cost begins at or before x
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= x)
            lo = mid;
        else
            hi = mid - 1;
    }
    ChunkSeq q;
    chunk_seq(a, lo, q);
    const int64_t head_cost = chunk_head_cost(q, a.group);
    const int64_t base = chunk_cost_base(q, a.group);
    p.unit = ChunkPos{lo, 0, 0, 0};
    p.rem = x - prefix[lo];
    p.unit.head = static_cast<int>(chunk_div(p.rem, head_cost));
    p.rem -= p.unit.head * head_cost;
    p.tiles = chunk_tiles(q, a.group);
    lo = 0, hi = p.tiles - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (chunk_cost_before(base, mid) <= p.rem)
            lo = mid;
        else
            hi = mid - 1;
    }
    p.unit.tile = lo;
    p.rem -= chunk_cost_before(base, lo);
    p.cost = chunk_tile_cost(base, lo);
    p.ns = chunk_steps(q, a.group, lo);
    return p;
}
// The cut between steps at cost x.
PKV_HD inline ChunkPos chunk_step_cut(const ChunkShape& a, const int64_t* prefix, int64_t x) {
    if (x >= prefix[a.batch]) return ChunkPos{a.batch, 0, 0, 0};
    ChunkPlace p = chunk_locate(a, prefix, x);
    p.unit.s = static_cast<int>(chunk_div(p.rem * p.ns, p.cost));
    if (p.unit.s < kMinPiece)
        p.unit.s = 0;
    else if (p.ns - p.unit.s < kMinPiece)
        p.unit = chunk_next_unit(a, p.unit, p.tiles);
    return p.unit;
}
// The cut between units nearest to cost x, and the cost before it.
PKV_HD inline ChunkPos chunk_unit_cut(const ChunkShape& a, const int64_t* prefix, int64_t x, int64_t& at) {
    at = prefix[a.batch];
    if (x >= at) return ChunkPos{a.batch, 0, 0, 0};
    ChunkPlace p = chunk_locate(a, prefix, x);
    at = x - p.rem;
    if (2 * p.rem < p.cost) return p.unit;
    at += p.cost;
    return chunk_next_unit(a, p.unit, p.tiles);
}

// CTAs (of `grid`) that get work.
PKV_HD inline int chunk_ctas(int64_t total, int group, int grid) {
    const int64_t most = chunk_div(total, static_cast<int64_t>(kMinSteps) * kChunkStep * group / 64);
    return most >= grid ? grid : (most < 1 ? 1 : static_cast<int>(most));
}
// Costliest unit of a sequence.
PKV_HD inline int64_t chunk_most(const ChunkSeq& q, int group) {
    const int tiles = chunk_tiles(q, group);
    if (tiles == 0) return 0;
    return chunk_tile_cost(chunk_cost_base(q, group), tiles - 1);
}
// Rounds of whole units, and the length of their pieces: a multiple of the
// costliest unit, so that units of one size are dealt evenly. At least three
// quarters of such a unit per CTA are left to even the totals out.
struct ChunkRounds {
    int rounds;
    int64_t piece;
};
PKV_HD inline ChunkRounds chunk_rounds(int64_t total, int64_t most, int ctas) {
    const int64_t share = chunk_div(total, ctas) - most * 3 / 4;
    ChunkRounds r{0, most};
    if (share < most) return r;
    const int64_t n = chunk_div(share, most);
    r.rounds = static_cast<int>(n < kMaxRounds ? n : kMaxRounds);
    if (n > kMaxRounds) r.piece = n / kMaxRounds * most;
    return r;
}
// What the rounds give CTA c; at[i]: the cost before the i-th cut of the rounds.
PKV_HD inline int64_t chunk_dealt(const int64_t* at, const ChunkRounds& r, int c, int ctas) {
    int64_t sum = 0;
    for (int k = 0; k < r.rounds; ++k) sum += at[k * ctas + c + 1] - at[k * ctas + c];
    return sum;
}
// The cut before CTA c in what is left of the axis from cost `from` on; `due`: what
// the CTAs before c still have to get, of `all`.
PKV_HD inline ChunkPos chunk_rest_cut(const ChunkShape& a, const int64_t* prefix, int64_t from, int64_t due, int64_t all, int c,
                                      int ctas) {
    if (c >= ctas) return ChunkPos{a.batch, 0, 0, 0};
    const int64_t rest = prefix[a.batch] - from;
    if (all <= 0) return chunk_step_cut(a, prefix, prefix[a.batch]);
    if ((rest >> 31) == 0 && (all >> 31) == 0) return chunk_step_cut(a, prefix, from + due * rest / all);
    return chunk_step_cut(a, prefix, from + static_cast<int64_t>(static_cast<double>(due) / static_cast<double>(all) * static_cast<double>(rest)));
}

// Walks the segments (unit, steps s0 .. s1 - 1) between two cuts.
struct ChunkSegment {
    ChunkPos at;  // unit; at.s is the first step
    int s1, ns;   // one past the last step; the unit's steps
    int tiles;
    ChunkSeq q;
    PKV_HD bool whole() const { return at.s == 0 && s1 == ns; }
};
PKV_HD inline bool chunk_segment(const ChunkShape& a, const ChunkPos& cur, const ChunkPos& end, ChunkSegment& g) {
    if (cur == end || cur.seq >= a.batch) return false;
    g.at = cur;
    chunk_seq(a, cur.seq, g.q);
    g.tiles = chunk_tiles(g.q, a.group);
    g.ns = chunk_steps(g.q, a.group, cur.tile);
    g.s1 = cur.same_unit(end) ? end.s : g.ns;
    return true;
}
// The position after segment g.
PKV_HD inline ChunkPos chunk_after(const ChunkShape& a, const ChunkSegment& g) {
    if (g.s1 < g.ns) return ChunkPos{g.at.seq, g.at.head, g.at.tile, g.s1};
    return chunk_next_unit(a, g.at, g.tiles);
}
// Walks all segments of a CTA: `ranges` holds its rounds' and its last range, two cuts each.
// chunk_walk_to finds the segment at the walker, chunk_walk also moves it on.
struct ChunkWalk {
    ChunkPos cur;
    int range;
};
PKV_HD inline ChunkWalk chunk_begin(const ChunkPos* ranges) { return ChunkWalk{ranges[0], 0}; }
PKV_HD inline bool chunk_walk_to(const ChunkShape& a, const ChunkPos* ranges, int count, ChunkWalk& w, ChunkSegment& g) {
    while (!chunk_segment(a, w.cur, ranges[2 * w.range + 1], g)) {
        if (++w.range >= count) return false;
        w.cur = ranges[2 * w.range];
    }
    return true;
}
PKV_HD inline bool chunk_walk(const ChunkShape& a, const ChunkPos* ranges, int count, ChunkWalk& w, ChunkSegment& g) {
    if (!chunk_walk_to(a, ranges, count, w, g)) return false;
    w.cur = chunk_after(a, g);
    return true;
}

}  // namespace
}  // namespace pkv
