// Causal attention of a chunk of new tokens over the int8 pools
// (pkv_multiquery_attention_q8 in include/pkv.h): all its calls but those of up to 16
// query rows per (sequence, KV head) of 128 on tables for many tokens, which run on the
// kernel that splits the cache (split_kernel_takes in pkv_api.cu).
//
// Mathematics, per query row and step of 128 tokens:
//     s_p = q' . k_p                    f16 x f16 -> fp32; q' is q times a power of two
//                                       per row (exact), k_p = kc_p (ks_p 2^-F) rounded
//                                       to f16 once, an eighth of a quantization step
//     x_p = s_p f                       f = |scale| log2(e) 2^F over the row's power
//     w_p = 2^(x_p - m)                 m: running maximum or up to 9 less, moved only
//                                       when a part's weights sum to more than f16 holds
//     l  += w_p;   O += w_p v_p         w rounded to f16; v_p = vc_p (vs_p 2^-E)
//                                       rounded to f16; fp32 sums
// (m is the second largest of the maxima of a part's four groups of 16 tokens, but at most
// 9 below the largest. Behind one attention sink m lies 9 below it, so that f16 holds the
// weights of the tail: 11 bits down to 2^-23 of the sink's, some to 2^-34. Where no
// token stands out m is about the maximum, and a later token may outweigh it by 2^14 or
// so before m has to move, which costs about a step. With 7 below it everywhere, chunks of
// 512 on 8192 took 925 us, not 452, on scores of standard deviation 3.)
//     out = 2^E O / l
// F and E are one exponent each per piece of work, taken from the scales of its first
// block, that put K and V into the f16 range whatever their size. 32 tokens whose
// scales leave [2^-14, 2^8] times that (rows 2^22 apart; or infinities) are taken as
// bare codes; a step that holds such tokens, or absent ones, is slow: it takes
// x_p = s_p ks_p f in fp32, and w_p = 2^(x_p + log2(vs_p) - E - m) with l summed apart
// where V's codes are bare. That is exact over the whole float range, because the
// maximum is then taken over tokens the row sees.
//
// K's scale sits in the K operand, not in the softmax, because a factor per token
// costs every row a multiplication and a shared-memory broadcast, 1024 of the 2500
// cycles that a step's products take: the softmax would be the bound.
//
// Work (pkv_chunk_schedule.cuh): one persistent CTA per SM takes a range of
// (unit, step) pairs, a unit being 256 query rows of a (sequence, KV head) as
// two row halves A and B of 128. A unit cut by a range leaves fp32 pieces
// (O, m, l) in the workspace, which combine_kernel joins.
//
// Roles (24 warps). Warps 0-3 and 4-7: the softmax of halves A and B, one thread
// per query row. Warps 8-11 and 12-15: the converters of K and of V: codes and
// factors to scaled f16, in the 128-byte-swizzled layout the tensor cores read.
// Warps 16 and 17: one thread each issues S = Q K^T of A and of B; warps 18 and 19:
// O += P V of A and of B, in two parts of 64 tokens. Warps 20-23 run ahead: the
// segments, block ids, scales and the factors that follow from them.
//
// Tensor memory (512 columns): S of A and B, in two parts of 64 tokens (64 fp32
// columns each; the part's P is written over the first 32), O of A and B. The parts'
// buffers are independent: while the softmax takes one, the other's products and
// next scores run. Shared memory: Q 64 KB, two stages of K of 32 KB each, three of V
// of 16 KB, the next step's codes 32 KB.
//
// What bounds it: the tensor pipe is busy 72 % of the time (56 % at its product rate: a
// score product of 64 tokens reads 6 KB of operands for 32 cycles), the schedulers issue
// in 60 % of the slots, and both halves' chains of scores, softmax and products are
// about as long as a step, 3700 cycles against 2500 for the products alone. An
// instruction costs a warp 7 cycles, the price of sharing a scheduler and the
// instruction cache. So everything that is done once per step or segment sits in warps
// of its own, and waits and issuing loops are as short as they go. 8 sequences of 8192
// tokens, 512 of them new, 32 query heads on 8 of 128: 421 to 426 us in a captured graph,
// 1250 to 1265 TFLOP/s of the visible pairs (the cuBLAS rate is 1956), and 453 us, 1176,
// called among other work; one of 65536 tokens, 256 new, 64 heads on 8: 413 to 419 and
// 461 us, 1310 to 1329 and 1190 TFLOP/s. Chunks of other sizes are also bound by how
// evenly the work is split (pkv_chunk_schedule.cuh). Tiles of at most 128 rows are not
// bound by the products: half B idles, and half A's chain takes 1.6 us a step, about as
// long as a step of both halves. Scores far apart take longer, because m has to move: of
// standard deviation 3, 439 us for the first, of 6, 1620. Slower, for the first: scores as
// one product of 128 tokens 520 (against 425: a half's softmax waits for all of it); the
// halves' softmax in turns 535, half B held back by a part 442 (against 423); eight warps
// for K instead of four 518 (against 502).
// Small calls are bound by the chain before the first product: 2.5 us to plan, 4 for
// the table, the scales and the codes, one after another; 14 us for 40 new tokens on
// 200.
#include <math.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"

#include "pkv_chunk_schedule.cuh"

namespace pkv {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
// The K factor of an absent token (a block id outside the pool): a NaN that no
// arithmetic produces.
constexpr uint32_t kAbsent = 0x7fc0dead;

__device__ __forceinline__ float ninf() { return __int_as_float(0xff800000); }

// How far (log2) m may lie below the maximum, and what a part's weights may sum to: the
// largest f16, no weight is above the sum; 64 that sum to more hold one above 2^9.9, so
// that m then moves.
constexpr float kHeadroom = 9.f;
constexpr float kMostSum = 65504.f;
// Where V's codes are bare, m is the maximum of x_p + log2(vs_p) - E, and l, which takes
// 2^(x_p - m), may leave the float range. So that it does not, that logarithm counts as
// kLeastLack at least in the maximum (of a V scale 2^-96 of the others' or zero: its
// values have that much less weight in the f16 range), and |E| is at most kMostLack (l
// holds 2^-112 and more beside V scales of up to 2^52, whatever the first block's).
constexpr float kLeastLack = -96.f;
constexpr int kMostLack = 60;

constexpr int kMaxPieces = 512;  // CTAs of a launch, and pieces of a unit, at most

template <int D>
struct Cx {
    static constexpr int kSoftmaxWarps = 8;
    static constexpr int kConvertWarp = 8;  // K: 8 .. 11, V: 12 .. 15
    static constexpr int kScoreWarp = 16;   // 16, 17
    static constexpr int kValueWarp = 18;   // 18, 19
    static constexpr int kScaleWarp = 20;   // 20 .. 23
    static constexpr int kThreads = 768;
    static constexpr int kStages = 2;   // K stages (a step each)
    static constexpr int kParts = 3;    // V stages (64 tokens each)
    static constexpr int kRecords = 4;  // steps whose factors are laid out
    // Tables in flight: the scale warps write step n once the converters are done with
    // step n - kRecords; K's then are at most four steps ahead of the slower softmax
    // half (a fifth needs scores that need V parts which that half's products have
    // yet to release).
    static constexpr int kTables = kRecords + 5;
    static constexpr int kJobs = 8;     // segments laid out ahead
    static constexpr int kHalves = D / 64;                    // 128-byte column parts of a K or Q row
    static constexpr int kPartBytes = 128 * 128;              // 128 rows of one part
    static constexpr int kTileBytes = kHalves * kPartBytes;   // Q of one row half; one K stage
    static constexpr int kVPartBytes = D * 128;               // one V stage: 64 tokens of every coordinate
    static constexpr int kVecs = D / 16;                      // 16-code vectors of a converter lane and step
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kOffQ + 2 * kTileBytes;
    static constexpr int kOffV = kOffK + kStages * kTileBytes;
    static constexpr int kOffCodes = kOffV + kParts * kVPartBytes;  // the next step's codes: [8 warps][kVecs][32 lanes] vectors
    static constexpr int kOffTable = kOffCodes + 8 * kVecs * 512;
    // a step's table: 2^E, 2^F, whether it is a slow step, its number; the tokens' K factors [128] and,
    // in log2, what their V values lack [128] (for parts done with care)
    static constexpr int kTableBytes = 16 + 2 * 128 * 4;
    // a step's record: per token (hi, hi, lo, lo) of K's factor in f16 [128], V's factor in
    // f16 [128]; its 8 blocks' place in the pools, in vectors; whether there is such a step
    static constexpr int kOffRecord = kOffTable + kTables * kTableBytes;
    static constexpr int kRecordBytes = 128 * 8 + 128 * 2 + 8 * 8 + 16;
    static constexpr int kOffBars = kOffRecord + kRecords * kRecordBytes;
    // k_full, k_empty per K stage; v_full, v_empty per V stage; q_full per half;
    // s_full, p_full, pv_done per half and part; final per issuer; job_full, job_empty;
    // record_full, record_empty
    static constexpr int kNumBars = 2 * kStages + 2 * kParts + 2 + 3 * 4 + 4 + 2 * kJobs + 2 * kRecords;
    static constexpr int kOffJobs = kOffBars + (kNumBars + 1) / 2 * 16;
    static constexpr int kOffWalk = kOffJobs + kJobs * 48;
    static constexpr int kOffPlan = kOffWalk + (sizeof(ChunkWalk) + 15) / 16 * 16;
    static constexpr int kOffMisc = kOffPlan + 2 * (kMaxRounds + 1) * 16;
    static constexpr size_t kSmem = 1024 + kOffMisc + kThreads / 32 * 8 + 16;
    // scratch of the planning, over the operands: the rounds' cuts, then the costs before the sequences
    static constexpr int kOffPrefix = (kMaxRounds * kMaxPieces + 1) * 8;
    static_assert(kOffPrefix + (kMaxBatchPerLaunch + 1) * 8 <= kOffCodes, "planning scratch");
    static constexpr uint32_t kColS = 0;    // S of half x: 128 x
    static constexpr uint32_t kColO = 256;  // O of half x: 256 + 128 x
    static constexpr uint32_t kTmemCols = 512;
    static_assert(kSmem <= 227 * 1024, "shared memory");
};

// ---------------------------------------------------------------- workspace
// Per CTA a descriptor (first position of its range, flags) and two piece slots:
// 0 for a piece that begins inside a unit, 1 for one that begins a unit and is cut.
// A slot: O as [D / 4][256 rows] of four floats (a warp's lanes, one row each, write
// consecutive vectors), then the rows' m and l.
struct PieceInfo {
    ChunkPos start;
    int flags;  // 1: slot 0 written, 2: slot 1 written
    int pad[3];
};
static_assert(sizeof(PieceInfo) == 32, "layout");
__host__ __device__ constexpr size_t slot_floats(int d) { return static_cast<size_t>(kChunkRows) * (d + 2); }
__host__ __device__ constexpr size_t infos_bytes(int grid) { return (static_cast<size_t>(grid) * sizeof(PieceInfo) + 255) / 256 * 256; }
__device__ __forceinline__ float* slot_of(void* workspace, int grid, int d, int cta, int slot) {
    return reinterpret_cast<float*>(static_cast<char*>(workspace) + infos_bytes(grid)) + (static_cast<size_t>(cta) * 2 + slot) * slot_floats(d);
}

// Query of row R of a unit's sequence, and that row's place in q and out. (A division
// by the group as a multiplication: exact for rows below 2^26 and groups up to 1024.)
__device__ __forceinline__ int query_of(const ChunkArgs& a, int R) {
    return static_cast<int>((static_cast<uint64_t>(R) * a.group_inverse) >> 37);
}
__device__ __forceinline__ int64_t row_of_unit(const ChunkArgs& a, int q0, int head, int R) {
    const int t = query_of(a, R);
    return (static_cast<int64_t>(q0) + t) * a.q_heads + head * a.group + (R - t * a.group);
}

__device__ __forceinline__ ChunkShape shape_of(const ChunkArgs& a) {
    return ChunkShape{a.lens, a.qstart, a.batch, a.kv_heads, a.group, a.max_blocks, a.max_query_len};
}

// Sum of x over the threads before this one, the sum of all in `total` (one
// __syncthreads; scratch: an int64 per warp, free again after the next one).
template <int kThreads>
__device__ __forceinline__ int64_t block_sum(int64_t x, int64_t* scratch, int64_t& total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto scan = [lane](int64_t v) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t other = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += other;
        }
        return v;
    };
    const int64_t incl = scan(x);
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    const int64_t warps = scan(lane < kThreads / 32 ? scratch[lane] : 0);
    total = __shfl_sync(0xffffffffu, warps, 31);
    const int64_t before = __shfl_sync(0xffffffffu, warps, warp > 0 ? warp - 1 : 0);
    return (warp > 0 ? before : 0) + incl - x;
}

// This CTA's ranges (all threads; ends with __syncthreads): returns their number,
// 0 for a CTA without work. prefix: cost before each sequence; ranges: two cuts per
// range; at: scratch for the rounds' cuts and the CTAs' dues.
template <int kThreads>
__device__ int plan_ranges(const ChunkArgs& a, const ChunkShape& sh, int64_t* prefix, ChunkPos* ranges, int64_t* at, int64_t* scratch) {
    const int t = threadIdx.x, grid = gridDim.x, cta = blockIdx.x;
    // two sequences per thread
    int64_t mine[2], most = 0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int i = 2 * t + e;
        mine[e] = 0;
        if (i < a.batch) {
            ChunkSeq q;
            if (!chunk_seq(sh, i, q) && cta == 0) atomicOr(a.status, PKV_DEVERR_RANGE);
            mine[e] = chunk_head_cost(q, a.group) * a.kv_heads;
            most = max(most, chunk_most(q, a.group));
        }
    }
    auto largest = [](int64_t v) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
        return v;
    };
    most = largest(most);
    if ((t & 31) == 0) at[t >> 5] = most;  // (not yet used for the cuts)
    int64_t total;
    const int64_t before = block_sum<kThreads>(mine[0] + mine[1], scratch, total);
    most = largest((t & 31) < kThreads / 32 ? at[t & 31] : 0);
    if (2 * t <= a.batch) prefix[2 * t] = before;
    if (2 * t + 1 <= a.batch) prefix[2 * t + 1] = before + mine[0];
    __syncthreads();
    const int ctas = chunk_ctas(total, a.group, grid);
    if (total == 0 || cta >= ctas) return 0;
    const ChunkRounds r = chunk_rounds(total, most, ctas);
    int64_t from = 0, due0 = cta, due1 = cta + 1, all = ctas;
    if (r.rounds > 0) {
        for (int i = t; i <= r.rounds * ctas; i += kThreads) {
            int64_t cost;
            chunk_unit_cut(sh, prefix, static_cast<int64_t>(i) * r.piece, cost);
            at[i] = cost;
        }
        __syncthreads();
        from = at[r.rounds * ctas];
        const int64_t left = t < ctas ? chunk_div(total, ctas) - chunk_dealt(at, r, t, ctas) : 0;
        const int64_t due = block_sum<kThreads>(left > 0 ? left : 0, scratch, all);
        __syncthreads();
        if (t == cta) at[0] = due;
        if (t == cta + 1) at[1] = due;
        __syncthreads();
        due0 = at[0];
        due1 = at[1];
    }
    if (t < 2 * (r.rounds + 1)) {
        int64_t cost;
        const int k = t >> 1, e = t & 1;
        ranges[t] = k < r.rounds ? chunk_unit_cut(sh, prefix, (static_cast<int64_t>(k) * ctas + cta + e) * r.piece, cost)
                                 : chunk_rest_cut(sh, prefix, from, e ? due1 : due0, all, cta + e, ctas);
    }
    __syncthreads();
    return r.rounds + 1;
}

// ---------------------------------------------------------------- conversions
// Two codes (+ 128, bytes of f16s 1024 + code + 128) as f16x2, exactly.
__device__ __forceinline__ __half2 codes_f16x2(uint32_t h) {
    const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
    return __hsub2(*reinterpret_cast<const __half2*>(&h), bias);
}
__device__ __forceinline__ uint32_t bits(const __half2& x) { return *reinterpret_cast<const uint32_t*>(&x); }
__device__ __forceinline__ __half2 half2_of(uint32_t x) { return *reinterpret_cast<const __half2*>(&x); }
// Eight codes of one token times hi + lo (the scale to 22 bits): one rounding but for
// that of the small term.
__device__ __forceinline__ uint4 k_values(uint32_t w0, uint32_t w1, __half2 hi, __half2 lo) {
    w0 ^= 0x80808080u;
    w1 ^= 0x80808080u;
    const __half2 c0 = codes_f16x2(__byte_perm(w0, 0x64646464u, 0x5140)), c1 = codes_f16x2(__byte_perm(w0, 0x64646464u, 0x7362));
    const __half2 c2 = codes_f16x2(__byte_perm(w1, 0x64646464u, 0x5140)), c3 = codes_f16x2(__byte_perm(w1, 0x64646464u, 0x7362));
    return make_uint4(bits(__hfma2(c0, hi, __hmul2(c0, lo))), bits(__hfma2(c1, hi, __hmul2(c1, lo))),
                      bits(__hfma2(c2, hi, __hmul2(c2, lo))), bits(__hfma2(c3, hi, __hmul2(c3, lo))));
}
// Eight codes of one coordinate times their tokens' factors.
__device__ __forceinline__ uint4 v_values(uint32_t w0, uint32_t w1, const uint4& f) {
    w0 ^= 0x80808080u;
    w1 ^= 0x80808080u;
    return make_uint4(bits(__hmul2(codes_f16x2(__byte_perm(w0, 0x64646464u, 0x5140)), half2_of(f.x))),
                      bits(__hmul2(codes_f16x2(__byte_perm(w0, 0x64646464u, 0x7362)), half2_of(f.y))),
                      bits(__hmul2(codes_f16x2(__byte_perm(w1, 0x64646464u, 0x5140)), half2_of(f.z))),
                      bits(__hmul2(codes_f16x2(__byte_perm(w1, 0x64646464u, 0x7362)), half2_of(f.w))));
}
// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }
// The exponent that takes the largest of some scales (its bits; not an infinity) to 1/2 .. 1.
__device__ __forceinline__ int range_exponent(uint32_t most) { return max(-125, min(125, static_cast<int>(most >> 23) - 126)); }
// Whether a scale leaves [2^(e - 14), 2^(e + 8)] (bits compare as the floats do).
__device__ __forceinline__ bool leaves_range(uint32_t scale, int e) {
    return scale < static_cast<uint32_t>(max(e - 14, -126) + 127) << 23 || scale > static_cast<uint32_t>(min(e + 8, 127) + 127) << 23;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// kind::f16 with f16 A and B, fp32 accumulator, both K-major.
__host__ __device__ constexpr uint32_t umma_idesc_f16(int M, int N) {
    return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
// Sixteen scaled scores, -inf where the token is absent or not seen (columns taddr ..
// taddr + 15, K factors c, row factor f, the first `seen` of them seen). The factors are
// multiplied first: one of them may be as large as the other is small.
__device__ __forceinline__ void careful_scores(uint32_t taddr, const float* c, float f, int seen, float (&x)[16]) {
    uint32_t v[16];
    tmem_ld16(taddr, v);
    tmem_ld_wait();
#pragma unroll
    for (int e = 0; e < 16; ++e)
        x[e] = e >= seen || __float_as_uint(c[e]) == kAbsent ? ninf() : __uint_as_float(v[e]) * (c[e] * f);
}
// Waits until the phase of this parity has completed, for kProbes probes at most; false:
// it has not, and the role gives up, as does, in as much time, every role that depends
// on it. A failing probe holds the thread for 1.4 us where nothing happens (6 s together)
// and for 150 cycles or so where barriers of the CTA are arrived at (0.3 s together). That
// is thousands of steps, and every wait but one lasts a few steps at most; the one is half
// B's for the next segment while half A alone takes one of any length (next_job, which
// renews it as long as steps are laid out). One probe in a loop is all there is: the
// kernel's two dozen waits share the instruction cache with its loops, and a role reports
// at its end (a clock and the report in each wait: 487 us instead of 481 for 8 sequences by
// 512 new tokens).
constexpr int kProbes = 1 << 22;
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) {
#pragma unroll 1
    for (int n = 0; n < kProbes; ++n)
        if (mbar_try_wait(bar, parity)) return true;
    return false;
}
// wait by a whole warp, with one answer for all its lanes.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
#pragma unroll 1
    for (int n = 0; n < kProbes; ++n)
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return false;
}
__device__ __forceinline__ void report_timeout(const ChunkArgs& a) { atomicOr(a.status, PKV_DEVERR_TIMEOUT); }
// 16 bytes from global to shared memory, asynchronously.
__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copy_wait_all() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// One lane of a converged warp. Where the issuers choose theirs this way, and not as
// lane 0, the compiler knows that the branch holds one thread and keeps its loop in
// uniform registers (8 sequences by 512 new tokens: 444 us, as lane 0 465).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}

// ---------------------------------------------------------------- segments
// A segment as the roles need it. The first of the scale warps, ahead of all others, walks
// the CTA's ranges and lays the next segment out in shared memory; the others read it
// there. (Walking in each role cost a dependent chain of global loads at every
// segment, and its code.)
struct __align__(16) Job {
    int seq, head;
    int s0, s1;   // steps; s1 == 0: no more segments
    int n, q0;    // tokens and first query row of the sequence
    int before;   // its tokens ahead of the chunk
    int r0;       // first row of the unit
    int rows;     // rows of the unit, at most 256
    int piece;    // 0: the whole unit; 1: begins inside it (slot 0), 2: begins it and is cut (slot 1)
    int pad[2];
};
static_assert(sizeof(Job) == 48, "layout");

// The next segment of a warp's sequence of them (`count`: how many it has taken).
// All lanes of the warp, or kLanes = 1: one thread. False at the end (job.s1 == 0) and
// where the wait ran out (job.s1 < 0): with kWhileSteps, where no step was laid out for the
// CTA while it lasted (the scale warps stay a few steps ahead of the products).
template <int D, int kLanes, bool kWhileSteps = false>
__device__ __forceinline__ bool next_job(uint8_t* smem, uint64_t* job_full, uint64_t* job_empty, int& count, Job& job) {
    using C = Cx<D>;
    const int slot = count % C::kJobs;
    const uint32_t parity = static_cast<uint32_t>(count / C::kJobs) & 1u;
    if (kWhileSteps) {
        uint32_t before = 0;
        for (bool again = false; !warp_wait(&job_full[slot], parity); again = true) {
            uint32_t now = 0;  // the steps in the tables add up to more with every one
#pragma unroll 1
            for (int t = 0; t < C::kTables; ++t)
                now += *reinterpret_cast<const volatile uint32_t*>(smem + C::kOffTable + t * C::kTableBytes + 12);
            now = __shfl_sync(0xffffffffu, now, 0);
            if (again && now == before) {
                job.s1 = -1;
                return false;
            }
            before = now;
        }
    } else if (!(kLanes == 32 ? warp_wait(&job_full[slot], parity) : wait(&job_full[slot], parity))) {
        job.s1 = -1;
        return false;
    }
    job = *reinterpret_cast<const Job*>(smem + C::kOffJobs + slot * sizeof(Job));
    if (kLanes == 32) __syncwarp();
    if (kLanes == 1 || (threadIdx.x & 31) == 0) mbar_arrive(&job_empty[slot]);
    ++count;
    return job.s1 > 0;
}

// Lays out the segment after `count` others (one thread).
template <int D>
__device__ __forceinline__ void lay_out_job(const ChunkArgs& a, uint8_t* smem, uint64_t* job_full, uint64_t* job_empty, int ranges, int count) {
    using C = Cx<D>;
    const int slot = count % C::kJobs;
    if (count >= C::kJobs && !wait(&job_empty[slot], static_cast<uint32_t>(count / C::kJobs - 1) & 1u)) return;
    ChunkWalk& walk = *reinterpret_cast<ChunkWalk*>(smem + C::kOffWalk);
    ChunkSegment g;
    Job job{};
    const bool more = chunk_walk_to(shape_of(a), reinterpret_cast<const ChunkPos*>(smem + C::kOffPlan), ranges, walk, g);
    if (more) {
        job.seq = g.at.seq;
        job.head = g.at.head;
        job.s0 = g.at.s;
        job.s1 = g.s1;
        job.n = g.q.n;
        job.q0 = g.q.q0;
        job.before = g.q.n - g.q.nq;
        job.r0 = g.at.tile * kChunkRows;
        job.rows = min(kChunkRows, g.q.nq * a.group - job.r0);
        job.piece = g.whole() ? 0 : g.at.s > 0 ? 1 : 2;
    }
    *reinterpret_cast<Job*>(smem + C::kOffJobs + slot * sizeof(Job)) = job;
    mbar_arrive(&job_full[slot]);
    if (more) walk.cur = chunk_after(shape_of(a), g);  // while the others begin with this one
}

// ---------------------------------------------------------------- scales
// Four warps, ahead of all others: block ids, scales, and what follows from them. Warp w
// takes the CTA's steps w, w + 4, ...: four steps' chains of loads (id, then scales) are
// in flight, and none holds up the converters. (In the converters' own loop this was
// 2000 of 5200 cycles a step; with a quarter of every step per warp 2900 of 3300 where
// one row half is in use, because each step's chain then followed on the last one's.)
// Lane l holds tokens l, 32 + l, 64 + l, 96 + l; 32 of them at a time are taken as bare codes.
template <int D>
__device__ __forceinline__ void scale_role(const ChunkArgs& a, uint8_t* smem, int ranges, uint64_t* job_full, uint64_t* job_empty,
                                           uint64_t* full, uint64_t* empty) {
    using C = Cx<D>;
    const int lane = threadIdx.x & 31;
    const int w = (threadIdx.x >> 5) & 3;
    int jobs = 0;
    int base = 0;  // steps of the segments before
    int at = w;    // the warp's next step, of all the CTA's
    Job job;
    while (true) {
        if (w == 0) {
            if (lane == 0) lay_out_job<D>(a, smem, job_full, job_empty, ranges, jobs);
            __syncwarp();
        }
        if (!next_job<D, 32>(smem, job_full, job_empty, jobs, job)) break;
        const int steps = job.s1 - job.s0;
        const int32_t* trow = a.tables + static_cast<int64_t>(job.seq) * a.max_blocks;
        const int blocks = (job.n + 15) / 16;
        int ev = 0, ek = 0;  // E and F of the segment
        bool opened = false;
        for (; at < base + steps; at += 4) {
            const int step = job.s0 + at - base;
            // ---- its blocks (lanes 0 - 7); -1: past the end, -2: outside the pool
            int mine = -1, first = 0;
            const bool inside = lane < 8 && 8 * step + lane < blocks;
            if (inside) mine = __ldg(trow + 8 * step + lane);
            if (!opened) first = __ldg(trow + 8 * job.s0);
            if (inside && (mine < 0 || mine >= a.num_blocks)) {
                atomicOr(a.status, PKV_DEVERR_RANGE);
                mine = -2;
            }
            // an absent block's codes may be any (its tokens carry no weight): block 0 exists
            const int64_t row = static_cast<int64_t>(max(0, mine)) * a.kv_heads + job.head;
            float ks[4], vs[4];
            bool present[4], missing[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int id = __shfl_sync(0xffffffffu, mine, 2 * g + lane / 16);
                present[g] = id >= 0 && step * kChunkStep + 32 * g + lane < job.n;
                missing[g] = id == -2;
                const float* rec = a.scales + (static_cast<int64_t>(max(0, id)) * a.kv_heads + job.head) * 32 + (lane & 15);
                ks[g] = __ldg(rec);
                vs[g] = __ldg(rec + 16);
            }
            if (!opened) {
                // the scales of the segment's first block, K's in lanes 0-15 and V's in 16-31, give E and F
                opened = true;
                if (first < 0 || first >= a.num_blocks) first = 0;
                const float x = __ldg(a.scales + (static_cast<int64_t>(first) * a.kv_heads + job.head) * 32 + lane);
                const uint32_t size = __float_as_uint(job.s0 * kChunkStep + (lane & 15) < job.n ? x : 0.f) & 0x7fffffffu;
                const bool use = size < 0x7f800000u;
                ek = range_exponent(__reduce_max_sync(0xffffffffu, use && lane < 16 ? size : 0u));
                ev = max(-kMostLack, min(kMostLack, range_exponent(__reduce_max_sync(0xffffffffu, use && lane >= 16 ? size : 0u))));
            }
            const int slot = at % C::kRecords;
            if (!warp_wait(&empty[slot], (static_cast<uint32_t>(at / C::kRecords) & 1u) ^ 1u)) {
                report_timeout(a);
                return;
            }
            uint8_t* record = smem + C::kOffRecord + slot * C::kRecordBytes;
            float* tab = reinterpret_cast<float*>(smem + C::kOffTable + static_cast<uint32_t>(at) % C::kTables * C::kTableBytes);
            bool bare_k[4], bare_v[4], slow = false;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                bare_k[g] = __any_sync(0xffffffffu, present[g] && leaves_range(__float_as_uint(ks[g]) & 0x7fffffffu, ek));
                bare_v[g] = __any_sync(0xffffffffu, present[g] && leaves_range(__float_as_uint(vs[g]) & 0x7fffffffu, ev));
                slow = slow || bare_k[g] || bare_v[g] || missing[g];
                const float factor = !present[g] ? 0.f : bare_k[g] ? 1.f : ks[g] * exp2_int(-ek);
                const __half hi = __float2half(factor), lo = __float2half(factor - __half2float(hi));
                *reinterpret_cast<uint2*>(record + (32 * g + lane) * 8) = make_uint2(bits(__halves2half2(hi, hi)), bits(__halves2half2(lo, lo)));
                reinterpret_cast<__half*>(record + 1024)[32 * g + lane] =
                    __float2half(!present[g] ? 0.f : bare_v[g] ? copysignf(1.f, vs[g]) : vs[g] * exp2_int(-ev));
            }
            slow = __any_sync(0xffffffffu, slow);
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                tab[4 + 32 * g + lane] = missing[g] ? __uint_as_float(kAbsent) : bare_k[g] ? ks[g] : exp2_int(ek);
                tab[4 + 128 + 32 * g + lane] = 0.f;
            }
            if (slow) {
#pragma unroll
                for (int g = 0; g < 4; ++g)  // (-inf for a scale of zero)
                    if (bare_v[g] && present[g]) tab[4 + 128 + 32 * g + lane] = log2f(fabsf(vs[g])) - static_cast<float>(ev);
            }
            if (lane < 8) reinterpret_cast<int64_t*>(record + 1280)[lane] = row * D;
            if (lane == 0) {
                *reinterpret_cast<float4*>(tab) = make_float4(exp2_int(ev), exp2_int(ek), __uint_as_float(slow ? 1u : 0u), __int_as_float(at));
                *reinterpret_cast<int*>(record + 1344) = 1;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[slot]);
        }
        base += steps;
    }
    if (at != base) return;  // the record after the last says that there is none
    const int slot = at % C::kRecords;
    if (!warp_wait(&empty[slot], (static_cast<uint32_t>(at / C::kRecords) & 1u) ^ 1u)) {
        report_timeout(a);
        return;
    }
    if (lane == 0) {
        *reinterpret_cast<int*>(smem + C::kOffRecord + slot * C::kRecordBytes + 1344) = 0;
        mbar_arrive(&full[slot]);
    }
}

// ---------------------------------------------------------------- converters
// K's (IsV false) or V's four warps: every step of the CTA. Warp w takes tokens
// 32 w .. 32 w + 31 of a step (blocks 2 w, 2 w + 1). A lane copies the codes of the
// next step into its own slots of shared memory as it takes the current ones out of
// them (asynchronous copies: a step's time ahead, and no registers).
template <int D, bool IsV>
__device__ __forceinline__ void convert_role(const ChunkArgs& a, uint8_t* smem, uint64_t* rec_full, uint64_t* rec_empty, uint64_t* full,
                                             uint64_t* empty) {
    using C = Cx<D>;
    const int lane = threadIdx.x & 31;
    const int cw = (threadIdx.x >> 5) & 3;
    constexpr int kPerBlock = C::kVecs / 2;    // vectors of a lane in each of the warp's two blocks
    constexpr int kLanes = D / 16;             // lanes that hold one token's K row
    const uint4* codes = static_cast<const uint4*>(IsV ? a.v_codes : a.k_codes) + lane;
    uint8_t* mine = smem + C::kOffCodes + (((IsV ? 4 : 0) + cw) * C::kVecs * 32 + lane) * 16;  // vector i at + 512 i
    const uint4 *src0 = nullptr, *src1 = nullptr;  // the next step's two blocks of this warp
    int slot = 0, next_slot = 0;     // records of the step and of the next
    uint32_t parity = 0;             // of the next record
    int st = IsV ? cw >> 1 : 0;      // stage: V's of the half with this warp's tokens
    uint32_t st_parity = 1;
    bool failed = false;
    for (int it = -1;; ++it) {
        if (!warp_wait(&rec_full[next_slot], parity)) {
            failed = true;
            break;
        }
        const uint8_t* next = smem + C::kOffRecord + next_slot * C::kRecordBytes;
        const bool live = *reinterpret_cast<const int*>(next + 1344) != 0;
        if (live) {
            const longlong2 rows = *reinterpret_cast<const longlong2*>(next + 1280 + 16 * cw);
            src0 = codes + rows.x;
            src1 = codes + rows.y;
        }
        const uint8_t* record = smem + C::kOffRecord + slot * C::kRecordBytes;
        if (it < 0) {
            if (!live) return;
#pragma unroll 1
            for (int i = 0; i < C::kVecs; ++i)
                copy16_async(smem_u32(mine + 512 * i), i < kPerBlock ? src0 + 32 * i : src1 + 32 * (i - kPerBlock));
            copy_commit();
        } else {
            if (!warp_wait(&empty[st], st_parity)) {
                failed = true;
                break;
            }
            copy_wait_all();
            // Two vectors at a time, the next two on their way out of shared memory. (8
            // sequences by 512 new tokens: 425 us unrolled, rolled 444. It was the other way
            // round while the issuers' and the waits' code was twice as long: 627 and 546.)
            if (IsV) {
                // ---- coordinate rows, 64 tokens each: this warp's are 32 cw .. 32 cw + 31
                uint8_t* vd = smem + C::kOffV + st * C::kVPartBytes + lane * 128;
                const uint8_t* factors = record + 1024 + 64 * cw;
                uint4 x0 = *reinterpret_cast<const uint4*>(mine), x1 = *reinterpret_cast<const uint4*>(mine + 512);
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const uint4 f0 = *reinterpret_cast<const uint4*>(factors + 32 * b), f1 = *reinterpret_cast<const uint4*>(factors + 32 * b + 16);
                    uint8_t* c0 = vd + (((((2 * cw + b) & 3) * 2) ^ (lane & 7)) << 4);
                    uint8_t* c1 = vd + ((((((2 * cw + b) & 3) * 2) ^ (lane & 7)) << 4) ^ 16);
                    const uint4* src = b == 0 ? src0 : src1;
                    uint8_t* in = mine + 512 * kPerBlock * b;
#pragma unroll
                    for (int i = 0; i < kPerBlock; i += 2) {
                        const uint8_t* ahead = b * kPerBlock + i + 2 < C::kVecs ? in + 512 * (i + 2) : in;
                        const uint4 y0 = *reinterpret_cast<const uint4*>(ahead), y1 = *reinterpret_cast<const uint4*>(ahead + 512);
                        *reinterpret_cast<uint4*>(c0 + i * 32 * 128) = v_values(x0.x, x0.y, f0);
                        *reinterpret_cast<uint4*>(c1 + i * 32 * 128) = v_values(x0.z, x0.w, f1);
                        *reinterpret_cast<uint4*>(c0 + (i + 1) * 32 * 128) = v_values(x1.x, x1.y, f0);
                        *reinterpret_cast<uint4*>(c1 + (i + 1) * 32 * 128) = v_values(x1.z, x1.w, f1);
                        if (live) {
                            copy16_async(smem_u32(in + 512 * i), src + 32 * i);
                            copy16_async(smem_u32(in + 512 * (i + 1)), src + 32 * (i + 1));
                        }
                        x0 = y0;
                        x1 = y1;
                    }
                }
            } else {
                // ---- token rows: vector i of a lane lies in row 32 cw + i * (32 / kLanes) + lane / kLanes
                const int ch = lane % kLanes, sub = lane / kLanes;
                // lanes of the second column part take their halves in the other order: no bank is hit twice
                const int flip = ch >> 2;
                uint8_t* kd = smem + C::kOffK + st * C::kTileBytes + flip * C::kPartBytes + (32 * cw + sub) * 128;
                const int c0 = (ch & 3) * 2 + flip;
                const uint8_t* first = mine + 8 * flip;
                const uint8_t* second = mine + 8 * (flip ^ 1);
                const uint8_t* factors = record + (32 * cw + sub) * 8;
                constexpr int kRows = 32 / kLanes;  // token rows of a vector index
                struct Two {
                    uint2 x, y, f;
                };
                auto take = [&](int i) {
                    return Two{*reinterpret_cast<const uint2*>(first + 512 * i), *reinterpret_cast<const uint2*>(second + 512 * i),
                               *reinterpret_cast<const uint2*>(factors + i * kRows * 8)};
                };
                auto put = [&](int i, const Two& t) {
                    const int row8 = (i * kRows + sub) & 7;
                    uint8_t* rowp = kd + i * kRows * 128;
                    *reinterpret_cast<uint4*>(rowp + ((c0 ^ row8) << 4)) = k_values(t.x.x, t.x.y, half2_of(t.f.x), half2_of(t.f.y));
                    *reinterpret_cast<uint4*>(rowp + ((c0 ^ 1 ^ row8) << 4)) = k_values(t.y.x, t.y.y, half2_of(t.f.x), half2_of(t.f.y));
                };
                Two t0 = take(0), t1 = take(1);
#pragma unroll
                for (int i = 0; i < C::kVecs; i += 2) {
                    const int ahead = (i + 2) % C::kVecs;  // (after the last, values that are not used)
                    const Two n0 = take(ahead), n1 = take(ahead + 1);
                    put(i, t0);
                    put(i + 1, t1);
                    if (live) {
                        const uint4* src = i < kPerBlock ? src0 + 32 * i : src1 + 32 * (i - kPerBlock);
                        copy16_async(smem_u32(mine + 512 * i), src);
                        copy16_async(smem_u32(mine + 512 * (i + 1)), src + 32);
                    }
                    t0 = n0;
                    t1 = n1;
                }
            }
            copy_commit();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&full[st]);
                mbar_arrive(&rec_empty[slot]);
            }
            if (!live) break;
            st += IsV ? 2 : 1;
            if (st >= (IsV ? C::kParts : C::kStages)) {
                st -= IsV ? C::kParts : C::kStages;
                st_parity ^= 1u;
            }
        }
        slot = next_slot;
        if (++next_slot == C::kRecords) {
            next_slot = 0;
            parity ^= 1u;
        }
    }
    if (failed) report_timeout(a);
    copy_wait_all();
}

template <int D>
__global__ void __launch_bounds__(Cx<D>::kThreads, 1) chunk_q8_kernel(const ChunkArgs a) {
    using C = Cx<D>;
    extern __shared__ uint8_t smem_raw[];
    // by an offset: through an integer the compiler would lose that this is shared memory
    uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
    uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + C::kOffBars);
    uint64_t* k_empty = k_full + C::kStages;
    uint64_t* v_full = k_empty + C::kStages;
    uint64_t* v_empty = v_full + C::kParts;
    uint64_t* q_full = v_empty + C::kParts;   // [half]: Q rows in place
    uint64_t* s_full = q_full + 2;            // [half][part]: scores in tensor memory
    uint64_t* p_full = s_full + 4;            // [half][part]: weights written
    uint64_t* pv_done = p_full + 4;           // [half][part]: that product has completed
    uint64_t* final_bar = pv_done + 4;        // [issuer]: everything it issued has completed
    uint64_t* job_full = final_bar + 4;       // [slot]: segment laid out
    uint64_t* job_empty = job_full + C::kJobs;  // [slot]: read by the softmax, issuer and scale warps
    uint64_t* rec_full = job_empty + C::kJobs;  // [slot]: a step's factors laid out
    uint64_t* rec_empty = rec_full + C::kRecords;  // [slot]: read by the converters
    ChunkPos* ranges = reinterpret_cast<ChunkPos*>(smem + C::kOffPlan);  // two cuts per range
    int64_t* scratch = reinterpret_cast<int64_t*>(smem + C::kOffMisc);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc + C::kThreads / 32 * 8);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int grid = gridDim.x;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&k_full[s], 4);
            mbar_init(&k_empty[s], 2);  // both score issuers
        }
        for (int s = 0; s < C::kParts; ++s) {
            mbar_init(&v_full[s], 2);   // the two warps that hold its tokens
            mbar_init(&v_empty[s], 2);  // both value issuers
        }
        for (int x = 0; x < 2; ++x) mbar_init(&q_full[x], 4);
        for (int i = 0; i < 4; ++i) {
            mbar_init(&s_full[i], 2);  // the products' completion, and the issuer itself (it has seen the step's table)
            mbar_init(&p_full[i], 4);
            mbar_init(&pv_done[i], 1);
            mbar_init(&final_bar[i], 1);
        }
        for (int i = 0; i < C::kJobs; ++i) {
            mbar_init(&job_full[i], 1);
            mbar_init(&job_empty[i], 16);
        }
        for (int i = 0; i < C::kRecords; ++i) {
            mbar_init(&rec_full[i], 1);
            mbar_init(&rec_empty[i], 8);
        }
        fence_barrier_init();
    }
    grid_dependency_wait();  // lengths, tables, codes and the workspace may come from the kernel before
    allow_dependents();
    const ChunkShape sh = shape_of(a);
    const int count = plan_ranges<C::kThreads>(a, sh, reinterpret_cast<int64_t*>(smem + C::kOffPrefix), ranges, reinterpret_cast<int64_t*>(smem), scratch);
    PieceInfo* info = static_cast<PieceInfo*>(a.workspace) + blockIdx.x;
    if (threadIdx.x == 0) info->start = count > 0 ? ranges[2 * count - 2] : ChunkPos{a.batch, 0, 0, 0};
    if (count == 0) {  // nothing here
        if (threadIdx.x == 0) info->flags = 0;
        return;
    }
    if (threadIdx.x == 0) *reinterpret_cast<ChunkWalk*>(smem + C::kOffWalk) = chunk_begin(ranges);
    if (warp == C::kScoreWarp) {
        tmem_alloc(tmem_slot, C::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    // Registers: launched with 80 a thread, 61440 together, which 256 softmax threads at
    // 120, 256 converters at 64, 128 issuers at 40 and 128 threads for the scales at 72
    // share. The kernel for D = 128 spills nothing, that for 64 56 bytes. (A few spilled
    // words in a loop cost up to a tenth.)
    if (warp < C::kSoftmaxWarps) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 120;");
        // ------------------------------------------------ softmax: half x, query row 32 (warp % 4) + lane of it
        const int x = warp >> 2;
        const int rr = (warp & 3) * 32 + lane;
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t col_s = tmem + lane_base + C::kColS + 128 * x;
        const uint32_t col_o = tmem + lane_base + C::kColO + 128 * x;
        // A row of Q, of the output: kRowLanes lanes, 8 elements each; the warp's 32 rows
        // kRowsAtOnce at a time.
        constexpr int kRowLanes = D / 8, kRowsAtOnce = 32 / kRowLanes;
        auto row_of_lane = [&](int i) { return (warp & 3) * 32 + i * kRowsAtOnce + lane / kRowLanes; };
        auto row_slot = [&](int r, int chunk) {  // 16 bytes of row r of this half in shared memory
            return smem + C::kOffQ + x * C::kTileBytes + (chunk >> 3) * C::kPartBytes + r * 128 + (((chunk & 7) ^ (r & 7)) << 4);
        };
        int it = 0;      // steps this half has taken
        uint32_t table = 0;   // steps of the CTA
        int jobs = 0, flags = 0;
        bool ok = true;
        Job job;
        while (next_job<D, 32, true>(smem, job_full, job_empty, jobs, job)) {
            const int rows = job.rows - 128 * x;  // rows of the half, if positive
            const int steps = job.s1 - job.s0;
            if (rows <= 0) {
                table += steps;
                continue;
            }
            const int r0 = job.r0 + 128 * x;
            const bool row_ok = rr < rows;
            const int lim = row_ok ? job.before + query_of(a, r0 + rr) : -1;  // the last token the row sees
            // where the lane's row begins in q and out; rows are moved by several lanes each
            const int64_t own = row_ok ? row_of_unit(a, job.q0, job.head, r0 + rr) * D : -1;
            float row_f = 0.f;  // |scale| log2(e) over the power of two in q'
            {
                // whole rows into the warp's own slots, then a row per lane, in place (loops
                // rolled: this runs once per segment, mostly out of a cold instruction cache)
#pragma unroll 2
                for (int i = 0; i < kRowLanes; ++i) {
                    uint8_t* slot = row_slot(row_of_lane(i), lane % kRowLanes);
                    const int64_t from = __shfl_sync(0xffffffffu, own, row_of_lane(i) & 31);
                    if (from >= 0)
                        copy16_async(smem_u32(slot), static_cast<const __nv_bfloat16*>(a.q) + from + 8 * (lane % kRowLanes));
                    else
                        *reinterpret_cast<uint4*>(slot) = make_uint4(0u, 0u, 0u, 0u);
                }
                copy_commit();
                copy_wait_all();
                __syncwarp();
                // The row's largest goes to 2^14 .. 2^15 (a row with infinities is left as
                // it is); the scale's sign goes into q', a zero scale makes q' zero.
                uint32_t top = 0;
#pragma unroll 4
                for (int c = 0; c < kRowLanes; ++c) {
                    const uint4 v = *reinterpret_cast<const uint4*>(row_slot(rr, c));
                    top = __vmaxu2(top, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
                }
                const int ex = static_cast<int>(max(top >> 16, top & 0xffffu) >> 7);  // biased exponent
                const int shift = ex == 255 ? 0 : min(126, 141 - ex);                  // -113 .. 126
                const float mul = a.scale == 0.f ? 0.f : copysignf(exp2_int(shift), a.scale);
                row_f = (a.scale == 0.f ? 1.f : fabsf(a.scale)) * kLog2e * exp2_int(-shift);
#pragma unroll 2
                for (int c = 0; c < kRowLanes; ++c) {
                    uint4* slot = reinterpret_cast<uint4*>(row_slot(rr, c));
                    const uint4 v = *slot;
                    *slot = make_uint4(pack_f16x2(bf16lo_to_f32(v.x) * mul, bf16hi_to_f32(v.x) * mul),
                                       pack_f16x2(bf16lo_to_f32(v.y) * mul, bf16hi_to_f32(v.y) * mul),
                                       pack_f16x2(bf16lo_to_f32(v.z) * mul, bf16hi_to_f32(v.z) * mul),
                                       pack_f16x2(bf16lo_to_f32(v.w) * mul, bf16hi_to_f32(v.w) * mul));
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&q_full[x]);
            }
            const int warp_lim = __reduce_min_sync(0xffffffffu, lim);
            float m = ninf(), l = 0.f, unit = 1.f;
            for (int j = 0; j < steps; ++j, ++it, ++table) {
                const float* tab = reinterpret_cast<const float*>(smem + C::kOffTable + (table % C::kTables) * C::kTableBytes);
                const int seen = lim - (job.s0 + j) * kChunkStep + 1;  // tokens of the step the row sees
                const bool masked = (job.s0 + j) * kChunkStep + kChunkStep - 1 > warp_lim;
#pragma unroll 1
                for (int part = 0; part < 2; ++part) {
                    if (!warp_wait(&s_full[2 * x + part], it & 1)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const float4 modes = *reinterpret_cast<const float4*>(tab);
                    unit = modes.x;
                    // never 0 or infinite: a hidden score is -inf times it
                    const float f = fminf(fmaxf(row_f * modes.y, 1.2e-38f), 3e38f);
                    const int seen_part = seen - 64 * part;
                    const uint32_t col = col_s + 64 * part;
                    // Weights with the maximum as it stands: their sum tells whether it has to
                    // move (no pass over the scores for it; then, and in slow steps, the part
                    // is done with care, 16 tokens at a time).
                    bool careful = __float_as_uint(modes.z) != 0u;
                    if (!careful) {
                        if (__any_sync(0xffffffffu, m == ninf() && seen_part > 0)) {
                            // rows without a maximum (and so without weights yet): theirs is the part's
                            float mx = ninf(), second = ninf();
#pragma unroll 1
                            for (int c = 0; c < 64; c += 16) {
                                uint32_t v[16];
                                float group = ninf();
                                tmem_ld16(col + c, v);
                                tmem_ld_wait();
#pragma unroll
                                for (int e = 0; e < 16; ++e) group = e < seen_part - c ? fmaxf(group, __uint_as_float(v[e])) : group;
                                second = fmaxf(second, fminf(mx, group));
                                mx = fmaxf(mx, group);
                            }
                            if (m == ninf()) m = fmaxf(second * f, mx * f - kHeadroom);
                        }
                        uint32_t sv[32], pw[32];
                        const float base = m == ninf() ? 0.f : m;
                        const uint64_t nb2 = f32x2_pack(-base, -base), f2 = f32x2_pack(f, f);
                        uint64_t acc0 = f32x2_pack(0.f, 0.f), acc1 = acc0;
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            tmem_ld32(col + 32 * half, sv);
                            tmem_ld_wait();
                            if (masked) {
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    if (e >= seen_part - 32 * half) sv[e] = 0xff800000u;
                            }
#pragma unroll
                            for (int e = 0; e < 32; e += 2) {
                                float a0, a1;
                                f32x2_unpack(f32x2_fma(f32x2_pack(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1])), f2, nb2), a0, a1);
                                const float p0 = ex2(a0), p1 = ex2(a1);
                                pw[16 * half + e / 2] = pack_f16x2(p0, p1);
                                if ((e / 2) & 1)
                                    acc1 = f32x2_add(acc1, f32x2_pack(p0, p1));
                                else
                                    acc0 = f32x2_add(acc0, f32x2_pack(p0, p1));
                            }
                        }
                        float s0, s1;
                        f32x2_unpack(f32x2_add(acc0, acc1), s0, s1);
                        const float sum = s0 + s1;
                        // above it (or not a number) a weight may have left f16
                        careful = __any_sync(0xffffffffu, !(sum <= kMostSum));
                        if (!careful) {
                            l += sum;
                            tmem_st32(col, pw);
                        }
                    }
                    if (careful) {
                        const float* cp = tab + 4 + 64 * part;
                        float mx = ninf(), second = m;
#pragma unroll 1
                        for (int c = 0; c < 64; c += 16) {
                            float xe[16], group = ninf();
                            careful_scores(col + c, cp + c, row_f, seen_part - c, xe);
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                group = fmaxf(group, xe[e] == ninf() ? ninf() : xe[e] + fmaxf(cp[128 + c + e], kLeastLack));
                            second = fmaxf(second, fminf(mx, group));
                            mx = fmaxf(mx, group);
                        }
                        if (__any_sync(0xffffffffu, mx > m + kHeadroom)) {
                            float alpha = 1.f;
                            if (mx > m + kHeadroom) {
                                const float to = fmaxf(second, mx - kHeadroom);
                                alpha = m == ninf() ? 0.f : ex2(m - to);
                                m = to;
                                l *= alpha;
                            }
                            // O holds something once a part of this segment has been multiplied in:
                            // the last one is the other part, of this step or of the one before
                            if (j + part > 0) {
                                if (!warp_wait(&pv_done[2 * x + (part ^ 1)], (it - 1 + part) & 1)) {
                                    ok = false;
                                    break;
                                }
                                tc_fence_after();
#pragma unroll 1
                                for (int c = 0; c < D; c += 16) {
                                    uint32_t ov[16];
                                    tmem_ld16(col_o + c, ov);
                                    tmem_ld_wait();
#pragma unroll
                                    for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
                                    tmem_st16(col_o + c, ov);
                                }
                            }
                        }
                        const float base = m == ninf() ? 0.f : m;
                        // the weights overwrite scores that have been read
#pragma unroll 1
                        for (int c = 0; c < 64; c += 16) {
                            float xe[16];
                            careful_scores(col + c, cp + c, row_f, seen_part - c, xe);
                            uint32_t pw[8];
#pragma unroll
                            for (int e = 0; e < 16; e += 2) {
                                float w[2];
#pragma unroll
                                for (int u = 0; u < 2; ++u) {
                                    const float xu = xe[e + u], lack = cp[128 + c + e + u];
                                    w[u] = xu == ninf() ? 0.f : ex2(xu + lack - base);
                                    l += xu == ninf() ? 0.f : lack == 0.f ? w[u] : ex2(xu - base);
                                }
                                pw[e / 2] = pack_f16x2(w[0], w[1]);
                            }
                            tmem_st8(col + c / 2, pw);
                        }
                    }
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&p_full[2 * x + part]);
                }
                if (!ok) break;
            }
            if (!ok) break;
            // the products of the last step (part 1 completes after part 0)
            if (!warp_wait(&pv_done[2 * x + 1], (it - 1) & 1)) {
                ok = false;
                break;
            }
            tc_fence_after();
            if (job.piece == 0) {
                // through the shared memory of this warp's rows of Q, which the scores no longer need
                const float inv = l == 0.f ? 0.f : unit / l;
#pragma unroll 1
                for (int c = 0; c < D; c += 16) {
                    uint32_t ov[16];
                    tmem_ld16(col_o + c, ov);
                    tmem_ld_wait();
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            w[e] = pack_bf16x2(__uint_as_float(ov[8 * u + 2 * e]) * inv, __uint_as_float(ov[8 * u + 2 * e + 1]) * inv);
                        *reinterpret_cast<uint4*>(row_slot(rr, c / 8 + u)) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                __syncwarp();
#pragma unroll 2
                for (int i = 0; i < kRowLanes; ++i) {
                    const int64_t to = __shfl_sync(0xffffffffu, own, row_of_lane(i) & 31);
                    if (to >= 0)
                        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + to + 8 * (lane % kRowLanes)) =
                            *reinterpret_cast<const uint4*>(row_slot(row_of_lane(i), lane % kRowLanes));
                }
                __syncwarp();
            } else {
                flags |= job.piece;
                float* piece = slot_of(a.workspace, grid, D, blockIdx.x, job.piece - 1);
#pragma unroll 1
                for (int c = 0; c < D; c += 16) {
                    uint32_t ov[16];
                    tmem_ld16(col_o + c, ov);
                    tmem_ld_wait();
                    if (row_ok) {
#pragma unroll
                        for (int e = 0; e < 16; e += 4)
                            *reinterpret_cast<float4*>(piece + (c + e) * kChunkRows + 4 * (128 * x + rr)) =
                                make_float4(__uint_as_float(ov[e]) * unit, __uint_as_float(ov[e + 1]) * unit,
                                            __uint_as_float(ov[e + 2]) * unit, __uint_as_float(ov[e + 3]) * unit);
                    }
                }
                if (row_ok) {
                    piece[kChunkRows * D + 128 * x + rr] = m;
                    // (finite, or the joining would take 0 times it where the piece has no weight)
                    piece[kChunkRows * (D + 1) + 128 * x + rr] = fminf(l, 3e38f);
                }
            }
            tc_fence_before();  // the next segment's products overwrite O after this half's next arrival
        }
        if (threadIdx.x == 0) info->flags = ok ? flags : 0;  // half A takes part in every segment
        if (!ok || job.s1 != 0) report_timeout(a);
    } else if (warp < C::kScoreWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        if (warp < C::kConvertWarp + 4)
            convert_role<D, false>(a, smem, rec_full, rec_empty, k_full, k_empty);
        else
            convert_role<D, true>(a, smem, rec_full, rec_empty, v_full, v_empty);
    } else if (warp >= C::kScaleWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        scale_role<D>(a, smem, count, job_full, job_empty, rec_full, rec_empty);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        const int x = warp & 1;
        if (warp < C::kValueWarp) {
            // -------------------------------------------- scores S = Q K^T of half x (one thread)
            if (elect_one()) {
                constexpr uint32_t idS = umma_idesc_f16(128, 64);
                const uint64_t q_desc = umma_desc_sw128(smem_u32(smem + C::kOffQ + x * C::kTileBytes), 16, 1024);
                const uint64_t k_desc = umma_desc_sw128(smem_u32(smem + C::kOffK), 16, 1024);
                int step = 0, it = 0, segs = 0, jobs = 0;
                bool ok = true;
                Job job;
                while (ok && next_job<D, 1>(smem, job_full, job_empty, jobs, job)) {
                    const bool mine = job.rows > 128 * x;
                    if (mine) {
                        ok = wait(&q_full[x], segs & 1);
                        ++segs;
                    }
                    for (int j = job.s0; ok && j < job.s1; ++j, ++step) {
                        const int st = step & 1;
                        if (!wait(&k_full[st], (step >> 1) & 1)) {
                            ok = false;
                            break;
                        }
                        if (!mine) {
                            mbar_arrive(&k_empty[st]);
                            continue;
                        }
#pragma unroll 1
                        for (int part = 0; part < 2; ++part) {
                            // the part's weights of the step before lie over its scores
                            if (it > 0 && !wait(&pv_done[2 * x + part], (it - 1) & 1)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
                            const uint64_t kd = k_desc + ((st * C::kTileBytes + part * 64 * 128) >> 4);
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk) {
                                const uint32_t off = (kk >> 2) * C::kPartBytes + (kk & 3) * 32;
                                umma_bf16(tmem + C::kColS + 128 * x + 64 * part, q_desc + (off >> 4), kd + (off >> 4), idS, kk > 0 ? 1u : 0u);
                            }
                            if (part == 1) umma_commit(&k_empty[st]);
                            umma_commit(&s_full[2 * x + part]);
                            mbar_arrive(&s_full[2 * x + part]);
                        }
                        ++it;
                    }
                }
                umma_commit(&final_bar[x]);
                if (!wait(&final_bar[x], 0) || !ok || job.s1 != 0) report_timeout(a);
            }
        } else {
            // -------------------------------------------- values O += P V of half x (one thread)
            if (elect_one()) {
                constexpr uint32_t idO = umma_idesc_f16(128, D);
                const uint64_t v_desc = umma_desc_sw128(smem_u32(smem + C::kOffV), 16, 1024);
                int st = 0, it = 0, jobs = 0;
                uint32_t phase = 0;
                bool ok = true;
                Job job;
                while (ok && next_job<D, 1>(smem, job_full, job_empty, jobs, job)) {
                    const bool mine = job.rows > 128 * x;
                    for (int j = job.s0; ok && j < job.s1; ++j) {
#pragma unroll 1
                        for (int part = 0; part < 2; ++part) {
                            const int now = st;
                            const uint32_t parity = phase;
                            if (++st == C::kParts) {
                                st = 0;
                                phase ^= 1u;
                            }
                            if (!wait(&v_full[now], parity)) {
                                ok = false;
                                break;
                            }
                            if (!mine) {
                                mbar_arrive(&v_empty[now]);
                                continue;
                            }
                            if (!wait(&p_full[2 * x + part], it & 1)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
                            const uint64_t vd = v_desc + (now * C::kVPartBytes >> 4);
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                umma_bf16_ts(tmem + C::kColO + 128 * x, tmem + C::kColS + 128 * x + 64 * part + 8 * kk,
                                             vd + 2 * kk, idO,
                                             (j > job.s0 || part > 0 || kk > 0) ? 1u : 0u);
                            umma_commit(&pv_done[2 * x + part]);
                            umma_commit(&v_empty[now]);
                        }
                        if (mine) ++it;
                    }
                }
                umma_commit(&final_bar[2 + x]);
                if (!wait(&final_bar[2 + x], 0) || !ok || job.s1 != 0) report_timeout(a);
            }
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == C::kScoreWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

// ---------------------------------------------------------------- joining the pieces of cut units
// CTA (c, y): the unit that begins in CTA c's range and is cut at its end (slot 1
// of c, then slot 0 of the following CTAs while they begin inside it), columns
// 8 y .. 8 y + 7, a thread per row: out = sum_i O_i 2^(m_i - M) / sum_i l_i 2^(m_i - M).
template <int D>
__global__ void __launch_bounds__(kChunkRows) combine_kernel(const ChunkArgs a, int grid) {
    __shared__ int pieces[kMaxPieces];  // 2 cta + slot
    __shared__ int count;
    grid_dependency_wait();
    allow_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = blockIdx.x;
    const PieceInfo* infos = static_cast<const PieceInfo*>(a.workspace);
    if (c + 1 >= grid || !(infos[c].flags & 2)) return;
    const ChunkPos unit = infos[c + 1].start;
    if (warp == 0) {
        int n = 1;
        if (lane == 0) pieces[0] = 2 * c + 1;
        for (int k0 = c + 1; k0 < grid; k0 += 32) {
            const int k = k0 + lane;
            const bool in = k < grid && infos[k].start.same_unit(unit) && infos[k].start.s > 0;
            const unsigned int inside = __ballot_sync(0xffffffffu, in);
            const int run = __ffs(~inside) - 1;  // leading CTAs that begin inside the unit (-1: all 32)
            const bool use = in && (run < 0 || lane < run) && (infos[k].flags & 1);
            const unsigned int used = __ballot_sync(0xffffffffu, use);
            const int at = n + __popc(used & ((1u << lane) - 1u));
            if (use && at < kMaxPieces) pieces[at] = 2 * k;
            n += __popc(used);
            if (run >= 0) break;
        }
        if (lane == 0) count = min(n, kMaxPieces);
    }
    const ChunkShape sh = shape_of(a);
    ChunkSeq q;
    chunk_seq(sh, unit.seq, q);
    __syncthreads();
    const int r = threadIdx.x, R = unit.tile * kChunkRows + r;
    if (R >= q.nq * a.group) return;
    float top = ninf();
#pragma unroll 4
    for (int i = 0; i < count; ++i) top = fmaxf(top, slot_of(a.workspace, grid, D, pieces[i] >> 1, pieces[i] & 1)[kChunkRows * D + r]);
    const float base = top == ninf() ? 0.f : top;
    float l = 0.f, acc[8] = {};
#pragma unroll 2
    for (int i = 0; i < count; ++i) {
        const float* p = slot_of(a.workspace, grid, D, pieces[i] >> 1, pieces[i] & 1);
        const float4 o0 = *reinterpret_cast<const float4*>(p + (8 * blockIdx.y * kChunkRows + 4 * r));
        const float4 o1 = *reinterpret_cast<const float4*>(p + ((8 * blockIdx.y + 4) * kChunkRows + 4 * r));
        const float w = ex2(p[kChunkRows * D + r] - base);
        l += w * p[kChunkRows * (D + 1) + r];
        acc[0] += w * o0.x, acc[1] += w * o0.y, acc[2] += w * o0.z, acc[3] += w * o0.w;
        acc[4] += w * o1.x, acc[5] += w * o1.y, acc[6] += w * o1.z, acc[7] += w * o1.w;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int64_t row = row_of_unit(a, q.q0, unit.head, R);
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + row * D + 8 * blockIdx.y) =
        make_uint4(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv),
                   pack_bf16x2(acc[4] * inv, acc[5] * inv), pack_bf16x2(acc[6] * inv, acc[7] * inv));
}

// CTAs of a launch: one per SM (piece lists hold at most kMaxPieces).
int chunk_q8_ctas() { return device_sm_count() < kMaxPieces ? device_sm_count() : kMaxPieces; }

template <int D>
cudaError_t run_chunk(const ChunkArgs& a, cudaStream_t s) {
    const int grid = chunk_q8_ctas();
    cudaError_t e = cudaFuncSetAttribute(chunk_q8_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(Cx<D>::kSmem));
    if (e != cudaSuccess) return e;
    e = launch_pdl(chunk_q8_kernel<D>, dim3(grid), dim3(Cx<D>::kThreads), Cx<D>::kSmem, s, a);
    // a unit of three steps is never cut: tables that hold no more leave nothing to join
    if (e != cudaSuccess || a.max_blocks * 16 < 2 * kMinPiece * kChunkStep - kChunkStep + 1) return e;
    return launch_pdl(combine_kernel<D>, dim3(grid, D / 8), dim3(kChunkRows), 0, s, a, grid);
}

}  // namespace

size_t chunk_q8_workspace_bytes(int head_dim) {
    const int grid = chunk_q8_ctas();
    return infos_bytes(grid) + static_cast<size_t>(grid) * 2 * slot_floats(head_dim) * sizeof(float);
}

cudaError_t launch_chunk_q8(const ChunkArgs& a, cudaStream_t s) {
    return a.head_dim == 128 ? run_chunk<128>(a, s) : run_chunk<64>(a, s);
}

}  // namespace pkv
