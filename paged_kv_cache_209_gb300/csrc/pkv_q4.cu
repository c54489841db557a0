// Attention over the 4-bit cache, few query rows per (sequence, KV head)
// (pkv_decode_attention_q4, and pkv_multiquery_attention_q4 up to kMq4Rows rows; more
// rows run in tiles, pkv_chunk_q8.cu).
//
// Work: (sequence, KV head, block) units split over the CTAs by cost (pkv_schedule.cuh);
// a segment that a cut divides leaves pieces, which the last CTA to finish one merges.
// Bound by HBM: a unit is one record of 16 D + 128 bytes, read once.
//
// A record is contiguous, so a producer warp fetches each with one bulk copy into a ring
// of stages of two records (32 tokens); the query rows of a segment come the same way,
// ahead of its first records. Four consumer warps take stages in turn. Per stage, with
// the query rows of a (sequence, KV head) in tiles of 8:
//     S^T[16 tokens][8 rows] = K[16][D] Q^T[D][8]     (mma m16n8k16, bf16 -> fp32)
//     x = log2(e) scale S k_p,  P' = 2^(x - m) v_p,  l += 2^(x - m)
//     O^T[D][8] += V^T[D][16] P'^T[16][8]             (f16 -> fp32)
// k_p and v_p are the tokens' scales; m is a base, not a maximum, moved only where a P'
// would leave f16 (below).
//
// Codes become operands by one mask: a nibble n (code + 8) alone in the low bits of a bf16
// is n 2^-133, of an f16 n 2^-24, four bits higher 16 times that (in bf16 its top bit is the
// exponent's lowest, whose two ranges share their step). For K the 8 stays: S = 2^133 S' - 8
// sum(q), q's halves over 16 where the codes are 16-fold. For V it goes, by one subtraction
// per 256 tokens, because O runs over the whole context, where the sum of the eights would
// take the low bits of the rest. q rows are scaled by a power of two to a largest magnitude of
// 2^126 .. 2^127; sums are fp32.
//
// The products of such small operands are exact, but their sum is not: the 16 of an
// instruction are lined up by exponents that take an operand below the normal range for one
// at its end, and what lies 23 bits or more below the largest is cut. So a product with a code
// loses what is below 2^-18 of the largest q of its 16 dimensions (bf16, whose low bits are 7
// below the range's end; with f16's 10, which q would fit as well, 2^-15), and below 2^-15 of the
// largest P' of its 16 tokens (P' needs f16's bits). Four bits higher it is 16 times less; the
// eights are summed in both places for that.
//
// Three CTAs an SM of four consumer warps (two with two row tiles a warp, for the
// registers), each with a ring of eight stages, 35 KB: what one CTA of twelve consumers
// with one ring of the same size takes is 61 to 66 us against 56 (one producer, and stages
// that free up in order). With two row tiles 7 to 11 consumers an SM, rings of 12 and 16
// stages and two blocks at a time are all within 4 us of the 85.5.
//
// Measured, 32 query heads on 8 of 128, in a captured graph: 32 sequences of 8192 tokens 56.5
// us, 5.07 TB/s of records (the copy rate is 6.78); per token more 43.5 us for 8192, 6.57
// TB/s: the rest is the way to the first records (5 us), the CTAs of an SM ending up to 8 us
// apart, and joining the pieces (3 us). 32 of 131072 692 to 701 us, 6.5 TB/s; one of them 36.8. Two queries
// a sequence take the same; four 86.7 us, 3.3 TB/s, out of L2 as out of HBM: with two row tiles a
// warp there are two warps a scheduler, and one issues every 4.9 cycles (2.0 of them waiting on
// the instruction before, 0.7 on loads, 0.8 for its turn or an instruction), 300 times a block of
// which it takes 108: 81 us. No unit is full (issue slots 41 %, tensor pipe and ALU 37 %). Eight 154. 64 ragged contexts of up
// to 8191 tokens, 24 heads: 38.5 us, 3.6 TB/s. One of 1000 tokens: 9.1 us, all of it latency.
#include <math.h>
#include <mutex>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_q4.cuh"
#include "pkv_schedule.cuh"

namespace pkv {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kConsumers = 4;
constexpr int kThreads = (kConsumers + 1) * 32;
constexpr int kIssueLanes = 8;  // stages whose copies are issued together
// Cost of a segment shorter than kShortBlocks beside its blocks, in blocks, where there are
// blocks enough for every CTA (64 contexts of 1 to 8191 tokens: 38.5 us, 45.4 without; 40 of up to 6000
// with four queries 34.8, 35.9 with 16 and 38 with 12; 256 of up to 16384 231.4, 234 with 28; many equal
// short ones, which are not exempted, lose by it, 256 of 100 tokens 33.5 against 30.8, being cut more rarely).
constexpr int kSegmentCost = 20, kShortBlocks = 256;
// Where there are not, a CTA gets about this many blocks: of contexts of one length (one of 1000 tokens 9.1
// us; 9.3 with 8, 11.6 with 2, 9.6 with 24; 14 of 700 10.7, 14.0 with 8; 9 of 700 with four queries 13.7
// and 20; but 4 of 700 10.1 and 9.5, which no rule here tells from them), and of others (14 of up to 1100 19.0 us, 25.5 with 12) or where two
// warps share a block (one of 1024 tokens with eight queries 15.7, 17.4 with 12).
constexpr int kLeastAlike = 12, kLeastBlocks = 8;

// The base m of a row: where some P' = 2^(x - m) v would leave f16 it moves to the largest
// x + log2 |v| less kHeadroom, so that what is rounded to f16 lies high in its range for
// the tokens that make up the output, whatever the scales. A V scale counts as
// kTinyScale at least, so that l stays below 2^(16 + 96) times the tokens.
constexpr float kHeadroom = 8.f;
constexpr float kMostSum = 5.1922969e33f;        // 2^112
constexpr float kTinyScale = 1.2621774e-29f;     // 2^-96
// Stages (32 tokens) whose eights are summed in O before they are taken out again.
constexpr int kFold = 8;
constexpr int kMergeAhead = 8;  // pieces whose loads a merge has in flight
constexpr float kUnset = -3.0e38f;               // base of a row that has seen no token

// A piece of a segment, as the producer lays it out for the consumers.
struct __align__(16) Piece4 {
    int seq, head, q0, rows;        // rows: query rows of the segment, (query, head) pairs
    int n, nq, blk_from, blk_to;    // tokens and queries of the sequence; the piece's blocks (blk_to 0: no more pieces)
    int cut;                        // 0: the whole segment; else the workspace slot of the piece, plus 1
    int first_cta, pieces, slot0;   // (cut ones, at the end) where the segment's pieces lie: that CTA's slot slot0, then slot 0
                                    // of the following CTAs
};
static_assert(sizeof(Piece4) == 48, "layout");

// D: head_dim, R: tiles of 8 query rows of a warp.
template <int D, int R>
struct M4 {
    static constexpr int kRecord = q4_record_bytes(D);
    static constexpr int kStageBytes = 2 * kRecord;
    static constexpr int kCtas = R == 1 ? 3 : 2;              // an SM's, at 128 and 168 registers a thread
    static constexpr int kStages = D == 128 ? 8 : 16;
    // A stage always meets the same warp (one that ran ahead of the copies into another's stage would take the
    // parity of the round before for its own), and stages issued together are different ones.
    static_assert(kStages % kConsumers == 0 && kStages >= kIssueLanes, "ring");
    static constexpr int kRows = 8 * R;                       // query rows of a warp
    static constexpr int kQSlots = R == 1 ? 4 : 2;            // segments whose query rows are in work or on their way
    static constexpr int kStateFloats = kRows * (D + 2);      // a warp's O, m and l
    static constexpr int kOffBars = kStages * kStageBytes;    // full, empty per stage; q_full, q_empty per slot; state_full, state_empty
    static constexpr int kNumBars = 2 * kStages + 2 * kQSlots + 2;
    static constexpr int kOffFlags = kOffBars + (kNumBars + 1) / 2 * 16;  // per stage: which of its blocks exist; abort
    static constexpr int kOffState = (kOffFlags + (kStages + 1) * 4 + 15) / 16 * 16;
    static constexpr int kOffPieces = kOffState + kConsumers * kStateFloats * 4;  // per slot; then the cut ones, and their number
    static constexpr int kOffQ = kOffPieces + (kQSlots + 2) * sizeof(Piece4) + 16;
    static size_t smem_bytes(int warps_per_unit, int batch) {
        return 128 + kOffQ + kQSlots * kRows * warps_per_unit * D * 2 + (3 * static_cast<size_t>(batch) + 2) * 4;
    }
    static size_t most_smem_bytes() { return smem_bytes(R, kMaxBatchPerLaunch); }  // (warps_per_unit is at most R)
    static_assert(kOffBars % 16 == 0 && kOffQ % 16 == 0, "alignment");
};

// Bulk copy of `bytes` contiguous bytes (a multiple of 16) into shared memory, counted on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// Adds to a counter, ordered after what the warp has written and before what it reads next.
__device__ __forceinline__ int add_acq_rel(int* p, int v) {
    int old;
    asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
    return old;
}
// D = A B + C for bf16 A (16 x 16) and B (16 x 8), C and D apart.
__device__ __forceinline__ void mma_bf16_from(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1,
                                             float c0, float c1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %10, %11};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
}
// Larger, half by half, of a (not negative) and b's magnitude; a NaN stays.
__device__ __forceinline__ uint32_t larger_f16x2(uint32_t a, uint32_t b) {
    const __half2 r = __hmax2_nan(*reinterpret_cast<const __half2*>(&a), __habs2(*reinterpret_cast<const __half2*>(&b)));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// Workspace of one piece: per row tile O [8][D], then per consumer warp (each merges D / 4
// dimensions on its own) the rows' m [8] and l [8].
__host__ __device__ constexpr int piece_floats(int d) { return 8 * d + 4 * 16; }
__device__ __forceinline__ float* piece_of(const Q4Args& a, int d, int cta, int slot, int tile) {
    return a.partials + static_cast<long long>((cta * 2 + slot) * a.tiles + tile) * piece_floats(d);
}

// D / 16 values of row `rr` of a segment, dimensions d0 .., as bf16.
template <int D>
__device__ __forceinline__ void write_part(const Q4Args& a, int q0, int head, int rr, int d0, const float (&o)[D / 16], float l) {
    const int t = rr / a.group;
    const float inv = l == 0.f ? 0.f : 1.f / l;  // (a NaN, of a token that the row sees, stays)
    __nv_bfloat16* row = static_cast<__nv_bfloat16*>(a.out) +
                         ((static_cast<long long>(q0) + t) * a.q_heads + head * a.group + (rr - t * a.group)) * D + d0;
#pragma unroll
    for (int e = 0; e < D / 16; e += 4)
        *reinterpret_cast<uint2*>(row + e) = make_uint2(pack_bf16x2(o[e] * inv, o[e + 1] * inv), pack_bf16x2(o[e + 2] * inv, o[e + 3] * inv));
}

template <int D, int R>
__global__ void __launch_bounds__(kThreads, M4<D, R>::kCtas) mq4_kernel(const Q4Args a) {
    using C = M4<D, R>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 127u);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBars);
    uint64_t* empty = full + C::kStages;
    uint64_t* q_full = empty + C::kStages;
    uint64_t* q_empty = q_full + C::kQSlots;
    uint64_t* state_full = q_empty + C::kQSlots;  // every consumer warp has published its state of the piece
    uint64_t* state_empty = state_full + 1;    // and every one has taken its share of them
    int* present = reinterpret_cast<int*>(smem + C::kOffFlags);
    volatile int* abort_flag = present + C::kStages;
    float* state = reinterpret_cast<float*>(smem + C::kOffState);
    Piece4* slots = reinterpret_cast<Piece4*>(smem + C::kOffPieces);
    Piece4* cuts = slots + C::kQSlots;
    int* num_cuts = reinterpret_cast<int*>(cuts + 2);
    const int W = a.warps_per_unit, UL = kConsumers / W;  // unit lanes: stages in work at a time
    const int q_bytes = C::kRows * W * D * 2;
    uint8_t* q_rows = smem + C::kOffQ;
    int32_t* s_pre = reinterpret_cast<int32_t*>(q_rows + C::kQSlots * q_bytes);  // blocks, cost up to and with each sequence; length
    int32_t* s_cost = s_pre + a.batch;
    int32_t* s_len = s_cost + a.batch;
    int32_t* s_active = s_len + a.batch;  // sequences with blocks
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = a.group;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], W);
        }
        for (int s = 0; s < C::kQSlots; ++s) {
            mbar_init(&q_full[s], 1);
            mbar_init(&q_empty[s], kConsumers);
        }
        mbar_init(state_full, kConsumers);
        mbar_init(state_empty, kConsumers);
        *abort_flag = 0;
        fence_barrier_init();
    }
    grid_dependency_wait();
    allow_dependents();
    const int cap = a.max_blocks * 16;
    for (int i = threadIdx.x; i < a.batch; i += kThreads) {
        int n = a.lens[i];
        bool bad = n < 0 || n > cap;
        n = n < 0 ? 0 : (n > cap ? cap : n);
        // without query offsets: one query per sequence (row i), none for an empty context
        const int q0 = a.qstart != nullptr ? a.qstart[i] : i;
        long long nq = a.qstart != nullptr ? static_cast<long long>(a.qstart[i + 1]) - q0 : (n > 0 ? 1 : 0);
        if (q0 < 0 || nq < 0 || nq > n || nq > a.max_query_len) {
            bad = true;
            nq = 0;
        }
        if (bad) {
            if (blockIdx.x == 0) atomicOr(a.status, PKV_DEVERR_RANGE);
            if (a.qstart != nullptr) nq = 0;  // a malformed sequence has no queries
        }
        s_len[i] = n;
        s_pre[i] = nq > 0 ? (n + 15) >> 4 : 0;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        int blocks = 0, cost = 0, active = 0, longest = 0;
        for (int base = 0; base < a.batch; base += 32) {
            int x = base + lane < a.batch ? s_pre[base + lane] : 0;
            int y = x > 0 && x < kShortBlocks ? x + kSegmentCost : x;
            active += __popc(__ballot_sync(0xffffffffu, x > 0));
            longest = max(longest, x);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x1 = __shfl_up_sync(0xffffffffu, x, o), y1 = __shfl_up_sync(0xffffffffu, y, o);
                if (lane >= o) x += x1, y += y1;
            }
            if (base + lane < a.batch) {
                s_pre[base + lane] = x + blocks;
                s_cost[base + lane] = y + cost;
            }
            blocks += __shfl_sync(0xffffffffu, x, 31);
            cost += __shfl_sync(0xffffffffu, y, 31);
        }
        longest = __reduce_max_sync(0xffffffffu, longest);
        if (lane == 0) s_active[0] = active, s_active[1] = longest;
    }
    __syncthreads();
    if (a.qstart == nullptr) {
        // one query per sequence: an empty context gives a zero row
        const int vecs = a.q_heads * D / 8;
        for (int i = blockIdx.x; i < a.batch; i += gridDim.x) {
            if (s_len[i] != 0) continue;
            uint4* o = static_cast<uint4*>(a.out) + static_cast<long long>(i) * vecs;
            for (int e = threadIdx.x; e < vecs; e += kThreads) o[e] = make_uint4(0u, 0u, 0u, 0u);
        }
    }
    const long long U = static_cast<long long>(a.kv_heads) * s_pre[a.batch - 1];
    if (U == 0) return;
    const int cta = blockIdx.x;
    // Few blocks: fewer CTAs, as many for each segment, whose cuts then fall between segments of one
    // length (a CTA with two pieces takes them one after the other). (No range is empty, so a segment's
    // pieces lie in consecutive CTAs.)
    const bool alike = W == 1 && static_cast<long long>(s_active[0]) * s_active[1] == s_pre[a.batch - 1];
    // (two divisions by constants: one by either is a loop)
    long long ctas = alike ? U / kLeastAlike : U / kLeastBlocks;
    const bool few = ctas < gridDim.x;
    if (few) {
        const long long segments = static_cast<long long>(a.kv_heads) * s_active[0];
        ctas = ctas < 1 ? 1 : ctas >= segments ? ctas / segments * segments : ctas;
    } else {
        ctas = gridDim.x;
    }
    const bool weighted = !few && static_cast<long long>(a.kv_heads) * s_cost[a.batch - 1] >= ctas * (1 + kSegmentCost);
    if (cta >= ctas) return;

    if (warp == kConsumers) {
        // ------------------------------------------------ producer
        const uint64_t policy = l2_evict_first_policy(), q_policy = l2_evict_last_policy();
        const uint8_t* cache = static_cast<const uint8_t*>(a.cache);
        const long long block_bytes = static_cast<long long>(a.kv_heads) * C::kRecord;
        CostSplit split;
        split.init(s_pre, weighted ? s_cost : s_pre, a.batch, a.kv_heads, weighted ? 1 + kSegmentCost : 1, ctas);
        Walker wk;
        wk.init(s_pre, a.batch, a.kv_heads, split.start(cta), split.start(cta + 1));
        uint32_t k = 0;  // stages issued
        uint32_t pieces = 0;
        int ncut = 0;
        Piece pc;
        bool ok = true;
        while (ok) {
            const bool more = wk.next(pc);
            const int32_t* trow = a.tables + static_cast<long long>(pc.seq) * a.max_blocks + pc.blk_from;
            const int blocks = more ? pc.blk_to - pc.blk_from : 0;
            const uint8_t* head = cache + static_cast<long long>(pc.head) * C::kRecord;
            int cur = lane < blocks ? __ldg(trow + lane) : 0;
            const int slot = pieces % C::kQSlots;
            if (lane == 0 && pieces >= C::kQSlots) ok = mbar_wait(&q_empty[slot], (pieces / C::kQSlots - 1) & 1, a.status, abort_flag);
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            if (!more) {
                if (lane == 0) {
                    slots[slot].blk_to = 0;
                    *num_cuts = ncut;
                    mbar_arrive(&q_full[slot]);
                }
                break;
            }
            const int q0 = a.qstart != nullptr ? a.qstart[pc.seq] : pc.seq;
            const int nq = a.qstart != nullptr ? a.qstart[pc.seq + 1] - q0 : 1;
            if (lane == 0) {
                Piece4 p{pc.seq, pc.head, q0, nq * G, s_len[pc.seq], nq, pc.blk_from, pc.blk_to, 0, 0, 0, 0};
                if (!pc.complete) {
                    p.cut = pc.first ? 1 : 2;
                    cuts[ncut] = p;
                }
                slots[slot] = p;
                mbar_arrive_expect_tx(&q_full[slot], nq * G * D * 2);
            }
            __syncwarp();
            if (lane < nq)  // G rows of each query are contiguous
                bulk_load(q_rows + slot * q_bytes + lane * G * D * 2,
                          static_cast<const __nv_bfloat16*>(a.q) + ((static_cast<long long>(q0) + lane) * a.q_heads + pc.head * G) * D, G * D * 2,
                          &q_full[slot], q_policy);
            ++pieces;
            for (int b0 = 0; ok && b0 < blocks; b0 += 32) {
                const int nidx = b0 + 32 + lane;
                const int nxt = nidx < blocks ? __ldg(trow + nidx) : 0;
                const int stages = (min(32, blocks - b0) + 1) / 2;
                // in order, as many stages at once as are free from the first on, one a lane
                for (int e0 = 0; e0 < stages;) {
                    const int e = e0 + lane;
                    const uint32_t kk = k + lane;
                    const int s = static_cast<int>(kk % C::kStages);
                    const uint32_t par = ((kk / C::kStages) & 1) ^ 1u;
                    const bool probe = lane < kIssueLanes && e < stages && mbar_test_wait(&empty[s], par);
                    int n = __ffs(~__ballot_sync(0xffffffffu, probe)) - 1;
                    if (n == 0) {
                        bool waited = true;
                        if (lane == 0) waited = mbar_wait(&empty[s], par, a.status, abort_flag);
                        if (!__shfl_sync(0xffffffffu, waited, 0)) {  // nothing of this batch was issued
                            ok = false;
                            break;
                        }
                        n = 1;
                    }
                    const int id0 = __shfl_sync(0xffffffffu, cur, 2 * e & 31), id1 = __shfl_sync(0xffffffffu, cur, 2 * e + 1 & 31);
                    if (lane < n) {
                        const bool in1 = b0 + 2 * e + 1 < blocks;
                        const bool load0 = id0 >= 0 && id0 < a.num_blocks, load1 = in1 && id1 >= 0 && id1 < a.num_blocks;
                        if (!load0 || (in1 && !load1)) atomicOr(a.status, PKV_DEVERR_RANGE);
                        present[s] = (load0 ? 1 : 0) | (load1 ? 2 : 0);
                        if (load0 || load1)
                            mbar_arrive_expect_tx(&full[s], (load0 ? C::kRecord : 0) + (load1 ? C::kRecord : 0));
                        else
                            mbar_arrive(&full[s]);
                        uint8_t* st = smem + s * C::kStageBytes;
                        if (load0) bulk_load(st, head + id0 * block_bytes, C::kRecord, &full[s], policy);
                        if (load1) bulk_load(st + C::kRecord, head + id1 * block_bytes, C::kRecord, &full[s], policy);
                    }
                    __syncwarp();
                    k += n;
                    e0 += n;
                }
                cur = nxt;
            }
            if (!pc.complete) {  // where the segment's pieces lie (several divisions: not ahead of the copies)
                if (lane == 0) {
                    Piece4& p = cuts[ncut];
                    p.first_cta = static_cast<int>(split.cta_of(pc.seg_start));
                    p.pieces = static_cast<int>(split.cta_of(pc.seg_start + pc.seg_len - 1)) - p.first_cta + 1;
                    p.slot0 = pc.seg_start == split.start(p.first_cta) ? 0 : 1;
                }
                ++ncut;
            }
        }
        if (!ok && lane == 0) {  // after an abort: wait (bounded) for the copies still in flight
            for (uint32_t u = k > C::kStages ? k - C::kStages : 0; u < k; ++u)
                mbar_wait(&full[u % C::kStages], (u / C::kStages) & 1, a.status, nullptr);
            for (uint32_t u = pieces > C::kQSlots ? pieces - C::kQSlots : 0; u < pieces; ++u)
                mbar_wait(&q_full[u % C::kQSlots], (u / C::kQSlots) & 1, a.status, nullptr);
        }
        return;
    }

    // ---------------------------------------------------- consumers
    const int rg = warp % W;  // this warp's query rows: 8 R rg ..
    const int ul = warp / W;
    const int gid = lane >> 2, tig = lane & 3;
    const float scale_log2 = a.scale * kLog2e;
    uint32_t k = 0;
    for (uint32_t pieces = 0;; ++pieces) {
        const int slot = pieces % C::kQSlots;
        if (!mbar_wait(&q_full[slot], (pieces / C::kQSlots) & 1, a.status, abort_flag)) return;
        const Piece4* pc = slots + slot;
        const int blk_to = pc->blk_to;
        if (blk_to == 0) break;
        const int rows = pc->rows;
        const bool active = rg * C::kRows < rows;
        uint32_t qf[R][D / 16][2];
        float cf[R][2], kb[R][2];  // per column: 2^133, the power of two and the scale; what the eights add, 2^-133 of it
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int rr = rg * C::kRows + r * 8 + gid;
            const uint4* row = reinterpret_cast<const uint4*>(q_rows + slot * q_bytes + rr * (D * 2) + tig * (D / 2));
            uint4 w[D / 32];
            uint32_t top = 0;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                w[c] = rr < rows ? row[c] : make_uint4(0u, 0u, 0u, 0u);
                top = __vmaxu2(top, __vmaxu2(__vmaxu2(w[c].x & 0x7fff7fffu, w[c].y & 0x7fff7fffu), __vmaxu2(w[c].z & 0x7fff7fffu, w[c].w & 0x7fff7fffu)));
            }
            top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // the largest |q| lies in 2^e .. 2^(e + 1); its row is taken 2^(126 - e) times, by two factors
            const int e = max(static_cast<int>(max(top >> 16, top & 0xffffu) >> 7) - 127, -126);
            const int half = (126 - e) >> 1;
            const float up = __uint_as_float(static_cast<uint32_t>(127 + min(e, 127)) << 23), by0 = __uint_as_float(static_cast<uint32_t>(127 + half) << 23),
                        by1 = __uint_as_float(static_cast<uint32_t>(127 + 126 - e - half) << 23);
            float sum = 0.f;  // 2^-10 of q's
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t lo = h ? w[c].z : w[c].x, hi = h ? w[c].w : w[c].y;
                    const float q0 = bf16lo_to_f32(lo) * by0 * by1, q1 = bf16hi_to_f32(lo) * by0 * by1, q2 = bf16lo_to_f32(hi) * by0 * by1,
                                q3 = bf16hi_to_f32(hi) * by0 * by1;
                    qf[r][2 * c + h][0] = pack_bf16x2(q0, q1);
                    qf[r][2 * c + h][1] = pack_bf16x2(q2 * 0.0625f, q3 * 0.0625f);
                    sum = fmaf(q0, 9.765625e-4f, fmaf(q1, 9.765625e-4f, fmaf(q2, 9.765625e-4f, fmaf(q3, 9.765625e-4f, sum))));
                }
            }
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            // S^T columns 2 tig, 2 tig + 1 are the rows of lanes 8 tig and 8 tig + 4
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                cf[r][c] = __shfl_sync(0xffffffffu, up, 8 * tig + 4 * c) * (scale_log2 * 128.f);  // 2^(133 - 126)
                kb[r][c] = -7.52316385e-37f * __shfl_sync(0xffffffffu, sum, 8 * tig + 4 * c);     // 8 2^(10 - 133)
            }
        }
        // the last token each of the lane's columns sees
        int lim[R][2], least = 0x7fffffff;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int rr = rg * C::kRows + r * 8 + 2 * tig + c;
                lim[r][c] = rr < rows ? pc->n - pc->nq + rr / G : -1;
                if (rr < rows) least = min(least, lim[r][c]);
            }
        least = __reduce_min_sync(0xffffffffu, least);
        // O and z hold what the codes' eights add too, in o and in z alike; fold() takes it out
        float m[R][2], l[R][2], o[R][D / 16][4], z[R][4];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            m[r][0] = m[r][1] = kUnset;
            l[r][0] = l[r][1] = 0.f;
            z[r][0] = z[r][1] = z[r][2] = z[r][3] = 0.f;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) o[r][i][0] = o[r][i][1] = o[r][i][2] = o[r][i][3] = 0.f;
        }
        auto fold = [&]() {
#pragma unroll
            for (int r = 0; r < R; ++r) {
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    o[r][i][0] -= z[r][0];
                    o[r][i][1] -= z[r][1];
                    o[r][i][2] -= z[r][2];
                    o[r][i][3] -= z[r][3];
                }
                z[r][0] = z[r][1] = z[r][2] = z[r][3] = 0.f;
            }
        };
        const uint32_t k_end = k + (blk_to - pc->blk_from + 1) / 2;
        const int skip = (ul - static_cast<int>(k & (UL - 1))) & (UL - 1);
        k += skip;
        int s = static_cast<int>(k % C::kStages);
        uint32_t parity = (k / C::kStages) & 1;
        auto next_stage = [&]() {
            s += UL;
            if (s >= C::kStages) {
                s -= C::kStages;
                parity ^= 1u;
            }
        };
        int unfolded = 0;
        for (int blk = pc->blk_from + 2 * skip; blk < blk_to; blk += 2 * UL, next_stage()) {
            if (!mbar_wait(&full[s], parity, a.status, abort_flag)) return;
            const int there = present[s];
            if (active && there) {
                const uint8_t* st = smem + s * C::kStageBytes;
                // every token of the stage exists and every row sees it
                const bool whole = there == 3 && blk * 16 + 31 <= least;
                // (two blocks at a time with one tile of rows, to have several chains in flight; one with two tiles, for the registers)
                constexpr int kAt = R == 1 ? 2 : 1;
#pragma unroll
                for (int b0 = 0; b0 < 2; b0 += kAt) {
                    float sc[R][kAt][4];  // per block: tokens gid, gid + 8 by 2 columns
                    float f[R][4 * kAt];  // the scores' factors
                    float sv[2 * kAt];
#pragma unroll
                    for (int b = 0; b < kAt; ++b) {
                        const uint8_t* rec = st + (b0 + b) * C::kRecord;
                        uint32_t wa[D / 32], wb[D / 32];
                        if (D == 128) {
                            const uint4 u = *reinterpret_cast<const uint4*>(rec + gid * 64 + tig * 16), v = *reinterpret_cast<const uint4*>(rec + (gid + 8) * 64 + tig * 16);
                            wa[0] = u.x, wa[1] = u.y, wa[D / 32 - 2] = u.z, wa[D / 32 - 1] = u.w;
                            wb[0] = v.x, wb[1] = v.y, wb[D / 32 - 2] = v.z, wb[D / 32 - 1] = v.w;
                        } else {
                            const uint2 u = *reinterpret_cast<const uint2*>(rec + gid * 32 + tig * 8), v = *reinterpret_cast<const uint2*>(rec + (gid + 8) * 32 + tig * 8);
                            wa[0] = u.x, wa[1] = u.y;
                            wb[0] = v.x, wb[1] = v.y;
                        }
#pragma unroll
                        for (int c = 0; c < D / 32; ++c) {
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const uint32_t u = h ? wa[c] >> 8 : wa[c], v = h ? wb[c] >> 8 : wb[c];
#pragma unroll
                                for (int r = 0; r < R; ++r) {
                                    if (c + h == 0)
                                        mma_bf16_from(sc[r][b], u & 0x000f000fu, v & 0x000f000fu, u & 0x00f000f0u, v & 0x00f000f0u, qf[r][0][0], qf[r][0][1],
                                                     kb[r][0], kb[r][1]);
                                    else
                                        mma_bf16_16816(sc[r][b], u & 0x000f000fu, v & 0x000f000fu, u & 0x00f000f0u, v & 0x00f000f0u, qf[r][2 * c + h][0],
                                                      qf[r][2 * c + h][1]);
                                }
                            }
                        }
                        const float* scales = reinterpret_cast<const float*>(rec + q4_scales_offset(D));
                        const float ka = scales[gid], kc = scales[gid + 8];
                        // (an infinite K scale makes V's a NaN: it may take a score to -inf, where it would go unseen)
                        sv[2 * b] = fmaf(ka, 0.f, scales[16 + gid]);
                        sv[2 * b + 1] = fmaf(kc, 0.f, scales[24 + gid]);
#pragma unroll
                        for (int r = 0; r < R; ++r)
#pragma unroll
                            for (int e = 0; e < 4; ++e) f[r][4 * b + e] = (e & 2 ? kc : ka) * cf[r][e & 1];
                    }
                    uint4 vw[kAt][D / 64];
#pragma unroll
                    for (int b = 0; b < kAt; ++b)
#pragma unroll
                        for (int h = 0; h < D / 64; ++h)
                            vw[b][h] = *reinterpret_cast<const uint4*>(st + (b0 + b) * C::kRecord + q4_v_offset(D) + gid * 64 + tig * 16 + h * 512);
                    if (b0 + kAt == 2) {
                        __syncwarp();  // everything is in registers
                        if (lane == 0) mbar_arrive(&empty[s]);
                    }
                    if (!whole) {  // what a row does not see: a score of -inf
#pragma unroll
                        for (int i = 0; i < 2 * kAt; ++i) {
                            const int p = (blk + b0 + (i >> 1)) * 16 + 8 * (i & 1) + gid;
                            const bool in = (there >> (b0 + (i >> 1)) & 1) != 0;
#pragma unroll
                            for (int r = 0; r < R; ++r)
#pragma unroll
                                for (int c = 0; c < 2; ++c)
                                    if (!in || p > lim[r][c]) {
                                        sc[r][i >> 1][2 * (i & 1) + c] = __int_as_float(0xff800000);
                                        f[r][2 * i + c] = 1.f;
                                    }
                        }
                    }
                    float e[R][4 * kAt], sum[R][2];
                    uint32_t p[R][2 * kAt];
                    uint32_t top = 0;
                    float most = 0.f;
                    auto weights = [&]() {
#pragma unroll
                        for (int r = 0; r < R; ++r) {
#pragma unroll
                            for (int i = 0; i < 4 * kAt; ++i) e[r][i] = ex2(fmaf(sc[r][i >> 2][i & 3], f[r][i], -m[r][i & 1]));
#pragma unroll
                            for (int i = 0; i < 2 * kAt; ++i) {
                                p[r][i] = pack_f16x2(e[r][2 * i] * sv[i], e[r][2 * i + 1] * sv[i]);
                            }
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                sum[r][c] = e[r][c] + e[r][2 + c];
                                if (kAt == 2) sum[r][c] += e[r][4 * kAt - 4 + c] + e[r][4 * kAt - 2 + c];
                                sum[r][c] += l[r][c];
                                most = fmaxf(most, sum[r][c]);
                            }
                        }
                    };
                    // what a row does not see (the scores of -inf above) has no weight, whatever its scale
                    auto mask = [&]() {
#pragma unroll
                        for (int r = 0; r < R; ++r)
#pragma unroll
                            for (int i = 0; i < 2 * kAt; ++i)
                                p[r][i] &= (__float_as_uint(sc[r][i >> 1][2 * (i & 1)]) != 0xff800000u ? 0x0000ffffu : 0u) |
                                           (__float_as_uint(sc[r][i >> 1][2 * (i & 1) + 1]) != 0xff800000u ? 0xffff0000u : 0u);
                    };
                    weights();
                    if (!whole) mask();
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int i = 0; i < 2 * kAt; ++i) top = larger_f16x2(top, p[r][i]);
                    // some P' has left f16 (its exponent is full), or l grows beside tiny V scales
                    if (__any_sync(0xffffffffu, ((top + 0x04000400u) & 0x80008000u) != 0u || most > kMostSum)) {
                        float lg[2 * kAt];
#pragma unroll
                        for (int i = 0; i < 2 * kAt; ++i) lg[i] = fminf(__log2f(fmaxf(fabsf(sv[i]), kTinyScale)), 128.f);
#pragma unroll
                        for (int r = 0; r < R; ++r)
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                float j = kUnset;
#pragma unroll
                                for (int i = 0; i < 2 * kAt; ++i) j = fmaxf(j, sc[r][i >> 1][2 * (i & 1) + c] * f[r][2 * i + c] + lg[i]);
#pragma unroll
                                for (int off = 4; off < 32; off <<= 1) j = fmaxf(j, __shfl_xor_sync(0xffffffffu, j, off));
                                const float to = fmaxf(m[r][c], j - kHeadroom), al = ex2(m[r][c] - to);
                                m[r][c] = to;
                                l[r][c] *= al;
                                z[r][c] *= al;
                                z[r][2 + c] *= al;
#pragma unroll
                                for (int i = 0; i < D / 16; ++i) {
                                    o[r][i][c] *= al;
                                    o[r][i][2 + c] *= al;
                                }
                            }
                        weights();
                        if (!whole) mask();
                    }
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        l[r][0] = sum[r][0];
                        l[r][1] = sum[r][1];
#pragma unroll
                        for (int i = 0; i < 2 * kAt; ++i) p[r][i] = movmatrix_trans(p[r][i]);
                    }
#pragma unroll
                    for (int b = 0; b < kAt; ++b) {
#pragma unroll
                        for (int r = 0; r < R; ++r) mma_f16_16816(z[r], 0x00080008u, 0x00800080u, 0x00080008u, 0x00800080u, p[r][2 * b], p[r][2 * b + 1]);
#pragma unroll
                        for (int h = 0; h < D / 64; ++h) {
                            const uint32_t w[4] = {vw[b][h].x, vw[b][h].y, vw[b][h].z, vw[b][h].w};
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
#pragma unroll
                                for (int r = 0; r < R; ++r)
                                    mma_f16_16816(o[r][4 * h + j], w[j] & 0x000f000fu, w[j] & 0x00f000f0u, w[j] >> 8 & 0x000f000fu, w[j] >> 8 & 0x00f000f0u,
                                                  p[r][2 * b], p[r][2 * b + 1]);
                            }
                        }
                    }
                }
                if (++unfolded == kFold) {
                    fold();
                    unfolded = 0;
                }
            } else {
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[s]);
            }
        }
        fold();
        k = k_end;
        // ---- end of the piece: this warp's state into shared memory (O over 2^-24)
        if (pieces > 0 && !mbar_wait(state_empty, (pieces - 1) & 1, a.status, abort_flag)) return;
        float* own = state + warp * C::kStateFloats;
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) l[r][c] += __shfl_xor_sync(0xffffffffu, l[r][c], off);
                const int row = r * 8 + 2 * tig + c;
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
                    *reinterpret_cast<float2*>(own + row * D + 8 * (gid + 8 * (i >> 2)) + 2 * (i & 3)) =
                        make_float2(o[r][i][c] * 16777216.f, o[r][i][2 + c] * 1048576.f);
                if (gid == 0) {
                    own[C::kRows * D + row] = m[r][c];
                    own[C::kRows * (D + 1) + row] = l[r][c];
                }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(state_full);
        if (!mbar_wait(state_full, pieces & 1, a.status, abort_flag)) return;
        // ---- all unit lanes together; a warp takes D / 4 dimensions, a lane a quarter of them of one row of a tile
        const int tiles = (rows + 7) / 8;
        constexpr int kPer = D / 16;
        const int row8 = lane >> 2, d0 = warp * (D / 4) + (lane & 3) * kPer;
        for (int tile = 0; tile < tiles; ++tile) {
            const int row = tile % R * 8 + row8, group = tile / R;  // among the rows of that group's warps
            float M = kUnset, L = 0.f, O[kPer] = {};
            for (int u = 0; u < UL; ++u) M = fmaxf(M, state[(u * W + group) * C::kStateFloats + C::kRows * D + row]);
            for (int u = 0; u < UL; ++u) {
                const float* su = state + (u * W + group) * C::kStateFloats;
                const float wu = ex2(su[C::kRows * D + row] - M);
                L += wu * su[C::kRows * (D + 1) + row];
#pragma unroll
                for (int e = 0; e < kPer; e += 4) {
                    const float4 v = *reinterpret_cast<const float4*>(su + row * D + d0 + e);
                    O[e] += wu * v.x, O[e + 1] += wu * v.y, O[e + 2] += wu * v.z, O[e + 3] += wu * v.w;
                }
            }
            const int rr = tile * 8 + row8;
            if (pc->cut == 0) {
                if (rr < rows) write_part<D>(a, pc->q0, pc->head, rr, d0, O, L);
            } else {
                float* sl = piece_of(a, D, cta, pc->cut - 1, tile);
#pragma unroll
                for (int e = 0; e < kPer; e += 4) *reinterpret_cast<float4*>(sl + row8 * D + d0 + e) = make_float4(O[e], O[e + 1], O[e + 2], O[e + 3]);
                if ((lane & 3) == 0) {
                    sl[8 * D + warp * 16 + row8] = M;
                    sl[8 * D + warp * 16 + 8 + row8] = L;
                }
            }
        }
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(state_empty);
            mbar_arrive(&q_empty[slot]);
        }
    }
    // ---- announce this warp's share of the cut pieces; the warp that completes a count merges them
    const int ncut = *num_cuts;
    if (ncut == 0) return;
    __syncwarp();
    int old = 0;
    if (lane < ncut) old = add_acq_rel(a.counters + (static_cast<long long>(cuts[lane].seq) * a.kv_heads + cuts[lane].head) * kConsumers + warp, 1);
    __syncwarp();
    for (int i = 0; i < ncut; ++i) {
        const Piece4& pc = cuts[i];
        if (__shfl_sync(0xffffffffu, old, i) != pc.pieces - 1) continue;
        constexpr int kPer = D / 16;
        const int row8 = lane >> 2, d0 = warp * (D / 4) + (lane & 3) * kPer;
        for (int tile = 0; tile * 8 < pc.rows; ++tile) {
            float M = kUnset, L = 0.f, O[kPer] = {};
            for (int p0 = 0; p0 < pc.pieces; p0 += kMergeAhead) {
                // several pieces' loads in flight at once (past the last: the last again, without weight)
                float mp[kMergeAhead], lp[kMergeAhead];
                float4 v[kMergeAhead][kPer / 4];
#pragma unroll
                for (int u = 0; u < kMergeAhead; ++u) {
                    const int p = min(p0 + u, pc.pieces - 1);
                    const float* sl = piece_of(a, D, pc.first_cta + p, p == 0 ? pc.slot0 : 0, tile);
                    mp[u] = p0 + u < pc.pieces ? __ldcg(sl + 8 * D + warp * 16 + row8) : kUnset;
                    lp[u] = __ldcg(sl + 8 * D + warp * 16 + 8 + row8);
#pragma unroll
                    for (int e = 0; e < kPer; e += 4) v[u][e / 4] = __ldcg(reinterpret_cast<const float4*>(sl + row8 * D + d0 + e));
                }
                float to = M;
#pragma unroll
                for (int u = 0; u < kMergeAhead; ++u) to = fmaxf(to, mp[u]);
                const float keep = ex2(M - to);
                M = to;
                L *= keep;
#pragma unroll
                for (int e = 0; e < kPer; ++e) O[e] *= keep;
#pragma unroll
                for (int u = 0; u < kMergeAhead; ++u) {
                    const float w = p0 + u < pc.pieces ? ex2(mp[u] - to) : 0.f;
                    L += w * lp[u];
#pragma unroll
                    for (int e = 0; e < kPer; e += 4) {
                        O[e] += w * v[u][e / 4].x, O[e + 1] += w * v[u][e / 4].y;
                        O[e + 2] += w * v[u][e / 4].z, O[e + 3] += w * v[u][e / 4].w;
                    }
                }
            }
            if (tile * 8 + row8 < pc.rows) write_part<D>(a, pc.q0, pc.head, tile * 8 + row8, d0, O, L);
        }
        if (lane == 0) a.counters[(static_cast<long long>(pc.seq) * a.kv_heads + pc.head) * kConsumers + warp] = 0;
    }
}

// The kernel's shared-memory limit belongs to the function, which calls of all threads share: every call sets it to
// the largest launch's, so that none takes it away from another's launch.
template <int D, int R>
cudaError_t allow_smem() {
    return cudaFuncSetAttribute(mq4_kernel<D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(M4<D, R>::most_smem_bytes()));
}

template <int D, int R>
cudaError_t run_mq4(const Q4Args& a, cudaStream_t s) {
    using C = M4<D, R>;
    const size_t smem = C::smem_bytes(a.warps_per_unit, a.batch);
    const cudaError_t e = allow_smem<D, R>();
    if (e != cudaSuccess) return e;
    return launch_pdl(mq4_kernel<D, R>, dim3(a.num_ctas), dim3(kThreads), smem, s, a);
}

// Resident CTAs of an SM, at the largest launch; 0 where that could not be found out.
template <int D, int R>
int resident(int warps_per_unit) {
    const size_t smem = M4<D, R>::smem_bytes(warps_per_unit, kMaxBatchPerLaunch);
    int n = 0;
    if (allow_smem<D, R>() != cudaSuccess) return 0;
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, mq4_kernel<D, R>, kThreads, smem) == cudaSuccess && n > 0 ? n : 0;
}

}  // namespace

Q4Plan q4_plan(int head_dim, int rows) {
    Q4Plan p;
    p.tiles = (rows + 7) / 8;
    p.row_tiles = p.tiles == 1 ? 1 : 2;
    p.warps_per_unit = p.tiles <= 2 ? 1 : 2;
    p.tiles = p.row_tiles * p.warps_per_unit;
    static std::mutex mu;
    static int cache[2][3][64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) dev = 0;
    std::lock_guard<std::mutex> lock(mu);
    int& per_sm = cache[head_dim == 128][p.row_tiles + p.warps_per_unit - 2][dev];
    if (per_sm == 0) {
        if (head_dim == 128)
            per_sm = p.row_tiles == 1 ? resident<128, 1>(1) : resident<128, 2>(p.warps_per_unit);
        else
            per_sm = p.row_tiles == 1 ? resident<64, 1>(1) : resident<64, 2>(p.warps_per_unit);
    }
    p.num_ctas = (per_sm > 0 ? per_sm : 1) * device_sm_count();  // (what failed is not kept, and asked for again)
    return p;
}

size_t q4_partials_bytes(int head_dim, const Q4Plan& p) {
    return static_cast<size_t>(p.num_ctas) * 2 * p.tiles * piece_floats(head_dim) * sizeof(float);
}

cudaError_t launch_mq4(const Q4Args& a, const Q4Plan& p, cudaStream_t s) {
    if (a.head_dim == 128) return p.row_tiles == 1 ? run_mq4<128, 1>(a, s) : run_mq4<128, 2>(a, s);
    return p.row_tiles == 1 ? run_mq4<64, 1>(a, s) : run_mq4<64, 2>(a, s);
}

}  // namespace pkv
