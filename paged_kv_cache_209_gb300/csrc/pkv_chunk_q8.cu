// Causal attention of a chunk of new tokens over the int8 pools
// (pkv_multiquery_attention_q8 in include/pkv.h), for more than 32 query rows
// per (sequence, KV head) or head_dim 64.
//
// Mathematics, per query row and step of 128 tokens:
//     s_p = q' . k_p                    f16 x f16 -> fp32; q' is q times a power of two
//                                       per row (exact), k_p = kc_p (ks_p 2^-F) rounded
//                                       to f16 once, an eighth of a quantization step
//     x_p = s_p f                       f = |scale| log2(e) 2^F over the row's power
//     w_p = 2^(x_p - m)                 m: running maximum, moved only when a score
//                                       exceeds it by more than 8 (w <= 2^8)
//     l  += w_p;   O += w_p v_p         w rounded to f16; v_p = vc_p (vs_p 2^-E)
//                                       rounded to f16; fp32 sums
//     out = 2^E O / l
// F and E are one exponent each per piece of work, taken from its first step, that
// put K and V into the f16 range whatever their size. A step whose scales leave
// [2^-14, 2^8] times that (rows 2^22 apart; or infinities), or with absent tokens, is
// slow: it takes K's codes themselves and x_p = s_p ks_p f in fp32, and, where it is V
// that leaves the range, V's codes with w_p = 2^(x_p + log2(vs_p) - E - m) and l summed
// apart. That is exact over the whole float range, because the maximum is then
// taken over tokens the row sees.
//
// K's scale sits in the K operand, not in the softmax, because a factor per token
// costs every row a multiplication and a shared-memory broadcast, 1024 of the 2048
// cycles that a step's products take: the softmax would be the bound.
//
// Work (pkv_chunk_schedule.cuh): one persistent CTA per SM takes a range of
// (unit, step) pairs, a unit being 256 query rows of a (sequence, KV head) as
// two row halves A and B of 128. A unit cut by a range leaves fp32 pieces
// (O, m, l) in the workspace, which combine_kernel joins.
//
// Roles (20 warps). Warps 0-3 and 4-7: the softmax of halves A and B, one thread
// per query row. Warps 8-11 and 12-15: the converters of K and of V; they load
// the codes of the next step from global memory into registers while they turn
// the previous loads into scaled f16, in the 128-byte-swizzled layout the tensor
// cores read; K's also write the step's exponents and, for a slow step, its factors. Warps 16
// and 17: one thread each issues S = Q K^T of A and of B; warps 18 and 19: O += P V
// of A and of B, in two parts of 64 tokens. While the softmax of one half runs,
// the tensor cores work on the other.
//
// Tensor memory (512 columns): S of A and B (128 fp32 columns each; P is written
// over its first 64), O of A and B. Shared memory: Q 64 KB, two stages of K and
// of V of 32 KB each.
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

template <int D>
struct Cx {
    static constexpr int kSoftmaxWarps = 8;
    static constexpr int kConvertWarp = 8;  // K: 8 .. 11, V: 12 .. 15
    static constexpr int kScoreWarp = 16;   // 16, 17
    static constexpr int kValueWarp = 18;   // 18, 19
    static constexpr int kThreads = 640;
    static constexpr int kConverters = 128;  // threads that convert K, and V
    static constexpr int kStages = 2;     // K stages, and V stages
    static constexpr int kTables = 4;     // factor tables in flight
    static constexpr int kHalves = D / 64;                    // 128-byte column parts of a K or Q row
    static constexpr int kPartBytes = 128 * 128;              // 128 rows of one part
    static constexpr int kTileBytes = kHalves * kPartBytes;   // Q of one row half; one K stage
    static constexpr int kVPartBytes = D * 128;               // 64 tokens of every coordinate
    static constexpr int kVBytes = 2 * kVPartBytes;           // one V stage
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kOffQ + 2 * kTileBytes;
    static constexpr int kOffV = kOffK + kStages * kTileBytes;
    static constexpr int kOffTable = kOffV + kStages * kVBytes;
    // a step's table: 2^E, 2^F, 1 for a slow step; and for a slow step the K factors
    // [128] and log2(vs) - E [128] (0 unless V's scales leave the range)
    static constexpr int kTableBytes = 16 + 2 * 128 * 4;
    static constexpr int kOffScale = kOffTable + kTables * kTableBytes;  // f16 V factors [2][128]
    static constexpr int kOffReduce = kOffScale + 512;                   // K, V: [2][4 warps] of 32 bytes
    static constexpr int kOffBars = kOffReduce + 512;
    // k_full, k_empty, v_full, v_empty per stage; q_full, s_full per half;
    // p_full, pv_done per half and token part; final per issuer
    static constexpr int kNumBars = 4 * kStages + 2 * 2 + 2 * 4 + 4;
    static constexpr int kOffPrefix = kOffBars + kNumBars * 8;
    static constexpr int kOffPlan = kOffPrefix + (kMaxBatchPerLaunch + 1) * 8;
    static constexpr int kOffMisc = kOffPlan + (2 + kThreads / 32) * 16;
    static constexpr size_t kSmem = 1024 + kOffMisc + kThreads / 32 * 8 + 16;
    static constexpr uint32_t kColS = 0;    // S of half x: 128 x
    static constexpr uint32_t kColO = 256;  // O of half x: 256 + 128 x
    static constexpr uint32_t kTmemCols = 512;
    static_assert(kSmem <= 227 * 1024, "shared memory");
};

// ---------------------------------------------------------------- workspace
// Per CTA a descriptor (first position of its range, flags) and two piece slots:
// 0 for a piece that begins inside a unit, 1 for one that begins a unit and is cut.
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

__device__ __forceinline__ ChunkShape shape_of(const ChunkArgs& a) {
    return ChunkShape{a.lens, a.qstart, a.batch, a.kv_heads, a.group, a.max_blocks, a.max_query_len};
}

// Cost before each sequence (all threads, two sequences each; ends with __syncthreads).
__device__ void sum_costs(const ChunkArgs& a, const ChunkShape& sh, int64_t* prefix, int64_t* warp_sum) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int64_t mine[2], sum = 0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int i = 2 * threadIdx.x + e;
        mine[e] = 0;
        if (i < a.batch) {
            ChunkSeq q;
            if (chunk_seq(sh, i, q))
                mine[e] = chunk_head_cost(q, a.group) * a.kv_heads;
            else if (blockIdx.x == 0)
                atomicOr(a.status, PKV_DEVERR_RANGE);
        }
        sum += mine[e];
    }
    int64_t incl = sum;
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t other = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += other;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int64_t at = incl - sum;
    for (int w = 0; w < warp; ++w) at += warp_sum[w];
    if (2 * threadIdx.x <= a.batch) prefix[2 * threadIdx.x] = at;
    if (2 * threadIdx.x + 1 <= a.batch) prefix[2 * threadIdx.x + 1] = at + mine[0];
    __syncthreads();
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
// The exponent a segment takes from its first step's scales (bits of the largest and
// smallest): the largest, or beside an infinity the smallest, goes to 1/2 .. 1.
__device__ __forceinline__ int range_exponent(uint32_t most, uint32_t least) {
    const uint32_t ref = most < 0x7f800000u ? most : (least < 0x7f800000u ? least : 0x3f800000u);
    return max(-125, min(125, static_cast<int>(ref >> 23) - 126));
}
// Whether scales leave [2^(e - 14), 2^(e + 8)] (bits compare as the floats do).
__device__ __forceinline__ bool leaves_range(uint32_t most, uint32_t least, int e) {
    return least < static_cast<uint32_t>(max(e - 14, -126) + 127) << 23 || most > static_cast<uint32_t>(min(e + 8, 127) + 127) << 23;
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
// All `threads` of named barrier `id` meet; true if `ok` held for every one.
__device__ __forceinline__ bool named_barrier_all(int id, int threads, bool ok) {
    int r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.s32 p, %3, 0;\n\t"
        "barrier.cta.red.and.pred q, %1, %2, p;\n\t"
        "selp.s32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(id), "r"(threads), "r"(static_cast<int>(ok))
        : "memory");
    return r != 0;
}

// Eight scores of a slow step, scaled, -inf where the token is absent or not seen
// (columns taddr .. taddr + 7, K factors c, row factor f, the first `seen` of them seen).
__device__ __forceinline__ void slow_scores(uint32_t taddr, const float* c, float f, int seen, float (&x)[8]) {
    uint32_t v[8];
    tmem_ld8(taddr, v);
    tmem_ld_wait();
#pragma unroll
    for (int e = 0; e < 8; ++e)
        x[e] = e >= seen || __float_as_uint(c[e]) == kAbsent ? ninf() : __uint_as_float(v[e]) * c[e] * f;
}
// mbar_wait by a whole warp, with one answer for all its lanes.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, unsigned int* status, volatile int* abort) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, status, abort));
}

// ---------------------------------------------------------------- converters
// K's (IsV false) or V's four warps: every step of the CTA's range, one load
// ahead. Warp w takes tokens 32 w .. 32 w + 31 of a step (blocks 2 w, 2 w + 1), lane l
// the scales of token 32 w + l. The range of the scales decides a step's mode and a
// segment's exponents; both groups read V's scales and decide alike.
template <int D, bool IsV>
__device__ void convert_role(const ChunkArgs& a, const ChunkShape& sh, uint8_t* smem, const int64_t* prefix,
                             const ChunkPos* plan, ChunkPos* after, uint64_t* full, uint64_t* empty,
                             volatile int* abort_flag) {
    using C = Cx<D>;
    const int lane = threadIdx.x & 31;
    const int cw = (threadIdx.x >> 5) & 3;
    constexpr int kVecs = 32 * D / 16 / 32;    // 16-code vectors per lane and step
    constexpr int kPerBlock = kVecs / 2;       // of them in each of the warp's two blocks
    constexpr int kLanes = D / 16;             // lanes that hold one token's K row
    constexpr int kBlockVecs = D;              // vectors of one (block, head)
    constexpr int kBarrier = IsV ? 2 : 1;
    const uint4* codes = static_cast<const uint4*>(IsV ? a.v_codes : a.k_codes);
    uint32_t (*reduce)[4][8] = reinterpret_cast<uint32_t (*)[4][8]>(smem + C::kOffReduce + (IsV ? 256 : 0));

    // the segment being loaded (the position after it: in shared memory, one per warp, read once per segment)
    if (lane == 0) *after = plan[0];
    __syncwarp();
    int step = 0, last = 0;         // next step to load, one past the segment's last
    int n = 0, head = 0;            // its tokens, KV head
    const int32_t* trow = nullptr;  // its block table
    int ids = 0, ids_next = 0;      // lane l: id of block 32 b + l (-1: past the end, -2: outside the pool), b = step / 4; b + 1
    bool opens = false;             // the loaded step is its segment's first
    auto id_at = [&](int b) {
        if (b >= (n + 15) / 16) return -1;
        const int id = __ldg(trow + b);
        if (id >= 0 && id < a.num_blocks) return id;
        if (!IsV) atomicOr(a.status, PKV_DEVERR_RANGE);
        return -2;
    };
    auto open = [&]() {
        ChunkSegment g;
        const ChunkPos cur = *after;
        __syncwarp();
        if (!chunk_segment(sh, cur, plan[1], g)) return false;
        if (lane == 0) *after = chunk_after(sh, prefix, g);
        __syncwarp();
        step = g.at.s;
        last = g.s1;
        n = g.q.n;
        head = g.at.head;
        trow = a.tables + static_cast<int64_t>(g.at.seq) * a.max_blocks;
        ids = id_at(32 * (step >> 2) + lane);
        ids_next = id_at(32 * (step >> 2) + 32 + lane);
        opens = true;
        return true;
    };
    // the loaded step: codes; scales of the lane's token, whether it exists or lies in a block outside the pool
    uint4 w[kVecs];
    float ks = 0.f, vs = 0.f;
    bool present = false, missing = false;
    auto load = [&]() {
        const int b0 = (step & 3) * 8 + 2 * cw;
        const int id0 = __shfl_sync(0xffffffffu, ids, b0), id1 = __shfl_sync(0xffffffffu, ids, b0 + 1);
        // an absent block's codes may be any (its tokens carry no weight): block 0 exists
        const uint4* src0 = codes + (static_cast<int64_t>(max(0, id0)) * a.kv_heads + head) * kBlockVecs + lane;
        const uint4* src1 = codes + (static_cast<int64_t>(max(0, id1)) * a.kv_heads + head) * kBlockVecs + lane;
#pragma unroll
        for (int i = 0; i < kPerBlock; ++i) {
            w[i] = __ldg(src0 + 32 * i);
            w[kPerBlock + i] = __ldg(src1 + 32 * i);
        }
        const int id = lane < 16 ? id0 : id1;
        present = id >= 0 && step * kChunkStep + 32 * cw + lane < n;
        missing = id == -2;
        const float* rec = a.scales + (static_cast<int64_t>(max(0, id)) * a.kv_heads + head) * 32 + (lane & 15);
        if (!IsV) ks = __ldg(rec);
        vs = __ldg(rec + 16);
    };
    // moves on to the next step, if there is one, and loads it
    auto advance = [&]() {
        opens = false;
        if (++step >= last) {
            if (!open()) return false;
        } else if ((step & 3) == 0) {
            ids = ids_next;
            ids_next = id_at(32 * (step >> 2) + 32 + lane);
        }
        load();
        return true;
    };

    bool live = open();
    if (live) load();
    int ev = 0, ek = 0;  // E and F of the segment
    bool have = false;   // they are set
    for (int it = 0; live; ++it) {
        const int st = it & 1;
        if (opens) have = false;
        // ---- range of the scales of the tokens that exist; absent tokens
        const uint32_t vbits = __float_as_uint(vs) & 0x7fffffffu;
        const uint32_t kbits = __float_as_uint(ks) & 0x7fffffffu;
        {
            const uint32_t vm = __reduce_max_sync(0xffffffffu, present ? vbits : 0u);
            const uint32_t vl = __reduce_min_sync(0xffffffffu, present ? vbits : 0xffffffffu);
            if (lane == 0) *reinterpret_cast<uint2*>(&reduce[st][cw][0]) = make_uint2(vm, vl);
            if (!IsV) {
                const uint32_t km = __reduce_max_sync(0xffffffffu, present ? kbits : 0u);
                const uint32_t kl = __reduce_min_sync(0xffffffffu, present ? kbits : 0xffffffffu);
                const uint32_t miss = __any_sync(0xffffffffu, missing);
                if (lane == 0) *reinterpret_cast<uint4*>(&reduce[st][cw][4]) = make_uint4(km, kl, miss, 0u);
            }
        }
        const bool go = mbar_wait(&empty[st], static_cast<uint32_t>((it >> 1) & 1) ^ 1u, a.status, abort_flag);
        if (!named_barrier_all(kBarrier, C::kConverters, go)) break;
        uint32_t vmax = 0, vmin = 0xffffffffu, kmax = 0, kmin = 0xffffffffu, miss = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint2 r = *reinterpret_cast<const uint2*>(&reduce[st][i][0]);
            vmax = max(vmax, r.x);
            vmin = min(vmin, r.y);
            if (!IsV) {
                const uint4 t = *reinterpret_cast<const uint4*>(&reduce[st][i][4]);
                kmax = max(kmax, t.x);
                kmin = min(kmin, t.y);
                miss |= t.z;
            }
        }
        bool wide = false, slow = miss != 0;
        if (vmin != 0xffffffffu) {
            if (!have) {  // the segment's first step with tokens
                ev = range_exponent(vmax, vmin);
                if (!IsV) ek = range_exponent(kmax, kmin);
                have = true;
            }
            wide = leaves_range(vmax, vmin, ev);
            if (!IsV) slow |= wide || leaves_range(kmax, kmin, ek);
        }
        if (IsV) {
            __half* factors = reinterpret_cast<__half*>(smem + C::kOffScale) + 128 * st + 32 * cw;
            factors[lane] = __float2half(!present ? 0.f : wide ? 1.f : vs * exp2_int(-ev));
            __syncwarp();
            // ---- coordinate rows, 64 tokens each: this warp's are 32 cw .. 32 cw + 31
            uint8_t* vd = smem + C::kOffV + st * C::kVBytes + (cw >> 1) * C::kVPartBytes + lane * 128;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const uint4* f = reinterpret_cast<const uint4*>(factors + 16 * b);
                const uint4 f0 = f[0], f1 = f[1];
                const int c0 = ((2 * cw + b) & 3) * 2;
#pragma unroll
                for (int i = 0; i < kPerBlock; ++i) {
                    const uint4& x = w[b * kPerBlock + i];
                    *reinterpret_cast<uint4*>(vd + i * 32 * 128 + ((c0 ^ (lane & 7)) << 4)) = v_values(x.x, x.y, f0);
                    *reinterpret_cast<uint4*>(vd + i * 32 * 128 + (((c0 + 1) ^ (lane & 7)) << 4)) = v_values(x.z, x.w, f1);
                }
            }
        } else {
            float* tab = reinterpret_cast<float*>(smem + C::kOffTable + (it & (C::kTables - 1)) * C::kTableBytes);
            if (cw == 0 && lane == 0)
                *reinterpret_cast<float4*>(tab) = make_float4(exp2_int(ev), exp2_int(ek), slow ? 1.f : 0.f, 0.f);
            if (slow) {
                tab[4 + 32 * cw + lane] = missing ? __uint_as_float(kAbsent) : present ? ks : 0.f;
                // a scale below the normal range counts as its smallest number
                tab[4 + 128 + 32 * cw + lane] = present && wide ? log2f(vbits < 0x00800000u ? 1.17549435e-38f : vs) - static_cast<float>(ev) : 0.f;
            }
            const float factor = !present ? 0.f : slow ? 1.f : ks * exp2_int(-ek);
            const __half hi = __float2half(factor);
            const uint32_t pair = bits(__halves2half2(hi, __float2half(factor - __half2float(hi))));  // (hi, lo) of the lane's token
            // ---- token rows: vector i of a lane lies in row 32 cw + i * (32 / kLanes) + lane / kLanes
            const int ch = lane % kLanes, sub = lane / kLanes;
            // lanes of the second column part write their halves in the other order: no bank is hit twice
            const int flip = ch >> 2;
            uint8_t* kd = smem + C::kOffK + st * C::kTileBytes + flip * C::kPartBytes + (32 * cw + sub) * 128;
            const int c0 = (ch & 3) * 2 + flip;
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                // (the row modulo 8 alternates between two values at head_dim 128)
                const int row8 = (i * (32 / kLanes) + sub) & 7;
                const uint32_t f = __shfl_sync(0xffffffffu, pair, i * (32 / kLanes) + sub);
                const __half2 fh = half2_of(__byte_perm(f, f, 0x1010)), fl = half2_of(__byte_perm(f, f, 0x3232));
                const uint4 x0 = k_values(w[i].x, w[i].y, fh, fl), x1 = k_values(w[i].z, w[i].w, fh, fl);
                uint8_t* rowp = kd + i * (32 / kLanes) * 128;
                *reinterpret_cast<uint4*>(rowp + ((c0 ^ row8) << 4)) = flip ? x1 : x0;
                *reinterpret_cast<uint4*>(rowp + ((c0 ^ 1 ^ row8) << 4)) = flip ? x0 : x1;
            }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[st]);
        live = advance();
    }
}

template <int D>
__global__ void __launch_bounds__(Cx<D>::kThreads, 1) chunk_q8_kernel(const ChunkArgs a) {
    using C = Cx<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + C::kOffBars);
    uint64_t* k_empty = k_full + C::kStages;
    uint64_t* v_full = k_empty + C::kStages;
    uint64_t* v_empty = v_full + C::kStages;
    uint64_t* q_full = v_empty + C::kStages;  // [half]: Q rows in place
    uint64_t* s_full = q_full + 2;            // [half]: scores in tensor memory
    uint64_t* p_full = s_full + 2;            // [half][part]: weights written
    uint64_t* pv_done = p_full + 4;           // [half][part]: that product has completed
    uint64_t* final_bar = pv_done + 4;        // [issuer]: everything it issued has completed
    int64_t* prefix = reinterpret_cast<int64_t*>(smem + C::kOffPrefix);
    ChunkPos* plan = reinterpret_cast<ChunkPos*>(smem + C::kOffPlan);  // [0] first position, [1] end, [2 + warp] where a warp is
    int64_t* warp_sum = reinterpret_cast<int64_t*>(smem + C::kOffMisc);
    volatile int* abort_flag = reinterpret_cast<int*>(smem + C::kOffMisc + C::kThreads / 32 * 8);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc + C::kThreads / 32 * 8 + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int grid = gridDim.x;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&k_full[s], C::kConverters / 32);
            mbar_init(&k_empty[s], 2);  // both score issuers
            mbar_init(&v_full[s], C::kConverters / 32);
            mbar_init(&v_empty[s], 2);  // both value issuers
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(&q_full[x], 4);
            mbar_init(&s_full[x], 2);  // the products' completion, and the issuer itself (it has seen the step's table)
            for (int p = 0; p < 2; ++p) {
                mbar_init(&p_full[2 * x + p], 4);
                mbar_init(&pv_done[2 * x + p], 1);
            }
        }
        for (int i = 0; i < 4; ++i) mbar_init(&final_bar[i], 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    grid_dependency_wait();  // lengths, tables, codes and the workspace may come from the kernel before
    allow_dependents();
    const ChunkShape sh = shape_of(a);
    sum_costs(a, sh, prefix, warp_sum);
    const int ctas = chunk_ctas(prefix[a.batch], a.group, grid);
    if (lane == 0 && warp < 2) plan[warp] = chunk_cut(sh, prefix, static_cast<int>(blockIdx.x) + warp, ctas);
    __syncthreads();
    const ChunkPos first = plan[0], end = plan[1];
    PieceInfo* info = static_cast<PieceInfo*>(a.workspace) + blockIdx.x;
    if (first == end || first.seq >= a.batch) {  // nothing here
        if (threadIdx.x == 0) {
            info->start = first;
            info->flags = 0;
        }
        return;
    }
    if (warp == C::kScoreWarp) {
        tmem_alloc(tmem_slot, C::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    // Registers: launched with 96 a thread, 61440 together, which 256 softmax
    // threads at 144, 256 converters at 72 and 128 issuers at 48 share.
    if (warp < C::kSoftmaxWarps) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 144;");
        // ------------------------------------------------ softmax: half x, query row 32 (warp % 4) + lane of it
        const int x = warp >> 2;
        const int rr = (warp & 3) * 32 + lane;
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t col_s = tmem + lane_base + C::kColS + 128 * x;
        const uint32_t col_o = tmem + lane_base + C::kColO + 128 * x;
        int it = 0;      // steps this half has taken
        int table = 0;   // steps of the CTA
        int flags = 0;
        bool ok = true;
        ChunkPos cur = first;
        ChunkSegment g;
        while (ok && chunk_segment(sh, cur, end, g)) {
            cur = chunk_after(sh, prefix, g);
            const int h = g.at.head;
            const int r0 = g.at.tile * kChunkRows + 128 * x;
            const int rows = g.q.nq * a.group - r0;  // rows of the half, if positive
            const int steps = g.s1 - g.at.s;
            if (rows <= 0) {
                table += steps;
                continue;
            }
            const bool row_ok = rr < rows;
            const int t = (r0 + rr) / a.group;
            const int64_t row = (static_cast<int64_t>(g.q.q0) + t) * a.q_heads + h * a.group + (r0 + rr - t * a.group);
            const int lim = row_ok ? g.q.n - g.q.nq + t : -1;  // the last token the row sees
            float row_f = 0.f;  // |scale| log2(e) over the power of two in q'
            {
                const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + row * D);
                uint4 v[D / 8];
                uint32_t top = 0;  // largest |q|, per half word
#pragma unroll
                for (int c = 0; c < D / 8; ++c) {
                    v[c] = row_ok ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
                    top = __vmaxu2(top, __vmaxu2(__vmaxu2(v[c].x & 0x7fff7fffu, v[c].y & 0x7fff7fffu),
                                                 __vmaxu2(v[c].z & 0x7fff7fffu, v[c].w & 0x7fff7fffu)));
                }
                // the row's largest goes to 2^14 .. 2^15 (a row with infinities is left as it is);
                // the scale's sign goes into q', a zero scale makes q' zero
                const int ex = static_cast<int>(max(top >> 16, top & 0xffffu) >> 7);  // biased exponent
                const int shift = ex == 255 || ex == 0 ? 0 : min(126, 141 - ex);  // -113 .. 126
                const float mul = a.scale == 0.f ? 0.f : copysignf(exp2_int(shift), a.scale);
                row_f = (a.scale == 0.f ? 1.f : fabsf(a.scale)) * kLog2e * exp2_int(-shift);
                uint8_t* qs = smem + C::kOffQ + x * C::kTileBytes + rr * 128;
#pragma unroll
                for (int c = 0; c < D / 8; ++c) {
                    const uint4 h = make_uint4(pack_f16x2(bf16lo_to_f32(v[c].x) * mul, bf16hi_to_f32(v[c].x) * mul),
                                               pack_f16x2(bf16lo_to_f32(v[c].y) * mul, bf16hi_to_f32(v[c].y) * mul),
                                               pack_f16x2(bf16lo_to_f32(v[c].z) * mul, bf16hi_to_f32(v[c].z) * mul),
                                               pack_f16x2(bf16lo_to_f32(v[c].w) * mul, bf16hi_to_f32(v[c].w) * mul));
                    *reinterpret_cast<uint4*>(qs + (c >> 3) * C::kPartBytes + (((c & 7) ^ (rr & 7)) << 4)) = h;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&q_full[x]);
            }
            const int warp_lim = __reduce_min_sync(0xffffffffu, lim);
            float m = ninf(), l = 0.f, unit = 1.f;
            for (int j = 0; j < steps; ++j, ++it, ++table) {
                if (!warp_wait(&s_full[x], it & 1, a.status, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const float* tab = reinterpret_cast<const float*>(smem + C::kOffTable + (table & (C::kTables - 1)) * C::kTableBytes);
                const float4 modes = *reinterpret_cast<const float4*>(tab);
                unit = modes.x;
                const bool plain = modes.z == 0.f;
                // never 0 or infinite: a hidden score is -inf times it
                const float f = plain ? fminf(fmaxf(row_f * modes.y, 1.2e-38f), 3e38f) : row_f;
                const int seen = lim - (g.at.s + j) * kChunkStep + 1;  // tokens of the step the row sees
                const bool masked = (g.at.s + j + 1) * kChunkStep - 1 > warp_lim;
#pragma unroll 1
                for (int part = 0; part < 2; ++part) {
                    const float* cp = tab + 4 + 64 * part;  // of a slow step
                    const int seen_part = seen - 64 * part;
                    const uint32_t col = col_s + 64 * part;
                    float sx[64];
                    float mx;
                    if (plain) {
                        {
                            uint32_t lo[32], hi[32];
                            tmem_ld32(col, lo);
                            tmem_ld32(col + 32, hi);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                sx[e] = __uint_as_float(lo[e]);
                                sx[32 + e] = __uint_as_float(hi[e]);
                            }
                        }
                        if (masked) {
#pragma unroll
                            for (int e = 0; e < 64; ++e)
                                if (e >= seen_part) sx[e] = ninf();
                        }
                        float m1[21];
#pragma unroll
                        for (int k = 0; k < 21; ++k) m1[k] = fmax3(sx[3 * k], sx[3 * k + 1], sx[3 * k + 2]);
#pragma unroll
                        for (int k = 0; k < 7; ++k) m1[k] = fmax3(m1[3 * k], m1[3 * k + 1], m1[3 * k + 2]);
                        mx = fmax3(fmax3(m1[0], m1[1], m1[2]), fmax3(m1[3], m1[4], m1[5]), fmaxf(m1[6], sx[63])) * f;
                    } else {
                        mx = ninf();
#pragma unroll 1
                        for (int c = 0; c < 64; c += 8) {
                            float xe[8];
                            slow_scores(col + c, cp + c, f, seen_part - c, xe);
#pragma unroll
                            for (int e = 0; e < 8; ++e) mx = fmaxf(mx, xe[e] == ninf() ? ninf() : xe[e] + cp[128 + c + e]);
                        }
                    }
                    const bool resc = mx > m + 8.f;
                    // O holds something once a part of this segment has been multiplied in
                    if (__any_sync(0xffffffffu, resc)) {
                        float alpha = 1.f;
                        if (resc) {
                            const float mn = fmaxf(m, mx);
                            alpha = m == ninf() ? 0.f : ex2(m - mn);
                            m = mn;
                            l *= alpha;
                        }
                        if (j + part > 0) {
                            // part 0: the products of the step before completed ahead of these scores
                            if (part == 1 && !warp_wait(&pv_done[2 * x], it & 1, a.status, abort_flag)) {
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
                    if (plain) {
                        const uint64_t nb2 = f32x2_pack(-base, -base), f2 = f32x2_pack(f, f);
                        uint64_t acc0 = f32x2_pack(0.f, 0.f), acc1 = acc0;
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            uint32_t pw[16];
#pragma unroll
                            for (int e = 0; e < 32; e += 2) {
                                float a0, a1;
                                f32x2_unpack(f32x2_fma(f32x2_pack(sx[32 * half + e], sx[32 * half + e + 1]), f2, nb2), a0, a1);
                                const float p0 = ex2(a0), p1 = ex2(a1);
                                pw[e / 2] = pack_f16x2(p0, p1);
                                if ((e / 2) & 1)
                                    acc1 = f32x2_add(acc1, f32x2_pack(p0, p1));
                                else
                                    acc0 = f32x2_add(acc0, f32x2_pack(p0, p1));
                            }
                            tmem_st16(col_s + 32 * part + 16 * half, pw);
                        }
                        float s0, s1;
                        f32x2_unpack(f32x2_add(acc0, acc1), s0, s1);
                        l += s0 + s1;
                    } else {
                        // the weights overwrite scores that have been read
#pragma unroll 1
                        for (int c = 0; c < 64; c += 8) {
                            float xe[8], w[8];
                            slow_scores(col + c, cp + c, f, seen_part - c, xe);
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                w[e] = xe[e] == ninf() ? 0.f : ex2(xe[e] + cp[128 + c + e] - base);
                                l += xe[e] == ninf() ? 0.f : ex2(xe[e] - base);
                            }
                            const uint32_t pw[4] = {pack_f16x2(w[0], w[1]), pack_f16x2(w[2], w[3]), pack_f16x2(w[4], w[5]),
                                                    pack_f16x2(w[6], w[7])};
                            tmem_st4(col_s + 32 * part + c / 2, pw);
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
            if (!warp_wait(&pv_done[2 * x + 1], (it - 1) & 1, a.status, abort_flag)) {
                ok = false;
                break;
            }
            tc_fence_after();
            if (g.whole()) {
                const float inv = l == 0.f ? 0.f : unit / l;
                __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + row * D;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t ov[32];
                    tmem_ld32(col_o + c, ov);
                    tmem_ld_wait();
                    if (row_ok) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            uint32_t w[4];
#pragma unroll
                            for (int u = 0; u < 4; ++u)
                                w[u] = pack_bf16x2(__uint_as_float(ov[e + 2 * u]) * inv, __uint_as_float(ov[e + 2 * u + 1]) * inv);
                            *reinterpret_cast<uint4*>(dst + c + e) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                }
            } else {
                const int slot = g.at.s > 0 ? 0 : 1;
                flags |= 1 << slot;
                float* piece = slot_of(a.workspace, grid, D, blockIdx.x, slot);
                float* dst = piece + (128 * x + rr) * D;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t ov[32];
                    tmem_ld32(col_o + c, ov);
                    tmem_ld_wait();
                    if (row_ok) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<float4*>(dst + c + e) =
                                make_float4(__uint_as_float(ov[e]) * unit, __uint_as_float(ov[e + 1]) * unit,
                                            __uint_as_float(ov[e + 2]) * unit, __uint_as_float(ov[e + 3]) * unit);
                    }
                }
                if (row_ok) {
                    piece[kChunkRows * D + 128 * x + rr] = m;
                    piece[kChunkRows * (D + 1) + 128 * x + rr] = l;
                }
            }
            tc_fence_before();  // the next segment's products overwrite O after this half's next arrival
        }
        if (threadIdx.x == 0) {  // half A takes part in every segment
            info->start = first;
            info->flags = ok ? flags : 0;
        }
    } else if (warp < C::kScoreWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        ChunkPos* after = plan + 2 + warp;  // every warp its own
        if (warp < C::kConvertWarp + 4)
            convert_role<D, false>(a, sh, smem, prefix, plan, after, k_full, k_empty, abort_flag);
        else
            convert_role<D, true>(a, sh, smem, prefix, plan, after, v_full, v_empty, abort_flag);
    } else if (warp < C::kValueWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
        // ------------------------------------------------ scores S = Q K^T of half x (one thread)
        const int x = warp - C::kScoreWarp;
        if (lane == 0) {
            constexpr uint32_t idS = umma_idesc_f16(128, 128);
            const uint32_t q_base = smem_u32(smem + C::kOffQ + x * C::kTileBytes);
            int step = 0, it = 0, segs = 0;
            bool ok = true;
            ChunkPos cur = first;
            ChunkSegment g;
            while (ok && chunk_segment(sh, cur, end, g)) {
                cur = chunk_after(sh, prefix, g);
                const bool mine = g.q.nq * a.group - g.at.tile * kChunkRows > 128 * x;
                if (mine) {
                    if (!mbar_wait(&q_full[x], segs & 1, a.status, abort_flag)) break;
                    ++segs;
                }
                for (int j = g.at.s; j < g.s1; ++j, ++step) {
                    const int st = step & 1;
                    if (mine && it > 0 && !mbar_wait(&pv_done[2 * x + 1], (it - 1) & 1, a.status, abort_flag)) {
                        ok = false;
                        break;
                    }
                    if (!mbar_wait(&k_full[st], (step >> 1) & 1, a.status, abort_flag)) {
                        ok = false;
                        break;
                    }
                    if (!mine) {
                        mbar_arrive(&k_empty[st]);
                        continue;
                    }
                    tc_fence_after();
                    const uint32_t k_base = smem_u32(smem + C::kOffK + st * C::kTileBytes);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = (kk >> 2) * C::kPartBytes + (kk & 3) * 32;
                        umma_bf16(tmem + C::kColS + 128 * x, umma_desc_sw128(q_base + off, 16, 1024),
                                  umma_desc_sw128(k_base + off, 16, 1024), idS, kk > 0 ? 1u : 0u);
                    }
                    umma_commit(&k_empty[st]);
                    umma_commit(&s_full[x]);
                    mbar_arrive(&s_full[x]);
                    ++it;
                }
            }
            umma_commit(&final_bar[x]);
            mbar_wait(&final_bar[x], 0, a.status, nullptr);
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
        // ------------------------------------------------ values O += P V of half x (one thread)
        const int x = warp - C::kValueWarp;
        if (lane == 0) {
            constexpr uint32_t idO = umma_idesc_f16(128, D);
            int step = 0, it = 0;
            bool ok = true;
            ChunkPos cur = first;
            ChunkSegment g;
            while (ok && chunk_segment(sh, cur, end, g)) {
                cur = chunk_after(sh, prefix, g);
                const bool mine = g.q.nq * a.group - g.at.tile * kChunkRows > 128 * x;
                for (int j = g.at.s; ok && j < g.s1; ++j, ++step) {
                    const int st = step & 1;
                    if (!mbar_wait(&v_full[st], (step >> 1) & 1, a.status, abort_flag)) {
                        ok = false;
                        break;
                    }
                    if (!mine) {
                        mbar_arrive(&v_empty[st]);
                        continue;
                    }
                    const uint32_t v_base = smem_u32(smem + C::kOffV + st * C::kVBytes);
#pragma unroll 1
                    for (int part = 0; part < 2; ++part) {
                        if (!mbar_wait(&p_full[2 * x + part], it & 1, a.status, abort_flag)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma_bf16_ts(tmem + C::kColO + 128 * x, tmem + C::kColS + 128 * x + 32 * part + 8 * kk,
                                         umma_desc_sw128(v_base + part * C::kVPartBytes + kk * 32, 16, 1024), idO,
                                         (j > g.at.s || part > 0 || kk > 0) ? 1u : 0u);
                        umma_commit(&pv_done[2 * x + part]);
                    }
                    if (!ok) break;
                    umma_commit(&v_empty[st]);
                    ++it;
                }
            }
            umma_commit(&final_bar[2 + x]);
            mbar_wait(&final_bar[2 + x], 0, a.status, nullptr);
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
// of c, then slot 0 of the following CTAs while they begin inside it), rows
// 32 y .. 32 y + 31, a warp per row: out = sum_i O_i 2^(m_i - M) / sum_i l_i 2^(m_i - M).
constexpr int kCombineRows = 32;
constexpr int kCombineThreads = 256;
constexpr int kMaxPieces = 1024;

template <int D>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(const ChunkArgs a, int grid) {
    __shared__ int pieces[kMaxPieces];  // 2 cta + slot
    __shared__ int count;
    grid_dependency_wait();
    allow_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = blockIdx.x;
    const PieceInfo* infos = static_cast<const PieceInfo*>(a.workspace);
    if (!(infos[c].flags & 2) || c + 1 >= grid) return;
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
    __syncthreads();
    const ChunkShape sh = shape_of(a);
    ChunkSeq q;
    chunk_seq(sh, unit.seq, q);
    const int r0 = unit.tile * kChunkRows;
    const int rows = min(kChunkRows, q.nq * a.group - r0);
    constexpr int kPer = D / 32;
    for (int r = blockIdx.y * kCombineRows + warp; r < min(rows, static_cast<int>(blockIdx.y + 1) * kCombineRows); r += kCombineThreads / 32) {
        float top = ninf();
        for (int i = lane; i < count; i += 32) {
            const float* p = slot_of(a.workspace, grid, D, pieces[i] >> 1, pieces[i] & 1);
            top = fmaxf(top, p[kChunkRows * D + r]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float base = top == ninf() ? 0.f : top;
        float l = 0.f, acc[kPer];
#pragma unroll
        for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
        for (int i = 0; i < count; ++i) {
            const float* p = slot_of(a.workspace, grid, D, pieces[i] >> 1, pieces[i] & 1);
            const float w = ex2(p[kChunkRows * D + r] - base);
            l += w * p[kChunkRows * (D + 1) + r];
            const float* src = p + r * D + lane * kPer;
#pragma unroll
            for (int e = 0; e < kPer; ++e) acc[e] += w * src[e];
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int t = (r0 + r) / a.group;
        const int64_t row = (static_cast<int64_t>(q.q0) + t) * a.q_heads + unit.head * a.group + (r0 + r - t * a.group);
        uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + row * D) + lane * (kPer / 2);
#pragma unroll
        for (int e = 0; e < kPer; e += 2) dst[e / 2] = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
    }
}

// CTAs of a launch: one per SM (piece lists hold at most kMaxPieces).
int chunk_q8_ctas() { return device_sm_count() < kMaxPieces ? device_sm_count() : kMaxPieces; }

template <int D>
cudaError_t run_chunk(const ChunkArgs& a, cudaStream_t s) {
    const int grid = chunk_q8_ctas();
    cudaError_t e = cudaFuncSetAttribute(chunk_q8_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(Cx<D>::kSmem));
    if (e != cudaSuccess) return e;
    e = launch_pdl(chunk_q8_kernel<D>, dim3(grid), dim3(Cx<D>::kThreads), Cx<D>::kSmem, s, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(combine_kernel<D>, dim3(grid, kChunkRows / kCombineRows), dim3(kCombineThreads), 0, s, a, grid);
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
