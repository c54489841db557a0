// Causal attention of a chunk of new tokens over the int8 pools
// (pkv_multiquery_attention_q8 in include/pkv.h), for more than 32 query rows
// per (sequence, KV head) or head_dim 64.
//
// Mathematics, per query row and step of 128 tokens:
//     s_p = q . kc_p                    bf16 x bf16 -> fp32 (q and the codes exact)
//     x_p = s_p * c_p,  c_p = ks_p * scale * log2(e)                        fp32
//     w_p = 2^(x_p - m)                 m: running maximum, moved only when a
//                                       score exceeds it by more than 8 (w <= 2^8)
//     l  += w_p;   O += w_p v_p         w rounded to f16; v_p = vc_p (vs_p 2^-E)
//                                       rounded to f16; fp32 sums
//     out = 2^E O / l
// E is one exponent per piece of work, taken from its first step, that puts V
// into the f16 range whatever its size. A later step whose V scales leave
// [2^-14, 2^8] 2^E (rows 2^22 apart; or infinities) takes the codes themselves as
// v_p and moves the scale into the weight, w_p = 2^(x_p + log2(vs_p) - E - m), with
// l summed apart: slower, and exact over the whole float range, because the
// maximum is then taken over tokens the row sees.
//
// Work (pkv_chunk_schedule.cuh): one persistent CTA per SM takes a range of
// (unit, step) pairs, a unit being 256 query rows of a (sequence, KV head) as
// two row halves A and B of 128. A unit cut by a range leaves fp32 pieces
// (O, m, l) in the workspace, which combine_kernel joins.
//
// Roles (20 warps). Warps 0-3 and 4-7: the softmax of halves A and B, one thread
// per query row. Warps 8-11 and 12-15: the converters of K and of V; they load
// the codes of the next step from global memory into registers while they turn
// the previous loads into bf16 (K) or scaled f16 (V), in the 128-byte-swizzled
// layout the tensor cores read; K's also write the step's factors c_p. Warps 16
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
// The factor c of an absent token (a block id outside the pool): a NaN that no
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
    // a table: c [128], log2(vs) - E [128] (0 unless the step is wide; written for
    // wide steps and for those with absent tokens), then 2^E and 1 for such a step
    static constexpr int kTableBytes = 2 * 128 * 4 + 16;
    static constexpr int kOffScale = kOffTable + kTables * kTableBytes;  // f16 V factors [2][128]
    static constexpr int kOffReduce = kOffScale + 512;                   // K, V: [2][4 warps] of 16 bytes
    static constexpr int kOffBars = kOffReduce + 256;
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
// Two codes (bytes 0 and 2 of `h`, the others 0x43) -> bf16x2, exactly: the byte
// under exponent 0x43 without its top bit is 128 + (code mod 128); the top bit
// alone is 128, or 256 for a negative code.
__device__ __forceinline__ uint32_t codes_bf16x2(uint32_t h) {
    const uint32_t a = h & 0xff7fff7fu, b = h & 0xff80ff80u;
    const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}
// Two codes + 128 (bytes 0 and 2, the others 0x64: 1024 + code + 128 in f16)
// times two f16 factors.
__device__ __forceinline__ uint32_t codes_f16x2(uint32_t h, uint32_t factors) {
    const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
    const __half2 r = __hmul2(__hsub2(*reinterpret_cast<const __half2*>(&h), bias), *reinterpret_cast<const __half2*>(&factors));
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint4 codes8_bf16(uint32_t w0, uint32_t w1) {
    return make_uint4(codes_bf16x2(__byte_perm(w0, 0x43434343u, 0x5140)), codes_bf16x2(__byte_perm(w0, 0x43434343u, 0x7362)),
                      codes_bf16x2(__byte_perm(w1, 0x43434343u, 0x5140)), codes_bf16x2(__byte_perm(w1, 0x43434343u, 0x7362)));
}
__device__ __forceinline__ uint4 codes8_f16(uint32_t w0, uint32_t w1, const uint4& f) {
    w0 ^= 0x80808080u;
    w1 ^= 0x80808080u;
    return make_uint4(codes_f16x2(__byte_perm(w0, 0x64646464u, 0x5140), f.x), codes_f16x2(__byte_perm(w0, 0x64646464u, 0x7362), f.y),
                      codes_f16x2(__byte_perm(w1, 0x64646464u, 0x5140), f.z), codes_f16x2(__byte_perm(w1, 0x64646464u, 0x7362), f.w));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint64_t f32x2_mul(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
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

// Eight scores of a step that is not plain, scaled, -inf where the token is absent or not
// seen (columns taddr .. taddr + 7, factors c, the first `seen` of them seen).
__device__ __forceinline__ void slow_scores(uint32_t taddr, const float* c, int seen, float (&x)[8]) {
    uint32_t v[8];
    tmem_ld8(taddr, v);
    tmem_ld_wait();
#pragma unroll
    for (int e = 0; e < 8; ++e)
        x[e] = e >= seen || __float_as_uint(c[e]) == kAbsent ? ninf() : __uint_as_float(v[e]) * c[e];
}
// mbar_wait by a whole warp, with one answer for all its lanes.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, unsigned int* status, volatile int* abort) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, status, abort));
}

// ---------------------------------------------------------------- converters
// K's (IsV false) or V's four warps: every step of the CTA's range, one load
// ahead. The V scales' range decides a step's mode and a segment's exponent; both
// groups read the scales and decide alike.
template <int D, bool IsV>
__device__ void convert_role(const ChunkArgs& a, const ChunkShape& sh, uint8_t* smem, const int64_t* prefix,
                             const ChunkPos* plan, ChunkPos* after, uint64_t* full, uint64_t* empty,
                             volatile int* abort_flag) {
    using C = Cx<D>;
    const int lane = threadIdx.x & 31;
    const int cw = (threadIdx.x >> 5) & 3;
    const int tid = cw * 32 + lane;
    constexpr int kVecs = 128 * D / 16 / C::kConverters;  // 16-code vectors per thread and step
    constexpr int kBlockVecs = D;                         // vectors of one (block, head)
    constexpr int kBarrier = IsV ? 2 : 1;
    const uint4* codes = static_cast<const uint4*>(IsV ? a.v_codes : a.k_codes);
    uint32_t (*reduce)[4][4] = reinterpret_cast<uint32_t (*)[4][4]>(smem + C::kOffReduce + (IsV ? 128 : 0));
    const float cscale = a.scale * kLog2e;

    // the segment being loaded (the position after it: in shared memory, one per warp, read once per segment)
    if (lane == 0) *after = plan[0];
    __syncwarp();
    int step = 0, last = 0;            // next step to load, one past the segment's last
    int n = 0, head = 0;               // its tokens, KV head
    const int32_t* trow = nullptr;     // its block table
    int ids = 0, ids_next = 0;         // lane l: id of block 32 b + l (-1: past the end, -2: outside the pool), b = step / 4; b + 1
    bool opens = false;                // the loaded step is its segment's first
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
    // the loaded step: codes, scales of token `tid`, whether it exists or lies in a block outside the pool
    uint4 w[kVecs];
    float ks = 0.f, vs = 0.f;
    bool present = false, missing = false;
    auto load = [&]() {
        const int b0 = (step & 3) * 8;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int v = tid + i * C::kConverters;
            // an absent block's codes may be any (its tokens carry no weight): block 0 exists
            const int id = max(0, __shfl_sync(0xffffffffu, ids, b0 + v / kBlockVecs));
            w[i] = __ldg(codes + (static_cast<int64_t>(id) * a.kv_heads + head) * kBlockVecs + v % kBlockVecs);
        }
        const int id = __shfl_sync(0xffffffffu, ids, b0 + (tid >> 4));
        present = id >= 0 && step * kChunkStep + tid < n;
        missing = id == -2;
        const float* rec = a.scales + (static_cast<int64_t>(max(0, id)) * a.kv_heads + head) * 32 + (tid & 15);
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
    int exponent = 0;   // E of the segment
    bool have = false;  // E is set
    for (int it = 0; live; ++it) {
        const int st = it & 1;
        if (opens) have = false;
        // ---- range of the V scales of the tokens that exist; absent tokens
        const uint32_t vbits = __float_as_uint(vs) & 0x7fffffffu;
        const uint32_t wmax = __reduce_max_sync(0xffffffffu, present ? vbits : 0u);
        const uint32_t wmin = __reduce_min_sync(0xffffffffu, present ? vbits : 0xffffffffu);
        const uint32_t wmiss = __any_sync(0xffffffffu, missing);
        if (lane == 0) *reinterpret_cast<uint4*>(reduce[st][cw]) = make_uint4(wmax, wmin, wmiss, 0u);
        __half* factors = reinterpret_cast<__half*>(smem + C::kOffScale) + 128 * st;
        const float before = __uint_as_float(static_cast<uint32_t>(127 - exponent) << 23);
        if (IsV) factors[tid] = __float2half(present ? vs * before : 0.f);  // right unless E or the mode changes below
        const bool go = mbar_wait(&empty[st], static_cast<uint32_t>((it >> 1) & 1) ^ 1u, a.status, abort_flag);
        if (!named_barrier_all(kBarrier, C::kConverters, go)) break;
        uint32_t vmax = 0, vmin = 0xffffffffu, miss = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 r = *reinterpret_cast<const uint4*>(reduce[st][i]);
            vmax = max(vmax, r.x);
            vmin = min(vmin, r.y);
            miss |= r.z;
        }
        bool wide = false;
        const int old = exponent;
        if (vmin != 0xffffffffu) {
            if (!have) {
                // the first step with tokens: its largest scale (smallest, beside an infinity) goes to 1/2 .. 1
                const uint32_t ref = vmax < 0x7f800000u ? vmax : (vmin < 0x7f800000u ? vmin : 0x3f800000u);
                exponent = max(-125, min(125, static_cast<int>(ref >> 23) - 126));
                have = true;
            }
            // outside [2^(E - 14), 2^(E + 8)] (bits compare as the floats do)
            const int lo = max(exponent - 14, -126) + 127, hi = min(exponent + 8, 127) + 127;
            wide = vmin < static_cast<uint32_t>(lo) << 23 || vmax > static_cast<uint32_t>(hi) << 23;
        }
        if (IsV) {
            if (wide || exponent != old) {
                const float down = __uint_as_float(static_cast<uint32_t>(127 - exponent) << 23);
                factors[tid] = __float2half(!present ? 0.f : wide ? 1.f : vs * down);
                if (!named_barrier_all(kBarrier, C::kConverters, true)) break;
            }
            // ---- coordinate rows, 64 tokens each
            uint8_t* vd = smem + C::kOffV + st * C::kVBytes;
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const int v = tid + i * C::kConverters;
                const int block = v / kBlockVecs, d = v % kBlockVecs;
                const uint4* f = reinterpret_cast<const uint4*>(factors + 16 * block);
                uint8_t* rowp = vd + (block >> 2) * C::kVPartBytes + d * 128;
                const int c0 = (block & 3) * 2;
                *reinterpret_cast<uint4*>(rowp + ((c0 ^ (d & 7)) << 4)) = codes8_f16(w[i].x, w[i].y, f[0]);
                *reinterpret_cast<uint4*>(rowp + (((c0 + 1) ^ (d & 7)) << 4)) = codes8_f16(w[i].z, w[i].w, f[1]);
            }
        } else {
            uint8_t* tab = smem + C::kOffTable + (it & (C::kTables - 1)) * C::kTableBytes;
            float* cs = reinterpret_cast<float*>(tab);
            cs[tid] = missing ? __uint_as_float(kAbsent) : present ? ks * cscale : 0.f;
            if (wide || miss)  // a scale below the normal range counts as its smallest number
                cs[128 + tid] = present && wide ? log2f(vbits < 0x00800000u ? 1.17549435e-38f : vs) - static_cast<float>(exponent) : 0.f;
            if (tid == 0) {
                cs[256] = __uint_as_float(static_cast<uint32_t>(127 + exponent) << 23);
                reinterpret_cast<int*>(tab)[257] = wide || miss;
            }
            // ---- token rows
            uint8_t* kd = smem + C::kOffK + st * C::kTileBytes;
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const int v = tid + i * C::kConverters;
                const int token = v / (D / 16), ch = v % (D / 16);
                const uint4 lo = codes8_bf16(w[i].x, w[i].y), hi = codes8_bf16(w[i].z, w[i].w);
                uint8_t* rowp = kd + (ch >> 2) * C::kPartBytes + token * 128;
                // lanes of the second column part write their halves in the other order: no bank is hit twice
                const int flip = (ch >> 2) & 1;
                const int c0 = (ch & 3) * 2 + flip;
                *reinterpret_cast<uint4*>(rowp + ((c0 ^ (token & 7)) << 4)) = flip ? hi : lo;
                *reinterpret_cast<uint4*>(rowp + (((c0 ^ 1) ^ (token & 7)) << 4)) = flip ? lo : hi;
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
            {
                const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + row * D);
                uint8_t* qs = smem + C::kOffQ + x * C::kTileBytes + rr * 128;
#pragma unroll
                for (int c = 0; c < D / 8; ++c) {
                    const uint4 v = row_ok ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
                    *reinterpret_cast<uint4*>(qs + (c >> 3) * C::kPartBytes + (((c & 7) ^ (rr & 7)) << 4)) = v;
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
                const uint8_t* tab = smem + C::kOffTable + (table & (C::kTables - 1)) * C::kTableBytes;
                const float* cs = reinterpret_cast<const float*>(tab);
                unit = cs[256];
                const bool plain = reinterpret_cast<const int*>(tab)[257] == 0;
                const int seen = lim - (g.at.s + j) * kChunkStep + 1;  // tokens of the step the row sees
                const bool masked = (g.at.s + j + 1) * kChunkStep - 1 > warp_lim;
#pragma unroll 1
                for (int part = 0; part < 2; ++part) {
                    const float* cp = cs + 64 * part;
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
#pragma unroll
                        for (int e = 0; e < 64; e += 4) {
                            const ulonglong2 c4 = *reinterpret_cast<const ulonglong2*>(cp + e);
                            f32x2_unpack(f32x2_mul(f32x2_pack(sx[e], sx[e + 1]), c4.x), sx[e], sx[e + 1]);
                            f32x2_unpack(f32x2_mul(f32x2_pack(sx[e + 2], sx[e + 3]), c4.y), sx[e + 2], sx[e + 3]);
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
                        mx = fmax3(fmax3(m1[0], m1[1], m1[2]), fmax3(m1[3], m1[4], m1[5]), fmaxf(m1[6], sx[63]));
                    } else {
                        mx = ninf();
#pragma unroll 1
                        for (int c = 0; c < 64; c += 8) {
                            float xe[8];
                            slow_scores(col + c, cp + c, seen_part - c, xe);
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
                        const uint64_t nb2 = f32x2_pack(-base, -base);
                        uint64_t acc0 = f32x2_pack(0.f, 0.f), acc1 = acc0;
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            uint32_t pw[16];
#pragma unroll
                            for (int e = 0; e < 32; e += 2) {
                                float a0, a1;
                                f32x2_unpack(f32x2_add(f32x2_pack(sx[32 * half + e], sx[32 * half + e + 1]), nb2), a0, a1);
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
                            slow_scores(col + c, cp + c, seen_part - c, xe);
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
            constexpr uint32_t idS = umma_idesc_bf16(128, 128, false, false);
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
