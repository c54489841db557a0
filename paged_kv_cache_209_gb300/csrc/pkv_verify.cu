// Verification of drafted tokens against the target's probabilities
// (pkv_verify_drafts in include/pkv.h).
//
// Sequence i keeps its leading drafts with u_j q_j(x_j) < p_j(x_j) -- both sides
// products of two 24-bit significands, exact in float64, so the decision is the
// one of exact arithmetic -- and draws one more token from r = max(p_a - q_a, 0)
// (the rejected position) or r = p_k (none rejected): the lowest index whose
// running sum exceeds w * sum(r).
//
// Sums. A draw next to a border must not depend on how the sum was split, so
// running sums carry far more than float32: entries, lanes, segments and slices are
// added in pairs of floats (the exact error of each addition is kept, about 2^-46
// relative), in a fixed order. Sums in float64 cost too much on this part (two
// additions per SM and clock, and a long latency) even where they are few: for the
// segments and slices alone 40 of 80 us on 200 sequences of 50001 entries, for the
// walk through the drawn segment 4 us of one sequence's 12.
//
// A cluster of CTAs per sequence, each with a slice of the vocabulary: the warps
// take the slice's segments in turn (32 loads of each row in flight per lane) and
// leave their sums in shared memory; the CTAs read one another's totals through
// distributed shared memory, and the one whose slice holds the draw finds the segment
// and scans its entries again (from L2). One launch, nothing in global memory but
// the results. What bounds it: a few sequences, the chain of the acceptance test, the
// row, the totals and the segment (7.3 us for one of 32000 entries); many, the latency of
// the loads with few warps to hide it: 32 sequences are 256 CTAs of 4 warps, under 7 warps
// an SM, whose loads are of one element a lane (32 of 131072 float32 entries: 11.5 us,
// 39 % of the copy rate; issue slots 18 % used, ALU and FMA pipes 10 %, DRAM 18 %, the
// stalls are long-scoreboard and barrier).
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kSeg = 256;         // entries per segment
constexpr int kPer = kSeg / 32;   // of them per lane
constexpr int kGroup = 4;         // segments a warp loads at once
constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCtas = 8;       // per cluster (the portable maximum)
constexpr int kMaxSegs = kMaxVocab / kSeg;

__device__ __forceinline__ float load_prob(const float* p, int64_t i) { return __ldg(p + i); }
__device__ __forceinline__ float load_prob(const __nv_bfloat16* p, int64_t i) {
    return __bfloat162float(p[i]);
}

// The mass an entry of r carries: a finite number above zero, else none.
__device__ __forceinline__ float mass_of(float x) { return x > 0.f && x <= 3.402823466e38f ? x : 0.f; }

// r at index v: the target row alone, or less the draft's row (or less the
// certain draft's 1 at token x). Both rows are always loaded, without a branch
// between the loads of a warp; with nothing to subtract q is p and counts zero times.
template <typename T>
struct Rest {
    const T* p;
    const T* q;
    float times;  // 1, or 0: nothing to subtract
    int certain;  // >= 0: the draft was certain of this token
    __device__ __forceinline__ float at(int v) const {
        float x = fmaf(-times, load_prob(q, v), load_prob(p, v));
        if (v == certain) x -= 1.f;
        return mass_of(x);
    }
    __device__ __forceinline__ void alone() {
        q = p;
        times = 0.f;
        certain = -1;
    }
};

// s + c += x with s the rounded sum and c the accumulated rounding errors.
__device__ __forceinline__ void add_two(float& s, float& c, float x) {
    const float t = s + x;
    const float z = t - s;
    c += (s - (t - z)) + (x - z);
    s = t;
}
// A sum and its rounding errors.
struct Pair {
    float s, c;
    // s - o.s is exact where the two lie close
    __device__ __forceinline__ bool operator>(const Pair& o) const { return (s - o.s) + (c - o.c) > 0.f; }
};
__device__ __forceinline__ Pair operator+(const Pair& a, const Pair& b) {
    Pair r{a.s, a.c};
    add_two(r.s, r.c, b.s);
    r.c += b.c;
    return r;
}
__device__ __forceinline__ Pair shuffle_up(const Pair& x, int o) {
    return Pair{__shfl_up_sync(0xffffffffu, x.s, o), __shfl_up_sync(0xffffffffu, x.c, o)};
}
__device__ __forceinline__ Pair shuffle(const Pair& x, int lane) {
    return Pair{__shfl_sync(0xffffffffu, x.s, lane), __shfl_sync(0xffffffffu, x.c, lane)};
}
// Inclusive sums over the warp's lanes, in a fixed order; `before`: the exclusive ones.
__device__ __forceinline__ Pair warp_scan(Pair x, int lane, Pair& before) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Pair other = shuffle_up(x, o);
        if (lane >= o) x = other + x;
    }
    before = shuffle_up(x, 1);
    if (lane == 0) before = Pair{0.f, 0.f};
    return x;
}
__device__ __forceinline__ Pair ld_cluster_pair(uint32_t addr) {
    Pair v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.s), "=f"(v.c) : "r"(addr) : "memory");
    return v;
}

// The masses of segments sg .. sg + kGroup - 1 below `end` into seg_sum;
// returns their sum (the same in every lane). All loads go out before the first sum.
template <typename T>
__device__ Pair group_sum(const Rest<T>& r, int sg, int end, int vocab, int lane, Pair* seg_sum) {
    float x[kGroup][kPer];
    const int v0 = sg * kSeg + lane;
    const int limit = min(vocab, end * kSeg);
    if ((sg + kGroup) * kSeg <= limit) {
#pragma unroll
        for (int g = 0; g < kGroup; ++g)
#pragma unroll
            for (int e = 0; e < kPer; ++e) x[g][e] = r.at(v0 + g * kSeg + 32 * e);
    } else {
#pragma unroll
        for (int g = 0; g < kGroup; ++g)
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                const int v = v0 + g * kSeg + 32 * e;
                x[g][e] = v < limit ? r.at(v) : 0.f;
            }
    }
    Pair sum[kGroup];
#pragma unroll
    for (int g = 0; g < kGroup; ++g) {
        sum[g] = Pair{x[g][0], 0.f};
#pragma unroll
        for (int e = 1; e < kPer; ++e) add_two(sum[g].s, sum[g].c, x[g][e]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
        for (int g = 0; g < kGroup; ++g)
            sum[g] = sum[g] + Pair{__shfl_xor_sync(0xffffffffu, sum[g].s, o), __shfl_xor_sync(0xffffffffu, sum[g].c, o)};
    }
    Pair all{0.f, 0.f};
#pragma unroll
    for (int g = 0; g < kGroup; ++g) {
        if (lane == 0 && sg + g < end) seg_sum[g] = sum[g];
        all = all + sum[g];
    }
    return all;
}

// The draw inside segment sg (one warp): the lowest index whose running sum, from
// `before` on, exceeds `aim`, else the last index with mass. `stage`: kSeg floats.
template <typename T>
__device__ int segment_draw(const Rest<T>& r, int sg, int vocab, int lane, const Pair& before, const Pair& aim, float* stage) {
    // entry i lies at i + i / kPer: a lane's kPer consecutive entries meet no bank twice
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        const int i = 32 * e + lane, v = sg * kSeg + i;
        stage[i + i / kPer] = v < vocab ? r.at(v) : 0.f;
    }
    __syncwarp();
    const float* x = stage + lane * (kPer + 1);
    Pair mine{0.f, 0.f}, lanes_before;
#pragma unroll
    for (int e = 0; e < kPer; ++e) add_two(mine.s, mine.c, x[e]);
    warp_scan(mine, lane, lanes_before);
    Pair cum = before + lanes_before;
    int hit = INT_MAX, last = -1;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        add_two(cum.s, cum.c, x[e]);
        if (x[e] > 0.f) {
            last = sg * kSeg + lane * kPer + e;
            if (cum > aim && hit == INT_MAX) hit = last;
        }
    }
    hit = __reduce_min_sync(0xffffffffu, hit);
    last = __reduce_max_sync(0xffffffffu, last);
    return hit != INT_MAX ? hit : last;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) verify_kernel(const VerifyArgs a) {
    __shared__ Pair seg_sum[kMaxSegs];
    __shared__ Pair warp_total[kWarps];
    __shared__ Pair cta_total[2];  // of the two attempts
    __shared__ float stage[kSeg + 32];
    __shared__ int shared_kept, shared_empty;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ctas = static_cast<int>(cluster_size());
    const int rank = static_cast<int>(cluster_ctarank());
    const int i = blockIdx.x / ctas;
    grid_dependency_wait();
    allow_dependents();
    const int t0 = a.query_start[i], d0 = a.draft_start[i];
    const int64_t rows = static_cast<int64_t>(a.query_start[i + 1]) - t0;
    const int64_t k64 = static_cast<int64_t>(a.draft_start[i + 1]) - d0;
    const bool idle = rows == 0 && k64 == 0;
    const bool bad = !idle && (k64 < 0 || k64 > a.max_draft_len || rows != k64 + 1 || t0 < 0 || d0 < 0 ||
                               t0 + rows > a.num_target_rows || d0 + k64 > a.num_draft_rows);
    int* out = a.out_tokens + static_cast<int64_t>(i) * (a.max_draft_len + 1);
    if (idle || bad) {  // for the whole cluster
        if (rank == 0) {
            for (int j = threadIdx.x; j <= a.max_draft_len; j += kThreads) out[j] = -1;
            if (threadIdx.x == 0) {
                a.num_accepted[i] = bad ? -1 : 0;
                if (a.new_lens != nullptr) a.new_lens[i] = a.lens[i];
                if (bad) atomicOr(a.status, PKV_DEVERR_RANGE);
            }
        }
        return;
    }
    const int k = static_cast<int>(k64);
    const T* target = static_cast<const T*>(a.target) + t0 * a.target_stride;
    const T* draft = a.draft == nullptr ? nullptr : static_cast<const T*>(a.draft) + d0 * a.draft_stride;
    if (warp == 0) {
        int kept = k;
        for (int base = 0; base < k && kept == k; base += 32) {
            const int j = base + lane;
            bool keep = true;
            if (j < k) {
                const int x = a.draft_tokens[d0 + j];
                const float u = a.accept[d0 + j];
                if (x < 0 || x >= a.vocab) {
                    if (rank == 0) atomicOr(a.status, PKV_DEVERR_RANGE);
                    keep = false;
                } else {
                    const double p = load_prob(target + j * a.target_stride, x);
                    const double q = draft == nullptr ? 1.0 : static_cast<double>(load_prob(draft + j * a.draft_stride, x));
                    keep = static_cast<double>(u) * q < p;
                }
            }
            const unsigned int no = __ballot_sync(0xffffffffu, !keep);
            if (no != 0) kept = base + __ffs(no) - 1;
        }
        if (lane == 0) shared_kept = kept;
    }
    __syncthreads();
    const int kept = shared_kept;
    const int segs = (a.vocab + kSeg - 1) / kSeg;
    const int first = static_cast<int>(static_cast<int64_t>(segs) * rank / ctas);
    const int end = static_cast<int>(static_cast<int64_t>(segs) * (rank + 1) / ctas);
    Rest<T> r;
    r.p = target + kept * a.target_stride;
    r.alone();
    const bool less = kept < k;  // a draft was rejected
    if (less && draft != nullptr) {
        r.q = draft + kept * a.draft_stride;
        r.times = 1.f;
    }
    if (less && draft == nullptr) r.certain = a.draft_tokens[d0 + kept];
    int y = -1;
    bool writer = rank == 0;  // who writes the results: the CTA that holds the draw, or the first if there is none
    // a second attempt, on p itself, where max(p - q, 0) holds nothing
    for (int attempt = 0; attempt < 2; ++attempt) {
        Pair mine{0.f, 0.f};
        for (int sg = first + warp * kGroup; sg < end; sg += kWarps * kGroup)
            mine = mine + group_sum(r, sg, end, a.vocab, lane, seg_sum + (sg - first));
        if (lane == 0) warp_total[warp] = mine;
        __syncthreads();
        if (threadIdx.x == 0) {
            Pair sum = warp_total[0];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) sum = sum + warp_total[w];
            cta_total[attempt] = sum;
        }
        cluster_sync();
        if (warp == 0) {
            // the CTAs' totals, one per lane
            Pair at{0.f, 0.f}, ctas_before;
            if (lane < ctas) at = ld_cluster_pair(mapa_shared(smem_u32(&cta_total[attempt]), lane));
            const Pair incl = warp_scan(at, lane, ctas_before);
            const Pair total = shuffle(incl, 31);
            const bool some = total.s > 0.f;
            if (lane == 0) shared_empty = !some;
            if (some) {
                const double product = static_cast<double>(a.sample[i]) * (static_cast<double>(total.s) + static_cast<double>(total.c));
                Pair aim{static_cast<float>(product), 0.f};
                aim.c = static_cast<float>(product - static_cast<double>(aim.s));
                // the CTA that holds the draw: the first whose running sum exceeds the aim, else the last with mass
                const unsigned int above = __ballot_sync(0xffffffffu, at.s > 0.f && incl > aim);
                const unsigned int mass = __ballot_sync(0xffffffffu, at.s > 0.f);
                const int holder = above != 0 ? __ffs(above) - 1 : 31 - __clz(mass);
                writer = rank == holder;
                if (writer) {
                    // its segment, likewise
                    Pair run = shuffle(ctas_before, rank), sg_before = run;
                    int sg = -1;
                    for (int s0 = 0; s0 < end - first; s0 += 32) {
                        const Pair x = s0 + lane < end - first ? seg_sum[s0 + lane] : Pair{0.f, 0.f};
                        Pair lanes_before;
                        const Pair seg_incl = warp_scan(x, lane, lanes_before);
                        const unsigned int over = __ballot_sync(0xffffffffu, x.s > 0.f && run + seg_incl > aim);
                        const unsigned int full = __ballot_sync(0xffffffffu, x.s > 0.f);
                        if (full != 0) {
                            const int l = over != 0 ? __ffs(over) - 1 : 31 - __clz(full);
                            sg = first + s0 + l;
                            sg_before = run + shuffle(lanes_before, l);
                        }
                        if (over != 0) break;
                        run = run + shuffle(seg_incl, 31);
                    }
                    y = segment_draw(r, sg, a.vocab, lane, sg_before, aim, stage);
                }
            }
        }
        if (!less) break;
        __syncthreads();
        if (!shared_empty) break;
        r.alone();
    }
    cluster_arrive();
    if (writer && warp == 0) {
        for (int j = lane; j <= a.max_draft_len; j += 32)
            out[j] = j < kept ? a.draft_tokens[d0 + j] : (j == kept ? y : -1);
        if (lane == 0) {
            a.num_accepted[i] = kept;
            if (a.new_lens != nullptr) a.new_lens[i] = a.lens[i] - (k - kept);
        }
    }
    cluster_wait();  // a CTA's total stays until the whole cluster has read it
}

// Checked mode: the rows of every sequence and its draft tokens.
__global__ void check_verify_kernel(const VerifyArgs a, unsigned int* verdict) {
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < a.batch; i += gridDim.x * blockDim.x) {
        const int64_t t0 = a.query_start[i], d0 = a.draft_start[i];
        const int64_t rows = a.query_start[i + 1] - t0, k = a.draft_start[i + 1] - d0;
        if (rows == 0 && k == 0) continue;
        if (k < 0 || k > a.max_draft_len || rows != k + 1 || t0 < 0 || d0 < 0 || t0 + rows > a.num_target_rows ||
            d0 + k > a.num_draft_rows) {
            atomicOr(verdict, kVerdictRange);
            continue;
        }
        for (int64_t j = d0; j < d0 + k; ++j)
            if (a.draft_tokens[j] < 0 || a.draft_tokens[j] >= a.vocab) atomicOr(verdict, kVerdictRange);
    }
}

}  // namespace

// CTAs of a cluster: one load of every warp each, fewer when the sequences alone
// come to several CTAs per SM. One sequence of 32000 entries / 32 of 131072 / 200 of
// 50001 in bf16, in us: 1 CTA each 13.9 / 41.0 / 24.2, 2 10.3 / 24.1 / 19.4,
// 4 8.4 / 15.0 / 19.2, 8 7.6 / 11.6 / 24.1, by this rule 7.6 / 11.6 / 19.1.
static int cluster_of(const VerifyArgs& a) {
    const int segs = (a.vocab + kSeg - 1) / kSeg;
    int c = kMaxCtas;
    while (c > 1 && (2 * segs < c * kWarps * kGroup || static_cast<int64_t>(a.batch) * c > 8 * static_cast<int64_t>(device_sm_count()))) c /= 2;
    return c;
}

cudaError_t launch_verify(const VerifyArgs& a, int dtype, cudaStream_t s) {
    const int c = cluster_of(a);
    const dim3 grid(static_cast<unsigned>(a.batch) * c), cluster(c, 1, 1);
    if (dtype == PKV_F32) return launch_pdl_cluster(verify_kernel<float>, grid, dim3(kThreads), cluster, 0, s, a);
    return launch_pdl_cluster(verify_kernel<__nv_bfloat16>, grid, dim3(kThreads), cluster, 0, s, a);
}

cudaError_t launch_check_verify(const VerifyArgs& a, unsigned int* verdict, cudaStream_t s) {
    check_verify_kernel<<<(a.batch + 127) / 128, 128, 0, s>>>(a, verdict);
    return cudaGetLastError();
}

}  // namespace pkv
