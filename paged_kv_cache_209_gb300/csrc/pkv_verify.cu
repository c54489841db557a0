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
// running sums carry far more than float32: a lane adds its entries of a
// kSeg-entry segment in two floats (the exact error of each addition is kept,
// about 2^-46 relative), the lanes' sums and the segments' sums are added in
// float64 in a fixed order. float64 per entry would be bound by the FP64 pipe:
// two additions per SM and clock on this part, against 32 entries per SM and
// clock that HBM delivers.
//
// One CTA per sequence: the warps take the segments in turn and leave their
// sums in shared memory, one warp finds the segment that holds the draw, and
// scans its entries again (from L2).
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kSeg = 1024;                       // entries per segment
constexpr int kMaxSegs = kMaxVocab / kSeg;
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ float load_prob(const float* p, int64_t i) { return __ldg(p + i); }
__device__ __forceinline__ float load_prob(const __nv_bfloat16* p, int64_t i) {
    return __bfloat162float(p[i]);
}

// The mass an entry of r carries: a finite number above zero, else none.
__device__ __forceinline__ float mass_of(float x) { return x > 0.f && x <= 3.402823466e38f ? x : 0.f; }

// r at index v: the target row alone, or less the draft's row (or less the
// certain draft's 1 at token x).
template <typename T>
struct Rest {
    const T* p;
    const T* q;   // null: nothing to subtract
    int certain;  // >= 0: the draft was certain of this token
    __device__ __forceinline__ float at(int v) const {
        float x = load_prob(p, v);
        if (q != nullptr) x -= load_prob(q, v);
        if (v == certain) x -= 1.f;
        return mass_of(x);
    }
};

// s + c += x with s the rounded sum and c the accumulated rounding errors.
__device__ __forceinline__ void add_two(float& s, float& c, float x) {
    const float t = s + x;
    const float z = t - s;
    c += (s - (t - z)) + (x - z);
    s = t;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) verify_kernel(const VerifyArgs a) {
    __shared__ double seg_sum[kMaxSegs];
    __shared__ int info[4];  // kept drafts, 1 if a draft was rejected, rows of the sequence, bad
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int i = blockIdx.x;
    grid_dependency_wait();
    allow_dependents();
    const int t0 = a.query_start[i], d0 = a.draft_start[i];
    const int64_t rows = static_cast<int64_t>(a.query_start[i + 1]) - t0;
    const int64_t k64 = static_cast<int64_t>(a.draft_start[i + 1]) - d0;
    const bool idle = rows == 0 && k64 == 0;
    const bool bad = !idle && (k64 < 0 || k64 > a.max_draft_len || rows != k64 + 1 || t0 < 0 || d0 < 0 ||
                               t0 + rows > a.num_target_rows || d0 + k64 > a.num_draft_rows);
    int* out = a.out_tokens + static_cast<int64_t>(i) * (a.max_draft_len + 1);
    if (idle || bad) {
        for (int j = threadIdx.x; j <= a.max_draft_len; j += kThreads) out[j] = -1;
        if (threadIdx.x == 0) {
            a.num_accepted[i] = bad ? -1 : 0;
            if (a.new_lens != nullptr) a.new_lens[i] = a.lens[i];
            if (bad) atomicOr(a.status, PKV_DEVERR_RANGE);
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
                if (x < 0 || x >= a.vocab) {
                    atomicOr(a.status, PKV_DEVERR_RANGE);
                    keep = false;
                } else {
                    const double p = load_prob(target + j * a.target_stride, x);
                    const double q = draft == nullptr ? 1.0 : static_cast<double>(load_prob(draft + j * a.draft_stride, x));
                    keep = static_cast<double>(a.accept[d0 + j]) * q < p;
                }
            }
            const unsigned int no = __ballot_sync(0xffffffffu, !keep);
            if (no != 0) kept = base + __ffs(no) - 1;
        }
        if (lane == 0) info[0] = kept;
    }
    __syncthreads();
    const int kept = info[0];
    const int segs = (a.vocab + kSeg - 1) / kSeg;
    Rest<T> r;
    r.p = target + kept * a.target_stride;
    r.q = kept < k && draft != nullptr ? draft + kept * a.draft_stride : nullptr;
    r.certain = kept < k && draft == nullptr ? a.draft_tokens[d0 + kept] : -1;
    int y = -1;
    // second try, on p itself, where max(p - q, 0) holds nothing
    for (int attempt = 0; attempt < 2; ++attempt) {
        for (int sg = warp; sg < segs; sg += kWarps) {
            float s = 0.f, c = 0.f;
            for (int v = sg * kSeg + lane; v < min(a.vocab, (sg + 1) * kSeg); v += 32) add_two(s, c, r.at(v));
            double sum = static_cast<double>(s) + static_cast<double>(c);
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane == 0) seg_sum[sg] = sum;
        }
        __syncthreads();
        double total = 0.0;
        for (int sg = 0; sg < segs; ++sg) total += seg_sum[sg];
        if (total > 0.0) {
            if (warp == 0) {
                const double aim = static_cast<double>(a.sample[i]) * total;
                // the first segment whose running sum exceeds the aim, else the last that holds anything
                double before = 0.0, run = 0.0;
                int at = -1;
                for (int sg = 0; sg < segs; ++sg) {
                    if (!(seg_sum[sg] > 0.0)) continue;
                    at = sg;
                    before = run;
                    run += seg_sum[sg];
                    if (run > aim) break;
                }
                // its entries, 32 consecutive ones per lane
                const int v0 = at * kSeg + lane * (kSeg / 32);
                double mine = 0.0;
                for (int e = 0; e < kSeg / 32; ++e) mine += v0 + e < a.vocab ? r.at(v0 + e) : 0.f;
                double incl = mine;
                for (int o = 1; o < 32; o <<= 1) {
                    const double other = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += other;
                }
                double cum = before + (incl - mine);
                int hit = INT_MAX, last = -1;
                for (int e = 0; e < kSeg / 32; ++e) {
                    const float x = v0 + e < a.vocab ? r.at(v0 + e) : 0.f;
                    cum += x;
                    if (x > 0.f) {
                        last = v0 + e;
                        if (cum > aim && hit == INT_MAX) hit = v0 + e;
                    }
                }
                hit = __reduce_min_sync(0xffffffffu, hit);
                last = __reduce_max_sync(0xffffffffu, last);
                y = hit != INT_MAX ? hit : last;
            }
            break;
        }
        if (attempt == 0) {
            if (r.q == nullptr && r.certain < 0) break;  // it was p already
            r.q = nullptr;
            r.certain = -1;
            __syncthreads();
        }
    }
    if (warp == 0) {
        for (int j = lane; j <= a.max_draft_len; j += 32)
            out[j] = j < kept ? a.draft_tokens[d0 + j] : (j == kept ? y : -1);
        if (lane == 0) {
            a.num_accepted[i] = kept;
            if (a.new_lens != nullptr) a.new_lens[i] = a.lens[i] - (k - kept);
        }
    }
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

cudaError_t launch_verify(const VerifyArgs& a, int dtype, cudaStream_t s) {
    if (dtype == PKV_F32) return launch_pdl(verify_kernel<float>, dim3(a.batch), dim3(kThreads), 0, s, a);
    return launch_pdl(verify_kernel<__nv_bfloat16>, dim3(a.batch), dim3(kThreads), 0, s, a);
}

cudaError_t launch_check_verify(const VerifyArgs& a, unsigned int* verdict, cudaStream_t s) {
    check_verify_kernel<<<(a.batch + 127) / 128, 128, 0, s>>>(a, verdict);
    return cudaGetLastError();
}

}  // namespace pkv
