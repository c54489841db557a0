// pkv_plan_step (include/pkv.h): where a step's new tokens go. Per sequence with n
// tokens, m new ones and h blocks, max(0, ceil((n + m) / 16) - h) blocks come off the
// stack of free blocks, in sequence order, the top first; token n + t lies at slot
// block((n + t) / 16) * 16 + (n + t) % 16.
//
// Every CTA reads all lengths (12 bytes a sequence, out of L2) and sums them up in
// shared memory, so that nothing waits on another CTA; then each writes its share of the
// rows, of the sequences and of the new table entries, whose sequences it finds by
// bisection in those sums. Bound by latency: lengths in, two scans, a bisection, the
// block's id, rows out: 3.4 us for 32 sequences, 5.1 for 1000 of which some are prompts, in
// a captured graph, a row a thread (four, which share a bisection: 5.4 and 9.3). Called
// from Python 7 to 12, the host's share being 5.5 to 8, more than the GPU's.
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ int64_t warp_scan(int64_t v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t other = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += other;
    }
    return v;
}

// The last i with sums[i] <= x (sums[0] = 0; x < sums[n]).
__device__ __forceinline__ int find(const int32_t* sums, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sums[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kThreads) plan_kernel(const PlanArgs a) {
    extern __shared__ int32_t sums[];
    int32_t* row_sum = sums;                   // rows before each sequence, and all
    int32_t* need_sum = sums + a.batch + 1;    // blocks taken before each sequence, and all
    __shared__ int64_t warp_rows[kWarps], warp_need[kWarps];
    grid_dependency_wait();
    allow_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t most = static_cast<int64_t>(a.max_blocks) * 16;
    auto valid = [&](int64_t n, int64_t m, int64_t h) { return n >= 0 && m >= 0 && h >= 0 && h <= a.max_blocks && n <= 16 * h && n + m <= most; };
    const int64_t left = *a.free_count;
    int64_t rows = 0, need = 0;  // before this turn's sequences
    bool bad = false;
    for (int i0 = 0; i0 < a.batch; i0 += kThreads) {
        const int i = i0 + threadIdx.x;
        int64_t m = 0, take = 0;
        if (i < a.batch) {
            const int64_t n = a.lens[i], h = a.held[i];
            m = a.new_tokens[i];
            if (valid(n, m, h)) {
                take = max((n + m + 15) / 16 - h, int64_t(0));
            } else {
                m = 0;
                bad = true;
            }
        }
        const int64_t mr = warp_scan(m, lane), mt = warp_scan(take, lane);
        if (lane == 31) {
            warp_rows[warp] = mr;
            warp_need[warp] = mt;
        }
        __syncthreads();
        const int64_t wr = warp_scan(warp_rows[lane], lane), wt = warp_scan(warp_need[lane], lane);
        const int64_t r = rows + __shfl_sync(0xffffffffu, wr, max(warp - 1, 0)) * (warp > 0) + mr - m;
        const int64_t t = need + __shfl_sync(0xffffffffu, wt, max(warp - 1, 0)) * (warp > 0) + mt - take;
        if (i < a.batch) {
            row_sum[i] = static_cast<int32_t>(r);
            need_sum[i] = static_cast<int32_t>(t);
        }
        rows += __shfl_sync(0xffffffffu, wr, 31);
        need += __shfl_sync(0xffffffffu, wt, 31);
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        row_sum[a.batch] = static_cast<int32_t>(rows);
        need_sum[a.batch] = static_cast<int32_t>(need);
    }
    __syncthreads();
    const bool count_ok = left >= 0 && left <= a.free_capacity;
    const bool planned = count_ok && rows <= a.num_rows && need <= left;
    if (blockIdx.x == 0) {
        bad = bad || !count_ok || rows > a.num_rows;
        if (bad) atomicOr(a.status, PKV_DEVERR_RANGE);
        if (threadIdx.x == 0) {
            a.result[0] = planned ? static_cast<int32_t>(rows) : 0;
            a.result[1] = count_ok && need > left ? static_cast<int32_t>(min(need - left, int64_t(0x7fffffff))) : 0;
            *a.new_free_count = static_cast<int32_t>(planned ? left - need : left);
            a.query_start[a.batch] = planned ? static_cast<int32_t>(rows) : 0;
        }
    }
    const int64_t at = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x, stride = static_cast<int64_t>(gridDim.x) * kThreads;
    // ---- sequences
    for (int64_t i = at; i < a.batch; i += stride) {
        const int32_t m = row_sum[i + 1] - row_sum[i], take = need_sum[i + 1] - need_sum[i];
        a.query_start[i] = planned ? row_sum[i] : 0;
        a.new_lens[i] = a.lens[i] + (planned ? m : 0);
        a.new_held[i] = a.held[i] + (planned ? take : 0);
    }
    auto inside = [&](int32_t id) { return id >= 0 && id < a.num_blocks; };
    // ---- new table entries
    if (planned) {
        for (int64_t k = at; k < need; k += stride) {
            const int i = find(need_sum, a.batch, static_cast<int>(k));
            const int32_t id = a.free_blocks[left - 1 - k];
            if (!inside(id)) atomicOr(a.status, PKV_DEVERR_RANGE);
            a.tables[static_cast<int64_t>(i) * a.max_blocks + a.held[i] + (k - need_sum[i])] = inside(id) ? id : -1;
        }
    }
    // ---- rows
    for (int64_t r = at; r < a.num_rows; r += stride) {
        int64_t slot = -1;
        int32_t pos = -1;
        if (planned && r < rows) {
            const int i = find(row_sum, a.batch, static_cast<int>(r));
            const int h = a.held[i];
            pos = a.lens[i] + static_cast<int>(r - row_sum[i]);
            const int b = pos >> 4;
            const int32_t id = b < h ? a.tables[static_cast<int64_t>(i) * a.max_blocks + b]
                                     : a.free_blocks[left - 1 - need_sum[i] - (b - h)];
            if (inside(id))
                slot = static_cast<int64_t>(id) * 16 + (pos & 15);
            else
                atomicOr(a.status, PKV_DEVERR_RANGE);
        }
        a.slots[r] = slot;
        a.positions[r] = pos;
    }
}

// Checked mode, one CTA: every sequence, the rows and the blocks.
__global__ void __launch_bounds__(kThreads) check_plan_kernel(const PlanArgs a, unsigned int* verdict) {
    __shared__ unsigned long long rows, need;
    if (threadIdx.x == 0) rows = need = 0;
    __syncthreads();
    const int64_t most = static_cast<int64_t>(a.max_blocks) * 16;
    for (int i = threadIdx.x; i < a.batch; i += kThreads) {
        const int64_t n = a.lens[i], m = a.new_tokens[i], h = a.held[i];
        if (n < 0 || m < 0 || h < 0 || h > a.max_blocks || n > 16 * h || n + m > most) {
            atomicOr(verdict, kVerdictRange);
            continue;
        }
        atomicAdd(&rows, static_cast<unsigned long long>(m));
        atomicAdd(&need, static_cast<unsigned long long>(max((n + m + 15) / 16 - h, int64_t(0))));
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        const int64_t left = *a.free_count;
        if (left < 0 || left > a.free_capacity || rows > static_cast<unsigned long long>(a.num_rows)) atomicOr(verdict, kVerdictRange);
        else if (need > static_cast<unsigned long long>(left)) atomicOr(verdict, kVerdictBlocks);
    }
}

}  // namespace

cudaError_t launch_check_plan(const PlanArgs& a, unsigned int* verdict, cudaStream_t s) {
    check_plan_kernel<<<1, kThreads, 0, s>>>(a, verdict);
    return cudaGetLastError();
}

cudaError_t launch_plan(const PlanArgs& a, cudaStream_t s) {
    auto sums_bytes = [](int batch) { return 2 * (static_cast<size_t>(batch) + 1) * sizeof(int32_t); };
    const size_t smem = sums_bytes(a.batch);
    if (smem > 40 * 1024) {
        // (to the largest launch's: the limit is the function's, and another thread may be about to launch)
        const cudaError_t e = cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(sums_bytes(PKV_MAX_PLAN_BATCH)));
        if (e != cudaSuccess) return e;
    }
    const int64_t want = (a.num_rows + kThreads - 1) / kThreads, most = device_sm_count();
    return launch_pdl(plan_kernel, dim3(static_cast<unsigned>(want < 1 ? 1 : want < most ? want : most)), dim3(kThreads), smem, s, a);
}

}  // namespace pkv
