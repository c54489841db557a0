// Attention over the 4-bit cache (pkv_decode_attention_q4, pkv_multiquery_attention_q4 in
// include/pkv.h).
//
// One warp per query row and head: an online softmax over the row's tokens, a lane
// holding D / 32 dimensions.
#include <math.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_q4.cuh"

namespace pkv {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ninf() { return __int_as_float(0xff800000); }

template <int D>
__global__ void __launch_bounds__(128) attend_q4_kernel(const Q4Args a) {
    constexpr int kPer = D / 32;
    grid_dependency_wait();
    allow_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t items = static_cast<int64_t>(a.batch) * a.max_query_len * a.q_heads;
    for (int64_t x = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5); x < items; x += static_cast<int64_t>(gridDim.x) * 4) {
        const int h = static_cast<int>(x % a.q_heads);
        const int t = static_cast<int>(x / a.q_heads % a.max_query_len);
        const int i = static_cast<int>(x / a.q_heads / a.max_query_len);
        const int64_t n = a.lens[i];
        const int64_t q0 = a.qstart ? a.qstart[i] : i, nq = a.qstart ? a.qstart[i + 1] - q0 : 1;
        if (n < 0 || n > static_cast<int64_t>(a.max_blocks) * 16 || q0 < 0 || nq < 0 || (a.qstart && nq > n) || nq > a.max_query_len) {
            if (t == 0 && h == 0 && lane == 0) atomicOr(a.status, PKV_DEVERR_RANGE);
            continue;
        }
        if (t >= nq) continue;
        const int head = h / a.group;
        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + ((q0 + t) * a.q_heads + h) * D + lane * kPer;
        float qv[kPer], o[kPer] = {}, m = ninf(), l = 0.f;
#pragma unroll
        for (int e = 0; e < kPer; ++e) qv[e] = __bfloat162float(q[e]) * a.scale * kLog2e;
        const int64_t last = a.qstart ? n - nq + t : n - 1;
        for (int64_t p = 0; p <= last; ++p) {
            const int32_t id = a.tables[static_cast<int64_t>(i) * a.max_blocks + (p >> 4)];
            if (id < 0 || id >= a.num_blocks) {
                if (lane == 0) atomicOr(a.status, PKV_DEVERR_RANGE);
                continue;
            }
            const uint8_t* rec = static_cast<const uint8_t*>(a.cache) + (static_cast<int64_t>(id) * a.kv_heads + head) * q4_record_bytes(D);
            const int s = static_cast<int>(p & 15);
            const float* scales = reinterpret_cast<const float*>(rec + q4_scales_offset(D));
            float dot = 0.f, v[kPer];
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                const int d = lane * kPer + e, w = d & 7, nib = (w >> 1) + 4 * (w & 1);
                dot += qv[e] * static_cast<float>(((rec[s * (D / 2) + (d >> 3) * 4 + (nib >> 1)] >> (4 * (nib & 1))) & 15) - 8);
                v[e] = static_cast<float>(((rec[q4_v_offset(D) + q4_v_byte(d >> 3, w >> 1, s)] >> (4 * (w & 1))) & 15) - 8);
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
            const float x2 = dot * scales[s], to = fmaxf(m, x2);
            const float keep = m == ninf() ? 0.f : ex2(m - to), e2 = ex2(x2 - to);
            l = l * keep + e2;
            m = to;
#pragma unroll
            for (int e = 0; e < kPer; ++e) o[e] = o[e] * keep + e2 * (v[e] * scales[16 + s]);
        }
        const float inv = l > 0.f ? 1.f / l : 0.f;
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + ((q0 + t) * a.q_heads + h) * D + lane * kPer;
#pragma unroll
        for (int e = 0; e < kPer; ++e) out[e] = __float2bfloat16_rn(o[e] * inv);
    }
}

}  // namespace

cudaError_t launch_attend_q4(const Q4Args& a, cudaStream_t s) {
    const int64_t items = static_cast<int64_t>(a.batch) * a.max_query_len * a.q_heads;
    const int64_t want = (items + 3) / 4, most = static_cast<int64_t>(device_sm_count()) * 64;
    const dim3 grid(static_cast<unsigned>(want < most ? want : most));
    return a.head_dim == 128 ? launch_pdl(attend_q4_kernel<128>, grid, dim3(128), 0, s, a) : launch_pdl(attend_q4_kernel<64>, grid, dim3(128), 0, s, a);
}

}  // namespace pkv
