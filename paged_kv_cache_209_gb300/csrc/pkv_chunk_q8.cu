// Causal attention of a chunk of new tokens over the int8 pools
// (pkv_multiquery_attention_q8 in include/pkv.h), for more than 32 query rows
// per (sequence, KV head) or head_dim 64.
//
// First form: one warp per query row, float32 arithmetic, the running maximum
// and sum of an online softmax over 16-token blocks.
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kWarps = 8;

template <int D>
__global__ void __launch_bounds__(32 * kWarps) chunk_q8_simple_kernel(const ChunkArgs a) {
    constexpr int kPer = D / 32;
    grid_dependency_wait();
    allow_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int i = blockIdx.y;
    const int n = a.lens[i], q0 = a.qstart[i];
    const int64_t nq = static_cast<int64_t>(a.qstart[i + 1]) - q0;
    if (n < 0 || n > a.max_blocks * 16 || q0 < 0 || nq < 0 || nq > n || nq > a.max_query_len) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.status, PKV_DEVERR_RANGE);
        return;
    }
    const int64_t r = static_cast<int64_t>(blockIdx.x) * kWarps + warp;  // query t * heads + head
    if (r >= nq * a.q_heads) return;
    const int t = static_cast<int>(r / a.q_heads), hq = static_cast<int>(r - static_cast<int64_t>(t) * a.q_heads);
    const int h = hq / a.group;
    const int seen = n - static_cast<int>(nq) + t + 1;
    const int64_t row = (static_cast<int64_t>(q0) + t) * a.q_heads + hq;
    float q[kPer], o[kPer];
    for (int e = 0; e < kPer; ++e) {
        q[e] = __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[row * D + lane * kPer + e]);
        o[e] = 0.f;
    }
    float m = __int_as_float(0xff800000), l = 0.f;
    const float c = a.scale * 1.4426950408889634f;
    const int32_t* table = a.tables + static_cast<int64_t>(i) * a.max_blocks;
    for (int b = 0; b * 16 < seen; ++b) {
        const int bid = table[b];
        if (bid < 0 || bid >= a.num_blocks) {
            if (lane == 0) atomicOr(a.status, PKV_DEVERR_RANGE);
            continue;
        }
        const int64_t bh = static_cast<int64_t>(bid) * a.kv_heads + h;
        const int8_t* kc = static_cast<const int8_t*>(a.k_codes) + bh * 16 * D;
        const int8_t* vc = static_cast<const int8_t*>(a.v_codes) + bh * 16 * D;
        const int cnt = min(16, seen - b * 16);
        for (int tt = 0; tt < cnt; ++tt) {
            float s = 0.f;
            for (int e = 0; e < kPer; ++e) s += q[e] * static_cast<float>(kc[tt * D + lane * kPer + e]);
            for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
            const float x = s * a.scales[bh * 32 + tt] * c;
            if (x > m) {
                const float alpha = ex2(m - x);
                m = x;
                l *= alpha;
                for (int e = 0; e < kPer; ++e) o[e] *= alpha;
            }
            const float p = ex2(x - m);
            l += p;
            const float w = p * a.scales[bh * 32 + 16 + tt];
            for (int e = 0; e < kPer; ++e) o[e] += w * static_cast<float>(vc[(lane * kPer + e) * 16 + tt]);
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int e = 0; e < kPer; ++e)
        static_cast<__nv_bfloat16*>(a.out)[row * D + lane * kPer + e] = __float2bfloat16(o[e] * inv);
}

}  // namespace

size_t chunk_q8_workspace_bytes(int, int, int) { return 256; }

cudaError_t launch_chunk_q8(const ChunkArgs& a, cudaStream_t s) {
    const int64_t rows = static_cast<int64_t>(a.max_query_len) * a.q_heads;
    const dim3 grid(static_cast<unsigned>((rows + kWarps - 1) / kWarps), a.batch);
    return a.head_dim == 128 ? launch_pdl(chunk_q8_simple_kernel<128>, grid, dim3(32 * kWarps), 0, s, a)
                             : launch_pdl(chunk_q8_simple_kernel<64>, grid, dim3(32 * kWarps), 0, s, a);
}

}  // namespace pkv
