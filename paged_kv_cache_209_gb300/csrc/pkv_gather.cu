// Reading tokens back out of the paged cache (pkv_gather, pkv_gather_q8 and
// pkv_gather_q4 in include/pkv.h): a token range of each sequence becomes packed rows
// [row][KV head][head_dim] of K and of V. Pure data movement, bound by HBM: per
// row 2 Hkv D elements written and as many read (2 Hkv (D + 4) bytes for int8).
//
// One warp takes one item, a (sequence, block, KV head): 16 rows that are
// contiguous in the pool. The items of a launch are numbered through prefix sums
// over the sequences' block counts (in shared memory), head fastest, so that
// warps working at the same time write neighbouring rows; the sequence of an
// item is found by bisection. Nothing is launched for table entries that no
// sequence uses.
//
// Int8 V codes lie coordinate by coordinate ([D][16 tokens]): a lane loads the
// 16 tokens of D / 32 neighbouring coordinates and the warp writes one token's
// whole row at a time.
//
// 32 sequences of 8192 int8 tokens, 8 KV heads of 128: 1.63 GB in 257 us, 94 % of
// the measured copy rate; 64 ragged bf16 sequences 126 us, 97 %; 300 tokens 5 us. The
// same 32 sequences of a 4-bit cache: 1.36 GB in 221 us, 91 %, 2.43 GB in float32 in 381 us,
// 94 %; 300 tokens 3.5 us (one warp for both sides of a record: 225, 376, 4.3).
#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_q4.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// Four times the CTAs that fit an SM, so that the last ones even the SMs out. bf16, 64
// ragged sequences / int8, 32 of 8192 tokens, in us: 8 per SM 133 / 260, 16 128 / 259,
// 32 126 / 257, 64 126 / 263, one item per warp 126 / 282 (each CTA sums the block
// counts anew).
constexpr int kCtasPerSm = 32;

// The token range of sequence i; false when it leaves the context, the table or
// the outputs.
__device__ __forceinline__ bool range_of(const GatherArgs& a, int i, int64_t& first, int64_t& row0, int64_t& rows) {
    const int64_t n = a.lens[i];
    first = a.token_start == nullptr ? 0 : a.token_start[i];
    row0 = a.row_start[i];
    rows = a.row_start[i + 1] - row0;
    return n >= 0 && n <= static_cast<int64_t>(a.max_blocks) * 16 && first >= 0 && rows >= 0 && first + rows <= n &&
           row0 >= 0 && row0 + rows <= a.num_rows;
}

// Exclusive prefix sums of the sequences' block counts: prefix[i] .. prefix[batch]
// (all threads; ends with __syncthreads). Below 2^31: the host bounds the blocks
// of a launch's tables.
__device__ void count_blocks(const GatherArgs& a, int* prefix) {
    __shared__ int warp_sum[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kPer = kMaxBatchPerLaunch / kThreads;
    int mine[kPer], sum = 0;
    for (int e = 0; e < kPer; ++e) {
        const int i = threadIdx.x * kPer + e;
        mine[e] = 0;
        if (i < a.batch) {
            int64_t first, row0, rows;
            if (!range_of(a, i, first, row0, rows)) {
                if (blockIdx.x == 0) atomicOr(a.status, PKV_DEVERR_RANGE);
            } else if (rows > 0) {
                mine[e] = static_cast<int>(((first + rows - 1) >> 4) - (first >> 4)) + 1;
            }
        }
        sum += mine[e];
    }
    int incl = sum;
    for (int o = 1; o < 32; o <<= 1) {
        const int other = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += other;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int at = incl - sum;
    for (int w = 0; w < warp; ++w) at += warp_sum[w];
    for (int e = 0; e < kPer; ++e) {
        const int i = threadIdx.x * kPer + e;
        if (i <= a.batch) prefix[i] = at;
        at += mine[e];
    }
    if (threadIdx.x == kThreads - 1 && a.batch == kMaxBatchPerLaunch) prefix[kMaxBatchPerLaunch] = at;
    __syncthreads();
}

// One item: its block's place in the pool, and which of its 16 rows go where.
struct Item {
    int64_t chunk;  // block id * heads + head
    int64_t row;    // output row of the block's token 0 (may lie before the range)
    int lo, hi;     // tokens lo .. hi - 1 of the block
    int head;
};

__device__ __forceinline__ bool item_of(const GatherArgs& a, const int* prefix, int64_t index, int lane, Item& it) {
    const int unit = static_cast<int>(index / a.kv_heads);
    it.head = static_cast<int>(index - static_cast<int64_t>(unit) * a.kv_heads);
    int i = 0;  // the last sequence with prefix[i] <= unit
    for (int step = kMaxBatchPerLaunch / 2; step > 0; step >>= 1)
        if (i + step < a.batch && prefix[i + step] <= unit) i += step;
    const int64_t first = a.token_start == nullptr ? 0 : a.token_start[i];
    const int64_t row0 = a.row_start[i];
    const int64_t rows = a.row_start[i + 1] - row0;
    const int64_t block = (first >> 4) + unit - prefix[i];
    it.lo = static_cast<int>(max(first - block * 16, int64_t(0)));
    it.hi = static_cast<int>(min(first + rows - block * 16, int64_t(16)));
    it.row = row0 + block * 16 - first;
    const int id = a.tables[static_cast<int64_t>(i) * a.max_blocks + block];
    if (id < 0 || id >= a.num_blocks) {
        if (lane == 0) atomicOr(a.status, PKV_DEVERR_RANGE);
        return false;
    }
    it.chunk = static_cast<int64_t>(id) * a.kv_heads + it.head;
    return true;
}

// Byte `b` of four codes (each xor 0x80, i.e. code + 128) as a float, exactly:
// 2^23 + code + 128 has the byte in its lowest bits.
template <int b>
__device__ __forceinline__ float code_f32(uint32_t biased) {
    return __uint_as_float(__byte_perm(biased, 0x4B000000u, 0x7650 | b)) - 8388736.f;
}

__device__ __forceinline__ void store8(float* dst, const float (&x)[8]) {
    reinterpret_cast<float4*>(dst)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(dst)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* dst, const float (&x)[8]) {
    *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void store_coords(float* dst, const float (&x)[4]) {
    *reinterpret_cast<float4*>(dst) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store_coords(float* dst, const float (&x)[2]) {
    *reinterpret_cast<float2*>(dst) = make_float2(x[0], x[1]);
}
__device__ __forceinline__ void store_coords(__nv_bfloat16* dst, const float (&x)[4]) {
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
}
__device__ __forceinline__ void store_coords(__nv_bfloat16* dst, const float (&x)[2]) {
    *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(x[0], x[1]);
}

template <int D, typename Out>
__global__ void __launch_bounds__(kThreads) gather_q8_kernel(const GatherArgs a) {
    __shared__ int prefix[kMaxBatchPerLaunch + 1];
    grid_dependency_wait();
    allow_dependents();
    count_blocks(a, prefix);
    const int lane = threadIdx.x & 31;
    const int64_t items = static_cast<int64_t>(prefix[a.batch]) * a.kv_heads;
    const int64_t stride = static_cast<int64_t>(a.kv_heads) * D;  // elements from a token's row to the next
    constexpr int kLanes = D / 16;         // lanes that hold one K row, 16 codes each
    constexpr int kRows = 32 / kLanes;     // K rows of one load
    constexpr int kCoords = D / 32;        // V coordinates of a lane
    for (int64_t x = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); x < items;
         x += static_cast<int64_t>(gridDim.x) * kWarps) {
        Item it;
        if (!item_of(a, prefix, x, lane, it)) continue;
        const uint4* kc = static_cast<const uint4*>(a.k) + it.chunk * D;  // 16 rows of D bytes = D vectors
        const uint4* vc = static_cast<const uint4*>(a.v) + it.chunk * D;
        const float sc = __ldg(a.scales + it.chunk * 32 + lane);  // K scales in lanes 0-15, V in 16-31
        uint4 kv[16 / kRows], vv[kCoords];
#pragma unroll
        for (int r = 0; r < 16 / kRows; ++r) kv[r] = __ldcs(kc + r * 32 + lane);
#pragma unroll
        for (int e = 0; e < kCoords; ++e) vv[e] = __ldcs(vc + lane * kCoords + e);
        Out* ko = static_cast<Out*>(a.k_out) + it.row * stride + it.head * D + (lane % kLanes) * 16;
#pragma unroll
        for (int r = 0; r < 16 / kRows; ++r) {
            const int t = r * kRows + lane / kLanes;
            const float s = __shfl_sync(0xffffffffu, sc, t);
            if (t < it.lo || t >= it.hi) continue;
            const uint32_t w[4] = {kv[r].x ^ 0x80808080u, kv[r].y ^ 0x80808080u, kv[r].z ^ 0x80808080u,
                                   kv[r].w ^ 0x80808080u};
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const uint32_t p = w[2 * half], q = w[2 * half + 1];
                const float y[8] = {code_f32<0>(p) * s, code_f32<1>(p) * s, code_f32<2>(p) * s, code_f32<3>(p) * s,
                                    code_f32<0>(q) * s, code_f32<1>(q) * s, code_f32<2>(q) * s, code_f32<3>(q) * s};
                store8(ko + t * stride + half * 8, y);
            }
        }
        Out* vo = static_cast<Out*>(a.v_out) + it.row * stride + it.head * D + lane * kCoords;
#pragma unroll
        for (int g = 0; g < 4; ++g) {  // tokens 4g .. 4g + 3: one word of every coordinate
            uint32_t w[kCoords];
#pragma unroll
            for (int e = 0; e < kCoords; ++e)
                w[e] = (g == 0 ? vv[e].x : g == 1 ? vv[e].y : g == 2 ? vv[e].z : vv[e].w) ^ 0x80808080u;
            float y[4][kCoords];
#pragma unroll
            for (int e = 0; e < kCoords; ++e) {
                y[0][e] = code_f32<0>(w[e]);
                y[1][e] = code_f32<1>(w[e]);
                y[2][e] = code_f32<2>(w[e]);
                y[3][e] = code_f32<3>(w[e]);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int t = 4 * g + u;
                const float s = __shfl_sync(0xffffffffu, sc, 16 + t);
#pragma unroll
                for (int e = 0; e < kCoords; ++e) y[u][e] *= s;
                if (t >= it.lo && t < it.hi) store_coords(vo + t * stride, y[u]);
            }
        }
    }
}

// Nibble p of a word of 4-bit codes (code + 8), as the code, exactly: 2^23 + nibble has it
// in its lowest bits.
__device__ __forceinline__ float nibble_f32(uint32_t w, int p) {
    return __uint_as_float((w >> (4 * p) & 15u) | 0x4B000000u) - 8388616.f;
}

__device__ __forceinline__ void store16(float* dst, const float (&x)[4]) { store_coords(dst, x); }
__device__ __forceinline__ void store16(__nv_bfloat16* dst, const float (&x)[8]) { store8(dst, x); }

// A 4-bit record is 16 rows of D / 8 words of K and D / 8 octets of 16 words of V (pkv_q4.cuh). A
// warp takes one side of a record: K's rows as they come, of V 16 bytes at a time, an octet's four tokens
// of one quad. A lane writes 16 bytes at a time, an octet in bf16, half of one in float32 (whose
// halves lie in neighbouring lanes, so that every line that a store touches is written whole).
template <int D, typename Out>
__global__ void __launch_bounds__(kThreads) gather_q4_kernel(const GatherArgs a) {
    __shared__ int prefix[kMaxBatchPerLaunch + 1];
    grid_dependency_wait();
    allow_dependents();
    count_blocks(a, prefix);
    const int lane = threadIdx.x & 31;
    const int64_t items = static_cast<int64_t>(prefix[a.batch]) * a.kv_heads * 2;
    const int64_t stride = static_cast<int64_t>(a.kv_heads) * D;  // elements from a token's row to the next
    constexpr int kDims = 16 / sizeof(Out);  // of a store
    constexpr int kParts = 8 / kDims;        // of an octet
    constexpr int kWords = D / 16;           // K words of a lane
    const int part = lane % kParts;
    for (int64_t x = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); x < items;
         x += static_cast<int64_t>(gridDim.x) * kWarps) {
        Item it;
        if (!item_of(a, prefix, x >> 1, lane, it)) continue;
        const bool is_v = (x & 1) != 0;
        const uint8_t* rec = static_cast<const uint8_t*>(a.k) + it.chunk * q4_record_bytes(D);
        const float sc = __ldg(reinterpret_cast<const float*>(rec + q4_scales_offset(D)) + 16 * is_v + (lane & 15));
        Out* out = static_cast<Out*>(is_v ? a.v_out : a.k_out) + it.row * stride + it.head * D + kDims * part;
        if (!is_v) {
            uint32_t k[kWords];
#pragma unroll
            for (int r = 0; r < kWords; ++r) k[r] = __ldcs(reinterpret_cast<const uint32_t*>(rec) + 32 * r + lane);
#pragma unroll
            for (int r = 0; r < kWords * kParts; ++r) {
                const int word = (32 * r + lane) / kParts, t = word / (D / 8);
                const float s = __shfl_sync(0xffffffffu, sc, t);
                const uint32_t w = __shfl_sync(0xffffffffu, k[r / kParts], word % 32) >> (2 * kDims * part);
                float y[kDims];
#pragma unroll
                for (int e = 0; e < kDims; ++e) y[e] = nibble_f32(w, e / 2 + 4 * (e & 1)) * s;
                if (t >= it.lo && t < it.hi) store16(out + t * stride + word % (D / 8) * 8, y);
            }
        } else {
            constexpr int kLoads = D / 64 * kParts;  // of kDims / 2 words each
            uint32_t v[kLoads][kDims / 2];
#pragma unroll
            for (int r = 0; r < kLoads; ++r) {
                const uint32_t* from = reinterpret_cast<const uint32_t*>(rec + q4_v_offset(D)) + (32 * r + lane) * (kDims / 2);
                if (kDims == 8) {
                    const uint4 w = __ldcs(reinterpret_cast<const uint4*>(from));
                    v[r][0] = w.x, v[r][1] = w.y, v[r][kDims / 2 - 2] = w.z, v[r][kDims / 2 - 1] = w.w;
                } else {
                    const uint2 w = __ldcs(reinterpret_cast<const uint2*>(from));
                    v[r][0] = w.x, v[r][1] = w.y;
                }
            }
#pragma unroll
            for (int r = 0; r < kLoads; ++r) {
                const int vec = (32 * r + lane) / kParts, quad = vec & 3, o = vec >> 2;
#pragma unroll
                for (int u = 0; u < 4; ++u) {  // tokens 2 quad, + 1, + 8, + 9
                    const int t = 2 * quad + (u & 1) + 8 * (u >> 1);
                    const float s = __shfl_sync(0xffffffffu, sc, t);
                    float y[kDims];
#pragma unroll
                    for (int e = 0; e < kDims; ++e) y[e] = nibble_f32(v[r][e / 2], 4 * (u & 1) + 2 * (u >> 1) + (e & 1)) * s;
                    if (t >= it.lo && t < it.hi) store16(out + t * stride + 8 * o, y);
                }
            }
        }
    }
}

// Rows of kVecs 16-byte vectors, copied as they are: an item's rows are 16 kVecs
// consecutive vectors of the pool.
template <int kVecs>
__global__ void __launch_bounds__(kThreads) gather_kernel(const GatherArgs a) {
    __shared__ int prefix[kMaxBatchPerLaunch + 1];
    grid_dependency_wait();
    allow_dependents();
    count_blocks(a, prefix);
    const int lane = threadIdx.x & 31;
    const int64_t items = static_cast<int64_t>(prefix[a.batch]) * a.kv_heads;
    const int64_t stride = static_cast<int64_t>(a.kv_heads) * kVecs;
    for (int64_t x = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); x < items;
         x += static_cast<int64_t>(gridDim.x) * kWarps) {
        Item it;
        if (!item_of(a, prefix, x, lane, it)) continue;
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            const uint4* src = static_cast<const uint4*>(side ? a.v : a.k) + it.chunk * 16 * kVecs + lane;
            uint4* dst = static_cast<uint4*>(side ? a.v_out : a.k_out) + it.row * stride + it.head * kVecs;
            uint4 w[kVecs / 2];
#pragma unroll
            for (int e = 0; e < kVecs / 2; ++e) w[e] = __ldcs(src + 32 * e);
#pragma unroll
            for (int e = 0; e < kVecs / 2; ++e) {
                const int v = 32 * e + lane, t = v / kVecs;
                if (t >= it.lo && t < it.hi) dst[t * stride + v % kVecs] = w[e];
            }
        }
    }
}

// Checked mode: the ranges (the blocks of whole contexts are checked apart).
__global__ void check_gather_kernel(const GatherArgs a, unsigned int* verdict) {
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < a.batch; i += gridDim.x * blockDim.x) {
        int64_t first, row0, rows;
        if (!range_of(a, i, first, row0, rows)) atomicOr(verdict, kVerdictRange);
    }
}

}  // namespace

cudaError_t launch_gather(const GatherArgs& a, const pkv_cache_desc& d, int out_dtype, cudaStream_t s) {
    // at most one item per KV head for every 16 rows, and two more per sequence; two warps an item of a 4-bit cache
    const int64_t units = (a.num_rows / 16 + 2 * static_cast<int64_t>(a.batch)) * (d.dtype == PKV_INT4 ? 2 : 1);
    const int64_t want = (units * d.num_kv_heads + kWarps - 1) / kWarps;
    const int64_t most = static_cast<int64_t>(device_sm_count()) * kCtasPerSm;
    const dim3 grid(static_cast<unsigned>(want < most ? want : most)), block(kThreads);
    const bool wide = d.head_dim == 128;
    if (d.dtype == PKV_F32)
        return wide ? launch_pdl(gather_kernel<32>, grid, block, 0, s, a) : launch_pdl(gather_kernel<16>, grid, block, 0, s, a);
    if (d.dtype == PKV_BF16)
        return wide ? launch_pdl(gather_kernel<16>, grid, block, 0, s, a) : launch_pdl(gather_kernel<8>, grid, block, 0, s, a);
    if (d.dtype == PKV_INT4 && out_dtype == PKV_F32)
        return wide ? launch_pdl(gather_q4_kernel<128, float>, grid, block, 0, s, a)
                    : launch_pdl(gather_q4_kernel<64, float>, grid, block, 0, s, a);
    if (d.dtype == PKV_INT4)
        return wide ? launch_pdl(gather_q4_kernel<128, __nv_bfloat16>, grid, block, 0, s, a)
                    : launch_pdl(gather_q4_kernel<64, __nv_bfloat16>, grid, block, 0, s, a);
    if (out_dtype == PKV_F32)
        return wide ? launch_pdl(gather_q8_kernel<128, float>, grid, block, 0, s, a)
                    : launch_pdl(gather_q8_kernel<64, float>, grid, block, 0, s, a);
    return wide ? launch_pdl(gather_q8_kernel<128, __nv_bfloat16>, grid, block, 0, s, a)
                : launch_pdl(gather_q8_kernel<64, __nv_bfloat16>, grid, block, 0, s, a);
}

cudaError_t launch_check_gather(const GatherArgs& a, unsigned int* verdict, cudaStream_t s) {
    check_gather_kernel<<<(a.batch + 127) / 128, 128, 0, s>>>(a, verdict);
    return cudaGetLastError();
}

}  // namespace pkv
