// Rotary positions (pkv_rotary_table, pkv_append_rotary in include/pkv.h) and the
// quantizing append of the 4-bit cache (pkv_append_q4: the same kernel without
// positions or queries).
//
// A row of q or k, of which the first R dimensions turn, with c_i and s_i the table's
// cosine and sine of its position:
//     y_a = x_a c_i - x_b s_i,   y_b = x_b c_i + x_a s_i,   i < R / 2
// over the pairs (a, b) = (i, i + R / 2), or (2 i, 2 i + 1). The products of a bf16 and a
// float32 are exact in float64, so y is that difference rounded to float64, then to
// float32 and to bf16: a value that does not depend on the order of operations, and so
// neither do the codes of a cache that quantizes it. FP64 is slow on this part: a float32
// difference comes with a bound on its error, and only where the bf16 roundings of both
// ends differ (one value in some 2^14) float64 decides.
#include <math.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_q4.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256;

// x c - y s as described above, for bf16 x and y held in float32: a bf16 in float32.
__device__ __forceinline__ float turned(__nv_bfloat16, float x, float c, float y, float s) {
    const float p = y * s;
    const float r = fmaf(x, c, -p);
    // each rounding is off by at most 2^-24 of its result (2^-150 below the normal range)
    const float off = fmaf(fabsf(p) + fabsf(r), 1.1920929e-7f, 2.8026e-45f);
    const uint32_t ends = pack_bf16x2(r - off, r + off);
    if ((ends & 0xffffu) == ends >> 16) return bf16hi_to_f32(ends);
    const double exact = static_cast<double>(x) * c - static_cast<double>(y) * s;
    return __bfloat162float(__float2bfloat16_rn(static_cast<float>(exact)));
}
// float32 rows: the product's error joins the sum (one rounding, and one of a small term).
__device__ __forceinline__ float turned(float, float x, float c, float y, float s) {
    const float p = y * s;
    return fmaf(x, c, -p) - fmaf(y, s, -p);
}

// Eight elements of a row, in float32.
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    x[0] = bf16lo_to_f32(w.x), x[1] = bf16hi_to_f32(w.x), x[2] = bf16lo_to_f32(w.y), x[3] = bf16hi_to_f32(w.y);
    x[4] = bf16lo_to_f32(w.z), x[5] = bf16hi_to_f32(w.z), x[6] = bf16lo_to_f32(w.w), x[7] = bf16hi_to_f32(w.w);
}
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                              pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ float value(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float value(float x) { return x; }

enum { kWhole = 0, kHalves = 1, kNeighbours = 2, kAny = 3 };

// A lane takes two vectors of 8 dimensions of a row: va and vb. Where pairs lie R / 2
// apart and that is a multiple of 8, lane i < R / 16 takes vectors i and i + R / 16, the
// others two of the rest; else 2 lane and 2 lane + 1.
struct Place {
    int va, vb;
    bool turns;  // (kHalves) the two vectors are pairs
};
template <int kMode>
__device__ __forceinline__ Place place_of(int lane, int R) {
    if (kMode != kHalves) return {2 * lane, 2 * lane + 1, true};
    const int part = R / 16;
    if (lane < part) return {lane, lane + part, true};
    return {2 * lane, 2 * lane + 1, false};
}

// The turned row (`row`: its first element; `cs`: its table row), in the lane's vectors.
template <int kMode, typename T>
__device__ __forceinline__ void turn(const T* row, const float* cs, int R, bool interleaved, const Place& at, float (&a)[8], float (&b)[8]) {
    load8(row + 8 * at.va, a);
    load8(row + 8 * at.vb, b);
    if (kMode == kWhole) return;
    const int half = R / 2;
    if (kMode == kHalves) {
        if (!at.turns) return;
        float c[8], s[8];
        load8(cs + 8 * at.va, c);
        load8(cs + half + 8 * at.va, s);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float x = a[e], y = b[e];
            a[e] = turned(T{}, x, c[e], y, s[e]);
            b[e] = turned(T{}, y, c[e], x, -s[e]);
        }
    } else if (kMode == kNeighbours) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            float (&v)[8] = u ? b : a;
            const int first = 8 * (u ? at.vb : at.va);
            if (first >= R) break;
            const float4 c = *reinterpret_cast<const float4*>(cs + first / 2), s = *reinterpret_cast<const float4*>(cs + half + first / 2);
            const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float x = v[2 * e], y = v[2 * e + 1];
                v[2 * e] = turned(T{}, x, cc[e], y, ss[e]);
                v[2 * e + 1] = turned(T{}, y, cc[e], x, -ss[e]);
            }
        }
    } else {
        // any even R: the partner of every dimension is read apart
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            float (&v)[8] = u ? b : a;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int d = 8 * (u ? at.vb : at.va) + e;
                if (d >= R) continue;
                const int i = interleaved ? d / 2 : d % half;
                const bool second = interleaved ? (d & 1) != 0 : d >= half;
                const int other = interleaved ? d ^ 1 : second ? d - half : d + half;
                const float y = value(row[other]), c = cs[i], s = cs[half + i];
                v[e] = turned(T{}, v[e], c, y, second ? -s : s);
            }
        }
    }
}

// Words of a 4-bit record for 8 dimensions: K's word, and V's bytes.
__device__ __forceinline__ uint32_t k_word(const int (&c)[8]) {
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) w |= static_cast<uint32_t>(c[e] + 8) << (4 * (e / 2 + 4 * (e & 1)));
    return w;
}

// One row per D / 16 lanes: q's rows, then k's, then v's of a token. kCache: the pkv_dtype
// of the pools, or PKV_INT4.
template <int D, int kMode, int kCache, typename T>
__global__ void __launch_bounds__(kThreads) append_rotary_kernel(const RotaryAppendArgs a) {
    constexpr int kLanes = D / 16;
    constexpr int kRows = kThreads / kLanes;  // rows of a CTA
    grid_dependency_wait();  // q, k, v, and a block copied onto the slots' block, come from the kernels before
    allow_dependents();
    const int lane = threadIdx.x % kLanes;
    const uint32_t heads = a.q_heads + 2 * a.kv_heads;
    const uint32_t rows = static_cast<uint32_t>(a.num_tokens) * heads;
    const Place at = place_of<kMode>(lane, a.rotary_dim);
    // (whole warps take part in every turn of the loop)
    for (uint32_t r0 = blockIdx.x * kRows; r0 < rows; r0 += gridDim.x * kRows) {
        const uint32_t r = r0 + threadIdx.x / kLanes;
        const uint32_t token = min(r, rows - 1) / heads;
        const int h = static_cast<int>(min(r, rows - 1) - token * heads);
        const bool is_q = h < a.q_heads, is_v = h >= a.q_heads + a.kv_heads;
        const int head = is_q ? h : is_v ? h - a.q_heads - a.kv_heads : h - a.q_heads;
        const int64_t slot = a.slots[token];
        const int pos = kMode == kWhole ? 0 : a.positions[token];
        const bool placed = kMode == kWhole || (pos >= 0 && pos < a.num_positions);
        const bool bad = slot >= a.num_slots || (!placed && (pos >= a.num_positions || slot >= 0));
        if (bad && h == 0 && lane == 0 && r < rows) atomicOr(a.status, PKV_DEVERR_RANGE);
        const bool live = r < rows && placed && (is_q || (slot >= 0 && slot < a.num_slots));
        const T* row = is_q ? static_cast<const T*>(a.q) + token * a.q_stride : is_v ? static_cast<const T*>(a.v) + token * a.v_stride
                                                                                  : static_cast<const T*>(a.k) + token * a.k_stride;
        row += head * D;
        float x[8] = {}, y[8] = {};
        if (live) {
            if (is_v)
                turn<kWhole>(row, nullptr, 0, false, at, x, y);
            else
                turn<kMode>(row, a.table + static_cast<int64_t>(pos) * a.rotary_dim, a.rotary_dim, a.interleaved != 0, at, x, y);
        }
        if (kMode == kAny) __syncwarp();  // q may turn in place, and its dimensions are read by two lanes
        if (is_q) {
            if (live) {
                T* out = static_cast<T*>(a.q_out) + token * a.q_out_stride + head * D;
                store8(out + 8 * at.va, x);
                store8(out + 8 * at.vb, y);
            }
        }
        if (kCache == PKV_F32 || kCache == PKV_BF16) {
            if (!is_q && live) {
                T* out = static_cast<T*>(is_v ? a.v_cache : a.k_cache) + (((slot >> 4) * a.kv_heads + head) * 16 + (slot & 15)) * D;
                store8(out + 8 * at.va, x);
                store8(out + 8 * at.vb, y);
            }
            continue;
        }
        // ---- quantized: the row's largest over its lanes (all lanes of the warp are here)
        float top = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, fmaxf(fabsf(x[e]), fabsf(y[e])));
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (is_q || !live) continue;
        constexpr float kLimit = kCache == PKV_INT4 ? 7.f : 127.f;
        // (a zero row's scale is 0 in a 4-bit cache, 1 in an int8 one)
        const float scale = kCache == PKV_INT4 ? top * kQ4Step : top > 0.f ? __fdiv_rn(top, kLimit) : 1.f;
        int cx[8], cy[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            cx[e] = scale > 0.f ? exact_code(x[e], scale, kLimit) : 0;
            cy[e] = scale > 0.f ? exact_code(y[e], scale, kLimit) : 0;
        }
        const int64_t chunk = (slot >> 4) * a.kv_heads + head;
        const int t = static_cast<int>(slot & 15);
        if (kCache == PKV_INT4) {
            uint8_t* rec = static_cast<uint8_t*>(a.k_cache) + chunk * q4_record_bytes(D);
            if (is_v) {
                uint8_t* v = rec + q4_v_offset(D);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[q4_v_byte(at.va, j, t)] = static_cast<uint8_t>((cx[2 * j] + 8) | (cx[2 * j + 1] + 8) << 4);
                    v[q4_v_byte(at.vb, j, t)] = static_cast<uint8_t>((cy[2 * j] + 8) | (cy[2 * j + 1] + 8) << 4);
                }
            } else {
                uint32_t* k = reinterpret_cast<uint32_t*>(rec + t * (D / 2));
                k[at.va] = k_word(cx);
                k[at.vb] = k_word(cy);
            }
            if (lane == 0) reinterpret_cast<float*>(rec + q4_scales_offset(D))[(is_v ? 16 : 0) + t] = scale;
        } else {
            if (is_v) {
                int8_t* v = static_cast<int8_t*>(a.v_cache) + chunk * D * 16 + t;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    v[(8 * at.va + e) * 16] = static_cast<int8_t>(cx[e]);
                    v[(8 * at.vb + e) * 16] = static_cast<int8_t>(cy[e]);
                }
            } else {
                int8_t* k = static_cast<int8_t*>(a.k_cache) + (chunk * 16 + t) * D;
                auto word = [](const int* c) {
                    return (c[0] & 255u) | (c[1] & 255u) << 8 | (c[2] & 255u) << 16 | static_cast<uint32_t>(c[3]) << 24;
                };
                *reinterpret_cast<uint2*>(k + 8 * at.va) = make_uint2(word(cx), word(cx + 4));
                *reinterpret_cast<uint2*>(k + 8 * at.vb) = make_uint2(word(cy), word(cy + 4));
            }
            if (lane == 0) a.scales[(chunk * 2 + (is_v ? 1 : 0)) * 16 + t] = scale;
        }
    }
}

template <int D, int kMode, int kCache, typename T>
cudaError_t run_append(const RotaryAppendArgs& a, cudaStream_t s) {
    const int64_t rows = a.num_tokens * (a.q_heads + 2 * a.kv_heads);
    constexpr int kRows = kThreads / (D / 16);
    const int64_t want = (rows + kRows - 1) / kRows, most = static_cast<int64_t>(device_sm_count()) * 16;
    return launch_pdl(append_rotary_kernel<D, kMode, kCache, T>, dim3(static_cast<unsigned>(want < most ? want : most)), dim3(kThreads), 0, s, a);
}
template <int D, int kCache, typename T>
cudaError_t run_mode(const RotaryAppendArgs& a, cudaStream_t s) {
    const int R = a.rotary_dim;
    if (R == 0) return run_append<D, kWhole, kCache, T>(a, s);
    if (!a.interleaved && R % 16 == 0) return run_append<D, kHalves, kCache, T>(a, s);
    if (a.interleaved && R % 8 == 0) return run_append<D, kNeighbours, kCache, T>(a, s);
    return run_append<D, kAny, kCache, T>(a, s);
}

// ---------------------------------------------------------------- the table
// Row p: factor cos(p f_i), i < half, then factor sin(p f_i). The angle in turns is p f_i
// / (2 pi) modulo 1: with g = f_i / (2 pi) as a 64-bit binary fraction that is p g modulo
// 2^64, an integer product, exact however far p is (g is off by 2^-53 of itself).
__device__ __forceinline__ uint64_t turn_fraction(double frequency) {
    const double turns = fabs(frequency) * 0.15915494309189533577;
    const uint64_t g = static_cast<uint64_t>((turns - floor(turns)) * 18446744073709551616.0);  // (an exact difference)
    return frequency < 0.0 ? 0 - g : g;
}
__global__ void __launch_bounds__(kThreads) rotary_table_kernel(const double* __restrict__ frequencies, int half, int64_t first,
                                                                int64_t positions, float factor, float* __restrict__ table) {
    grid_dependency_wait();
    allow_dependents();
    const int64_t all = positions * half;
    for (int64_t x = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; x < all; x += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int64_t p = x / half;
        const int i = static_cast<int>(x - p * half);
        const uint64_t g = turn_fraction(frequencies[i]);
        const int64_t part = static_cast<int64_t>(static_cast<uint64_t>(first + p) * g);  // of a turn, -1/2 .. 1/2
        float s, c;
        sincospif(__ll2float_rn(part) * 1.0842021724855044e-19f, &s, &c);  // 2^-63: half turns
        table[p * 2 * half + i] = c * factor;
        table[p * 2 * half + half + i] = s * factor;
    }
}

// Checked mode.
__global__ void check_positions_kernel(const int32_t* positions, const int64_t* slots, int64_t n, int32_t num_positions,
                                       unsigned int* verdict) {
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * blockDim.x)
        if (positions[i] >= num_positions || (positions[i] < 0 && slots[i] >= 0)) atomicOr(verdict, kVerdictRange);
}

}  // namespace

cudaError_t launch_check_positions(const int32_t* positions, const int64_t* slots, int64_t num_tokens, int32_t num_positions,
                                   unsigned int* verdict, cudaStream_t s) {
    check_positions_kernel<<<64, kThreads, 0, s>>>(positions, slots, num_tokens, num_positions, verdict);
    return cudaGetLastError();
}

bool rotary_frequencies(int R, double base, const pkv_rotary_scaling* scaling, double* out) {
    constexpr double kTurn = 6.283185307179586476925;
    if (R < 2 || R > 8192 || R % 2 || !(base > 1.0) || !isfinite(base)) return false;
    pkv_rotary_scaling s{};
    s.stretch = 1.0;
    if (scaling != nullptr) s = *scaling;
    if (s.kind < PKV_ROTARY_PLAIN || s.kind > PKV_ROTARY_RAMP) return false;
    if (s.kind != PKV_ROTARY_PLAIN && (!(s.stretch >= 1.0) || !isfinite(s.stretch))) return false;
    if (s.kind == PKV_ROTARY_BASE) {
        if (R == 2) return false;
        base *= pow(s.stretch, R / (R - 2.0));
        if (!isfinite(base)) return false;
    }
    double first = 0.0, last = 0.0;  // PKV_ROTARY_RAMP: where the mix begins and ends
    if (s.kind == PKV_ROTARY_TURNS || s.kind == PKV_ROTARY_RAMP) {
        if (!(s.original_context > 0.0) || !isfinite(s.original_context) || !(s.low_turns > 0.0) || !(s.high_turns > s.low_turns) ||
            !isfinite(s.high_turns))
            return false;
        // f_i makes n turns over the context where i = (R / 2) ln(context / (2 pi n)) / ln(base)
        auto makes = [&](double n) { return R / 2.0 * log(s.original_context / (kTurn * n)) / log(base); };
        first = fmax(floor(makes(s.high_turns)), 0.0);
        last = fmin(ceil(makes(s.low_turns)), R / 2.0 - 1.0);
    }
    for (int i = 0; i < R / 2; ++i) {
        const double f = pow(base, -2.0 * i / R);
        double keep = 1.0;  // share of f itself, the rest of f / stretch
        if (s.kind == PKV_ROTARY_LINEAR) keep = 0.0;
        if (s.kind == PKV_ROTARY_TURNS)
            keep = fmin(fmax((s.original_context * f / kTurn - s.low_turns) / (s.high_turns - s.low_turns), 0.0), 1.0);
        if (s.kind == PKV_ROTARY_RAMP) keep = 1.0 - fmin(fmax((i - first) / fmax(last - first, 1e-3), 0.0), 1.0);
        const bool mixed = s.kind == PKV_ROTARY_LINEAR || s.kind == PKV_ROTARY_TURNS || s.kind == PKV_ROTARY_RAMP;
        out[i] = mixed ? f * (keep + (1.0 - keep) / s.stretch) : f;
    }
    return true;
}

cudaError_t launch_append_rotary(const RotaryAppendArgs& a, const pkv_cache_desc& d, cudaStream_t s) {
    const bool wide = d.head_dim == 128;
    switch (d.dtype) {
        case PKV_F32: return wide ? run_mode<128, PKV_F32, float>(a, s) : run_mode<64, PKV_F32, float>(a, s);
        case PKV_BF16: return wide ? run_mode<128, PKV_BF16, __nv_bfloat16>(a, s) : run_mode<64, PKV_BF16, __nv_bfloat16>(a, s);
        case PKV_INT8: return wide ? run_mode<128, PKV_INT8, __nv_bfloat16>(a, s) : run_mode<64, PKV_INT8, __nv_bfloat16>(a, s);
        default: return wide ? run_mode<128, PKV_INT4, __nv_bfloat16>(a, s) : run_mode<64, PKV_INT4, __nv_bfloat16>(a, s);
    }
}

cudaError_t launch_rotary_table(const double* frequencies, int half, int64_t first, int64_t positions, float factor, float* table,
                                cudaStream_t s) {
    const int64_t want = (positions * half + kThreads - 1) / kThreads, most = static_cast<int64_t>(device_sm_count()) * 16;
    return launch_pdl(rotary_table_kernel, dim3(static_cast<unsigned>(want < most ? want : most)), dim3(kThreads), 0, s, frequencies, half,
                      first, positions, factor, table);
}

}  // namespace pkv
