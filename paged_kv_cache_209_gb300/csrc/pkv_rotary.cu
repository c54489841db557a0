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
// difference, two values at a time, comes with a bound on its error, and only where the
// bf16 roundings of both ends differ (one value in some 2^14) a difference of float32
// pairs decides, and float64 where that leaves a tie open.
//
// The append is pure streaming by its bytes (q in and out, k and v in, the pools' share
// out), and bound by its instructions, most of all by the exact rounding. Measured in a
// captured graph: 4096 tokens of 32 + 2 x 8 heads of 128 into a 4-bit cache 22.6 us, 88 MB
// at 3.9 TB/s (27.9 while V's codes went byte by byte; 16 with the rounding of one float32, inexact), into int8 pools 24.6,
// bf16 20.3 (101 MB, 5.0 TB/s), float32 31.1 (neighbouring pairs 34.1; 201 MB, 6.5 TB/s). Ragged prompts of 24 + 2 x 8 heads
// into bf16 pools 27.8 us, 5.3 TB/s; a decode step of 32 tokens 2.4 us. K and V alone, 4096 tokens of 24 heads: 19.6 us into a 4-bit
// cache without positions (64 MB, floor 9.4), 26.0 with them, 27.7 into int8 pools: 23 instructions an element for the
// quantizing (issue slots and ALU 71 % busy). A warp that goes from unit to unit with the next one's rows on their way took
// 1.8 us more for the first, 2.7 for the ragged prompts.
#include <math.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_q4.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 64;        // of the append's CTAs
constexpr int kAppendCtas = 14;     // an SM's at least: 72 registers a thread (at 96 registers and 10 CTAs 4096 tokens into a 4-bit
                                    // cache and their gather took 1.2 us more, of 38.2)
constexpr int kTableThreads = 256;  // of the table's, at most kTableCtas an SM
constexpr int kTableCtas = 8;       // (131072 x 64 angles: 11.3 us; 12.7 with 4, 12.1 with 16)
// Rows of an SM below which a warp takes one batch of heads, not two: a decode step's 32 tokens of
// 32 + 2 x 8 heads take 6.5 us so with their gather, 7.2 with two.
constexpr int kFew = 64;

// x c - y s rounded to float32 and to bf16. The exact value is s1 + lo, but for an error of lo's last
// bit: products and difference by their errors, which fused operations give exactly. Where that
// leaves open which float32 is nearest (one value in a thousand that come here), and near the ends of
// the float range, float64 decides.
__device__ __noinline__ float turned_exactly(float x, float c, float y, float s) {
    const float h = x * c, p = y * s, s1 = h - p, back = s1 - h;
    const float lo = ((h - (s1 - back)) - (p + back)) + (fmaf(x, c, -h) - fmaf(y, s, -p));
    const float r = s1 + lo, t = lo - (r - s1);
    const float half_step = __uint_as_float(__float_as_uint(r) & 0x7f800000u) * 5.9604645e-8f;  // 2^-24
    if (fabsf(lo) <= 4e-4f * fabsf(s1) && fabsf(t) < 0.999f * half_step && fabsf(r) > 1e-28f && fabsf(r) < 1e38f)
        return __bfloat162float(__float2bfloat16_rn(r));
    return __bfloat162float(__float2bfloat16_rn(static_cast<float>(static_cast<double>(x) * c - static_cast<double>(y) * s)));
}
// x c - y s as described above, for bf16 x and y held in float32: a bf16 in float32.
__device__ __forceinline__ float turned(__nv_bfloat16, float x, float c, float y, float s) {
    const float p = y * s;
    const float r = fmaf(x, c, -p);
    // each rounding is off by at most 2^-24 of its result (2^-150 below the normal range)
    const float off = fmaf(fabsf(p) + fabsf(r), 1.1920929e-7f, 2.8026e-45f);
    const uint32_t ends = pack_bf16x2(r - off, r + off);
    if ((ends & 0xffffu) == ends >> 16 && (ends & 0x7f80u) != 0x7f80u) return bf16hi_to_f32(ends);
    return turned_exactly(x, c, y, s);
}
// float32 rows: the product's error joins the sum (one rounding, and one of a small term). Where the result is not
// finite the product alone may have left the range, or been an infinity's: then float64 (turned_wide).
__device__ __forceinline__ float turned(float, float x, float c, float y, float s) {
    const float p = y * s;
    return fmaf(x, c, -p) - fmaf(y, s, -p);
}
__device__ __noinline__ float turned_wide(float x, float c, float y, float s) {
    return static_cast<float>(static_cast<double>(x) * c - static_cast<double>(y) * s);
}
__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= 3.402823466e38f; }

// Eight elements of a row as they are stored: words of two (bf16), or one each.
template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
    uint32_t w[4];
    __device__ __forceinline__ void load(const void* p) {
        const uint4 v = *static_cast<const uint4*>(p);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    }
    __device__ __forceinline__ void store(void* p) const { *static_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]); }
    __device__ __forceinline__ float get(int e) const { return e & 1 ? bf16hi_to_f32(w[e / 2]) : bf16lo_to_f32(w[e / 2]); }
    __device__ __forceinline__ void set(int e, float x) {  // (of a value that bf16 holds)
        w[e / 2] = e & 1 ? w[e / 2] & 0xffffu | __float_as_uint(x) : w[e / 2] & 0xffff0000u | __float_as_uint(x) >> 16;
    }
};
template <>
struct Eight<float> {
    float w[8];
    __device__ __forceinline__ void load(const void* p) {
        const float4 u = static_cast<const float4*>(p)[0], v = static_cast<const float4*>(p)[1];
        w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w, w[4] = v.x, w[5] = v.y, w[6] = v.z, w[7] = v.w;
    }
    __device__ __forceinline__ void store(void* p) const {
        static_cast<float4*>(p)[0] = make_float4(w[0], w[1], w[2], w[3]);
        static_cast<float4*>(p)[1] = make_float4(w[4], w[5], w[6], w[7]);
    }
    __device__ __forceinline__ float get(int e) const { return w[e]; }
    __device__ __forceinline__ void set(int e, float x) { w[e] = x; }
};
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

// The lane's cosines and sines of a token: kHalves of the pairs of both vectors, kNeighbours
// of va's four pairs, then vb's.
template <int kMode>
__device__ __forceinline__ void load_angles(const float* cs, int R, const Place& at, float (&c)[8], float (&s)[8]) {
    const int half = R / 2;
    auto four = [](const float* p, float (&x)[8], int to) {
        const float4 v = *reinterpret_cast<const float4*>(p);
        x[to] = v.x, x[to + 1] = v.y, x[to + 2] = v.z, x[to + 3] = v.w;
    };
    if (kMode == kHalves && at.turns) {
        four(cs + 8 * at.va, c, 0), four(cs + 8 * at.va + 4, c, 4);
        four(cs + half + 8 * at.va, s, 0), four(cs + half + 8 * at.va + 4, s, 4);
    }
    if (kMode == kNeighbours) {
        if (8 * at.va < R) four(cs + 4 * at.va, c, 0), four(cs + half + 4 * at.va, s, 0);
        if (8 * at.vb < R) four(cs + 4 * at.vb, c, 4), four(cs + half + 4 * at.vb, s, 4);
    }
}

// Two values r, off by at most `off` each, as bf16; false if a rounding is not decided by that.
__device__ __forceinline__ bool decided(uint64_t r, uint64_t off, uint32_t& word) {
    float a, b, c, d;
    f32x2_unpack(f32x2_sub(r, off), a, b);
    f32x2_unpack(f32x2_add(r, off), c, d);
    word = pack_bf16x2(c, d);
    return pack_bf16x2(a, b) == word;
}

// (The pairs that a lane's halves leave open, one at a time: short code, as few lanes come here. 4096 tokens 21.9
// us, 23.3 with every pair's own code; of neighbours, whose words hold whole pairs, 27.6 so and 28.4 one at a time.)
__device__ __forceinline__ float pick(const float (&v)[8], int e) {
    float x = v[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) x = e == i ? v[i] : x;
    return x;
}
__device__ __forceinline__ uint32_t pick(const uint32_t (&v)[4], int i) { return i == 0 ? v[0] : i == 1 ? v[1] : i == 2 ? v[2] : v[3]; }
// Two elements' words x and y (their partners) turned by (c0, s0) and (c1, s1).
__device__ __forceinline__ uint32_t turned_pair(uint32_t x, uint32_t y, float c0, float s0, float c1, float s1) {
    const float lo = turned_exactly(bf16lo_to_f32(x), c0, bf16lo_to_f32(y), s0), hi = turned_exactly(bf16hi_to_f32(x), c1, bf16hi_to_f32(y), s1);
    return __float_as_uint(lo) >> 16 | (__float_as_uint(hi) & 0xffff0000u);
}

// Turns the lane's vectors of a row of bf16s, two elements at a time. `size`: the largest of the
// lane's |c| and |s|. With X the larger of a pair's magnitudes, |y s| <= X size and |r| <= 2
// X size, so r = x c - y s is off by at most 2^-24 (|y s| + |r|) <= 3 2^-24 X size (and 2^-149
// below the normal range). Taken as X size first, the bound is infinite, and nothing decided, where a product may leave the
// range though y does not.
template <int kMode>
__device__ __forceinline__ void turn(Eight<__nv_bfloat16>& a, Eight<__nv_bfloat16>& b, const float (&c)[8], const float (&s)[8], float size,
                                     const Place& at, int R) {
    const uint64_t size2 = f32x2_pack(size, size), part = f32x2_pack(2.0e-7f, 2.0e-7f), least = f32x2_pack(2.8026e-45f, 2.8026e-45f);  // (3.36 2^-24)
    if (kMode == kHalves) {
        if (!at.turns) return;
        uint32_t open = 0;
        Eight<__nv_bfloat16> x = a, y = b;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x0 = x.get(2 * i), x1 = x.get(2 * i + 1), y0 = y.get(2 * i), y1 = y.get(2 * i + 1);
            const uint64_t xx = f32x2_pack(x0, x1), yy = f32x2_pack(y0, y1), cc = f32x2_pack(c[2 * i], c[2 * i + 1]), ss = f32x2_pack(s[2 * i], s[2 * i + 1]);
            const uint64_t off = f32x2_fma(f32x2_mul(f32x2_pack(fmaxf(fabsf(x0), fabsf(y0)), fmaxf(fabsf(x1), fabsf(y1))), size2), part, least);
            if (!decided(f32x2_fma(xx, cc, f32x2_mul(yy, f32x2_mul(ss, f32x2_pack(-1.f, -1.f)))), off, a.w[i])) open |= 1u << i;
            if (!decided(f32x2_fma(yy, cc, f32x2_mul(xx, ss)), off, b.w[i])) open |= 16u << i;
        }
#pragma unroll 1
        while (open) {
            const int bit = __ffs(open) - 1, i = bit & 3;
            open &= open - 1;
            const bool second = bit >= 4;
            const uint32_t xw = pick(x.w, i), yw = pick(y.w, i);
            const float s0 = pick(s, 2 * i), s1 = pick(s, 2 * i + 1);
            const uint32_t w = turned_pair(second ? yw : xw, second ? xw : yw, pick(c, 2 * i), second ? -s0 : s0, pick(c, 2 * i + 1), second ? -s1 : s1);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (bit == j) a.w[j] = w;
                if (bit == 4 + j) b.w[j] = w;
            }
        }
    } else if (kMode == kNeighbours) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            Eight<__nv_bfloat16>& v = u ? b : a;
            if (8 * (u ? at.vb : at.va) >= R) break;
            uint32_t open = 0;
            const Eight<__nv_bfloat16> x = v;
            float o[4];
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                const uint64_t top = f32x2_pack(fmaxf(fabsf(x.get(2 * i)), fabsf(x.get(2 * i + 1))), fmaxf(fabsf(x.get(2 * i + 2)), fabsf(x.get(2 * i + 3))));
                f32x2_unpack(f32x2_fma(f32x2_mul(top, size2), part, least), o[i], o[i + 1]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x0 = x.get(2 * i), x1 = x.get(2 * i + 1), cc = c[4 * u + i], ss = s[4 * u + i];
                if (!decided(f32x2_fma(f32x2_pack(x0, x1), f32x2_pack(cc, cc), f32x2_mul(f32x2_pack(x1, x0), f32x2_pack(-ss, ss))), f32x2_pack(o[i], o[i]), v.w[i]))
                    open |= 1u << i;
            }
            if (open) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (open >> i & 1) {
                        const float x0 = x.get(2 * i), x1 = x.get(2 * i + 1);
                        v.set(2 * i, turned_exactly(x0, c[4 * u + i], x1, s[4 * u + i]));
                        v.set(2 * i + 1, turned_exactly(x1, c[4 * u + i], x0, -s[4 * u + i]));
                    }
            }
        }
    }
}
// float32: by turned(), or with kWide by turned_wide().
template <int kMode, bool kWide>
__device__ __forceinline__ void turn_f32(Eight<float>& a, Eight<float>& b, const float (&c)[8], const float (&s)[8], const Place& at, int R) {
    auto one = [](float x, float c, float y, float s) { return kWide ? turned_wide(x, c, y, s) : turned(x, x, c, y, s); };
    if (kMode == kHalves) {
        if (!at.turns) return;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float x = a.w[e], y = b.w[e];
            a.w[e] = one(x, c[e], y, s[e]);
            b.w[e] = one(y, c[e], x, -s[e]);
        }
    } else if (kMode == kNeighbours) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            Eight<float>& v = u ? b : a;
            if (8 * (u ? at.vb : at.va) >= R) break;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float x = v.w[2 * e], y = v.w[2 * e + 1];
                v.w[2 * e] = one(x, c[4 * u + e], y, s[4 * u + e]);
                v.w[2 * e + 1] = one(y, c[4 * u + e], x, -s[4 * u + e]);
            }
        }
    }
}
template <int kMode>
__device__ __forceinline__ void turn(Eight<float>& a, Eight<float>& b, const float (&c)[8], const float (&s)[8], float, const Place& at, int R) {
    turn_f32<kMode, false>(a, b, c, s, at, R);
}
// Any even R: the partner of every dimension is read apart (`row`: the row's first element, `cs`: the table's row).
template <typename T>
__device__ __forceinline__ void turn_any(Eight<T>& a, Eight<T>& b, const Place& at, int R, const T* row, const float* cs, bool interleaved) {
    const int half = R / 2;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        Eight<T>& v = u ? b : a;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int d = 8 * (u ? at.vb : at.va) + e;
            if (d >= R) continue;
            const int i = interleaved ? d / 2 : d % half;
            const bool second = interleaved ? (d & 1) != 0 : d >= half;
            const int other = interleaved ? d ^ 1 : second ? d - half : d + half;
            const float y = value(row[other]), w = cs[half + i];
            float r = turned(T{}, v.get(e), cs[i], y, second ? -w : w);
            if (sizeof(T) == 4 && !finite(r)) r = turned_wide(v.get(e), cs[i], y, second ? -w : w);
            v.set(e, r);
        }
    }
}

// The codes of a row of bf16s, int8 (two's complement) or 4-bit (code + 8): the nearest
// integer c to x / scale, ties to even. x times 1 / scale gives c or a neighbour. x - c scale is
// exact in float32 (a multiple of the scale's last bit, below twice the scale; both taken
// far above the subnormal range first), and its magnitude against scale / 2 says whether
// c has to move: the two compare as integers, where an odd c counts as one more, which
// breaks ties to even. Needs no clipping: |x| <= limit scale but for a rounding.
template <int kCache>
struct Codes {
    float scale, inverse, lift;
    uint32_t half;
    __device__ __forceinline__ explicit Codes(float s) {
        lift = s < 1e-20f ? 1.2089258e24f : 1.f;  // 2^80
        scale = s * lift;
        inverse = scale > 0.f ? __fdividef(1.f, scale) : 0.f;
        half = __float_as_uint(scale * 0.5f);
    }
    __device__ __forceinline__ uint32_t operator()(float x) const {
        constexpr float kShift = 12582912.f + (kCache == PKV_INT4 ? 8.f : 0.f);  // 1.5 2^23: an integer sits in its low bits
        x *= lift;
        const float shifted = fmaf(x, inverse, kShift);
        const float rest = fmaf(-(shifted - kShift), scale, x);
        uint32_t c = __float_as_uint(shifted);
        if ((__float_as_uint(rest) & 0x7fffffffu) + (c & 1u) > half) c += __float_as_int(rest) >> 31 | 1;
        return c & (kCache == PKV_INT4 ? 15u : 255u);
    }
};
__device__ __forceinline__ uint32_t k_word(const uint32_t (&c)[8]) {  // of a 4-bit record
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) w |= c[e] << (4 * (e / 2 + 4 * (e & 1)));
    return w;
}

// The scale of the row that D / 16 lanes hold (all lanes of the warp). (A zero row's is 0 in a 4-bit cache, 1 in an int8
// one, NaN that of a row with a NaN or an infinity, whose values are then no numbers whatever their codes. The codes of
// such a row cleared as well: 4096 tokens of 24 heads 26.3 us, so 25.7.)
template <int D, int kCache>
__device__ __forceinline__ float row_scale(const Eight<__nv_bfloat16>& x, const Eight<__nv_bfloat16>& y) {
    float top = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = fmax3_nan(top, fabsf(x.get(e)), fabsf(y.get(e)));
#pragma unroll
    for (int o = 1; o < D / 16; o <<= 1) top = fmax_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    top = fmaf(top, 0.f, top);  // NaN for an infinity
    return kCache == PKV_INT4 ? top * kQ4Step : top == 0.f ? 1.f : __fdiv_rn(top, 127.f);
}
// Whether an append's V goes by windows of 16 tokens.
constexpr bool by_windows(int cache, int batch) { return (cache == PKV_INT4 || cache == PKV_INT8) && batch > 1; }

// Where a byte of a block's V codes (one head) lies while it is put together in shared memory: pieces
// of 16 bytes change places so that lanes of different octets meet different banks.
template <int kCache>
__device__ __forceinline__ int staged(int byte) {
    const int piece = byte >> 4;
    return (piece ^ (kCache == PKV_INT4 ? piece >> 3 & 3 : piece >> 3 & 7)) << 4 | (byte & 15);
}
// Byte of octet o's dimension 8 o + e (a pair of dimensions of a 4-bit code) of token t.
template <int kCache>
__device__ __forceinline__ int v_byte(int o, int e, int t) {
    return kCache == PKV_INT4 ? q4_v_byte(o, e >> 1, t) : (8 * o + e) * 16 + t;
}

// V of the 16 tokens from 16 `window` on, one head, quantized. A byte of a block's V codes is one token's, its
// words are several's: stored token by token, K and V of 4096 tokens of 24 heads take 47.7 us into a 4-bit cache and
// 115 into an int8 one, so 26.0 and 27.7. Where 16 tokens that follow one another fill a block, the warp whose window holds their first puts
// the block together in shared memory; tokens of no such block are stored byte by byte.
template <int D, int kMode, int kCache>
__device__ __forceinline__ void append_v_window(const RotaryAppendArgs& a, uint32_t window, int head, uint8_t* stage) {
    constexpr int kLanes = D / 16, kRows = 32 / kLanes, kSteps = 16 / kRows;
    constexpr int kStep = kCache == PKV_INT4 ? 2 : 1;                 // dimensions of a byte
    constexpr int kBytes = (kCache == PKV_INT4 ? 8 : 16) * D;         // of the block's V codes
    const int lane32 = threadIdx.x & 31, lane = lane32 % kLanes, row = lane32 / kLanes;
    const int64_t r0 = static_cast<int64_t>(window) * 16;
    auto slot_of = [&](int64_t r) -> int64_t {  // -1: nothing is stored
        if (r < 0 || r >= a.num_tokens) return -1;
        const int64_t s = a.slots[r];
        const int pos = kMode == kWhole ? 0 : a.positions[r];
        return s >= 0 && s < a.num_slots && (kMode == kWhole || (pos >= 0 && pos < a.num_positions)) ? s : -1;
    };
    // rows r0 - 16 .. r0 + 31, and which of them go on where the row before left off in its block
    const int64_t s0 = slot_of(r0 - 16 + lane32), s1 = lane32 < 16 ? slot_of(r0 + 16 + lane32) : -1;
    int64_t p0 = __shfl_up_sync(0xffffffffu, s0, 1), p1 = __shfl_up_sync(0xffffffffu, s1, 1);
    const int64_t last = __shfl_sync(0xffffffffu, s0, 31);
    if (lane32 == 0) p0 = -2, p1 = last;
    const uint32_t goes0 = __ballot_sync(0xffffffffu, (s0 & 15) != 0 && s0 >= 0 && s0 == p0 + 1 && p0 >= 0);
    const uint32_t goes1 = __ballot_sync(0xffffffffu, (s1 & 15) != 0 && s1 >= 0 && s1 == p1 + 1 && p1 >= 0);
    const uint64_t goes = goes0 | static_cast<uint64_t>(goes1) << 32;
    const uint32_t whole = __ballot_sync(0xffffffffu, s0 >= 0 && (s0 & 15) == 0 && (goes >> (lane32 + 1) & 0x7fff) == 0x7fff);
    // the window's tokens: some end a block that began before it, some are alone, the rest belongs to a block that begins here
    const int alone = (whole & 0xfffeu) != 0 ? 31 - __clz(whole & 0xfffeu) : 0;
    const int begins = whole >> 16 != 0 ? __ffs(whole >> 16) - 1 : 16;
    const __nv_bfloat16* from = static_cast<const __nv_bfloat16*>(a.v) + head * D + 8 * lane;  // octets lane and lane + kLanes
    uint8_t* pool = static_cast<uint8_t*>(kCache == PKV_INT4 ? a.k_cache : a.v_cache);
    auto codes_at = [&](int64_t slot) {
        const int64_t chunk = (slot >> 4) * a.kv_heads + head;
        return kCache == PKV_INT4 ? pool + chunk * q4_record_bytes(D) + q4_v_offset(D) : pool + chunk * kBytes;
    };
    auto scales_at = [&](int64_t slot) {
        const int64_t chunk = (slot >> 4) * a.kv_heads + head;
        return (kCache == PKV_INT4 ? reinterpret_cast<float*>(pool + chunk * q4_record_bytes(D) + q4_scales_offset(D)) : a.scales + chunk * 32) + 16;
    };
    // a row's codes, byte by byte to put(byte, code); its scale
    auto quantize = [&](const Eight<__nv_bfloat16>(&x)[2], int t, auto put) {
        const float scale = row_scale<D, kCache>(x[0], x[1]);
        const Codes<kCache> code(scale);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 8; e += kStep)
                put(v_byte<kCache>(lane + kLanes * i, e, t), kStep == 2 ? code(x[i].get(e)) | code(x[i].get(e + kStep - 1)) << 4 : code(x[i].get(e)));
        return scale;
    };
    if (begins < 16) {
        const int64_t slot = __shfl_sync(0xffffffffu, s0, 16 + begins);
        Eight<__nv_bfloat16> x[kSteps][2];
#pragma unroll
        for (int b = 0; b < kSteps; ++b) {
            const __nv_bfloat16* p = from + (r0 + begins + b * kRows + row) * a.v_stride;
            x[b][0].load(p), x[b][1].load(p + 8 * kLanes);
        }
        float* scales = scales_at(slot);
#pragma unroll
        for (int b = 0; b < kSteps; ++b) {
            const int t = b * kRows + row;
            const float scale = quantize(x[b], t, [&](int byte, uint32_t c) { stage[staged<kCache>(byte)] = static_cast<uint8_t>(c); });
            if (lane == 0) scales[t] = scale;
        }
        __syncwarp();
        uint8_t* to = codes_at(slot);
#pragma unroll
        for (int i = 16 * lane32; i < kBytes; i += 512) *reinterpret_cast<uint4*>(to + i) = *reinterpret_cast<const uint4*>(stage + staged<kCache>(i));
    }
    for (int b = alone; b < begins; b += kRows) {
        const int64_t slot = __shfl_sync(0xffffffffu, s0, 16 + min(b + row, 15));
        const bool live = b + row < begins && slot >= 0;
        Eight<__nv_bfloat16> x[2] = {};
        if (live) {
            const __nv_bfloat16* p = from + (r0 + b + row) * a.v_stride;
            x[0].load(p), x[1].load(p + 8 * kLanes);
        }
        uint8_t* to = codes_at(live ? slot : 0);
        const int t = static_cast<int>(slot & 15);
        const float scale = quantize(x, t, [&](int byte, uint32_t c) {
            if (live) to[byte] = static_cast<uint8_t>(c);
        });
        if (live && lane == 0) scales_at(slot)[t] = scale;
    }
}

// One warp takes a unit: kBatch times kRows heads of one token, all of q, of k or of v, D / 16 lanes a
// row, all of its loads in flight at once. Units are numbered token by token, so that what runs at
// a time reads and writes memory that lies together. Where there are many rows, a quantizing cache's V goes
// by windows of 16 tokens, which come first. kCache: the pkv_dtype of the pools, or PKV_INT4.
template <int D, int kMode, int kCache, typename T, int kBatch>
__global__ void __launch_bounds__(kThreads, kAppendCtas) append_rotary_kernel(const RotaryAppendArgs a) {
    constexpr int kLanes = D / 16;
    constexpr int kRows = 32 / kLanes;
    constexpr int kHeads = kBatch * kRows;
    constexpr bool kWindows = by_windows(kCache, kBatch);
    grid_dependency_wait();  // q, k, v, and a block copied onto the slots' block, come from the kernels before
    allow_dependents();
    const uint32_t lane = threadIdx.x % kLanes, row = threadIdx.x % 32 / kLanes;
    const uint32_t q_units = (a.q_heads + kHeads - 1) / kHeads, kv_units = (a.kv_heads + kHeads - 1) / kHeads;
    const uint32_t units = q_units + (kWindows ? 1 : 2) * kv_units;  // of a token
    uint32_t w = blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
    if (kWindows) {
        __shared__ alignas(16) uint8_t stage[kWindows ? kThreads / 32 : 1][kWindows ? (kCache == PKV_INT4 ? 8 : 16) * D : 16];
        const uint32_t windows = static_cast<uint32_t>((a.num_tokens + 15) / 16) * a.kv_heads;
        if (w < windows) {
            const uint32_t window = w / a.kv_heads;
            append_v_window<D, kMode, kCache>(a, window, w - window * a.kv_heads, stage[threadIdx.x / 32]);
            return;
        }
        w -= windows;
    }
    const uint32_t token = w / units, unit = w - token * units;
    if (token >= static_cast<uint32_t>(a.num_tokens)) return;
    const Place at = place_of<kMode>(lane, a.rotary_dim);
    const bool is_q = unit < q_units, is_v = unit >= q_units + kv_units;
    const int heads = is_q ? a.q_heads : a.kv_heads;
    const int head0 = (unit - (is_q ? 0 : is_v ? q_units + kv_units : q_units)) * kHeads + row;  // of this lane's heads, kRows apart
    const T* from = (is_q ? static_cast<const T*>(a.q) + token * a.q_stride
                          : is_v ? static_cast<const T*>(a.v) + token * a.v_stride : static_cast<const T*>(a.k) + token * a.k_stride) + head0 * D;
    Eight<T> in[kBatch][2];
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
        if (head0 + b * kRows < heads) {
            in[b][0].load(from + b * kRows * D + 8 * at.va);
            in[b][1].load(from + b * kRows * D + 8 * at.vb);
        }
    const int64_t slot = a.slots[token];
    const int pos = kMode == kWhole ? 0 : a.positions[token];
    const bool placed = kMode == kWhole || (pos >= 0 && pos < a.num_positions);
    const bool bad = slot >= a.num_slots || (!placed && (pos >= a.num_positions || slot >= 0));
    if (bad && unit == 0 && lane + row == 0) atomicOr(a.status, PKV_DEVERR_RANGE);
    if (!placed || (!is_q && (slot < 0 || slot >= a.num_slots))) return;  // (the whole warp)
    const float* cs = a.table + static_cast<int64_t>(pos) * a.rotary_dim;
    float c[8] = {}, s[8] = {}, size = 0.f;
    if ((kMode == kHalves || kMode == kNeighbours) && !is_v) {
        load_angles<kMode>(cs, a.rotary_dim, at, c, s);
#pragma unroll
        for (int e = 0; e < 8; ++e) size = fmax3(size, fabsf(c[e]), fabsf(s[e]));
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
        const int head = head0 + b * kRows;
        if (head - static_cast<int>(row) >= heads) break;  // (no row of the warp)
        const bool live = head < heads;
        Eight<T> x{}, y{};
        if (live) {
            x = in[b][0];
            y = in[b][1];
            if (!is_v) {
                if (kMode == kAny)
                    turn_any<T>(x, y, at, a.rotary_dim, from + b * kRows * D, cs, a.interleaved != 0);
                else if (kMode != kWhole)
                    turn<kMode>(x, y, c, s, size, at, a.rotary_dim);
                if constexpr (sizeof(T) == 4 && (kMode == kHalves || kMode == kNeighbours)) {
                    float top = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) top = fmax3_nan(top, fabsf(x.get(e)), fabsf(y.get(e)));
                    if (!finite(top)) {  // (the row as it was, read again)
                        x.load(from + b * kRows * D + 8 * at.va);
                        y.load(from + b * kRows * D + 8 * at.vb);
                        turn_f32<kMode, true>(x, y, c, s, at, a.rotary_dim);
                    }
                }
            }
        }
        if (kMode == kAny) __syncwarp();  // q may turn in place, its dimensions read by two lanes
        if (is_q) {
            if (live) {
                T* out = static_cast<T*>(a.q_out) + token * a.q_out_stride + head * D;
                x.store(out + 8 * at.va);
                y.store(out + 8 * at.vb);
            }
            continue;
        }
        if constexpr (kCache == PKV_F32 || kCache == PKV_BF16) {
            if (live) {
                T* out = static_cast<T*>(is_v ? a.v_cache : a.k_cache) + (((slot >> 4) * a.kv_heads + head) * 16 + (slot & 15)) * D;
                x.store(out + 8 * at.va);
                y.store(out + 8 * at.vb);
            }
        } else {
            // ---- quantized (all lanes of the warp are here)
            const float scale = row_scale<D, kCache>(x, y);
            if (!live) continue;
            const Codes<kCache> code(scale);
            uint32_t cx[8], cy[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                cx[e] = code(x.get(e));
                cy[e] = code(y.get(e));
            }
            const int64_t chunk = (slot >> 4) * a.kv_heads + head;
            const int t = static_cast<int>(slot & 15);
            if (kCache == PKV_INT4) {
                uint8_t* rec = static_cast<uint8_t*>(a.k_cache) + chunk * q4_record_bytes(D);
                if (is_v) {
                    uint8_t* v = rec + q4_v_offset(D);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        v[q4_v_byte(at.va, j, t)] = static_cast<uint8_t>(cx[2 * j] | cx[2 * j + 1] << 4);
                        v[q4_v_byte(at.vb, j, t)] = static_cast<uint8_t>(cy[2 * j] | cy[2 * j + 1] << 4);
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
                    auto word = [](const uint32_t* c) { return c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24; };
                    *reinterpret_cast<uint2*>(k + 8 * at.va) = make_uint2(word(cx), word(cx + 4));
                    *reinterpret_cast<uint2*>(k + 8 * at.vb) = make_uint2(word(cy), word(cy + 4));
                }
                if (lane == 0) a.scales[(chunk * 2 + (is_v ? 1 : 0)) * 16 + t] = scale;
            }
        }
    }
}

template <int D, int kMode, int kCache, typename T, int kBatch>
cudaError_t run_batch(const RotaryAppendArgs& a, cudaStream_t s) {
    constexpr int kHeads = kBatch * 32 / (D / 16), kWarps = kThreads / 32;
    constexpr bool kWindows = by_windows(kCache, kBatch);
    const int64_t units = a.num_tokens * ((a.q_heads + kHeads - 1) / kHeads + (kWindows ? 1 : 2) * ((a.kv_heads + kHeads - 1) / kHeads)) +
                          (kWindows ? (a.num_tokens + 15) / 16 * a.kv_heads : 0);
    return launch_pdl(append_rotary_kernel<D, kMode, kCache, T, kBatch>, dim3(static_cast<unsigned>((units + kWarps - 1) / kWarps)), dim3(kThreads), 0, s, a);
}
template <int D, int kMode, int kCache, typename T>
cudaError_t run_append(const RotaryAppendArgs& a, cudaStream_t s) {
    // two batches of a warp's loads in flight (4096 tokens of 32 + 2 x 8 heads, a 4-bit cache, with their gather, 38.2 us
    // then: 4.6 more with one, 1.8 with four)
    constexpr int kBatch = kMode == kAny ? 1 : 2;
    // few rows: every warp takes as few as it can, so that they spread over the SMs
    const int64_t rows = a.num_tokens * (a.q_heads + 2 * a.kv_heads);
    if (kBatch == 1 || rows < static_cast<int64_t>(device_sm_count()) * kFew) return run_batch<D, kMode, kCache, T, 1>(a, s);
    return run_batch<D, kMode, kCache, T, kBatch>(a, s);
}
template <int D, int kCache, typename T>
cudaError_t run_mode(const RotaryAppendArgs& a, cudaStream_t s) {
    const int R = a.rotary_dim;
    if constexpr (kCache == PKV_INT4) {  // pkv_append_q4
        if (R == 0) return run_append<D, kWhole, kCache, T>(a, s);
    }
    if (!a.interleaved && R % 16 == 0) return run_append<D, kHalves, kCache, T>(a, s);
    if (a.interleaved && R % 8 == 0) return run_append<D, kNeighbours, kCache, T>(a, s);
    return run_append<D, kAny, kCache, T>(a, s);
}

// ---------------------------------------------------------------- the table
// Row p: factor cos(p f_i), i < half, then factor sin(p f_i). The angle in turns is p f_i
// / (2 pi) modulo 1: with g = f_i / (2 pi) as a 64-bit binary fraction that is p g modulo
// 2^64, an integer product, exact however far p is (g is off by 2^-53 of itself). A thread
// keeps kV neighbouring frequencies and adds (step g) from one of its rows to the next.
// Of the fraction the upper 32 bits give the quarter turn and the angle from there, at most
// an eighth of a turn, whose sine and cosine are their Taylor polynomials of degree 9 and 8
// (off by 1.8e-9 and 2.5e-8 at most).
__device__ __forceinline__ uint64_t turn_fraction(double frequency) {
    const double turns = fabs(frequency) * 0.15915494309189533577;
    const uint64_t g = static_cast<uint64_t>((turns - floor(turns)) * 18446744073709551616.0);  // (an exact difference)
    return frequency < 0.0 ? 0 - g : g;
}
__device__ __forceinline__ void cos_sin(uint64_t part, float factor, float& c, float& s) {
    const uint32_t u = static_cast<uint32_t>(part >> 32);
    const uint32_t quarter = (u + 0x20000000u) >> 30;
    const float x = static_cast<float>(static_cast<int32_t>(u - (quarter << 30))) * 1.46291807926716e-9f;  // 2 pi / 2^32
    const float t = x * x;
    float ps = fmaf(t, 1.f / 362880.f, -1.f / 5040.f), pc = fmaf(t, 1.f / 40320.f, -1.f / 720.f);
    ps = fmaf(t, ps, 1.f / 120.f), pc = fmaf(t, pc, 1.f / 24.f);
    ps = fmaf(t, ps, -1.f / 6.f), pc = fmaf(t, pc, -0.5f);
    ps = fmaf(t * x, ps, x), pc = fmaf(t, pc, 1.f);
    const bool swap = (quarter & 1) != 0;
    c = __uint_as_float(__float_as_uint((swap ? ps : pc) * factor) ^ ((quarter + 1) & 2) << 30);
    s = __uint_as_float(__float_as_uint((swap ? pc : ps) * factor) ^ (quarter & 2) << 30);
}
template <int kV>
__global__ void __launch_bounds__(kTableThreads) rotary_table_kernel(const double* __restrict__ frequencies, int half, int64_t first,
                                                                int64_t positions, float factor, float* __restrict__ table) {
    extern __shared__ uint64_t turns[];  // double arithmetic is slow here: once a frequency
    grid_dependency_wait();
    allow_dependents();
    for (int i = threadIdx.x; i < half; i += kTableThreads) turns[i] = turn_fraction(frequencies[i]);
    __syncthreads();
    const int64_t per_row = half / kV;
    const int64_t thread = static_cast<int64_t>(blockIdx.x) * kTableThreads + threadIdx.x;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kTableThreads / per_row;  // rows (the last threads may have none)
    int64_t p = thread / per_row;
    const int i = static_cast<int>(thread - p * per_row) * kV;
    if (p >= step || p >= positions) return;
    uint64_t at[kV], by[kV];
#pragma unroll
    for (int e = 0; e < kV; ++e) {
        at[e] = static_cast<uint64_t>(first + p) * turns[i + e];
        by[e] = static_cast<uint64_t>(step) * turns[i + e];
    }
    float* row = table + p * 2 * half + i;
    for (; p < positions; p += step, row += step * 2 * half) {
        float c[kV], s[kV];
#pragma unroll
        for (int e = 0; e < kV; ++e) {
            cos_sin(at[e], factor, c[e], s[e]);
            at[e] += by[e];
        }
        if (kV == 4) {
            *reinterpret_cast<float4*>(row) = make_float4(c[0], c[1], c[2], c[kV - 1]);
            *reinterpret_cast<float4*>(row + half) = make_float4(s[0], s[1], s[2], s[kV - 1]);
        } else {
            row[0] = c[0];
            row[half] = s[0];
        }
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
        last = fmin(ceil(makes(s.low_turns)), R - 1.0);  // (past the last pair: the ramp goes on there, and that pair keeps its share)
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
    const int64_t threads = positions * half / (half % 4 ? 1 : 4);
    const int64_t want = (threads + kTableThreads - 1) / kTableThreads, most = static_cast<int64_t>(device_sm_count()) * kTableCtas;
    // (at least a row's threads)
    const int64_t row = (half / (half % 4 ? 1 : 4) + kTableThreads - 1) / kTableThreads;
    const dim3 grid(static_cast<unsigned>(want < row ? row : want < most ? want : most));
    const size_t smem = static_cast<size_t>(half) * sizeof(uint64_t);
    if (half % 4) return launch_pdl(rotary_table_kernel<1>, grid, dim3(kTableThreads), smem, s, frequencies, half, first, positions, factor, table);
    return launch_pdl(rotary_table_kernel<4>, grid, dim3(kTableThreads), smem, s, frequencies, half, first, positions, factor, table);
}

}  // namespace pkv
