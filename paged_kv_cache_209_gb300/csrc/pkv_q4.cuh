// The 4-bit cache: how a (block, KV head) record holds its 16 tokens, and how a row is
// quantized.
//
// A record is one contiguous piece of 16 D + 128 bytes (2176 at head_dim 128, a multiple
// of 128), so that a kernel fetches a block of a head with one bulk copy where three
// pools (K codes, V codes, scales) would take three:
//     [0, 8 D)           K codes, a token's row of D / 2 bytes after the other
//     [8 D, 16 D)        V codes
//     [16 D, 16 D + 128) 16 K scales, then 16 V scales, float32
// A code c, -7 .. 7, is the nibble c + 8; nibbles p and p + 4 of a 32-bit word are what
// one mask takes out as the two halves of an f16x2.
//     K: nibble p of a row's word w is dimension 8 w + 2 (p % 4) + p / 4;
//     V: word (o, q, j), o < D / 8, q < 4, j < 4, holds in nibble p dimension
//        8 o + 2 j + p % 2 of token 2 q + p / 4 + 8 (p / 2 % 2).
// The lane of a tensor-core fragment that holds tokens 2 q, 2 q + 1, 2 q + 8, 2 q + 9
// reads 16 bytes of V for each of its octets, and a byte of K or V holds one token only,
// so that tokens of a block are appended by different threads without a
// read-modify-write.
#pragma once

#include <stdint.h>

namespace pkv {
namespace {

__host__ __device__ constexpr int q4_record_bytes(int head_dim) { return 16 * head_dim + 128; }
__host__ __device__ constexpr int q4_v_offset(int head_dim) { return 8 * head_dim; }
__host__ __device__ constexpr int q4_scales_offset(int head_dim) { return 16 * head_dim; }
// Byte of word (o, q, j) of V that holds token t's codes of dimensions 8 o + 2 j (low
// nibble) and 8 o + 2 j + 1.
__host__ __device__ constexpr int q4_v_byte(int o, int j, int t) {
    return o * 64 + ((t & 7) >> 1) * 16 + j * 4 + 2 * (t & 1) + (t >> 3);
}

// A row's scale over its largest magnitude: 1/7 rounded to float32. (The quotient by 7, at
// up to twice the instructions, is at most two roundings away, and codes are decided
// against the stored scale either way.)
constexpr float kQ4Step = 0.142857149243354797f;

}  // namespace
}  // namespace pkv
