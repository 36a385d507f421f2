// Shared by the kernels of the 4-bit cache: its layout and the widening of codes.
//
//   codes  uint8 [num_blocks, H_kv, block_size, 64]: the 128 codes of one
//          token's row of one KV head, dim 2j in the low nibble of byte j, dim
//          2j + 1 in the high one
//   params bf16 [num_blocks, H_kv, block_size, 128 / group, 2]: (scale, offset)
//          of each group of dims
//
// Code n stands for bf16(scale * (16 + n) + offset). The 16 is there because a
// nibble placed in mantissa bits 3..6 of a bf16 with exponent 2^4 reads as
// 16 + n: one shift and one three-input logic operation widen two codes, and
// one packed fma per two codes applies the group's parameters.
#pragma once

#include "ptx.cuh"

namespace pkv {

constexpr int kQ4D = 128;                // head dim (the only one supported)
constexpr int kQ4RowBytes = kQ4D / 2;    // code bytes of one row

__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// (x & mask) | bits in one instruction. With both constants immediate the
// compiler makes two of it, which took a third of the widening's time.
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t bits) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(x), "r"(mask), "r"(bits));
  return d;
}

// The eight codes of a word as bf16 16 + n: p[i] holds nibble i (low half) and
// nibble i + 4 (high half).
__device__ __forceinline__ void q4_pairs(uint32_t w, uint32_t (&p)[4]) {
  constexpr uint32_t kMask = 0x00780078u, kSixteen = 0x41804180u;
  p[0] = and_or(w << 3, kMask, kSixteen);
  p[1] = and_or(w >> 1, kMask, kSixteen);
  p[2] = and_or(w >> 5, kMask, kSixteen);
  p[3] = and_or(w >> 9, kMask, kSixteen);
}

// A params word (scale in the low half, offset in the high one) with its scale,
// or its offset, in both halves; and the same of two words' scales or offsets.
__device__ __forceinline__ uint32_t q4_dup_scale(uint32_t pw) { return __byte_perm(pw, pw, 0x1010); }
__device__ __forceinline__ uint32_t q4_dup_offset(uint32_t pw) { return __byte_perm(pw, pw, 0x3232); }
__device__ __forceinline__ uint32_t q4_low_halves(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x5410); }
__device__ __forceinline__ uint32_t q4_high_halves(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7632); }

// The eight bf16 values of a code word, in dim order.
__device__ __forceinline__ uint4 q4_widen(uint32_t w, uint32_t pw) {
  uint32_t p[4];
  q4_pairs(w, p);
  const uint32_t s = q4_dup_scale(pw), b = q4_dup_offset(pw);
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = fma_bf16x2(p[i], s, b);
  return make_uint4(q4_low_halves(p[0], p[1]), q4_low_halves(p[2], p[3]),
                    q4_high_halves(p[0], p[1]), q4_high_halves(p[2], p[3]));
}

}  // namespace pkv
