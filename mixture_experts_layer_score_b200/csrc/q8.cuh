// q8.cuh -- the 8-bit form of a matrix: e4m3 values with one power of two (an e8m0 byte s
// standing for 2^(s-127)) per block of 128 values, the smallest 2^k with
// max|block| <= 448 2^k and k >= -126 (448 is e4m3's largest value). Powers of two make
// the scaling itself exact, so the only rounding is the one to e4m3, and they are what
// the block-scaled tcgen05.mma takes. A block that holds an infinity or a NaN becomes NaN
// as a whole (byte 255, values 0x7F): a product that reads it gives NaN, not a finite row.
#pragma once

#include <stdint.h>

namespace dsmoe {

constexpr int kQ8Block = 128;
// Scale bytes of a row of C values: whole 32-bit words, so that a row of scales can be
// read a word (four blocks, 512 values) at a time. Bytes past the last block hold 1.0.
__host__ __device__ constexpr int q8_scale_cols(int C) { return 4 * ((C + 511) / 512); }
constexpr uint8_t kQ8PadScale = 127;

// The scale byte for the bit pattern of max|block| (fp32 patterns of non-negative values
// order like the values, NaN above infinity). Adding 0x1FFFFF carries into the exponent
// exactly where the mantissa is above 1.75 = 448 / 256.
__device__ __forceinline__ uint32_t q8_scale_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7F800000u) return 255u;
  const int s = static_cast<int>((amax_bits + 0x1FFFFFu) >> 23) - 8;
  return static_cast<uint32_t>(s < 1 ? 1 : s);
}
// 2^(127-s), what a value of the block is multiplied by (s in [1, 247], so it is normal).
__device__ __forceinline__ float q8_inv_scale(uint32_t s) {
  return s == 255u ? 1.0f : __uint_as_float((254u - s) << 23);
}

// Two e4m3 values, a in the low byte; round to nearest even. |a|, |b| <= 448 here.
__device__ __forceinline__ uint32_t q8_pack2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ uint32_t q8_pack4(float a, float b, float c, float d) {
  return q8_pack2(a, b) | (q8_pack2(c, d) << 16);
}
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

}  // namespace dsmoe
