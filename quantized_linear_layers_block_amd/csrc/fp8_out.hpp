// Quantizing float32 results to E4M3 segments of 128 with one scale each (the recipe's 1x128
// activation rule, applied in the kernel that computes the values).
#pragma once
#include "common.hpp"

namespace ql {

// One segment's scale, from the bits of its largest magnitude.
//   float32 scales: s = amax / 448, codes E4M3(v / s)
//   power of two:   s = 2^e, e the smallest integer with amax <= 448 * 2^e (0 for a zero segment),
//                   clamped to [-127, 127], stored as the byte e + 127
// A code is E4M3((v * up) * r): r is the rounded reciprocal of s (exact for powers of two), so the
// quotient is within 2^-23 of v / s before its one rounding to 4 bits; up keeps r finite where s is
// below float32's normal range.  A segment that holds an Inf or NaN gets the scale NaN (0xFF).
struct Fp8Seg {
  float up, r;
  uint32_t stored;
};
template <bool POW2>
__device__ __forceinline__ Fp8Seg fp8_seg_scale(uint32_t amax_bits) {
  Fp8Seg o;
  if (POW2) {
    // the carry out of the low 21 mantissa bits: 448 = 1.75 * 2^8
    const int e127 = (int)((amax_bits + 0x1FFFFFu) >> 23) - 8;
    uint32_t b = amax_bits == 0 ? 127u : (uint32_t)(e127 < 0 ? 0 : e127);
    o.up = 1.0f;
    o.r = b == 254 ? 0x1p-127f : __uint_as_float((254u - b) << 23);  // 2^(127 - b); b <= 247 for finite values
    o.stored = amax_bits >= 0x7F800000u ? 0xFFu : b;
  } else {
    const float s = __uint_as_float(amax_bits) / 448.0f;
    o.up = s < 0x1p-100f ? 0x1p100f : 1.0f;
    o.r = s > 0.0f ? 1.0f / (s * o.up) : 0.0f;
    o.stored = amax_bits >= 0x7F800000u ? 0x7FC00000u : __float_as_uint(s);
  }
  return o;
}

__device__ __forceinline__ float fp8_scaled(float v, const Fp8Seg& s) {
  return __builtin_amdgcn_fmed3f((v * s.up) * s.r, -448.0f, 448.0f);
}
__device__ __forceinline__ uint32_t fp8_encode4(const float* v, const Fp8Seg& s) {
  return e4m3_pack4(fp8_scaled(v[0], s), fp8_scaled(v[1], s), fp8_scaled(v[2], s), fp8_scaled(v[3], s));
}
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

}  // namespace ql
