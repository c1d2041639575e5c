// 8-bit floating point (OCP e4m3 and e5m2) shared by the quantisers.
#pragma once

#include "common.hpp"

namespace nms {

// The scale of a block from the bits of its largest finite magnitude: the exponent of the smallest
// power of two, at least 2^-126, that is >= amax / max, with max = 1.75 * 2^8 (e4m3) or
// 1.75 * 2^15 (e5m2).  It follows from the exponent of amax and whether its significand exceeds
// 1.75, so it is exact, and so is the division by it.
__device__ inline int block_exponent(uint32_t amax_bits, bool e5m2) {
  if (amax_bits == 0) return 0;
  const int e = (int)(amax_bits >> 23) - 127 - (e5m2 ? 15 : 8) + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return e < -126 ? -126 : e;
}
__device__ inline float power2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Bits of |x| for the block maximum: infinities and NaN do not count.
__device__ inline uint32_t finite_bits(float x) {
  const uint32_t u = __float_as_uint(x) & 0x7FFFFFFFu;
  return u < 0x7F800000u ? u : 0u;
}

// Four values times inv, rounded to nearest even, as four bytes.  An infinite value becomes NaN, as
// a NaN does (e4m3 has no infinity; an overflow in a gradient stays visible in both formats).
template <bool E5M2>
__device__ inline uint32_t pack4(const float (&x)[4], float inv) {
  float y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = fabsf(x[i]) < __builtin_inff() ? x[i] * inv : __builtin_nanf("");
  if constexpr (E5M2) {
    const int lo = __builtin_amdgcn_cvt_pk_bf8_f32(y[0], y[1], 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_bf8_f32(y[2], y[3], lo, true);
  } else {
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], lo, true);
  }
}

}  // namespace nms
