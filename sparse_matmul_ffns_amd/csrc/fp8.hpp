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

// Eight consecutive elements as they lie in memory, and what the quantisers do with them.  The
// conversion instructions divide by a power-of-two scale and round to nearest even in one step, from
// bf16 pairs or from fp32 pairs; NaN becomes NaN.  An infinity is turned into NaN first (clean), in
// blocks that hold one, and neither counts for the block's maximum.
typedef unsigned short us2 __attribute__((ext_vector_type(2)));
typedef short s2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

template <typename T> struct Raw8;

template <> struct Raw8<uint16_t> {
  uint32_t w[4];
  typedef us2 Max;             // of |x|, for the columns 2 i (low) and 2 i + 1
  static constexpr int NMAX = 4;
  __device__ void zero() { w[0] = w[1] = w[2] = w[3] = 0; }
  __device__ void gate(const Raw8& g) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = __uint_as_float(g.w[i] << 16) > 0.f ? 0xFFFFu : 0u;
      const uint32_t hi = __uint_as_float(g.w[i] & 0xFFFF0000u) > 0.f ? 0xFFFF0000u : 0u;
      w[i] &= lo | hi;
    }
  }
  __device__ Max mag(int i) const { return __builtin_bit_cast(us2, w[i] & 0x7FFF7FFFu); }
  // largest |x| of the eight, as fp32 bits
  __device__ uint32_t row_max() const {
    const us2 m = __builtin_elementwise_max(__builtin_elementwise_max(mag(0), mag(1)),
                                            __builtin_elementwise_max(mag(2), mag(3)));
    return (uint32_t)(m[0] > m[1] ? m[0] : m[1]) << 16;
  }
  __device__ static uint32_t column(const Max (&m)[NMAX], int q) { return (uint32_t)m[q >> 1][q & 1] << 16; }
  __device__ void clean() {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = (w[i] & 0x7FFFu) >= 0x7F80u ? 0x7FC0u : w[i] & 0xFFFFu;
      const uint32_t hi = (w[i] & 0x7FFF0000u) >= 0x7F800000u ? 0x7FC00000u : w[i] & 0xFFFF0000u;
      w[i] = lo | hi;
    }
  }
  // of a cleaned vector: |x| with NaN as 0
  __device__ Max mag_finite(int i) const {
    us2 m = mag(i);
    m[0] = m[0] >= 0x7F80 ? 0 : m[0];
    m[1] = m[1] >= 0x7F80 ? 0 : m[1];
    return m;
  }
};

template <> struct Raw8<uint32_t> {
  uint32_t w[8];
  typedef uint32_t Max;
  static constexpr int NMAX = 8;
  __device__ void zero() {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 0;
  }
  __device__ void gate(const Raw8& g) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __uint_as_float(g.w[i]) > 0.f ? w[i] : 0u;
  }
  __device__ Max mag(int i) const { return w[i] & 0x7FFFFFFFu; }
  __device__ uint32_t row_max() const {
    uint32_t m = mag(0);
#pragma unroll
    for (int i = 1; i < 8; ++i) m = umax2(m, mag(i));
    return m;
  }
  __device__ static uint32_t column(const Max (&m)[NMAX], int q) { return m[q]; }
  __device__ void clean() {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = mag(i) >= 0x7F800000u ? 0x7FC00000u : w[i];
  }
  __device__ Max mag_finite(int i) const { return mag(i) >= 0x7F800000u ? 0u : mag(i); }
};

__device__ inline us2 vmax(us2 a, us2 b) { return __builtin_elementwise_max(a, b); }
__device__ inline uint32_t vmax(uint32_t a, uint32_t b) { return umax2(a, b); }

// Four bytes of a / scale .. d / scale.
template <bool E5M2>
__device__ inline uint32_t cvt4(bf16x2 ab, bf16x2 cd, float scale) {
  s2 r = {0, 0};
  if constexpr (E5M2) {
    r = __builtin_amdgcn_cvt_scalef32_pk_bf8_bf16(r, ab, scale, false);
    r = __builtin_amdgcn_cvt_scalef32_pk_bf8_bf16(r, cd, scale, true);
  } else {
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, ab, scale, false);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, cd, scale, true);
  }
  return __builtin_bit_cast(uint32_t, r);
}
template <bool E5M2>
__device__ inline uint32_t cvt4(float a, float b, float c, float d, float scale) {
  s2 r = {0, 0};
  if constexpr (E5M2) {
    r = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(r, a, b, scale, false);
    r = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(r, c, d, scale, true);
  } else {
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, a, b, scale, false);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, c, d, scale, true);
  }
  return __builtin_bit_cast(uint32_t, r);
}
// The eight elements of a row.
template <bool E5M2>
__device__ inline u32x2 pack_row(const Raw8<uint16_t>& x, float scale) {
  auto b = [&](int i) { return __builtin_bit_cast(bf16x2, x.w[i]); };
  return u32x2{cvt4<E5M2>(b(0), b(1), scale), cvt4<E5M2>(b(2), b(3), scale)};
}
template <bool E5M2>
__device__ inline u32x2 pack_row(const Raw8<uint32_t>& x, float scale) {
  auto f = [&](int i) { return __uint_as_float(x.w[i]); };
  return u32x2{cvt4<E5M2>(f(0), f(1), f(2), f(3), scale), cvt4<E5M2>(f(4), f(5), f(6), f(7), scale)};
}
// Column q of eight rows.
template <bool E5M2>
__device__ inline u32x2 pack_column(const Raw8<uint16_t> (&x)[8], int q, float scale) {
  auto b = [&](int i) {   // rows 2 i, 2 i + 1
    return __builtin_bit_cast(bf16x2, __builtin_amdgcn_perm(x[2 * i + 1].w[q >> 1], x[2 * i].w[q >> 1],
                                                            q & 1 ? 0x07060302u : 0x05040100u));
  };
  return u32x2{cvt4<E5M2>(b(0), b(1), scale), cvt4<E5M2>(b(2), b(3), scale)};
}
template <bool E5M2>
__device__ inline u32x2 pack_column(const Raw8<uint32_t> (&x)[8], int q, float scale) {
  auto f = [&](int i) { return __uint_as_float(x[i].w[q]); };
  return u32x2{cvt4<E5M2>(f(0), f(1), f(2), f(3), scale), cvt4<E5M2>(f(4), f(5), f(6), f(7), scale)};
}

}  // namespace nms
