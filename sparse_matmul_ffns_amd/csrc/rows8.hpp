// Eight consecutive elements of a row, for kernels that read and write whole rows.
//
// A vector of eight is loaded and stored in 16-byte accesses (fp32: two) whatever its address: global
// memory takes them at any multiple of the element size, so rows of an odd width need no path of their own.
// Only the vector that a row ends in is taken element by element (TAIL: the row's width is not a multiple of eight).
#pragma once

#include "common.hpp"

namespace nms {

typedef __bf16 bf16v8 __attribute__((ext_vector_type(8)));
typedef float f32v8 __attribute__((ext_vector_type(8)));

// As they lie in memory.
template <typename T>
struct Row8 {
  static constexpr int NW = sizeof(T) * 2;
  uint32_t w[NW];
  template <bool TAIL>
  __device__ inline void load(const T* p, int64_t c, int64_t D) {
    if (!TAIL || c + 8 <= D) {
      __builtin_memcpy(w, p + c, sizeof(w));
    } else {
#pragma unroll
      for (int i = 0; i < NW; ++i) w[i] = 0;
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (c + q < D) w[q * NW / 8] |= (uint32_t)p[c + q] << (sizeof(T) == 2 ? 16 * (q & 1) : 0);
    }
  }
  template <bool TAIL>
  __device__ inline void store(T* p, int64_t c, int64_t D) const {
    if (!TAIL || c + 8 <= D) {
      __builtin_memcpy(p + c, w, sizeof(w));
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (c + q < D) p[c + q] = (T)(w[q * NW / 8] >> (sizeof(T) == 2 ? 16 * (q & 1) : 0));
    }
  }
  __device__ inline void get(float (&v)[8]) const {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      if constexpr (sizeof(T) == 2) v[q] = __uint_as_float(q & 1 ? w[q / 2] & 0xFFFF0000u : w[q / 2] << 16);
      else v[q] = __uint_as_float(w[q]);
    }
  }
  // bf16 rounded to nearest even
  __device__ inline void set(const float (&v)[8]) {
    if constexpr (sizeof(T) == 2) {
      f32v8 f;
#pragma unroll
      for (int q = 0; q < 8; ++q) f[q] = v[q];
      const bf16v8 h = __builtin_convertvector(f, bf16v8);
      __builtin_memcpy(w, &h, sizeof(w));
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) w[q] = __float_as_uint(v[q]);
    }
  }
};

template <typename T, bool TAIL = true>
__device__ inline void load8f(const T* p, int64_t c, int64_t D, float (&v)[8]) {
  Row8<T> r;
  r.template load<TAIL>(p, c, D);
  r.get(v);
}
template <typename T, bool TAIL = true>
__device__ inline void store8f(T* p, int64_t c, int64_t D, const float (&v)[8]) {
  Row8<T> r;
  r.set(v);
  r.template store<TAIL>(p, c, D);
}

}  // namespace nms
