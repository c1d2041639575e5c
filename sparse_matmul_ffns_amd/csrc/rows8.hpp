// Eight consecutive elements of a row, in fp32, for kernels that read and write whole rows.
//
// A vector of eight is loaded and stored in 16-byte (bf16) or twice 16-byte (fp32) accesses whatever its
// address: global memory takes 16-byte accesses at any multiple of the element size, so rows of an odd
// width need no path of their own; only the vector that the row ends in is taken element by element.
#pragma once

#include "common.hpp"

namespace nms {

template <typename T>
__device__ inline void load8f(const T* p, int64_t c, int64_t D, float (&v)[8]) {
  T b[8];
  if (c + 8 <= D) {
    __builtin_memcpy(b, p + c, sizeof(b));
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q) b[q] = c + q < D ? p[c + q] : (T)0;
  }
#pragma unroll
  for (int q = 0; q < 8; ++q) v[q] = Elem<T>::to_f32(b[q]);
}

typedef __bf16 bf16v8 __attribute__((ext_vector_type(8)));
typedef float f32v8 __attribute__((ext_vector_type(8)));

// v as T, bf16 rounded to nearest even
__device__ inline void convert8(const float (&v)[8], uint16_t (&b)[8]) {
  f32v8 f;
#pragma unroll
  for (int q = 0; q < 8; ++q) f[q] = v[q];
  const bf16v8 h = __builtin_convertvector(f, bf16v8);
  __builtin_memcpy(b, &h, sizeof(b));
}
__device__ inline void convert8(const float (&v)[8], uint32_t (&b)[8]) {
#pragma unroll
  for (int q = 0; q < 8; ++q) b[q] = __float_as_uint(v[q]);
}
template <typename T>
__device__ inline void store8f(T* p, int64_t c, int64_t D, const float (&v)[8]) {
  T b[8];
  convert8(v, b);
  if (c + 8 <= D) {
    __builtin_memcpy(p + c, b, sizeof(b));
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (c + q < D) p[c + q] = b[q];
  }
}

// Sum over the 64 lanes, the same in each of them and in the same order in every wave.
__device__ inline float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d >= 1; d /= 2) v += __shfl_xor(v, d);
  return v;
}

}  // namespace nms
