// The activations of the dense products and their derivatives, in fp32.
#pragma once

#include <type_traits>

#include "common.hpp"

namespace nms {

enum { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU_TANH = 2, ACT_SILU = 3 };

// 1 / (1 + exp(-x)): the exponential and the reciprocal are correct to one unit in the last place of
// fp32, and x enters the exponent rounded, so the result's relative error is below (|x| + 3) 2^-23 where it is
// a normal number, x > -87.3.  Below that the reciprocal (and from -88.7 on the exponential's infinity) gives 0, which is
// off by less than 2^-126: x sigmoid(x) then is -0, off by less than 88 2^-126 = 1.04e-36.  +-infinity give 1 and 0.
__device__ inline float sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(x * -1.44269504088896341f));
}

// 0.5 z (1 + tanh(u)) = z sigmoid(2 u), u = sqrt(2 / pi) (z + 0.044715 z^3)
constexpr float kGelu2 = 1.59576912160573071f, kGeluCube = 0.044715f;   // 2 sqrt(2 / pi)

template <int ACT>
__device__ inline float act_fwd(float z) {
  if constexpr (ACT == ACT_RELU) return z > 0.f ? z : 0.f;
  if constexpr (ACT == ACT_GELU_TANH) return z * sigmoid(kGelu2 * z * __builtin_fmaf(kGeluCube * z, z, 1.f));
  if constexpr (ACT == ACT_SILU) return z * sigmoid(z);
  return z;
}

// The derivatives of the smooth ones.  Beyond +-100 they are 0 or 1 in fp32 (the exponential there is 0 or
// infinite); z is held there, so that no intermediate is 0 times infinity; a NaN stays one.
template <int ACT>
__device__ inline float act_bwd(float z) {
  static_assert(ACT == ACT_GELU_TANH || ACT == ACT_SILU, "");
  const float c = fminf(fmaxf(z, -100.f), 100.f);
  float d;
  if constexpr (ACT == ACT_SILU) {
    const float s = sigmoid(c);
    d = s * __builtin_fmaf(c, 1.f - s, 1.f);
  } else {
    const float cc = c * c, s = sigmoid(kGelu2 * c * __builtin_fmaf(kGeluCube, cc, 1.f));
    d = __builtin_fmaf(c * s * (1.f - s), kGelu2 * __builtin_fmaf(3.f * kGeluCube, cc, 1.f), s);
  }
  return z != z ? z : d;
}

// v times the derivative; ReLU passes v or 0, so what is not finite in a masked place goes no further.
template <int ACT>
__device__ inline float act_gate(float v, float z) {
  if constexpr (ACT == ACT_NONE) return v;
  else if constexpr (ACT == ACT_RELU) return z > 0.f ? v : 0.f;
  else return v * act_bwd<ACT>(z);
}

// f with the activation as a constant
template <typename F>
__device__ inline void with_act(int act, F f) {
  switch (act) {
    case ACT_RELU: f(std::integral_constant<int, ACT_RELU>()); break;
    case ACT_GELU_TANH: f(std::integral_constant<int, ACT_GELU_TANH>()); break;
    case ACT_SILU: f(std::integral_constant<int, ACT_SILU>()); break;
    default: f(std::integral_constant<int, ACT_NONE>());
  }
}

}  // namespace nms
