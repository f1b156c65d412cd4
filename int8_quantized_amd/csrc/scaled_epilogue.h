// What the projections with scales per token and channel do with their integer
// sums: the scales, the bias and the activation, in 32 bits, rounded once.
#pragma once

#include <type_traits>

#include "decode.h"

namespace q8ta {

// 1 / (1 + e^-x).  e^-x = 2^y with y = -x log2(e) in two parts: rounded to one, y
// is off by 2^-24 of itself, and 2^y by up to 40 times that.
__device__ __forceinline__ float logistic(float x) {
  x = __builtin_fminf(x, 128.0f);   // (infinities have no parts; a NaN comes back with v)
  const float y = -x * 1.44269504f;
  const float rest = __builtin_fmaf(-x, 1.44269504f, -y) - x * 1.92596299e-8f;
  const float e = __builtin_amdgcn_exp2f(y);
  return __builtin_amdgcn_rcpf(1.0f + __builtin_fmaf(e, rest * 0.693147181f, e));
}

template <int ACT>
__device__ __forceinline__ float activate(float v) {
  if constexpr (ACT == kActRelu) return v < 0.0f ? 0.0f : v;
  // (e^-v passes the range of fp32: below -88 the value is under 2^-118 and taken as -0, here and in the tanh
  // form; both sides of the fraction times 2^-64 there, for fp32's range: five more instructions, 2048 x 4096 x
  // 11008 183 -> 189 us)
  if constexpr (ACT == kActSilu) return v < -88.0f ? -0.0f : v * logistic(v);
  // (the complement keeps the small outputs' bits)
  if constexpr (ACT == kActGelu) return 0.5f * v * erfcf(v * -0.707106781f);
  if constexpr (ACT == kActGeluTanh) {
    // (1 + tanh(z / 2)) / 2 = logistic(z)
    const float z = 1.59576912f * __builtin_fmaf(0.044715f * v * v, v, v);
    return z < -88.0f ? -0.0f : v * logistic(z);
  }
  return v;
}

// f(integral_constant) of the activation: one branch for all of a thread's outputs
// (with a branch at each of them the code does not fit the instruction cache).
template <int MATS, class F>
__device__ __forceinline__ void with_activation(int act, F&& f) {
  if constexpr (MATS == 1) {
    if (act == kActRelu) f(std::integral_constant<int, kActRelu>{});
    else f(std::integral_constant<int, kActNone>{});
  } else {
    if (act == kActSilu) f(std::integral_constant<int, kActSilu>{});
    else if (act == kActGelu) f(std::integral_constant<int, kActGelu>{});
    else if (act == kActGeluTanh) f(std::integral_constant<int, kActGeluTanh>{});
    else f(std::integral_constant<int, kActRelu>{});
  }
}

// (acc * token's scale) * channel's scale + bias, one rounding each.
__device__ __forceinline__ float scaled(int32_t acc, float xs, float ws, float bias) {
  float v = (float)acc * xs;
  v = v * ws;
  return v + bias;
}

}  // namespace q8ta
