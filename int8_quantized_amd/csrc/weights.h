// 64-bit weights exp((x - top) / T) of logits, for what draws tokens.
#pragma once

#include "decode.h"

namespace q8ta {

// 2^y for y <= 0: 2^n times a polynomial in the rest f of [-1/2, 1/2], 1 + f * q(f)
// with q of degree 8 through (2^f - 1) / f at nine Chebyshev points (off by
// 4e-14 at most; exactly 1 for y = 0).
__device__ __forceinline__ double exp2_poly(double f) {
  double q = 0x1.b63880f16b7cap-24;
  q = __builtin_fma(q, f, 0x1.63d1363459636p-20);
  q = __builtin_fma(q, f, 0x1.ffcb95155d9ebp-17);
  q = __builtin_fma(q, f, 0x1.4308ac85ac57dp-13);
  q = __builtin_fma(q, f, 0x1.5d87fe86fe9e8p-10);
  q = __builtin_fma(q, f, 0x1.3b2ab7181b748p-7);
  q = __builtin_fma(q, f, 0x1.c6b08d7047e52p-5);
  q = __builtin_fma(q, f, 0x1.ebfbdff823cedp-3);
  q = __builtin_fma(q, f, 0x1.62e42fefa39efp-1);
  return q;
}
__device__ __forceinline__ double exp2_of(double y) {
  y = __builtin_fmax(y, -1100.0);
  const double n = __builtin_rint(y);
  const double f = y - n;
  const double q = exp2_poly(f);
  return __builtin_ldexp(__builtin_fma(q, f, 1.0), (int)n);
}

struct Heat {
  double top, scale;   // largest logit, log2(e) / temperature
};
__device__ __forceinline__ Heat make_heat(float top, float temperature) {
  // 1 / T to the last bit or two, from the estimate by Newton steps (which have none for infinity)
  const double t = temperature;
  double y = __builtin_amdgcn_rcp(t);
#pragma unroll
  for (int i = 0; i < 2; ++i) y = __builtin_fma(__builtin_fma(-t, y, 1.0), y, y);
  return Heat{(double)top, temperature < INFINITY ? 1.4426950408889634 * y : 0.0};
}
// exp((x - top) / T): 1 for the largest itself (an infinite one too), 0 for -inf.
__device__ __forceinline__ double weight(const Heat& h, float x) {
  const double y = ((double)x - h.top) * h.scale;
  const double w = exp2_of(y);
  return (double)x == h.top ? 1.0 : (x == -INFINITY ? 0.0 : w);
}

// The same in 32 bits, for a finite top and a scale of near_scale: y = log2 of the weight is off by
// 2^-23 of itself (the difference's rounding and the multiply-add's), so the weight by 0.7 * 2^-23 of
// itself for each power of two below 1, and by 2^-23 for the exponential; the same way for equal logits.
struct Near {
  float top, scale, rest;   // the scale in two parts of one sign, so that -inf stays
};
// Temperatures from 2^-99 to 2^100: both parts are normal numbers above 0, and a difference that
// passes fp32's range is a weight of 0 (2^-2^28).
__device__ __forceinline__ bool near_scale(const Heat& h) { return h.scale >= 0x1p-100 && h.scale <= 0x1p100; }
__device__ __forceinline__ Near make_near(const Heat& h) {
  float hi = (float)h.scale;
  if ((double)hi > h.scale) hi = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, hi) - 1);
  // (a rest of 0 would make a NaN of -inf)
  return Near{(float)h.top, hi, __builtin_fmaxf((float)(h.scale - (double)hi), 0x1p-126f)};
}
// log2 of it; the weight is 2 to that.
__device__ __forceinline__ float near_log2(const Near& h, float x) {
  const float d = x - h.top;
  return __builtin_fmaf(d, h.scale, d * h.rest);
}

}  // namespace q8ta
