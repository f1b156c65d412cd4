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
  return Heat{(double)top, 1.4426950408889634 / (double)temperature};
}
// exp((x - top) / T): 1 for the largest itself (an infinite one too), 0 for -inf.
__device__ __forceinline__ double weight(const Heat& h, float x) {
  const double y = ((double)x - h.top) * h.scale;
  const double w = exp2_of(y);
  return (double)x == h.top ? 1.0 : (x == -INFINITY ? 0.0 : w);
}

}  // namespace q8ta
