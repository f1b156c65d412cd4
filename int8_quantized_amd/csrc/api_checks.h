// What the argument checks of the C entry points share.
#pragma once

#include <initializer_list>

#include "decode.h"

namespace q8ta {

constexpr int64_t kMaxElems = (int64_t)1 << 40;

inline q8ta_status hip_status(hipError_t e, const char* what) {
  if (e == hipSuccess) return Q8TA_OK;
  return report(Q8TA_ERR_HIP, "%s: HIP error %d (%s)", what, (int)e, hipGetErrorString(e));
}

inline bool dtype_ok(int d) { return d == Q8TA_F32 || d == Q8TA_F16 || d == Q8TA_BF16; }

// a * b * .. <= 2^40 for factors >= 1.
inline bool fits(std::initializer_list<int64_t> f) {
  int64_t left = kMaxElems;
  for (int64_t x : f) {
    if (x > left) return false;
    left /= x;
  }
  return true;
}

}  // namespace q8ta
