// q8ta_rope_append: rotary positions on the queries and keys of new tokens,
// the keys and values quantized into a paged int8 cache.
//
//   angle[t, p] = positions[t] * inv_freq[p]                   (64 bits)
//   (a, b) -> factor * (a cos - b sin, b cos + a sin)          pairs of the first rot elements
//   q_out = the turned queries, rounded to fp32 and from there to the type
//   row scale = amax / 127,  code = rint(x * 127 / amax)        turned keys, plain values
//
// Everything between the loads and the stores is 64-bit: an angle far past
// the trained length has no correct bits left in 32, and 16-bit inputs put
// x * 127 / amax exactly on a tie often enough that a rounded quotient would
// turn it the wrong way.  (The queries' step through fp32 can make a value next
// to a tie of a 16-bit type a tie: 2^-24 of the value more than half a step of
// the type.  Rounding once takes the kernel from 42 to 46 us for 8192 bf16 tokens x
// (32 + 16) heads x 128, so the step stays.)
//
// Layout: a row (one head of one token) belongs to LPR lanes, LPR the power
// of two at or above dim / 8; a lane holds 8 elements, which are four whole
// pairs in either layout (elements 4u.. and rot/2 + 4u.. of the half layout, 8u..
// of the interleaved one) or 8 elements past the rotated part, so turning
// needs no exchange and the row's amax is log2(LPR) lane moves.  A workgroup
// serves one token (or a share of its rows when there are few tokens): its
// rot / 2 cosines and sines are computed once, into LDS, and all its rows read
// them there.
//
// Bound by memory: 8191 tokens x (32 + 16) heads x 128, fp32, in 71 us, which is
// 4.95 TB/s of queries, keys, values, codes and scales (a 2 GiB copy runs at 4.9).
// One token (40 rows over 3 workgroups) takes 3.6 us, the time of its loads.
#include "decode.h"

namespace q8ta {
namespace {

constexpr int kNT = 256;
constexpr int kMaxPairs = 256;

typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

// Four consecutive elements.
__device__ __forceinline__ void load4(const float* p, float (&x)[4]) {
  const v4f v = *reinterpret_cast<const v4f*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = v[i];
}
template <class T>
__device__ __forceinline__ void load4(const T* p, float (&x)[4]) {
  const v2u v = *reinterpret_cast<const v2u*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = to_float(T{(uint16_t)(v[i / 2] >> (16 * (i % 2)))});
}
__device__ __forceinline__ void store4(float* p, const double* x) {
  v4f v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = (float)x[i];
  *reinterpret_cast<v4f*>(p) = v;
}
template <class T>
__device__ __forceinline__ void store4(T* p, const double* x) {
  v2u v;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    v[i] = (uint32_t)from_float<T>((float)x[2 * i]).bits |
           (uint32_t)from_float<T>((float)x[2 * i + 1]).bits << 16;
  *reinterpret_cast<v2u*>(p) = v;
}

// rint(x * 127 / top), 0 for a row of zeros.  Where the row holds an infinity
// or a NaN its scale does too; the codes are then any value of [-127, 127].
__device__ __forceinline__ int code_of(double x, double top) {
  const double q = __builtin_rint(x * 127.0 / (top > 0.0 ? top : 1.0));
  return (int)__builtin_fmin(__builtin_fmax(q, -127.0), 127.0);
}

// The larger magnitude; a NaN on either side stays (fmax would drop it).
__device__ __forceinline__ double top_of(double a, double b) { return a > b || a != a ? a : b; }

__device__ __forceinline__ double turn_first(double a, double b, double2 c) { return a * c.x - b * c.y; }
__device__ __forceinline__ double turn_second(double a, double b, double2 c) { return b * c.x + a * c.y; }

__device__ __forceinline__ double2 turn(const RopeArgs& a, int64_t t, int p) {
  const double angle = (double)a.positions[t] * a.inv_freq[p];
  double s, c;
  sincos(angle, &s, &c);
  return double2{c * a.factor, s * a.factor};
}

// Cache row of (slot, part, head): part 0 keys, 1 values; -1 for a slot
// outside the cache.
__device__ __forceinline__ int64_t cache_row(const RopeArgs& a, int64_t slot, int part, int head) {
  if (slot < 0 || slot >= a.pages * a.page) return -1;
  const int64_t pg = slot / a.page;
  return ((pg * 2 + part) * a.kv_heads + head) * a.page + (slot - pg * a.page);
}

template <class T, int LPR, bool INTER>
__global__ __launch_bounds__(kNT) void k_rope_append(RopeArgs a, int rows_per_block) {
  __shared__ double2 cs[kMaxPairs];
  const int tid = threadIdx.x;
  const int64_t t = blockIdx.x;
  const int pairs = a.rot / 2;
  for (int p = tid; p < pairs; p += kNT) cs[p] = turn(a, t, p);
  __syncthreads();
  const int64_t slot = a.slots[t];
  const int u = tid % LPR;
  const int rows = a.heads + 2 * a.kv_heads;
  const int r0 = blockIdx.y * rows_per_block;
  const int r1 = r0 + rows_per_block < rows ? r0 + rows_per_block : rows;
  const bool live = 8 * u < a.dim;
  // the two groups of four elements of this lane; pair p0 is its first
  const bool turned = 8 * u < a.rot;
  const int e0 = INTER || !turned ? 8 * u : 4 * u;
  const int e1 = INTER || !turned ? 8 * u + 4 : pairs + 4 * u;
  const int p0 = 4 * u;
  for (int r = r0 + tid / LPR; r < r1; r += kNT / LPR) {
    const bool is_q = r < a.heads, is_k = !is_q && r < a.heads + a.kv_heads;
    const int head = is_q ? r : (is_k ? r - a.heads : r - a.heads - a.kv_heads);
    const T* src = is_q ? (const T*)a.q + t * a.q_ts + head * a.q_hs
                        : (is_k ? (const T*)a.k + t * a.k_ts + head * a.k_hs
                                : (const T*)a.v + t * a.v_ts + head * a.v_hs);
    float f0[4] = {}, f1[4] = {};
    if (live) {
      load4(src + e0, f0);
      load4(src + e1, f1);
    }
    double x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = f0[i];
      x[4 + i] = f1[i];
    }
    if (turned && (is_q || is_k)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int ia = INTER ? 2 * i : i, ib = INTER ? 2 * i + 1 : 4 + i;
        const double xa = x[ia], xb = x[ib];
        const double2 c = cs[p0 + i];
        x[ia] = turn_first(xa, xb, c);
        x[ib] = turn_second(xa, xb, c);
      }
    }
    if (is_q) {
      if (live) {
        T* dst = (T*)a.q_out + (t * a.heads + head) * (int64_t)a.dim;
        store4(dst + e0, x);
        store4(dst + e1, x + 4);
      }
      continue;
    }
    double top = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = top_of(__builtin_fabs(x[i]), top);
#pragma unroll
    for (int m = LPR / 2; m > 0; m /= 2) top = top_of(__shfl_xor(top, m, LPR), top);
    const int64_t row = cache_row(a, slot, is_k ? 0 : 1, head);
    if (row < 0 || !live) continue;
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      w[h] = pack4(code_of(x[4 * h], top), code_of(x[4 * h + 1], top), code_of(x[4 * h + 2], top),
                   code_of(x[4 * h + 3], top));
    int8_t* dst = a.cache + row * a.dim;
    *reinterpret_cast<uint32_t*>(dst + e0) = w[0];
    *reinterpret_cast<uint32_t*>(dst + e1) = w[1];
    if (u == 0) a.scales[row] = (float)(top / 127.0);
  }
}

// Any dim, rot, stride and alignment: one wave per row, its elements taken
// singly (twice: for the amax and for the codes).
template <class T>
__global__ __launch_bounds__(64) void k_rope_append_any(RopeArgs a) {
  const int lane = threadIdx.x;
  const int64_t t = blockIdx.x;
  const int r = blockIdx.y;
  const bool is_q = r < a.heads, is_k = !is_q && r < a.heads + a.kv_heads;
  const int head = is_q ? r : (is_k ? r - a.heads : r - a.heads - a.kv_heads);
  const T* src = is_q ? (const T*)a.q + t * a.q_ts + head * a.q_hs
                      : (is_k ? (const T*)a.k + t * a.k_ts + head * a.k_hs
                              : (const T*)a.v + t * a.v_ts + head * a.v_hs);
  const int pairs = a.rot / 2;
  // f(e, x) for every element e of this lane
  auto each = [&](auto&& f) {
    if (is_q || is_k) {
      for (int p = lane; p < pairs; p += 64) {
        const int ea = a.interleaved ? 2 * p : p, eb = a.interleaved ? 2 * p + 1 : pairs + p;
        const double xa = to_float(src[ea]), xb = to_float(src[eb]);
        const double2 c = turn(a, t, p);
        f(ea, turn_first(xa, xb, c));
        f(eb, turn_second(xa, xb, c));
      }
      for (int e = a.rot + lane; e < a.dim; e += 64) f(e, (double)to_float(src[e]));
    } else {
      for (int e = lane; e < a.dim; e += 64) f(e, (double)to_float(src[e]));
    }
  };
  if (is_q) {
    T* dst = (T*)a.q_out + (t * a.heads + head) * (int64_t)a.dim;
    each([&](int e, double x) { dst[e] = from_float<T>((float)x); });
    return;
  }
  double top = 0.0;
  each([&](int, double x) { top = top_of(__builtin_fabs(x), top); });
#pragma unroll
  for (int m = 32; m > 0; m /= 2) top = top_of(__shfl_xor(top, m, 64), top);
  const int64_t row = cache_row(a, a.slots[t], is_k ? 0 : 1, head);
  if (row < 0) return;
  int8_t* dst = a.cache + row * a.dim;
  each([&](int e, double x) { dst[e] = (int8_t)code_of(x, top); });
  if (lane == 0) a.scales[row] = (float)(top / 127.0);
}

template <class T, int LPR>
hipError_t launch_vec(const RopeArgs& a, hipStream_t s) {
  const int rows = a.heads + 2 * a.kv_heads;
  // few tokens: a workgroup takes one round of rows, so that a step of one
  // token spreads over several CUs; many: it takes the whole token and
  // computes the cosines once
  const int rpb = a.tokens < 512 ? kNT / LPR : rows;
  const dim3 g((unsigned)a.tokens, (unsigned)((rows + rpb - 1) / rpb));
  if (a.interleaved) hipLaunchKernelGGL((k_rope_append<T, LPR, true>), g, dim3(kNT), 0, s, a, rpb);
  else hipLaunchKernelGGL((k_rope_append<T, LPR, false>), g, dim3(kNT), 0, s, a, rpb);
  return hipGetLastError();
}

template <class T>
hipError_t launch_type(const RopeArgs& a, hipStream_t s) {
  const int64_t strides = a.q_ts | a.q_hs | a.k_ts | a.k_hs | a.v_ts | a.v_hs;
  const uintptr_t ptrs = (uintptr_t)a.q | (uintptr_t)a.k | (uintptr_t)a.v | (uintptr_t)a.q_out;
  const bool vec = a.dim % 8 == 0 && a.rot % 8 == 0 && a.dim <= 512 && strides % 4 == 0 &&
                   ptrs % (4 * sizeof(T)) == 0 && (uintptr_t)a.cache % 4 == 0;
  if (!vec) {
    const dim3 g((unsigned)a.tokens, (unsigned)(a.heads + 2 * a.kv_heads));
    hipLaunchKernelGGL((k_rope_append_any<T>), g, dim3(64), 0, s, a);
    return hipGetLastError();
  }
  if (a.dim <= 64) return launch_vec<T, 8>(a, s);
  if (a.dim <= 128) return launch_vec<T, 16>(a, s);
  if (a.dim <= 256) return launch_vec<T, 32>(a, s);
  return launch_vec<T, 64>(a, s);
}

}  // namespace

hipError_t launch_rope_append(const RopeArgs& a, hipStream_t s) {
  // a launch has fewer than 2^32 threads: one for each 2^22 tokens
  const int64_t es = a.dtype == Q8TA_F32 ? 4 : 2;
  for (int64_t t0 = 0; t0 < a.tokens; t0 += (int64_t)1 << 22) {
    RopeArgs p = a;
    p.tokens = a.tokens - t0 < (int64_t)1 << 22 ? a.tokens - t0 : (int64_t)1 << 22;
    p.q = (const char*)a.q + t0 * a.q_ts * es;
    p.k = (const char*)a.k + t0 * a.k_ts * es;
    p.v = (const char*)a.v + t0 * a.v_ts * es;
    p.q_out = (char*)a.q_out + t0 * a.heads * a.dim * es;
    p.positions = a.positions + t0;
    p.slots = a.slots + t0;
    hipError_t e;
    switch (a.dtype) {
      case Q8TA_F32: e = launch_type<float>(p, s); break;
      case Q8TA_F16: e = launch_type<Half>(p, s); break;
      default: e = launch_type<Bfloat>(p, s);
    }
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace q8ta
