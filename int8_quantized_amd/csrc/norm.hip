// q8ta_norm_quantize and q8ta_quantize_per_token: what stands between two
// blocks, and the codes that the next projection takes, one scale a token.
//
//   b = x, or x / rms(x) * post_weight          rms(v) = sqrt(mean v^2 + eps)
//   h = residual_scale * residual + gate * b    rounded to the type: the new residual
//   z = h, or h / rms(h) * weight
//   scale = max |z| / 127,  code = rint(z * 127 / max |z|)
//
// Everything between the loads and the stores is 64-bit: a 16-bit value times
// 127 over another is a tie of the codes often enough that 32 bits would turn
// it the wrong way, and the sum h is what later blocks add to.  (64-bit
// multiply-adds run at the rate of 32-bit ones here.)  The division is a
// product with 127 / max, but next to a tie, where it is carried out.
//
// A workgroup takes one row and holds it in registers (8 * C elements a
// thread): x, residual and gate are read once, the sum and the codes written
// once, and the two or three sums over the row meet in LDS.  Rows too long for
// that are read again for each sum (k_norm_long).
//
// Measured: 8191 x 5120 bf16 with both norms, residual and gate 75 to 88 us from card to card, 294 MB at
// 3.3 to 3.9 TB/s (a copy of the same bytes 52); 4096 x 6144 40 us, 4.4; 4096 x 4096 30 us, 3.9;
// without the norm of x 65 (4.5), 34 (5.2) and 25 (4.7).  The vector instructions, 47 for an element, are
// busy over half of the time and the rows' barriers keep them and the loads from
// overlapping whole.  One row of 4096: 2.8 us, a chain of latencies.  The codes alone of bf16 rows: 1, 64 and
// 2048 of 11008 4.4, 5.7 and 26 us, of 16384 5.0, 6.6 and 36.  Workgroups that
// take row after row and load the next one early (their registers spill, 188 us), and
// 32-bit estimates of the codes, were no faster.
#include "decode.h"

namespace q8ta {
namespace {

typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

constexpr int kMaxThreads = 1024;

// Eight elements as they lie in memory.
template <class T>
struct Raw {
  v4u v[sizeof(T) / 2];
};
// From p on; `live` of them, zeros behind, where not VEC.
template <bool VEC, class T>
__device__ __forceinline__ Raw<T> load8(const T* p, int live) {
  Raw<T> r;
  if constexpr (VEC) {
#pragma unroll
    for (int j = 0; j < (int)sizeof(T) / 2; ++j) r.v[j] = reinterpret_cast<const v4u*>(p)[j];
  } else {
#pragma unroll
    for (int j = 0; j < (int)sizeof(T) / 2; ++j) r.v[j] = v4u{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i >= live) continue;
      if constexpr (sizeof(T) == 4) r.v[i / 4][i % 4] = __builtin_bit_cast(uint32_t, p[i]);
      else r.v[0][i / 2] |= (uint32_t)__builtin_bit_cast(uint16_t, p[i]) << (16 * (i % 2));
    }
  }
  return r;
}
template <class T>
__device__ __forceinline__ float element(const Raw<T>& r, int i) {
  if constexpr (sizeof(T) == 4) {
    const uint32_t w = r.v[i / 4][i % 4];
    return __builtin_bit_cast(float, w);
  } else {
    return to_float(T{(uint16_t)(r.v[0][i / 2] >> (16 * (i % 2)))});
  }
}
// (x is of the type already: no rounding)
template <bool VEC, class T>
__device__ __forceinline__ void store8(T* p, int live, const float (&x)[8]) {
  if constexpr (VEC) {
#pragma unroll
    for (int j = 0; j < (int)sizeof(T) / 2; ++j) {
      v4u v;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) v[i] = __builtin_bit_cast(uint32_t, x[4 * j + i]);
        else v[i] = (uint32_t)from_float<T>(x[2 * i]).bits | (uint32_t)from_float<T>(x[2 * i + 1]).bits << 16;
      }
      reinterpret_cast<v4u*>(p)[j] = v;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < live) p[i] = from_float<T>(x[i]);
  }
}

// (of magnitudes; a row that holds a NaN comes with an infinity in its place)
__device__ __forceinline__ double top_of(double a, double b) { return __builtin_fmax(a, b); }
__device__ __forceinline__ double plus_of(double a, double b) { return a + b; }

template <int CTRL>
__device__ __forceinline__ double row_move64(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)row_move<CTRL>((int32_t)(uint32_t)b);
  const uint32_t hi = (uint32_t)row_move<CTRL>((int32_t)(uint32_t)(b >> 32));
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double lane64(double v, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int32_t)(uint32_t)b, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int32_t)(uint32_t)(b >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// v of all lanes of a wave by `f`, the same in each.
template <class F>
__device__ __forceinline__ double over_wave(double v, F&& f) {
  v = f(v, row_move64<kDppMirror16>(v));
  v = f(v, row_move64<kDppMirror8>(v));
  v = f(v, row_move64<kDppRev4>(v));
  v = f(v, row_move64<kDppSwap1>(v));
  return f(f(lane64(v, 0), lane64(v, 16)), f(lane64(v, 32), lane64(v, 48)));
}
// The waves' values in `sh` by `f`, where 0 is none (every lane of the wave active).
template <class F>
__device__ __forceinline__ double over_waves(const double* sh, F&& f) {
  const int lane = threadIdx.x & 15;
  double v = lane < (int)blockDim.x / 64 ? sh[lane] : 0.0;
  v = f(v, row_move64<kDppMirror16>(v));
  v = f(v, row_move64<kDppMirror8>(v));
  v = f(v, row_move64<kDppRev4>(v));
  return f(v, row_move64<kDppSwap1>(v));
}
// v of all threads of the workgroup by `f`, in a fixed order.  `sh`: kMaxThreads / 64 doubles that
// no other call uses.
template <class F>
__device__ __forceinline__ double over_row(double v, double* sh, F&& f) {
  v = over_wave(v, f);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x / 64] = v;
  __syncthreads();
  return over_waves(sh, f);
}

// rint(p * 127 / top).  fast_code: in the high byte, of q = p * 127 / top with 24 bits behind the
// point and a half added, as the sum's low word; the lower bytes are the distance from the tie
// below, in 2^-24.  With inv = 127 / top the product's rounding differs from the
// quotient's by 2^-52 of it, which matters next to a tie: kNear says how near.
constexpr double kMagic = 6755399441055744.0;   // 1.5 * 2^52: the sum's low word is the nearest whole number
constexpr uint32_t kNear = 4;
__device__ __forceinline__ uint32_t fast_code(double p, double inv) {
  constexpr double kHalf = 0x1.8p28 + 0.5 + kNear / 2 * 0x1p-24;   // 1.5 * 2^(52 - 24)
  return (uint32_t)__builtin_bit_cast(uint64_t, __builtin_fma(p, inv, kHalf));
}
__device__ __forceinline__ uint32_t exact_code(double p, double top) {
  return (uint32_t)__builtin_bit_cast(uint64_t, p * 127.0 / top + kMagic);
}
// The high bytes of four words.
__device__ __forceinline__ uint32_t pack_high(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x0c0c0703), hi = __builtin_amdgcn_perm(d, c, 0x07030c0c);
  return lo | hi;
}

// 1 / x and 1 / sqrt(x) to the last bit or two, from the estimates by Newton steps.
__device__ __forceinline__ double reciprocal(double x) {
  double y = __builtin_amdgcn_rcp(x);
#pragma unroll
  for (int i = 0; i < 2; ++i) y = __builtin_fma(__builtin_fma(-x, y, 1.0), y, y);
  return y;
}
__device__ __forceinline__ double reciprocal_root(double x) {
  double y = __builtin_amdgcn_rsq(x);
#pragma unroll
  for (int i = 0; i < 2; ++i) y = __builtin_fma(__builtin_fma(-x * y, y, 1.0), 0.5 * y, y);
  return x == (double)__builtin_inff() ? 0.0 : y;   // (the steps would make a NaN of it)
}

// The row's scale; 127 / max goes to inv.  A row with a value that is not finite
// has the scale NaN and codes 0 (inv 0), as has one of zeros with the scale 0.
__device__ __forceinline__ float scale_of(double top) {
  if (!(top < (double)__builtin_inff())) return __builtin_nanf("");
  return (float)(top / 127.0);
}
__device__ __forceinline__ double inv_of(double top) {
  return top > 0.0 && top < (double)__builtin_inff() ? 127.0 * reciprocal(top) : 0.0;
}

// h = residual_scale * residual + gate * b as it is stored.
template <class T>
__device__ __forceinline__ float sum_of(double b, bool has_gate, float gate, bool has_res, float res,
                                        double res_scale) {
  if (has_gate) b = b * (double)gate;
  if (has_res) b = __builtin_fma((double)res, res_scale, b);
  return to_float(from_float<T>((float)b));
}

// C: groups of 8 elements a thread.
template <class T, int C, bool VEC>
__global__ __launch_bounds__(C > 2 ? 256 : kMaxThreads, C == 1 ? 8 : (C == 4 ? 3 : 4)) void k_norm(NormArgs a, double inv_n) {
  __shared__ double sh[3][kMaxThreads / 64];
  const int tid = threadIdx.x, nt = blockDim.x;
  const int64_t t = blockIdx.x;
  const int n = (int)a.n;
  Raw<T> xr[C], rr[C], gr[C];
  Raw<float> pw[C], w[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int e = 8 * (tid + c * nt);
    const int live = n - e, at = live > 0 ? e : 0;   // (threads past the row read its first elements)
    const int some = live > 0 ? live : 0;
    xr[c] = load8<VEC>((const T*)a.x + t * a.x_stride + at, some);
    if (a.residual) rr[c] = load8<VEC>((const T*)a.residual + t * a.residual_stride + at, some);
    if (a.gate) gr[c] = load8<VEC>((const T*)a.gate + t * a.gate_stride + at, some);
    if (a.post_weight) pw[c] = load8<VEC>(a.post_weight + at, some);
    if (a.weight) w[c] = load8<VEC>(a.weight + at, some);
  }
  double post = 1.0;
  if (a.post_weight) {
    double s = 0.0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (8 * (tid + c * nt) >= n) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const double v = element(xr[c], i);
        s = __builtin_fma(v, v, s);
      }
    }
    post = reciprocal_root(__builtin_fma(over_row(s, sh[0], plus_of), inv_n, a.eps));
  }
  float h[C][8];
  double s = 0.0;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    double y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = element(xr[c], i);
    if (a.post_weight) {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = y[i] * post * (double)element(pw[c], i);
    }
    if (a.gate) {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = y[i] * (double)element(gr[c], i);
    }
    if (a.residual) {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = __builtin_fma((double)element(rr[c], i), a.residual_scale, y[i]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) h[c][i] = to_float(from_float<T>((float)y[i]));
    const int e = 8 * (tid + c * nt);
    if (e >= n) continue;
    if (a.weight) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s = __builtin_fma((double)h[c][i], (double)h[c][i], s);
    }
    if (a.sum) store8<VEC>((T*)a.sum + t * a.n + e, n - e, h[c]);
  }
  // the codes need p = h * weight and the largest of them alone: rms(h) is a factor of both
  double p[C][8], top = 0.0, odd = 0.0;
#pragma unroll
  for (int c = 0; c < C; ++c) {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[c][i] = h[c][i];
    if (a.weight) {
#pragma unroll
      for (int i = 0; i < 8; ++i) p[c][i] = p[c][i] * (double)element(w[c], i);
    }
    if (8 * (tid + c * nt) >= n) continue;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      top = __builtin_fmax(top, __builtin_fabs(p[c][i]));
      odd = __builtin_fma(p[c][i], 0.0, odd);   // (a maximum would drop a NaN)
    }
  }
  top = over_wave(odd == 0.0 ? top : (double)__builtin_inff(), top_of);
  s = over_wave(s, plus_of);
  if ((tid & 63) == 0) {
    sh[1][tid / 64] = s;
    sh[2][tid / 64] = top;
  }
  __syncthreads();
  top = over_waves(sh[2], top_of);
  const double inv = inv_of(top);
  if (tid < 64) {   // (a whole wave: its lanes hold the parts)
    const double rstd = a.weight ? reciprocal_root(__builtin_fma(over_waves(sh[1], plus_of), inv_n, a.eps)) : 1.0;
    if (tid == 0) a.scales[t] = scale_of(top * rstd);
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int e = 8 * (tid + c * nt);
    if (e >= n) continue;
    uint32_t q[8], least = kNear;
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = fast_code(p[c][i], inv);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t r = q[i] & 0xffffff;
      least = r < least ? r : least;
    }
    if (least < kNear) {
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] = exact_code(p[c][i], top) << 24;
    }
    if (!(inv > 0.0)) {
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] = 0;
    }
    int8_t* dst = a.codes + t * a.n + e;
    if constexpr (VEC) {
      *reinterpret_cast<v2u*>(dst) = v2u{pack_high(q[0], q[1], q[2], q[3]), pack_high(q[4], q[5], q[6], q[7])};
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n - e) dst[i] = (int8_t)(q[i] >> 24);
    }
  }
}

// Rows of any length: the row is read again for each sum.  Every thread writes
// only what it alone has read, last (the sum may stand in x's or the residual's place).
// One element a lane and load, a workgroup a row whatever their number: the codes of 1, 64 and 2048
// bf16 rows of 28672 take 21, 22 and 157 us (1.1 TB/s), of 53248 36, 38 and 284; with both norms and a
// residual 20480 36, 38 and 328.  What bounds it: the loads' latency, a row's after the other's.
template <class T>
__global__ __launch_bounds__(kMaxThreads) void k_norm_long(NormArgs a, double inv_n) {
  __shared__ double sh[3][kMaxThreads / 64];
  const int tid = threadIdx.x;
  const int64_t t = blockIdx.x;
  const T* x = (const T*)a.x + t * a.x_stride;
  const T* res = (const T*)a.residual + t * a.residual_stride;
  const T* gate = (const T*)a.gate + t * a.gate_stride;
  double post = 1.0, rstd = 1.0;
  auto h_of = [&](int64_t e) {
    double b = to_float(x[e]);
    if (a.post_weight) b = b * post * (double)a.post_weight[e];
    return sum_of<T>(b, a.gate != nullptr, a.gate ? to_float(gate[e]) : 0.0f, a.residual != nullptr,
                     a.residual ? to_float(res[e]) : 0.0f, a.residual_scale);
  };
  auto p_of = [&](int64_t e, float h) { return a.weight ? (double)h * (double)a.weight[e] : (double)h; };
  if (a.post_weight) {
    double s = 0.0;
    for (int64_t e = tid; e < a.n; e += kMaxThreads) {
      const double v = to_float(x[e]);
      s = __builtin_fma(v, v, s);
    }
    post = reciprocal_root(__builtin_fma(over_row(s, sh[0], plus_of), inv_n, a.eps));
  }
  if (a.weight) {
    double s = 0.0;
    for (int64_t e = tid; e < a.n; e += kMaxThreads) {
      const double v = h_of(e);
      s = __builtin_fma(v, v, s);
    }
    rstd = reciprocal_root(__builtin_fma(over_row(s, sh[1], plus_of), inv_n, a.eps));
  }
  double top = 0.0, odd = 0.0;
  for (int64_t e = tid; e < a.n; e += kMaxThreads) {
    const double p = p_of(e, h_of(e));
    top = top_of(__builtin_fabs(p), top);
    odd = __builtin_fma(p, 0.0, odd);
  }
  if (!(odd == 0.0)) top = (double)__builtin_inff();
  top = over_row(top, sh[2], top_of);
  const double inv = inv_of(top);
  if (tid == 0) a.scales[t] = scale_of(top * rstd);
  for (int64_t e = tid; e < a.n; e += kMaxThreads) {
    const float h = h_of(e);
    const uint32_t q = inv > 0.0 ? exact_code(p_of(e, h), top) : 0;
    if (a.sum) ((T*)a.sum)[t * a.n + e] = from_float<T>(h);
    a.codes[t * a.n + e] = (int8_t)q;
  }
}

template <class T, int C>
void launch_regs(const NormArgs& a, bool vec, int threads, hipStream_t s) {
  const dim3 g((unsigned)a.tokens), b((unsigned)threads);
  if (vec) hipLaunchKernelGGL((k_norm<T, C, true>), g, b, 0, s, a, 1.0 / (double)a.n);
  else hipLaunchKernelGGL((k_norm<T, C, false>), g, b, 0, s, a, 1.0 / (double)a.n);
}

template <class T>
hipError_t launch_type(const NormArgs& a, hipStream_t s) {
  const int64_t strides = a.x_stride | (a.residual ? a.residual_stride : 0) | (a.gate ? a.gate_stride : 0);
  const uintptr_t ptrs = (uintptr_t)a.x | (uintptr_t)a.residual | (uintptr_t)a.gate | (uintptr_t)a.sum |
                         (uintptr_t)a.post_weight | (uintptr_t)a.weight;
  const bool vec = a.n % 8 == 0 && strides % 8 == 0 && ptrs % 16 == 0 && (uintptr_t)a.codes % 8 == 0;
  const int64_t groups = (a.n + 7) / 8;
  auto threads = [&](int c) { return (int)((groups + 64 * c - 1) / (64 * c)) * 64; };
  // 8 elements a thread where a row is a chain of latencies; where there are many, 16 (8 took 6 % more),
  // and 24 or 32 of 16 bits where four waves hold a row then, one a SIMD (8191 x 5120: 89 us with 16,
  // 82 with 24; 4096 x 6144 44 and 36; 4096 x 7168 48, with 32 42; 8192 x 8192 117 with 16 as with 32)
  if (groups <= 1024 && a.tokens < 512) {
    launch_regs<T, 1>(a, vec, threads(1), s);
    return hipGetLastError();
  }
  if constexpr (sizeof(T) == 2) {
    if (groups > 512 && groups < 1024) {
      if (groups <= 768) launch_regs<T, 3>(a, vec, threads(3), s);
      else launch_regs<T, 4>(a, vec, threads(4), s);
      return hipGetLastError();
    }
  }
  if (groups <= 2048) launch_regs<T, 2>(a, vec, threads(2), s);
  else hipLaunchKernelGGL((k_norm_long<T>), dim3((unsigned)a.tokens), dim3(kMaxThreads), 0, s, a,
                          1.0 / (double)a.n);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_quantize(const NormArgs& a, hipStream_t s) {
  // a launch has fewer than 2^32 threads: one for each 2^21 tokens
  const int64_t es = a.dtype == Q8TA_F32 ? 4 : 2, most = (int64_t)1 << 21;
  for (int64_t t0 = 0; t0 < a.tokens; t0 += most) {
    NormArgs p = a;
    p.tokens = a.tokens - t0 < most ? a.tokens - t0 : most;
    p.x = (const char*)a.x + t0 * a.x_stride * es;
    if (a.residual) p.residual = (const char*)a.residual + t0 * a.residual_stride * es;
    if (a.gate) p.gate = (const char*)a.gate + t0 * a.gate_stride * es;
    if (a.sum) p.sum = (char*)a.sum + t0 * a.n * es;
    p.codes = a.codes + t0 * a.n;
    p.scales = a.scales + t0;
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
