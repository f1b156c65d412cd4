// q8ta_linear_lora: the int8 projection with the low-rank adapters of many
// requests at once.
//
//   y[m, n] = (acc * s_in) * wscale[n] + bias[n] + sum_r B[a, n, r] t[m, r]
//   t[m, r] = adapter_scale[a] * s_in * sum_k A[a, r, k] (x[m, k] - zp),  a = ids[m]
//
// Two launches: k_lora_down forms t (a few hundred kilobytes), and the product
// with the weight adds B t where it turns its integer sums into the output, so
// the output is written once and the adapters cost their own bytes.
//
// k_lora_down: a workgroup takes 16 rows, one of the distinct adapters among
// them and 16 of its ranks; its waves share K and meet in LDS.  x - zp is a
// whole number of [-255, 255] and exact in fp16 and in bf16, so with the
// adapter's own 16-bit values the products are exact and the sums 32-bit.
//
// k_lora_rows: 16 * MT rows by 16 * FN channels, for the row counts of decode
// steps, where the weight stream is what has to be paid: the four waves take
// every fourth 64-byte step of K, weight and activation fragments come
// straight from memory into the operands of v_mfma_i32_16x16x64_i8 (16
// bytes a lane, the next step's loads ahead of this step's products), and
// their integer sums meet in LDS.
#include <type_traits>

#include "decode.h"

namespace q8ta {
namespace {

typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------------ t = A (x - zp)
// Eight codes (two words) less the zero point, as 16-bit values.
template <class AT>
__device__ __forceinline__ v4u less_zp(uint32_t w0, uint32_t w1, int zp) {
  v4u r;
  w0 ^= 0x80808080u;   // code + 128
  w1 ^= 0x80808080u;
  if constexpr (std::is_same<AT, Half>::value) {
    // under the exponent byte 0x64: 1024 + 128 + code
    const uint32_t k = 0x64646464u;
    const _Float16 c = (_Float16)(float)(-1152 - zp);
    const v2h c2 = v2h{c, c};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // (the pair in a scalar of its own: a bit cast of a vector's element
      // reads element 0)
      const uint32_t pair = __builtin_amdgcn_perm(i < 2 ? w0 : w1, k, i % 2 ? 0x00070006u : 0x00050004u);
      const v2h h = __builtin_bit_cast(v2h, pair) + c2;
      r[i] = __builtin_bit_cast(uint32_t, h);
    }
  } else {
    const float c = (float)(128 + zp);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = (i < 2 ? w0 : w1) >> (16 * (i % 2));
      const uint32_t lo = __builtin_bit_cast(uint32_t, (float)(w & 255) - c);
      const uint32_t hi = __builtin_bit_cast(uint32_t, (float)((w >> 8) & 255) - c);
      r[i] = __builtin_amdgcn_perm(hi, lo, 0x07060302u);
    }
  }
  return r;
}

template <class AT>
__device__ __forceinline__ v4f mfma16(v4u a, v4u b, v4f c) {
  if constexpr (std::is_same<AT, Half>::value)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a),
                                                  __builtin_bit_cast(v8h, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8b, a),
                                                   __builtin_bit_cast(v8b, b), c, 0, 0, 0);
}

constexpr int kDownWaves = 8;

template <class AT>
__global__ __launch_bounds__(64 * kDownWaves) void k_lora_down(LoraArgs a) {
  __shared__ float part[kDownWaves][16][17];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int64_t m0 = (int64_t)blockIdx.x * 16, M = a.lin.M, K = a.lin.K;
  const int slot = blockIdx.y, r0 = 16 * blockIdx.z;
  const int64_t m = m0 + n < M ? m0 + n : M - 1;
  const int id = m0 + n < M ? adapter_of(a, m) : -1;
  // the slot-th distinct adapter of the 16 rows
  uint64_t left = __ballot(id >= 0) & 0xffff;
  uint64_t mine = 0;
  int ad = -1;
  for (int s = 0; left != 0; ++s) {
    ad = __builtin_amdgcn_readlane(id, (uint32_t)__builtin_ctzll(left));
    mine = __ballot(id == ad) & 0xffff;
    if (s == slot) break;
    left &= ~mine;
  }
  if (left == 0) return;
  const int rank = rank_of(a, ad);
  const bool rok = r0 + n < rank;

  const int8_t* xr = a.lin.x + m * K;
  const AT* ar = (const AT*)a.a + ((int64_t)ad * a.rank + (rok ? r0 + n : 0)) * K;
  v4f acc = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  if (r0 < rank) {
    for (int64_t k = 64 * wave; k < K; k += 64 * kDownWaves) {
      const int64_t kk = k + 16 * g;
      const bool ok = kk < K;
      v4u x = v4u{0, 0, 0, 0}, p = x, q = x;
      if (ok) x = *reinterpret_cast<const v4u*>(xr + kk);
      if (ok && rok) {
        p = *reinterpret_cast<const v4u*>(ar + kk);
        q = *reinterpret_cast<const v4u*>(ar + kk + 8);
      }
      acc = mfma16<AT>(p, less_zp<AT>(x[0], x[1], a.lin.izp), acc);
      acc = mfma16<AT>(q, less_zp<AT>(x[2], x[3], a.lin.izp), acc);
    }
  }
  // register r of lane (n, g): rank 4g + r, row n
#pragma unroll
  for (int r = 0; r < 4; ++r) part[wave][n][4 * g + r] = acc[r];
  __syncthreads();
  if (tid < 256) {
    const int row = tid / 16, r = tid % 16;
    if ((mine >> row) & 1) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < kDownWaves; ++w) s += part[w][row][r];
      const float f = a.lin.rq.s_in * (a.ad_scales ? a.ad_scales[ad] : 1.0f);
      a.t[(m0 + row) * a.rank_pad + r0 + r] = r0 + r < rank ? s * f : 0.0f;
    }
  }
}

// ------------------------------------------------------------------ the product
template <class AT>
__device__ __forceinline__ float half_at(uint32_t w, int hi) {
  return to_float(AT{(uint16_t)(hi ? w >> 16 : w)});
}

// sum_r B[ad, n, r] t[r] over the adapter's rank.
template <class AT>
__device__ __forceinline__ float up_dot(const LoraArgs& a, int ad, int64_t n, const float* t) {
  const int rank = rank_of(a, ad);
  const AT* b = (const AT*)a.b + ((int64_t)ad * a.lin.N + n) * a.rank;
  float s = 0.0f;
  if (a.rank % 8 == 0 && ((uintptr_t)a.b & 15) == 0) {
    for (int r = 0; r < rank; r += 8) {   // t is 0 past the rank
      const v4u w = *reinterpret_cast<const v4u*>(b + r);
      const v4f t0 = *reinterpret_cast<const v4f*>(t + r);
      const v4f t1 = *reinterpret_cast<const v4f*>(t + r + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool in0 = r + 2 * i < rank, in1 = r + 2 * i + 1 < rank;
        const float ta = i < 2 ? t0[2 * i] : t1[2 * i - 4];
        const float tb = i < 2 ? t0[2 * i + 1] : t1[2 * i - 3];
        s = __builtin_fmaf(in0 ? half_at<AT>(w[i], 0) : 0.0f, ta, s);
        s = __builtin_fmaf(in1 ? half_at<AT>(w[i], 1) : 0.0f, tb, s);
      }
    }
  } else {
    for (int r = 0; r < rank; ++r) s = __builtin_fmaf(to_float(b[r]), t[r], s);
  }
  return s;
}

template <class AT, class YT, int MT, int FN>
__global__ __launch_bounds__(256) void k_lora_rows(LoraArgs a) {
  constexpr int BM = 16 * MT, BN = 16 * FN, kWaves = 4;
  __shared__ int32_t part[kWaves][BM][BN + 1];
  __shared__ int32_t wsum[kWaves][BN];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int64_t M = a.lin.M, N = a.lin.N, K = a.lin.K;
  const int64_t n0 = (int64_t)blockIdx.x * BN, m0 = (int64_t)blockIdx.y * BM;
  const int8_t* wp[FN];
  const int8_t* xp[MT];
#pragma unroll
  for (int i = 0; i < FN; ++i) {
    const int64_t c = n0 + 16 * i + n;
    wp[i] = a.lin.w + (c < N ? c : N - 1) * K;
  }
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const int64_t m = m0 + 16 * j + n;
    xp[j] = a.lin.x + (m < M ? m : M - 1) * K;
  }
  v4i acc[FN][MT] = {};
  int32_t ws[FN] = {};
  v4i wf[FN], xf[MT];
  auto load = [&](int64_t k) {
    const int64_t kk = k + 16 * g;
    const bool ok = kk < K;   // past K: the row's first bytes, cleared below
#pragma unroll
    for (int i = 0; i < FN; ++i) wf[i] = *reinterpret_cast<const v4i*>(wp[i] + (ok ? kk : 0));
#pragma unroll
    for (int j = 0; j < MT; ++j) xf[j] = *reinterpret_cast<const v4i*>(xp[j] + (ok ? kk : 0));
    if (!ok) {
#pragma unroll
      for (int i = 0; i < FN; ++i) wf[i] = v4i{0, 0, 0, 0};
    }
  };
  int64_t k = 64 * wave;
  if (k < K) load(k);
  for (; k < K; k += 64 * kWaves) {
    v4i wc[FN], xc[MT];
#pragma unroll
    for (int i = 0; i < FN; ++i) wc[i] = wf[i];
#pragma unroll
    for (int j = 0; j < MT; ++j) xc[j] = xf[j];
    if (k + 64 * kWaves < K) load(k + 64 * kWaves);
#pragma unroll
    for (int i = 0; i < FN; ++i) {
#pragma unroll
      for (int j = 0; j < MT; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wc[i], xc[j], acc[i][j], 0, 0, 0);
#pragma unroll
      for (int d = 0; d < 4; ++d)
        ws[i] = __builtin_amdgcn_sdot4(wc[i][d], 0x01010101, ws[i], false);
    }
  }
  // register r of lane (n, g): channel 4g + r, row n
#pragma unroll
  for (int i = 0; i < FN; ++i) {
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) part[wave][16 * j + n][16 * i + 4 * g + r] = acc[i][j][r];
    ws[i] += __shfl_xor(ws[i], 16);
    ws[i] += __shfl_xor(ws[i], 32);
    if (g == 0) wsum[wave][16 * i + n] = ws[i];
  }
  __syncthreads();
  for (int e = tid; e < BM * BN; e += 256) {
    const int row = e / BN, c = e % BN;
    const int64_t m = m0 + row, ch = n0 + c;
    if (m >= M || ch >= N) continue;
    int32_t s = 0, w = 0;
#pragma unroll
    for (int v = 0; v < kWaves; ++v) {
      s += part[v][row][c];
      w += wsum[v][c];
    }
    float y = (float)(s - a.lin.izp * w);
    y = y * a.lin.rq.s_in;
    y = y * a.lin.wscale[ch];
    y = y + (a.lin.bias ? a.lin.bias[ch] : 0.0f);
    const int ad = adapter_of(a, m);
    if (ad >= 0) y = y + up_dot<AT>(a, ad, ch, a.t + m * a.rank_pad);
    if (a.relu) y = __builtin_fmaxf(y, 0.0f);
    ((YT*)a.y)[m * N + ch] = from_float<YT>(y);
  }
}

// ------------------------------------------------------------------ odd K and alignment
// Rows of `bytes` bytes at any address into rows of `padded` bytes (a multiple
// of 16), zero past the row: one 16-byte chunk a thread.
__global__ __launch_bounds__(256) void k_pad_rows(const int8_t* __restrict__ src, int64_t rows,
                                                  int64_t bytes, int64_t padded,
                                                  int8_t* __restrict__ dst) {
  const int64_t per = padded / 16;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= rows * per) return;
  const int64_t row = i / per, at = (i - row * per) * 16;
  const int8_t* p = src + row * bytes;
  v4u v = v4u{0, 0, 0, 0};
  if (at + 16 <= bytes) {
    __builtin_memcpy(&v, p + at, 16);
  } else {
    for (int b = 0; b < 16 && at + b < bytes; ++b)
      v[b / 4] |= (uint32_t)(uint8_t)p[at + b] << (8 * (b % 4));
  }
  *reinterpret_cast<v4u*>(dst + i * 16) = v;
}

hipError_t pad_rows(const void* src, int64_t rows, int64_t bytes, int64_t padded, int8_t* dst,
                    hipStream_t s) {
  const int64_t n = rows * (padded / 16);
  hipLaunchKernelGGL(k_pad_rows, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s,
                     (const int8_t*)src, rows, bytes, padded, dst);
  return hipGetLastError();
}

template <class AT, class YT>
hipError_t launch_rows(const LoraArgs& a, hipStream_t s) {
  const int64_t M = a.lin.M, N = a.lin.N;
  if (M <= 16) {
    const dim3 g((unsigned)((N + 15) / 16), 1);
    hipLaunchKernelGGL((k_lora_rows<AT, YT, 1, 1>), g, dim3(256), 0, s, a);
  } else {
    const dim3 g((unsigned)((N + 31) / 32), (unsigned)((M + 63) / 64));
    hipLaunchKernelGGL((k_lora_rows<AT, YT, 4, 2>), g, dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

template <class AT>
hipError_t launch_adapter(const LoraArgs& a, hipStream_t s) {
  const int slots = a.adapters < 16 ? a.adapters : 16;
  const dim3 g((unsigned)((a.lin.M + 15) / 16), (unsigned)slots, (unsigned)(a.rank_pad / 16));
  hipLaunchKernelGGL((k_lora_down<AT>), g, dim3(64 * kDownWaves), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  switch (a.y_type) {
    case Q8TA_F32: return launch_rows<AT, float>(a, s);
    case Q8TA_F16: return launch_rows<AT, Half>(a, s);
    default: return launch_rows<AT, Bfloat>(a, s);
  }
}

}  // namespace

hipError_t launch_linear_lora(LoraArgs a, hipStream_t s) {
  const int64_t M = a.lin.M, N = a.lin.N, K = a.lin.K;
  const int64_t at = (int64_t)a.adapters * a.rank;
  const size_t t_bytes = ((size_t)M * a.rank_pad * 4 + 255) / 256 * 256;
  const bool pad = K % 16 != 0 ||
                   (((uintptr_t)a.lin.x | (uintptr_t)a.lin.w | (uintptr_t)a.a) & 15) != 0;
  const int64_t kp = (K + 63) / 64 * 64;
  const size_t bytes = t_bytes + (pad ? (size_t)(M + N + 2 * at) * kp : 0);
  void* ws = nullptr;
  hipError_t e = workspace_acquire(&ws, bytes, s);
  if (e != hipSuccess) return e;
  a.t = (float*)ws;
  if (pad) {
    int8_t* x = (int8_t*)ws + t_bytes;
    int8_t* w = x + M * kp;
    int8_t* ap = w + N * kp;
    e = pad_rows(a.lin.x, M, K, kp, x, s);
    if (e == hipSuccess) e = pad_rows(a.lin.w, N, K, kp, w, s);
    if (e == hipSuccess) e = pad_rows(a.a, at, 2 * K, 2 * kp, ap, s);
    a.lin.x = x;
    a.lin.w = w;
    a.a = ap;
    a.lin.K = kp;
  }
  if (e == hipSuccess)
    e = a.ad_type == Q8TA_F16 ? launch_adapter<Half>(a, s) : launch_adapter<Bfloat>(a, s);
  const hipError_t f = workspace_release(ws, s);
  return e != hipSuccess ? e : f;
}

}  // namespace q8ta
