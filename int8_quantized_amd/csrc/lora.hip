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
// steps, where the weight stream is what has to be paid, and for products of few
// large tiles: the waves take
// every WAVES-th 64-byte step of K, weight and activation fragments come
// straight from memory into the operands of v_mfma_i32_16x16x64_i8 (16
// bytes a lane, the next step's loads ahead of this step's products), and
// their integer sums meet in LDS.
//
// Measured: 1 x 4096 x 4096, rank 16: down 6.6 us and rows 6.3 (17 MB, 2.5 us at
// the rate of a bare read: two launches of one round trip each); 50 x 4096 x 11008
// with 24 adapters: 10 and 27 us (68 MB, 10 us: every workgroup reads all
// rows of x from its L2, and the adapters' rows are 64 bytes each); 2048 x 4096 x
// 11008, rank 64: down 20 us, GEMM with the epilogue 144 (108 without adapters).
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

constexpr int kDownWaves = 16;

// RB: blocks of 16 ranks a workgroup takes, D: 64-byte steps of K whose loads
// are in flight at once.
template <class AT, int RB, int D>
__global__ __launch_bounds__(64 * kDownWaves) void k_lora_down(LoraArgs a) {
  __shared__ float part[kDownWaves][16][16 * RB + 1];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int64_t m0 = (int64_t)blockIdx.x * 16, M = a.lin.M, K = a.lin.K;
  const int r0 = 16 * RB * blockIdx.z;
  const int64_t m = m0 + n < M ? m0 + n : M - 1;
  const int id = m0 + n < M ? adapter_of(a, m) : -1;
  const int8_t* xr = a.lin.x + m * K;
  // the distinct adapters of the 16 rows, this workgroup's every gridDim.y-th
  uint64_t left = __ballot(id >= 0) & 0xffff;
  for (int slot = 0; left != 0; ++slot) {
    const int ad = __builtin_amdgcn_readlane(id, (uint32_t)__builtin_ctzll(left));
    const uint64_t mine = __ballot(id == ad) & 0xffff;
    left &= ~mine;
    if (slot % gridDim.y != blockIdx.y) continue;
    const int rank = rank_of(a, ad);
    const AT* ar[RB];
    bool rok[RB];
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      const int r = r0 + 16 * i + n;
      rok[i] = r < rank;
      ar[i] = (const AT*)a.a + ((int64_t)ad * a.rank + (rok[i] ? r : 0)) * K;
    }
    v4f acc[RB] = {};
    if (r0 < rank) {
      for (int64_t k0 = 64 * wave; k0 < K; k0 += 64 * kDownWaves * D) {
        v4u x[D], p[D][RB][2];
#pragma unroll
        for (int d = 0; d < D; ++d) {
          const int64_t kk = k0 + 64 * kDownWaves * d + 16 * g;
          const bool ok = kk < K;
          x[d] = v4u{0, 0, 0, 0};
          if (ok) x[d] = *reinterpret_cast<const v4u*>(xr + kk);
#pragma unroll
          for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              p[d][i][h] = v4u{0, 0, 0, 0};
              if (ok && rok[i]) p[d][i][h] = *reinterpret_cast<const v4u*>(ar[i] + kk + 8 * h);
            }
        }
#pragma unroll
        for (int d = 0; d < D; ++d) {
          const v4u x0 = less_zp<AT>(x[d][0], x[d][1], a.lin.izp);
          const v4u x1 = less_zp<AT>(x[d][2], x[d][3], a.lin.izp);
#pragma unroll
          for (int i = 0; i < RB; ++i) {
            acc[i] = mfma16<AT>(p[d][i][0], x0, acc[i]);
            acc[i] = mfma16<AT>(p[d][i][1], x1, acc[i]);
          }
        }
      }
    }
    // register r of lane (n, g): rank 4g + r of the block, row n
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) part[wave][n][16 * i + 4 * g + r] = acc[i][r];
    __syncthreads();
    for (int e = tid; e < 256 * RB; e += 64 * kDownWaves) {
      const int row = e / (16 * RB), r = e % (16 * RB);
      if (((mine >> row) & 1) && r0 + r < a.rank_pad) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kDownWaves; ++w) s += part[w][row][r];
        const float f = a.lin.rq.s_in * (a.ad_scales ? a.ad_scales[ad] : 1.0f);
        const int64_t at = (m0 + row) * a.rank_pad + r0 + r;
        float t = r0 + r < rank ? s * f : 0.0f;
        if (!a.in_parts) {
          a.t[at] = t;
        } else {
          for (int q = 0; q < kLoraParts; ++q) {   // each the rounding of what is left
            const Bfloat h = from_float<Bfloat>(t);
            a.tp[q * M * a.rank_pad + at] = h.bits;
            t = t - to_float(h);
          }
        }
      }
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ the product
template <class AT>
__device__ __forceinline__ float half_at(uint32_t w, int hi) {
  return to_float(AT{(uint16_t)(hi ? w >> 16 : w)});
}

// sum_r B[ad, n, r] t[r] over the adapter's rank.  Rows of 16-byte chunks: the
// first kAhead come loaded (ahead: ready before t and the sums are), the others
// as many at once.
constexpr int kAhead = 4;
template <class AT>
__device__ __forceinline__ const AT* up_row(const LoraArgs& a, int ad, int64_t n) {
  return (const AT*)a.b + ((int64_t)ad * a.lin.N + n) * a.rank;
}
__device__ __forceinline__ void up_load(const void* row, int r, int rank, v4u (&w)[kAhead]) {
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    w[i] = v4u{0, 0, 0, 0};
    if (r + 8 * i < rank) w[i] = *reinterpret_cast<const v4u*>((const uint16_t*)row + r + 8 * i);
  }
}
template <class AT>
__device__ __forceinline__ float up_sum(const v4u (&w)[kAhead], int r, int rank, const float* t, float s) {
#pragma unroll
  for (int j = 0; j < kAhead; ++j) {
    const int at = r + 8 * j;
    if (at >= rank) break;   // t is 0 past the rank, up to a multiple of 16
    const v4f t0 = *reinterpret_cast<const v4f*>(t + at);
    const v4f t1 = *reinterpret_cast<const v4f*>(t + at + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool in0 = at + 2 * i < rank, in1 = at + 2 * i + 1 < rank;
      const float ta = i < 2 ? t0[2 * i] : t1[2 * i - 4];
      const float tb = i < 2 ? t0[2 * i + 1] : t1[2 * i - 3];
      const uint32_t pair = w[j][i];
      s = __builtin_fmaf(in0 ? half_at<AT>(pair, 0) : 0.0f, ta, s);
      s = __builtin_fmaf(in1 ? half_at<AT>(pair, 1) : 0.0f, tb, s);
    }
  }
  return s;
}

// D: steps of K whose loads are in flight ahead of the products.
template <class AT, class YT, int MT, int FN, int WAVES, int D>
__global__ __launch_bounds__(64 * WAVES) void k_lora_rows(LoraArgs a) {
  constexpr int BM = 16 * MT, BN = 16 * FN;
  __shared__ int32_t part[WAVES][BM][BN + 1];
  __shared__ int32_t wsum[WAVES][BN];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int64_t M = a.lin.M, N = a.lin.N, K = a.lin.K;
  const int64_t n0 = a.n0 + (int64_t)blockIdx.x * BN, m0 = (int64_t)blockIdx.y * BM;
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
  v4i wf[D][FN], xf[D][MT];
  // every load unconditional: chunks past K read the row's first bytes, and
  // the weights' are replaced by zeros when they are used
  auto load = [&](int64_t k, v4i (&w)[FN], v4i (&x)[MT]) {
    const int64_t kk = k + 16 * g < K ? k + 16 * g : 0;
#pragma unroll
    for (int i = 0; i < FN; ++i)
      w[i] = __builtin_nontemporal_load(reinterpret_cast<const v4i*>(wp[i] + kk));
#pragma unroll
    for (int j = 0; j < MT; ++j) x[j] = *reinterpret_cast<const v4i*>(xp[j] + kk);
  };
  constexpr int kStride = 64 * WAVES;
#pragma unroll
  for (int d = 0; d < D; ++d) load(64 * wave + kStride * d, wf[d], xf[d]);
  for (int64_t k0 = 64 * wave; k0 < K; k0 += kStride * D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const bool ok = k0 + kStride * d + 16 * g < K;
#pragma unroll
      for (int i = 0; i < FN; ++i) {
        const v4i w = ok ? wf[d][i] : v4i{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < MT; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w, xf[d][j], acc[i][j], 0, 0, 0);
#pragma unroll
        for (int e = 0; e < 4; ++e) ws[i] = __builtin_amdgcn_sdot4(w[e], 0x01010101, ws[i], false);
      }
      if (k0 + kStride * D < K) load(k0 + kStride * (D + d), wf[d], xf[d]);
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
  // this thread's outputs; the first chunks of their adapters' rows are on
  // their way while the waves' sums meet
  constexpr int E = (BM * BN + 64 * WAVES - 1) / (64 * WAVES);
  const bool vec = a.rank % 8 == 0 && ((uintptr_t)a.b & 15) == 0;
  int ad[E], rank[E];
  v4u ahead[E][kAhead];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int e = tid + i * 64 * WAVES;
    const int64_t m = m0 + e / BN, ch = n0 + e % BN;
    ad[i] = e < BM * BN && m < M && ch < N ? adapter_of(a, m) : -1;
    rank[i] = ad[i] >= 0 ? rank_of(a, ad[i]) : 0;
    if (vec) up_load(up_row<AT>(a, ad[i] >= 0 ? ad[i] : 0, ch < N ? ch : 0), 0, rank[i], ahead[i]);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int e = tid + i * 64 * WAVES;
    const int row = e / BN, c = e % BN;
    const int64_t m = m0 + row, ch = n0 + c;
    if (e >= BM * BN || m >= M || ch >= N) continue;
    int32_t s = 0, w = 0;
#pragma unroll
    for (int v = 0; v < WAVES; ++v) {
      s += part[v][row][c];
      w += wsum[v][c];
    }
    float y = (float)(s - a.lin.izp * w);
    y = y * a.lin.rq.s_in;
    y = y * a.lin.wscale[ch];
    y = y + (a.lin.bias ? a.lin.bias[ch] : 0.0f);
    if (rank[i] > 0) {
      const AT* b = up_row<AT>(a, ad[i], ch);
      const float* t = a.t + m * a.rank_pad;
      float up = 0.0f;
      if (vec) {
        up = up_sum<AT>(ahead[i], 0, rank[i], t, up);
        for (int r = 8 * kAhead; r < rank[i]; r += 8 * kAhead) {
          v4u more[kAhead];
          up_load(b, r, rank[i], more);
          up = up_sum<AT>(more, r, rank[i], t, up);
        }
      } else {
        for (int r = 0; r < rank[i]; ++r) up = __builtin_fmaf(to_float(b[r]), t[r], up);
      }
      y = y + up;
    }
    if (a.relu) y = y < 0.0f ? 0.0f : y;
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

// A launch has fewer than 2^32 threads in x (more are cut off without an
// error); what takes more goes in launches of up to this many.
constexpr int64_t kMostThreads = (int64_t)1 << 31;

hipError_t pad_rows(const void* src, int64_t rows, int64_t bytes, int64_t padded, int8_t* dst,
                    hipStream_t s) {
  const int64_t most = kMostThreads / (padded / 16);   // (a row of 2^31 bytes is 2^27 chunks)
  for (int64_t r0 = 0; r0 < rows; r0 += most) {
    const int64_t part = rows - r0 < most ? rows - r0 : most, n = part * (padded / 16);
    hipLaunchKernelGGL(k_pad_rows, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s,
                       (const int8_t*)src + r0 * bytes, part, bytes, padded, dst + r0 * padded);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <class AT, class YT, int MT, int FN, int WAVES, int D>
hipError_t launch_shape(LoraArgs a, hipStream_t s) {
  constexpr int64_t BN = 16 * FN, most = kMostThreads / (64 * WAVES);
  const int64_t tiles = (a.lin.N + BN - 1) / BN;
  for (int64_t t0 = 0; t0 < tiles; t0 += most) {
    a.n0 = t0 * BN;
    const dim3 g((unsigned)(tiles - t0 < most ? tiles - t0 : most),
                 (unsigned)((a.lin.M + 16 * MT - 1) / (16 * MT)));
    hipLaunchKernelGGL((k_lora_rows<AT, YT, MT, FN, WAVES, D>), g, dim3(64 * WAVES), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <class AT, class YT>
hipError_t launch_rows(const LoraArgs& a, hipStream_t s) {
  // Channels of a workgroup, in sixteens: the fewest rounds of 256 workgroups
  // times what one of them takes, which is about c + 1 (it reads its channels and
  // all rows).  4096 x 11008 with 24 adapters, 64 rows: 48 channels 39 us, 32 48, 16
  // 53; 4096 x 16384: 64, 50, 67; 4096 x 4096: 38, 31, 26.
  int c = 1;
  int64_t least = INT64_MAX;
  for (int i = 1; i <= 3; ++i) {
    const int64_t groups = (a.lin.N + 16 * i - 1) / (16 * i) * ((a.lin.M + 63) / 64), cost = (groups + 255) / 256 * (i + 1);
    if (cost <= least) {
      least = cost;
      c = i;
    }
  }
  if (a.lin.M <= 16) {
    if (c == 1) return launch_shape<AT, YT, 1, 1, 16, 4>(a, s);
    if (c == 2) return launch_shape<AT, YT, 1, 2, 8, 4>(a, s);
    return launch_shape<AT, YT, 1, 3, 8, 4>(a, s);
  }
  if (a.lin.M <= 32) {
    if (c == 1) return launch_shape<AT, YT, 2, 1, 8, 4>(a, s);
    if (c == 2) return launch_shape<AT, YT, 2, 2, 8, 4>(a, s);
    return launch_shape<AT, YT, 2, 3, 16, 2>(a, s);
  }
  if (c == 1) return launch_shape<AT, YT, 4, 1, 16, 2>(a, s);
  if (c == 2) return launch_shape<AT, YT, 4, 2, 8, 2>(a, s);
  return launch_shape<AT, YT, 4, 3, 8, 2>(a, s);
}

template <class AT>
hipError_t launch_down(const LoraArgs& a, hipStream_t s) {
  const unsigned tiles = (unsigned)((a.lin.M + 15) / 16);
  // 32 ranks a workgroup where there are many tiles (x is read once for them:
  // 2048 rows 17.8 us against 21.6), 16 with twice the loads in flight where a
  // launch is a chain of latencies (50 rows 10.0 against 13.4)
  const int rb = a.rank_pad > 16 && a.lin.M > 64 ? 2 : 1;
  const unsigned z = (unsigned)((a.rank_pad + 16 * rb - 1) / (16 * rb));
  // workgroups a tile's adapters are dealt over: up to 16, fewer where the
  // tiles alone fill the card
  unsigned slots = (unsigned)(a.adapters < 16 ? a.adapters : 16);
  const unsigned want = 1024 / (tiles * z) + 1;
  slots = slots < want ? slots : want;
  const dim3 g(tiles, slots, z), t(64 * kDownWaves);
  if (rb == 2) hipLaunchKernelGGL((k_lora_down<AT, 2, 2>), g, t, 0, s, a);
  else hipLaunchKernelGGL((k_lora_down<AT, 1, 4>), g, t, 0, s, a);
  return hipGetLastError();
}

template <class AT>
hipError_t launch_few(const LoraArgs& a, hipStream_t s) {
  switch (a.y_type) {
    case Q8TA_F32: return launch_rows<AT, float>(a, s);
    case Q8TA_F16: return launch_rows<AT, Half>(a, s);
    default: return launch_rows<AT, Bfloat>(a, s);
  }
}

// Which product: the eight-wave GEMM, the two-workgroup GEMM, or k_lora_rows.
// The GEMMs' tiles of 256 x 256 and 256 x 128 leave most of the card idle where there
// are few: up to about one round of k_lora_rows' workgroups that is the faster
// (K 4096: 128 x 2048 22 us against 50, 168 x 4113, 258 groups, 40 and 51, 256 x
// 4113, 344 groups, 56 and 48; K 1024: 1024 x 512 15 and 20).
char product_of(const LinearArgs& a) {
  if ((a.M + 63) / 64 * ((a.N + 47) / 48) <= 300 || a.M <= 64) return 'r';
  return gemm_w8_preferred(a) ? 'w' : 'x';
}

}  // namespace

hipError_t launch_linear_lora(LoraArgs a, hipStream_t s) {
  const int64_t M = a.lin.M, N = a.lin.N, K = a.lin.K;
  const int64_t at = (int64_t)a.adapters * a.rank;
  const int64_t kp = (K + 63) / 64 * 64;
  LinearArgs whole = a.lin;
  whole.K = kp;
  const bool pad = K % 16 != 0 ||
                   (((uintptr_t)a.lin.x | (uintptr_t)a.lin.w | (uintptr_t)a.a) & 15) != 0;
  const char product = product_of(pad ? whole : a.lin);
  a.in_parts = product != 'r';
  const size_t t_bytes =
      ((size_t)M * a.rank_pad * (a.in_parts ? 2 * kLoraParts : 4) + 255) / 256 * 256;
  const size_t bytes = t_bytes + (pad ? (size_t)(M + N + 2 * at) * kp : 0);
  void* ws = nullptr;
  hipError_t e = workspace_acquire(&ws, bytes, s);
  if (e != hipSuccess) return e;
  a.t = (float*)ws;
  a.tp = (uint16_t*)ws;
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
  const bool half = a.ad_type == Q8TA_F16;
  if (e == hipSuccess) e = half ? launch_down<Half>(a, s) : launch_down<Bfloat>(a, s);
  if (e == hipSuccess) {
    if (product == 'w') e = launch_gemm_w8_lora(a, s);
    else if (product == 'x') e = launch_gemm_mx_lora(a, s);
    else e = half ? launch_few<Half>(a, s) : launch_few<Bfloat>(a, s);
  }
  const hipError_t f = workspace_release(ws, s);
  return e != hipSuccess ? e : f;
}

}  // namespace q8ta
