// q8ta_linear_per_token and q8ta_gated_linear where there are few rows, and the
// choice of their kernels.
//
//   y[m, n] = (sum_k x[m, k] w[n, k] * xs[m]) * ws[n] + bias[n]
//   gated:  out[m, n] = act(y_gate[m, n]) * y_up[m, n]
//
// k_scaled_rows: 16 * MT rows by 16 * FN weight rows, for the row counts of decode
// steps, where the weight stream is what has to be paid: the waves take every
// WAVES-th 64-byte step of K, weight and activation fragments come straight
// from memory into the operands of v_mfma_i32_16x16x64_i8 (16 bytes a lane, D
// steps' loads in flight), and their integer sums meet in LDS.  The gated form
// has a channel's gate and up rows in one workgroup, so that the block is one
// launch and the two products never reach memory.
//
// Measured (weights that the caches of the card hold): 1 x 4096 x 4096 4.8 us (the best of 200 calls 4.5), 1 x
// 4096 x 11008 9.9 (8.6), gated 1 x 4096 x 11008 16.0 (15.3): the weights at 3.5, 4.6 and 5.6 TB/s; a kernel that
// but reads as many bytes takes 3.6, 7.5 and 13.9.  What is left is the join of the waves'
// sums and, with many rows, x, which every workgroup reads whole.
#include <cmath>
#include <type_traits>

#include "scaled_epilogue.h"

namespace q8ta {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));

typedef int v4i_any __attribute__((ext_vector_type(4), aligned(1)));

// FN: fragments of 16 weight rows, FN / MATS of each matrix.  ODD: any alignment and any K >= 16;
// a row's last chunk is then its last 16 bytes, those that the chunk before had as zeros in x.
template <class YT, int MATS, int MT, int FN, int WAVES, int D, bool ODD>
__global__ __launch_bounds__(64 * WAVES) void k_scaled_rows(ScaledArgs a) {
  constexpr int BM = 16 * MT, BN = 16 * FN, C = BN / MATS, H = FN / MATS;
  __shared__ int32_t part[WAVES][BM][BN + 1];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int64_t M = a.M, N = a.N, K = a.K;
  const int64_t n0 = a.n0 + (int64_t)blockIdx.x * C, m0 = (int64_t)blockIdx.y * BM;
  const int8_t* wp[FN];
  const int8_t* xp[MT];
#pragma unroll
  for (int i = 0; i < FN; ++i) {
    const int64_t c = n0 + 16 * (i % H) + n;
    wp[i] = a.w[i / H] + (c < N ? c : N - 1) * K;
  }
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const int64_t m = m0 + 16 * j + n;
    xp[j] = a.x + (m < M ? m : M - 1) * K;
  }
  v4i acc[FN][MT] = {};
  v4i wf[D][FN], xf[D][MT];
  // every load unconditional: chunks past K read the row's first bytes, and the
  // rows' are replaced by zeros when they are used
  using Chunk = std::conditional_t<ODD, v4i_any, v4i>;
  auto load = [&](int64_t k, v4i (&w)[FN], v4i (&x)[MT]) {
    int64_t kk = k + 16 * g < K ? k + 16 * g : 0;
    if (ODD && kk > K - 16) kk = K - 16;
#pragma unroll
    for (int i = 0; i < FN; ++i) w[i] = *reinterpret_cast<const Chunk*>(wp[i] + kk);
#pragma unroll
    for (int j = 0; j < MT; ++j) x[j] = *reinterpret_cast<const Chunk*>(xp[j] + kk);
  };
  constexpr int kStride = 64 * WAVES;
#pragma unroll
  for (int d = 0; d < D; ++d) load(64 * wave + kStride * d, wf[d], xf[d]);
  for (int64_t k0 = 64 * wave; k0 < K; k0 += kStride * D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int64_t kk = k0 + kStride * d + 16 * g;
      v4i keep = kk < K ? v4i{-1, -1, -1, -1} : v4i{0, 0, 0, 0};
      if (ODD && kk < K && kk > K - 16) {
        const int twice = (int)(kk - (K - 16));   // bytes of the chunk before, 1 to 15
#pragma unroll
        for (int i = 0; i < 4; ++i)
          keep[i] = twice >= 4 * i + 4 ? 0 : (twice <= 4 * i ? -1 : (int)(0xffffffffu << (8 * (twice - 4 * i))));
      }
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        const v4i x = xf[d][j] & keep;
#pragma unroll
        for (int i = 0; i < FN; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[d][i], x, acc[i][j], 0, 0, 0);
      }
      if (k0 + kStride * D < K) load(k0 + kStride * (D + d), wf[d], xf[d]);
    }
  }
  // register r of lane (n, g): weight row 4g + r, row n
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) part[wave][16 * j + n][16 * i + 4 * g + r] = acc[i][j][r];
  // this thread's outputs; their constants are on their way while the sums meet
  constexpr int E = (BM * C + 64 * WAVES - 1) / (64 * WAVES);
  float xs[E], ws[E][MATS], bi[E][MATS];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int e = tid + i * 64 * WAVES;
    const int64_t m = m0 + e / C, ch = n0 + e % C;
    const bool in = e < BM * C && m < M && ch < N;
    xs[i] = in ? a.xs[m] : 0.0f;
#pragma unroll
    for (int q = 0; q < MATS; ++q) {
      ws[i][q] = in ? a.ws[q][ch] : 0.0f;
      bi[i][q] = in && a.bias[q] ? a.bias[q][ch] : 0.0f;
    }
  }
  __syncthreads();
  with_activation<MATS>(a.act, [&](auto ACT) {
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int e = tid + i * 64 * WAVES;
    const int row = e / C, c = e % C;
    const int64_t m = m0 + row, ch = n0 + c;
    if (e >= BM * C || m >= M || ch >= N) continue;
    float y[MATS];
#pragma unroll
    for (int q = 0; q < MATS; ++q) {
      int32_t s = 0;
#pragma unroll
      for (int v = 0; v < WAVES; ++v) s += part[v][row][q * C + c];
      y[q] = scaled(s, xs[i], ws[i][q], bi[i][q]);
    }
    float out = activate<decltype(ACT)::value>(y[0]);
    if constexpr (MATS == 2) out = out * y[1];
    ((YT*)a.y)[m * N + ch] = from_float<YT>(out);
  }
  });
}

constexpr int64_t kMostThreads = (int64_t)1 << 31;   // of one launch

template <class YT, int MATS, int MT, int FN, int WAVES, int D, bool ODD>
hipError_t launch_shape(ScaledArgs a, hipStream_t s) {
  constexpr int64_t C = 16 * FN / MATS, most = kMostThreads / (64 * WAVES);
  const int64_t tiles = (a.N + C - 1) / C;
  for (int64_t t0 = 0; t0 < tiles; t0 += most) {
    a.n0 = t0 * C;
    const dim3 g((unsigned)(tiles - t0 < most ? tiles - t0 : most),
                 (unsigned)((a.M + 16 * MT - 1) / (16 * MT)));
    hipLaunchKernelGGL((k_scaled_rows<YT, MATS, MT, FN, WAVES, D, ODD>), g, dim3(64 * WAVES), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Of the matrices' 16-channel fragments a workgroup takes one each, and sixteen waves
// share K (1 x 4096 x 4096 4.5 us, with eight waves 5.4, with three fragments 7.9).  For
// up to 16 rows of the gated form three each, where that is fewer rounds of 256
// workgroups times what one takes (1 x 11008: 16.9 us against 18.4, 1 x 2048: 8.0
// and 4.3).  Plain loads: nontemporal ones took 10 to 20 % longer, also for weights that
// no cache holds.
// Channels of a workgroup:
int64_t channels_of(const ScaledArgs& a) {
  auto cost = [&](int64_t c) { return ((a.N + 16 * c - 1) / (16 * c) + 255) / 256 * (c + 1); };
  return a.mats == 2 && a.M <= 16 && cost(3) < cost(1) ? 48 : 16;
}

// (D: a wave's steps, up to what measured best: a load that is not needed is no smaller than one that is,
// 16 x 1024 x 11008 12.6 us with four at a time.  All of them at once where there are up to four; where there
// are more, two: 1 x 11008 x 4096 10.7 with four, 9.8 with two.)
template <class YT, bool ODD>
hipError_t launch_rows_of(const ScaledArgs& a, hipStream_t s) {
  const int64_t k16 = (a.K + 1023) / 1024;   // steps of one of sixteen waves
  if (a.mats == 2) {
    if (a.M <= 16) {
      if (channels_of(a) == 48)
        return k16 == 1 ? launch_shape<YT, 2, 1, 6, 16, 1, ODD>(a, s) : launch_shape<YT, 2, 1, 6, 16, 2, ODD>(a, s);
      return k16 == 1 ? launch_shape<YT, 2, 1, 2, 16, 1, ODD>(a, s) : launch_shape<YT, 2, 1, 2, 16, 2, ODD>(a, s);
    }
    if (a.M > 32) return launch_shape<YT, 2, 4, 2, 8, 2, ODD>(a, s);
    return k16 == 1 ? launch_shape<YT, 2, 2, 2, 16, 1, ODD>(a, s) : launch_shape<YT, 2, 2, 2, 16, 2, ODD>(a, s);
  }
  if (a.M <= 16) {
    if (k16 == 1) return launch_shape<YT, 1, 1, 1, 16, 1, ODD>(a, s);
    if (k16 == 2 || k16 > 4) return launch_shape<YT, 1, 1, 1, 16, 2, ODD>(a, s);
    return launch_shape<YT, 1, 1, 1, 16, 4, ODD>(a, s);
  }
  if (a.M <= 32) {
    if (k16 == 1) return launch_shape<YT, 1, 2, 1, 16, 1, ODD>(a, s);
    return k16 == 2 ? launch_shape<YT, 1, 2, 1, 16, 2, ODD>(a, s) : launch_shape<YT, 1, 2, 1, 16, 4, ODD>(a, s);
  }
  return k16 == 1 ? launch_shape<YT, 1, 4, 1, 16, 1, ODD>(a, s) : launch_shape<YT, 1, 4, 1, 16, 2, ODD>(a, s);
}

template <class YT>
hipError_t launch_rows(const ScaledArgs& a, hipStream_t s) {
  return a.odd ? launch_rows_of<YT, true>(a, s) : launch_rows_of<YT, false>(a, s);
}

// Which kernel, by an estimate of the time in us.  The tiles: a start, and for each 64-byte
// step the larger of its latency (which grows as the tiles fill the card) times the
// rounds of workgroups, and of all tiles' loads at the 10.7 TB/s at which they come from the
// L2s.  The row kernel, which reads all rows of x for each 16 channels: a start and, for each
// round of 256 workgroups, the rows of x and the weights' at 26 KB a us.  Where rows have no
// 16-byte alignment it reads them as they are, at odd addresses at about a third of the
// rate (1 x 4089 x 4096 7.9 us, 1 x 4096 x 4096 4.5), and the tiles pay for the copies of x and
// the weights.  The numbers are fitted to the measured times of all seven kernels at 1700
// sizes (1 to 2048 rows, K 64 to 11008, N 256 to 28000, one and two matrices): what it takes is
// 1 % slower than the fastest on average and 34 % at most (with copies 2 and 62 %).  Some of
// them, one matrix (us; the row kernel, 32 x 32 by eight waves, 64 x 64 by four, by one,
// 128 x 128, 256 x 128, 256 x 256; rows x K x N):
//   16 x 4096 x 4096     5.8  5.1  7.3  18   17   26   38
//   64 x 4096 x 4096    11.8  7.1  8.2  18   19   28   41
//   64 x 11008 x 4096   28    17   27   40   47   66   96
//   128 x 4096 x 11008    -    -   23   20   22   29   42
//   512 x 4096 x 4096     -   44   23   20   20   27   40
//   512 x 4096 x 11008    -    -   61   49   37   33   42
//   1000 x 4096 x 11008   -    -  119  104   65   62   52
struct Guess {
  double start, step, fill;
  int at_once, tn, bm;   // workgroups of a CU, the tile
};
constexpr Guess kGuess[] = {{2.4, 0.0964, 1.1, 1, 64, 64},     // in the order of kTile*
                            {1.9, 0.205, 0.86, 6, 64, 64},
                            {3.0, 0.386, 0.0, 3, 128, 128},
                            {3.0, 0.387, 0.06, 1, 256, 128},
                            {4.1, 0.569, 0.35, 1, 256, 256},
                            {2.4, 0.0323, 1.76, 1, 32, 32}};   // (for each matrix)
// Sets the tile, -1 for the row kernel.
void choose(ScaledArgs& a) {
  // (a tile's offsets are 32-bit)
  a.tile = -1;
  if (a.K > (int64_t)1 << 23) return;
  const double m = (double)a.M, k = (double)a.K, steps = std::ceil(k / 64);
  const double rows = std::ceil((double)a.N / 32) * 32 * a.mats;
  const int64_t own = channels_of(a);
  const bool bytes = a.odd && (a.K % 2 != 0 || ((uintptr_t)a.x | (uintptr_t)a.w[0] | (uintptr_t)a.w[a.mats - 1]) % 2 != 0);
  const double slab = (m + (double)(own * a.mats)) * k / 26500.0;
  double least = 1.5 + (double)((a.N + 256 * own - 1) / (256 * own)) * (bytes ? 1.5 + 2.8 * slab : slab);
  if (a.M > 64) least = INFINITY;
  const double copies = a.odd ? 7.0 + 0.7 * k / 1000 + 2.0 * a.mats * (double)a.N * k / 3.5e6 : 0.0;
  for (int i = 0; i < 6; ++i) {
    Guess g = kGuess[i];
    if (i == kTile32Split) {
      g.step *= a.mats;
      g.tn *= a.mats;
    }
    const double tiles = std::ceil(m / g.bm) * std::ceil(rows / g.tn);
    const double rounds = std::ceil(tiles / (256.0 * g.at_once)), fill = tiles < 256.0 ? tiles / 256.0 : 1.0;
    const double latency = g.step * rounds * (1.0 + g.fill * fill * fill);
    const double loads = tiles * (g.tn + g.bm) * 64 / 10.7e6;
    const double t = copies + g.start + steps * (latency > loads ? latency : loads);
    if (t < least) {
      a.tile = i;
      least = t;
    }
  }
  // Whole rounds of 256 x 256 tiles, and the columns that are left as 256 x 128 tiles where those
  // fit one round, which takes that tile's time.
  const int64_t c = 256 / a.mats, n = (a.N + c - 1) / c, ma = (a.M + 255) / 256, mb = (a.M + 127) / 128;
  a.columns = n;
  const int64_t whole = ma * n / 256, cols = whole * 256 / ma;
  if (whole == 0 || cols == n || (n - cols) * mb > 256 || ma * cols > 1 << 20) return;
  const Guess &g = kGuess[kTile256], &h = kGuess[kTile256x128];
  const double t = copies + g.start + steps * (g.step * (1.0 + g.fill) * (double)whole + h.step * (1.0 + h.fill));
  if (t < least) {
    a.tile = kTile256;
    a.columns = cols;
  }
}

// The rows of x and of the weights, K bytes each, one after the other in rows of kp, which end
// in zeros: a wave a row.
__global__ __launch_bounds__(256) void k_copy_rows(ScaledArgs a, int64_t kp, int8_t* to) {
  constexpr int kAhead = 4;
  const int lane = threadIdx.x & 63;
  const int64_t rows = a.M + a.mats * a.N, K = a.K;
  for (int64_t r = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / 64); r < rows;
       r += (int64_t)gridDim.x * 4) {
    const int8_t* src = r < a.M ? a.x + r * K : (r < a.M + a.N ? a.w[0] + (r - a.M) * K : a.w[1] + (r - a.M - a.N) * K);
    int8_t* dst = to + r * kp;
    int64_t k = 16 * lane;
    for (; k + 1024 * (kAhead - 1) + 16 <= K; k += 1024 * kAhead) {
      v4i v[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) v[u] = *reinterpret_cast<const v4i_any*>(src + k + 1024 * u);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) *reinterpret_cast<v4i*>(dst + k + 1024 * u) = v[u];
    }
    for (; k + 16 <= K; k += 1024) *reinterpret_cast<v4i*>(dst + k) = *reinterpret_cast<const v4i_any*>(src + k);
    if (k < K) {
      uint32_t v[4] = {};
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (k + i < K) v[i / 4] |= (uint32_t)(uint8_t)src[k + i] << (8 * (i % 4));
      *reinterpret_cast<v4i*>(dst + k) = v4i{(int)v[0], (int)v[1], (int)v[2], (int)v[3]};
    }
  }
}
hipError_t launch_copies(const ScaledArgs& a, int64_t kp, int8_t* to, hipStream_t s) {
  const int64_t blocks = (a.M + a.mats * a.N + 3) / 4, most = (int64_t)1 << 20;
  hipLaunchKernelGGL(k_copy_rows, dim3((unsigned)(blocks < most ? blocks : most)), dim3(256), 0, s, a, kp, to);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_scaled(ScaledArgs a, hipStream_t s) {
  const int64_t M = a.M, N = a.N, K = a.K, kp = (K + 15) / 16 * 16;
  uintptr_t ptrs = (uintptr_t)a.x | (uintptr_t)a.w[0];
  if (a.mats == 2) ptrs |= (uintptr_t)a.w[1];
  a.odd = K % 16 != 0 || ptrs % 16 != 0;
  choose(a);
  const bool rows = a.tile < 0, pad = a.odd && (!rows || K < 16);
  void* ws = nullptr;
  hipError_t e = hipSuccess;
  if (pad) {
    e = workspace_acquire(&ws, (size_t)(M + a.mats * N) * kp, s);
    if (e != hipSuccess) return e;
    int8_t* to = (int8_t*)ws;
    e = launch_copies(a, kp, to, s);
    a.x = to;
    to += M * kp;
    for (int q = 0; q < a.mats; ++q, to += N * kp) a.w[q] = to;
    a.K = kp;
    a.odd = false;
  }
  if (e == hipSuccess) {
    if (a.y_type == Q8TA_F32) e = rows ? launch_rows<float>(a, s) : launch_tiles_f32(a, s);
    else if (a.y_type == Q8TA_F16) e = rows ? launch_rows<Half>(a, s) : launch_tiles_f16(a, s);
    else e = rows ? launch_rows<Bfloat>(a, s) : launch_tiles_bf16(a, s);
  }
  if (!pad) return e;
  const hipError_t f = workspace_release(ws, s);
  return e != hipSuccess ? e : f;
}

}  // namespace q8ta
