// Matrix-core GEMM of q8ta_linear_per_token and q8ta_gated_linear for more rows
// than the row kernel of scaled.hip takes.
//
//   y[m, n] = (sum_k x[m, k] w[n, k] * xs[m]) * ws[n] + bias[n]
//   gated:  out[m, n] = act(y_gate[m, n]) * y_up[m, n]
//
//  * The products run as in the eight-wave GEMM of q8ta_linear (gemm_w8.hip):
//    64-byte K steps straight from memory into one of three LDS stages, each
//    a shared object of its own, 32x32x32 products of waves that own 32 * FN weight
//    rows by 64 rows of x, one barrier a step between its two slices, the loads two and
//    a half steps ahead.  There is no zero point here, so no sums of the weights.
//  * Weight rows are dealt out to the lanes so that the FN fragments of a lane
//    are neighbouring channels (fragment i of lane l: channel FN * l + i of the
//    wave's; gated: the first half gate, the second half up, of FN / 2 channels):
//    LDS row 32 * i + l is fetched from that weight row.  A lane then stores up to 16
//    bytes and half a wave a whole stretch of the row, straight from the
//    accumulators, and the gated block's two factors meet in one lane.
//  * K is a multiple of 16: chunks past it, in the last step only, come from 64
//    bytes of zeros.
//  * Rows past M or N read the last row; their products are not stored.
//
// Measured: 2048 x 4096 x 11008 97 to 103 us by the card's clock (1.8 to 1.9 Pop/s), gated 186 to 194
// (1.9 to 2.0), 8192^3 506 to 570 (1.9 to 2.2; a library's product 517): the matrix instructions, with the fragment reads and
// the loads between them, bound it.  Fewer rows: scaled.hip says which tile and why; a quarter
// to a half of the card's rate is left where one round of workgroups has to fetch all of
// its bytes from the L2s.  K split over workgroups, their sums joined by another launch, gained
// less than the launch and its memory cost.
#pragma once

#include <type_traits>

#include "scaled_epilogue.h"

namespace q8ta {
namespace {   // (each source that includes this has kernels of its own)

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));
typedef float v4f __attribute__((ext_vector_type(4)));
#define Q8TA_LDS(p) ((__attribute__((address_space(3))) void*)(p))

template <int B, int E>
struct Static {
  template <class F>
  __device__ __forceinline__ static void each(F&& f) {
    if constexpr (B < E) {
      f(std::integral_constant<int, B>{});
      Static<B + 1, E>::each(f);
    }
  }
};

// s_waitcnt immediate (gfx9 encoding): vmcnt <= vm, lgkmcnt 0, expcnt any.
constexpr int wait_vm_lgkm0(int vm) { return (vm & 15) | ((vm >> 4) << 14) | (7 << 4); }

__device__ int8_t g_zeros[64] __attribute__((aligned(64)));   // never written

// WAVES_N x WAVES_M waves of FN x FM fragments of 32 x 32.
template <int WAVES_N_, int WAVES_M_, int FN_, int FM_ = 2>
struct Tile {
  static constexpr int WAVES_N = WAVES_N_, WAVES_M = WAVES_M_, FN = FN_, FM = FM_;
  static constexpr int WAVES = WAVES_N * WAVES_M, NT = 64 * WAVES;
  static constexpr int TN = 32 * FN * WAVES_N, BM = 32 * FM * WAVES_M, BK = 64;
  static constexpr int NBW = TN / 16, NBX = BM / 16;            // 16-row blocks of one step
  static constexpr int NQ = (NBW + NBX + WAVES - 1) / WAVES;    // load instructions per wave and step
  // bytes per stage: the blocks at 1 KiB each (W first, then X), then the landing
  // place of the padding loads that even out the waves' counts; a fragment row's sums fit too
  static constexpr int STAGE = WAVES * NQ * 1024 > 128 * TN || WAVES > 1 ? WAVES * NQ * 1024 : 128 * TN;
};

__device__ __forceinline__ int swz4(int r, int c) { return c ^ ((r >> 2) & 3); }

struct Smem {
  int8_t *st0, *st1, *st2;
  float* xs;   // the tile's rows' scales
};

// Weight row r of a tile: which matrix, and the channel within the tile.
template <class T, int MATS>
__device__ __forceinline__ void row_of(int r, int& mat, int& ch) {
  constexpr int W = 32 * T::FN, H = T::FN / MATS;
  const int wave = r / W, i = r % W / 32, l = r % 32;
  mat = i / H;
  ch = wave * (W / MATS) + H * l + i % H;
}

template <class YT, int H>
__device__ __forceinline__ void put(YT* p, int live, bool vec, const float (&v)[H]) {
  if (vec && live >= H) {
    if constexpr (std::is_same<YT, float>::value) {
      if constexpr (H == 4) *reinterpret_cast<v4f*>(p) = v4f{v[0], v[1], v[2], v[3]};
      else if constexpr (H == 2) *reinterpret_cast<float2*>(p) = float2{v[0], v[1]};
      else p[0] = v[0];
    } else {
      uint16_t b[H];
#pragma unroll
      for (int i = 0; i < H; ++i) b[i] = from_float<YT>(v[i]).bits;
      if constexpr (H == 4)
        *reinterpret_cast<uint2*>(p) = uint2{b[0] | (uint32_t)b[1] << 16, b[2] | (uint32_t)b[3] << 16};
      else if constexpr (H == 2) *reinterpret_cast<uint32_t*>(p) = b[0] | (uint32_t)b[1] << 16;
      else p[0].bits = b[0];
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < H; ++i)
    if (i < live) p[i] = from_float<YT>(v[i]);
}

// Outputs of the tile's row m (row `at` of its sums, in the workgroup's order) from
// channel ch on, C of them.
template <int ACT, class YT, int MATS, int C>
__device__ __forceinline__ void finish(const ScaledArgs& a, int64_t m, int64_t ch, int live, bool vec, float xs,
                                       const int32_t (&sum)[MATS][C], const float (&ws)[MATS][C],
                                       const float (&bi)[MATS][C]) {
  float v[C];
#pragma unroll
  for (int i = 0; i < C; ++i) {
    v[i] = activate<ACT>(scaled(sum[0][i], xs, ws[0][i], bi[0][i]));
    if constexpr (MATS == 2) v[i] = v[i] * scaled(sum[MATS - 1][i], xs, ws[MATS - 1][i], bi[MATS - 1][i]);
  }
  if (m < a.M) put<YT, C>((YT*)a.y + m * a.N + ch, live, vec, v);
}

// The scales and biases of C channels from ch on.
template <int MATS, int C>
__device__ __forceinline__ void channels(const ScaledArgs& a, int64_t ch, int live, float (&ws)[MATS][C],
                                         float (&bi)[MATS][C]) {
#pragma unroll
  for (int q = 0; q < MATS; ++q)
#pragma unroll
    for (int i = 0; i < C; ++i) {
      ws[q][i] = i < live ? a.ws[q][ch + i] : 0.0f;
      bi[q][i] = i < live && a.bias[q] ? a.bias[q][ch + i] : 0.0f;
    }
}

// One tile of shape T: weight rows of the tile's TN / MATS channels from c0 on,
// rows bm0 .. of x.  SPLIT > 1: the tile is one wave's, and SPLIT waves take every SPLIT-th step
// of K, each with stages of its own; their sums meet in LDS.
template <class T, int MATS, class YT, int SPLIT>
__device__ __forceinline__ void scaled_tile(const ScaledArgs& a, const Smem& sm, int64_t c0, int64_t bm0) {
  constexpr int FN = T::FN, FM = T::FM, H = FN / MATS;
  constexpr int NR = FN + FM;   // fragment reads per slice
  constexpr int NP = FN * FM;   // products per slice
  constexpr int kReads = (NR + NP - 1) / NP;   // behind each product
  static_assert(SPLIT == 1 || T::WAVES == 1, "a split tile is one wave's");
  const int tid = threadIdx.x, lane = tid & 63;
  const int split = SPLIT > 1 ? __builtin_amdgcn_readfirstlane(tid >> 6) : 0;
  const int wave = SPLIT > 1 ? 0 : __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave / T::WAVES_M, wm = wave % T::WAVES_M;
  const int64_t M = a.M, N = a.N, K = a.K;
  const int steps = (int)((K + T::BK - 1) / T::BK);
  const int KT = (steps - split + SPLIT - 1) / SPLIT;   // this wave's: steps split, split + SPLIT, ..
  const int64_t k_first = (int64_t)split * T::BK;
  constexpr int64_t kStep = (int64_t)SPLIT * T::BK;
  const int wr0 = 32 * FN * wn, xr0 = 32 * FM * wm;
  const int lrow = lane & 31, kg = lane >> 5;

  // Load instruction q of this wave moves 16-row block wave * NQ + q of a step (W
  // blocks, X blocks, then padding: a repeat of the tile's first X rows).  Lane
  // l takes row l / 4 of the block and the chunk that belongs at chunk
  // position l % 4 of that LDS row.
  const int8_t* gb[T::NQ];
  uint32_t voff[T::NQ];
  const int br = lane >> 2, chunk = swz4(br, lane & 3);
  Static<0, T::NQ>::each([&](auto Q) {
    constexpr int q = decltype(Q)::value;
    const int blk = wave * T::NQ + q;
    if (blk < T::NBW) {
      int mat, ch, first;
      row_of<T, MATS>(16 * blk, mat, first);   // (a block's rows are of one matrix)
      row_of<T, MATS>(16 * blk + br, mat, ch);
      const int64_t n = c0 + ch < N ? c0 + ch : N - 1;
      gb[q] = (MATS == 2 && __builtin_amdgcn_readfirstlane(mat) ? a.w[MATS - 1] : a.w[0]) + c0 * K + k_first;
      voff[q] = (uint32_t)((n - c0) * K + 16 * chunk);
    } else {
      const int xb = blk < T::NBW + T::NBX ? blk - T::NBW : 0;
      const int64_t m = bm0 + 16 * xb + br;
      gb[q] = a.x + bm0 * K + k_first;
      voff[q] = (uint32_t)(((m < M ? m : M - 1) - bm0) * K + 16 * chunk);
    }
  });
  if (tid < T::BM) sm.xs[tid] = a.xs[bm0 + tid < M ? bm0 + tid : M - 1];

  auto stage = [&](auto SI) -> int8_t* {
    constexpr int si = decltype(SI)::value;
    if constexpr (si == 0) return sm.st0 + split * T::STAGE;
    else if constexpr (si == 1) return sm.st1 + split * T::STAGE;
    else return sm.st2 + split * T::STAGE;
  };
  const bool ragged = K % T::BK != 0 && split + (KT - 1) * SPLIT == steps - 1;   // the last step is this wave's
  const bool past = (int64_t)(steps - 1) * T::BK + 16 * chunk >= K;          // this lane's chunk of it
  auto issue = [&](int k, auto SI, auto END) {   // END: k may be the last step
    int8_t* d = stage(SI) + wave * T::NQ * 1024;
    if (decltype(END)::value && ragged && k == KT - 1) {
      Static<0, T::NQ>::each([&](auto Q) {
        constexpr int q = decltype(Q)::value;
        const int8_t* p = gb[q] + k * kStep + voff[q];
        __builtin_amdgcn_global_load_lds((const void*)(past ? g_zeros : p), Q8TA_LDS(d + q * 1024), 16, 0, 0);
      });
    } else {
      Static<0, T::NQ>::each([&](auto Q) {
        constexpr int q = decltype(Q)::value;
        __builtin_amdgcn_global_load_lds((const void*)(gb[q] + k * kStep + voff[q]),
                                         Q8TA_LDS(d + q * 1024), 16, 0, 0);
      });
    }
  };

  v16i acc[FN][FM];
  Static<0, FN>::each([&](auto I) {
    Static<0, FM>::each([&](auto J) { acc[decltype(I)::value][decltype(J)::value] = v16i{}; });
  });
  const int a_off = (wr0 + lrow) * T::BK;
  const int b_off = T::TN * T::BK + (xr0 + lrow) * T::BK;
  auto read_frag = [&](const int8_t* S, v4i (&af)[FN], v4i (&bf)[FM], auto KSI, auto R) {
    constexpr int ks = decltype(KSI)::value, r = decltype(R)::value;
    const int cpos = 16 * swz4(lrow, 2 * ks + kg);
    if constexpr (r < FN) af[r] = *reinterpret_cast<const v4i*>(S + a_off + r * 32 * T::BK + cpos);
    else bf[r - FN] = *reinterpret_cast<const v4i*>(S + b_off + (r - FN) * 32 * T::BK + cpos);
  };
  auto product = [&](const v4i (&af)[FN], const v4i (&bf)[FM], auto I, auto J) {
    constexpr int i = decltype(I)::value, j = decltype(J)::value;
    acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(bf[j], af[i], acc[i][j], 0, 0, 0);
  };
  constexpr std::integral_constant<int, 0> K0{};
  constexpr std::integral_constant<int, 1> K1{};

  // Step k, its slab in stage k % 3 and slice 0's fragments in registers: the
  // products of slice 0, each followed by a fragment read of slice 1; the wait
  // for this wave's part of step k + 1 and the barrier; the load of step k + 3 into the
  // stage that is free now; the products of slice 1, each followed by a
  // fragment read of step k + 1.
  v4i af[2][FN], bf[2][FM];
  auto body = [&](int k, auto SI, auto END) {
    constexpr int si = decltype(SI)::value;
    using SNX = std::integral_constant<int, (si + 1) % 3>;
    const int8_t* S = stage(SI);
    const int8_t* SN = stage(SNX{});
    Static<0, NP>::each([&](auto MI) {
      constexpr int m = decltype(MI)::value;
      product(af[0], bf[0], std::integral_constant<int, m / FM>{}, std::integral_constant<int, m % FM>{});
      Static<m * kReads, (m * kReads + kReads < NR ? m * kReads + kReads : NR)>::each(
          [&](auto R) { read_frag(S, af[1], bf[1], K1, R); });
      __builtin_amdgcn_sched_barrier(0);
    });
    __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0(T::NQ));
    if constexpr (SPLIT == 1) __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    issue(k + 3 < KT ? k + 3 : KT - 1, SI, END);
    __builtin_amdgcn_sched_barrier(0);
    Static<0, NP>::each([&](auto MI) {
      constexpr int m = decltype(MI)::value;
      product(af[1], bf[1], std::integral_constant<int, m / FM>{}, std::integral_constant<int, m % FM>{});
      Static<m * kReads, (m * kReads + kReads < NR ? m * kReads + kReads : NR)>::each(
          [&](auto R) { read_frag(SN, af[0], bf[0], K0, R); });
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  constexpr std::integral_constant<int, 0> S0{};
  constexpr std::integral_constant<int, 1> S1{};
  constexpr std::integral_constant<int, 2> S2{};
  constexpr std::true_type kEnd{};
  constexpr std::false_type kInner{};
  if (SPLIT == 1 || KT > 0) {
  issue(0, S0, kEnd);
  issue(KT > 1 ? 1 : 0, S1, kEnd);
  issue(KT > 2 ? 2 : KT - 1, S2, kEnd);
  __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0(2 * T::NQ));   // this wave's part of step 0
  if constexpr (SPLIT == 1) __builtin_amdgcn_s_barrier();
  Static<0, NR>::each([&](auto R) { read_frag(stage(S0), af[0], bf[0], K0, R); });
  // (the question for the last step has no place in the loop: 95 us became 105 with it)
  int k = 0;
  const int inner = ragged ? KT - 7 : KT - 3;
  for (; k <= inner; k += 3) {
    body(k, S0, kInner);
    body(k + 1, S1, kInner);
    body(k + 2, S2, kInner);
  }
  for (; k + 3 <= KT; k += 3) {
    body(k, S0, kEnd);
    body(k + 1, S1, kEnd);
    body(k + 2, S2, kEnd);
  }
  if (k < KT) body(k, S0, kEnd);
  if (k + 1 < KT) body(k + 1, S1, kEnd);
  }
  __builtin_amdgcn_s_waitcnt(0);
  YT* out = (YT*)a.y;
  if constexpr (SPLIT > 1) {
    // rows 32 j .. of this wave's sums into its part of stage j: [32][MATS][C]
    constexpr int C = T::TN / MATS;
    Static<0, FM>::each([&](auto J) {
      constexpr int j = decltype(J)::value;
      int32_t* to = reinterpret_cast<int32_t*>(stage(J));
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int row = 8 * (r / 4) + 4 * kg + r % 4;
#pragma unroll
        for (int i = 0; i < FN; ++i) to[row * T::TN + i / H * C + H * lrow + i % H] = acc[i][j][r];
      }
    });
    __syncthreads();
    constexpr int Q = C / 4;                        // groups of four channels
    constexpr int kRows = 64 * SPLIT / Q;           // rows of one pass
    const int64_t ch = c0 + 4 * (tid % Q);
    const int live = ch >= N ? 0 : (N - ch < 4 ? (int)(N - ch) : 4);
    const bool vec = N % 4 == 0 && ((uintptr_t)a.y & (4 * sizeof(YT) - 1)) == 0;
    float ws[MATS][4], bi[MATS][4];
    channels<MATS, 4>(a, ch, live, ws, bi);
    with_activation<MATS>(a.act, [&](auto ACT) {
#pragma unroll
      for (int u = 0; u < (T::BM + kRows - 1) / kRows; ++u) {
        const int row = tid / Q + kRows * u;
        if (row >= T::BM) break;
        const int8_t* from = row < 32 ? sm.st0 : sm.st1;
        int32_t sum[MATS][4] = {};
#pragma unroll
        for (int s = 0; s < SPLIT; ++s)
#pragma unroll
          for (int q = 0; q < MATS; ++q) {
            const v4i v = *reinterpret_cast<const v4i*>(
                from + s * T::STAGE + 4 * (row % 32 * T::TN + q * C + 4 * (tid % Q)));
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[q][i] += v[i];
          }
        finish<decltype(ACT)::value, YT, MATS, 4>(a, bm0 + row, ch, live, vec, sm.xs[row], sum, ws, bi);
      }
    });
    return;
  }
  __syncthreads();

  // lane l: channels ch .. ch + H - 1; register r of fragment (i, j): row xr0 +
  // 32 j + 8 (r / 4) + 4 (l / 32) + r % 4
  const int64_t ch = c0 + wn * (32 * FN / MATS) + H * lrow;
  const int live = ch >= N ? 0 : (N - ch < H ? (int)(N - ch) : H);
  const bool vec = N % H == 0 && ((uintptr_t)a.y & (H * sizeof(YT) - 1)) == 0;
  float ws[MATS][H], bi[MATS][H];
  channels<MATS, H>(a, ch, live, ws, bi);
  // a whole tile of fewer than 2^31 outputs: no bounds, wave-uniform row bases and one
  // 32-bit offset a lane
  const bool whole = vec && bm0 + T::BM <= M && c0 + T::TN / MATS <= N && M * N <= (int64_t)INT32_MAX;
  const uint32_t lane_off = (uint32_t)((bm0 + xr0 + 4 * kg) * N + ch);
  with_activation<MATS>(a.act, [&](auto ACT) {
  Static<0, FM>::each([&](auto J) {
    constexpr int j = decltype(J)::value;
    Static<0, 4>::each([&](auto G) {
      constexpr int g = decltype(G)::value;
      const int row = xr0 + 32 * j + 8 * g + 4 * kg;
      const v4f xs = *reinterpret_cast<const v4f*>(sm.xs + row);
      Static<0, 4>::each([&](auto R) {
        constexpr int r = decltype(R)::value;
        int32_t sum[MATS][H];
#pragma unroll
        for (int i = 0; i < FN; ++i) sum[i / H][i % H] = acc[i][j][4 * g + r];
        if (whole) {
          float v[H];
#pragma unroll
          for (int i = 0; i < H; ++i) {
            v[i] = activate<decltype(ACT)::value>(scaled(sum[0][i], xs[r], ws[0][i], bi[0][i]));
            if constexpr (MATS == 2) v[i] = v[i] * scaled(sum[MATS - 1][i], xs[r], ws[MATS - 1][i], bi[MATS - 1][i]);
          }
          put<YT, H>(out + (int64_t)(32 * j + 8 * g + r) * N + lane_off, H, true, v);
        } else {
          finish<decltype(ACT)::value, YT, MATS, H>(a, bm0 + row + r, ch, live, vec, xs[r], sum, ws, bi);
        }
      });
    });
  });
  });
}

// Workgroups below ta take tiles of shape TA (ma of them along M, M fastest), the
// rest tiles of shape TB from channel cb on: the columns left after whole rounds
// of TA tiles, in one launch.  Within each part the workgroups, which go
// round the 8 XCDs, are renumbered so that an XCD walks a contiguous run of tiles, which
// share slabs in its L2.
template <class TA, class TB, int MATS, class YT, int S = 1>
__global__ __launch_bounds__(TA::NT * S, 1) void k_gemm_scaled(ScaledArgs a, int ma, int ta, int mb, int tb,
                                                            int64_t cb) {
  static_assert(TA::NT == TB::NT, "one block size");
  constexpr int STAGE = TA::STAGE > TB::STAGE ? TA::STAGE : TB::STAGE;
  constexpr int BM = TA::BM > TB::BM ? TA::BM : TB::BM;
  __shared__ __attribute__((aligned(16))) int8_t st0[S * STAGE];
  __shared__ __attribute__((aligned(16))) int8_t st1[S * STAGE];
  __shared__ __attribute__((aligned(16))) int8_t st2[S * STAGE];
  __shared__ __attribute__((aligned(16))) float xs[BM];
  const Smem sm{st0, st1, st2, xs};
  auto remap = [](int b, int nt) {
    const int per = nt / 8;
    return b < per * 8 ? (b % 8) * per + (b / 8) : b;
  };
  const int b = blockIdx.x;
  if constexpr (!std::is_same<TA, TB>::value) {
    if (b < ta) {
      const int t = remap(b, ta);
      scaled_tile<TA, MATS, YT, S>(a, sm, (int64_t)(t / ma) * (TA::TN / MATS), (int64_t)(t % ma) * TA::BM);
      return;
    }
  }
  const int t = remap(b - ta, tb);
  scaled_tile<TB, MATS, YT, S>(a, sm, cb + (int64_t)(t / mb) * (TB::TN / MATS), (int64_t)(t % mb) * TB::BM);
}

using T256 = Tile<2, 4, 4>;   // 256 weight rows x 256 rows, waves of 128 x 64
using T128 = Tile<4, 2, 2>;   // 256 x 128, waves of 64 x 64
using T64 = Tile<2, 2, 2>;    // 128 x 128, four waves
using T32 = Tile<1, 1, 2>;    // 64 x 64, one wave, or four that share K
template <int MATS>
using T16 = Tile<1, 1, MATS, 1>;   // 32 channels x 32, eight waves (two matrices: six) that share K

// A launch has fewer than 2^32 threads: columns go in as many as it takes.
constexpr int64_t kMostTiles = (int64_t)1 << 21;

template <class T, int MATS, class YT, int S = 1>
hipError_t launch_one(const ScaledArgs& a, hipStream_t s) {
  constexpr int64_t C = T::TN / MATS;
  const int64_t m = (a.M + T::BM - 1) / T::BM, n = (a.N + C - 1) / C;
  const int64_t most = kMostTiles / m > 0 ? kMostTiles / m : 1;
  for (int64_t n0 = 0; n0 < n; n0 += most) {
    const int64_t part = n - n0 < most ? n - n0 : most;
    hipLaunchKernelGGL((k_gemm_scaled<T, T, MATS, YT, S>), dim3((unsigned)(m * part)), dim3(T::NT * S), 0, s, a, (int)m,
                       0, (int)m, (int)(m * part), n0 * C);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int MATS, class YT>
hipError_t launch_plan(const ScaledArgs& a, hipStream_t s) {
  switch (a.tile) {
    case kTile64Split: return launch_one<T32, MATS, YT, 4>(a, s);
    case kTile32Split: return launch_one<T16<MATS>, MATS, YT, MATS == 2 ? 6 : 8>(a, s);
    case kTile64: return launch_one<T32, MATS, YT>(a, s);
    case kTile128: return launch_one<T64, MATS, YT>(a, s);
    case kTile256x128: return launch_one<T128, MATS, YT>(a, s);
  }
  // Columns of whole tiles, then the others as 256 x 128 tiles, in the same launch: they start on
  // the CUs that the first whole tiles free.
  constexpr int64_t CN = T256::TN / MATS;
  static_assert(T128::TN == T256::TN, "one width");
  const int64_t ma = (a.M + T256::BM - 1) / T256::BM, mb = (a.M + T128::BM - 1) / T128::BM;
  const int64_t cols = a.columns, rest = (a.N + CN - 1) / CN - cols;
  if (rest == 0) return launch_one<T256, MATS, YT>(a, s);
  hipLaunchKernelGGL((k_gemm_scaled<T256, T128, MATS, YT>), dim3((unsigned)(ma * cols + mb * rest)),
                     dim3(T256::NT), 0, s, a, (int)ma, (int)(ma * cols), (int)mb, (int)(mb * rest), cols * CN);
  return hipGetLastError();
}

template <class YT>
hipError_t launch_mats(const ScaledArgs& a, hipStream_t s) {
  return a.mats == 2 ? launch_plan<2, YT>(a, s) : launch_plan<1, YT>(a, s);
}

}  // namespace
}  // namespace q8ta
