// q8ta_sample: one token a row by temperature, top-k, top-p and min-p from a
// given random number.
//
// The kept tokens are a prefix of the row in the order of falling logits
// (equal ones by index), so they are given by a border: a key (the logit's
// bits in an order-preserving form) and how many of the tokens with that very
// key are kept, lowest indices first.  No sort is needed: the border is found
// by selection, digit by digit of the key, on counts (top-k) and on sums of
// weights (top-p).
//
// Which token a random number meets depends on sums of up to vocab weights,
// and one weight's error can move a border or the token: weights are exp in 64
// bits, and are added as whole numbers (a weight of 1 is 2^shift), which makes
// every sum exact and independent of the order in which lanes and atomics add.
#include <cmath>

#include "decode.h"

namespace q8ta {
namespace {

constexpr int kNT = 1024;
constexpr int kWaves = kNT / 64;
typedef unsigned long long u64;

// Order-preserving: larger floats have larger keys; -0 and +0 have one key.
__device__ __forceinline__ uint32_t key_of(float x) {
  uint32_t b = __builtin_bit_cast(uint32_t, x + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

template <class T>
__device__ __forceinline__ float logit(const T* row, int i) {
  const float x = to_float(row[i]);
  return x != x ? -INFINITY : x;
}

struct Row {
  double top, inv_t;   // largest logit, 1 / temperature
  double one;          // 2^shift
};

// exp((x - top) / T), 0 for -inf and 1 for the largest itself.
__device__ __forceinline__ double weight(const Row& r, float x) {
  const double d = (double)x == r.top ? 0.0 : ((double)x - r.top) * r.inv_t;
  return x == -INFINITY ? 0.0 : exp(d);
}
__device__ __forceinline__ u64 units(const Row& r, double w) { return (u64)__builtin_rint(w * r.one); }

template <class V>
__device__ __forceinline__ V wave_sum(V v) {
#pragma unroll
  for (int m = 32; m > 0; m /= 2) v += __shfl_xor(v, m);
  return v;
}

// The border of the kept tokens: keys above `key`, and the first `ties` tokens
// that have it.
struct Border {
  uint32_t key;
  int64_t ties;
};

template <class T>
__global__ __launch_bounds__(kNT) void k_sample_any(SampleArgs a) {
  __shared__ u64 hist[256];
  __shared__ u64 sums[kWaves];
  __shared__ int counts[kWaves];
  __shared__ float tops[kWaves];
  __shared__ uint32_t sh_digit;
  __shared__ u64 sh_before;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int V = a.vocab;
  const T* row = (const T*)a.logits + (int64_t)blockIdx.x * a.row_stride;

  float mx = -INFINITY;
  for (int i = tid; i < V; i += kNT) mx = __builtin_fmaxf(mx, logit(row, i));
#pragma unroll
  for (int m = 32; m > 0; m /= 2) mx = __builtin_fmaxf(mx, __shfl_xor(mx, m));
  if (lane == 0) tops[wave] = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWaves; ++w) mx = __builtin_fmaxf(mx, tops[w]);
  if (mx == -INFINITY) {
    if (tid == 0) {
      a.tokens[blockIdx.x] = -1;
      if (a.logprobs) a.logprobs[blockIdx.x] = -INFINITY;
    }
    return;
  }
  const float temp = a.temperature[blockIdx.x];
  const int k = a.top_k ? a.top_k[blockIdx.x] : 0;
  const float p = a.top_p ? a.top_p[blockIdx.x] : 1.0f;
  const float mp = a.min_p ? a.min_p[blockIdx.x] : 0.0f;
  const bool greedy = !(temp > 0.0f);
  const uint32_t top_key = key_of(mx);
  const Row r{(double)mx, greedy ? 1.0 : 1.0 / (double)temp, __builtin_ldexp(1.0, a.shift)};

  // Tokens of `in`, by digits of their keys from the top: finds the key at
  // which the running sum of amount(x) (in the order of falling keys) passes
  // `goal`, and the sum before that key.
  auto select = [&](auto&& in, auto&& amount, auto&& passes, u64& before) -> uint32_t {
    uint32_t key = 0;
    u64 base = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      const uint32_t high = shift == 24 ? 0u : ~0u << (shift + 8);
      for (int i = tid; i < V; i += kNT) {
        const float x = logit(row, i);
        const uint32_t kx = key_of(x);
        if ((kx & high) == (key & high) && in(kx)) atomicAdd(&hist[(kx >> shift) & 255], (u64)amount(x));
      }
      __syncthreads();
      if (tid == 0) {
        u64 sum = base;
        int d = 255, last = -1;
        u64 last_sum = base;
        for (; d >= 0; --d) {
          if (hist[d] == 0) continue;
          last = d;
          last_sum = sum;
          if (passes(sum + hist[d])) break;
          sum += hist[d];
        }
        sh_digit = (uint32_t)(last < 0 ? 0 : last);
        sh_before = last_sum;
      }
      __syncthreads();
      key |= sh_digit << shift;
      base = sh_before;
      __syncthreads();
    }
    before = base;
    return key;
  };

  Border cut{0u, INT64_MAX};   // everything
  if (greedy || !(1.0f >= mp)) {
    cut = Border{top_key, 1};
  } else {
    if (k > 0 && k < V) {
      u64 before;
      cut.key = select([](uint32_t) { return true; }, [](float) { return 1; },
                       [&](u64 c) { return c >= (u64)k; }, before);
      cut.ties = k - (int64_t)before;
    }
    if (!(p >= 1.0f)) {
      // weight of the first k tokens
      u64 s = 0;
      int t = 0;
      float xt = 0.0f;
      for (int i = tid; i < V; i += kNT) {
        const float x = logit(row, i);
        const uint32_t kx = key_of(x);
        if (kx > cut.key) s += units(r, weight(r, x));
        if (kx == cut.key) {
          ++t;
          xt = x;
        }
      }
      const u64 wt = t ? units(r, weight(r, xt)) : 0;   // one weight for all of that key
      s = wave_sum(s);
      u64 tie = wt;
#pragma unroll
      for (int m = 32; m > 0; m /= 2) {
        const u64 o = __shfl_xor(tie, m);
        tie = tie > o ? tie : o;
      }
      t = wave_sum(t);
      __syncthreads();
      if (lane == 0) {
        sums[wave] = s;
        counts[wave] = t;
        hist[wave] = tie;
      }
      __syncthreads();
      u64 total = 0, w_tie = 0;
      int64_t n_tie = 0;
      for (int w = 0; w < kWaves; ++w) {
        total += sums[w];
        n_tie += counts[w];
        w_tie = hist[w] > w_tie ? hist[w] : w_tie;
      }
      total += (u64)(n_tie < cut.ties ? n_tie : cut.ties) * w_tie;
      __syncthreads();
      const double goal = (double)p * (double)total;
      // the first token whose sum of weights before it reaches the goal is out
      u64 before;
      const uint32_t key_k = cut.key;
      const uint32_t key = select([&](uint32_t kx) { return kx >= key_k; },
                                  [&](float x) { return units(r, weight(r, x)); },
                                  [&](u64 c) { return (double)c >= goal; }, before);
      float x = 0.0f;   // back from the key
      const uint32_t bits = key & 0x80000000u ? key & 0x7fffffffu : ~key;
      x = __builtin_bit_cast(float, bits);
      const u64 w = units(r, weight(r, x));
      // ties kept: the j with before + j * w < goal
      int64_t keep = INT64_MAX;
      if (w > 0) {
        const double left = (goal - (double)before) / (double)w;
        keep = left <= 0.0 ? 0 : (int64_t)__builtin_ceil(left);
        while (keep > 0 && !((double)(before + (u64)(keep - 1) * w) < goal)) --keep;
        while ((double)(before + (u64)keep * w) < goal) ++keep;
      }
      if (key > key_k) cut = Border{key, keep};
      else if (keep < cut.ties) cut.ties = keep;
      if (cut.key == top_key && cut.ties < 1) cut.ties = 1;
    }
  }

  // In the vocabulary's order: sixteen stretches, one a wave, then sixteen of
  // the stretch that holds the token, until one is a wave's.  above / ties:
  // weight of the keys above the border, tokens at it.
  const bool has_min = !greedy && mp > 0.0f && 1.0f >= mp;
  auto kept = [&](float x, uint32_t kx, bool& tie) -> u64 {
    tie = false;
    if (kx < cut.key) return 0;
    const double w = greedy ? 1.0 : weight(r, x);
    if (has_min && !(w >= (double)mp)) return 0;
    tie = kx == cut.key;
    return units(r, w);
  };
  int lo = 0, len = V;
  u64 base = 0;               // weight before the stretch
  int64_t ties = cut.ties;    // ties still to keep
  double goal = -1.0;
  u64 all = 0;
  while (true) {
    const int step = len <= 64 ? 64 : ((len + kWaves - 1) / kWaves + 63) / 64 * 64;
    const int s0 = lo + wave * step;
    const int s1 = s0 + step < lo + len ? s0 + step : lo + len;
    u64 above = 0, w_tie = 0;
    int n_tie = 0;
    for (int i = s0 + lane; i < s1; i += 64) {
      const float x = logit(row, i);
      bool tie;
      const u64 w = kept(x, key_of(x), tie);
      if (tie) {
        ++n_tie;
        w_tie = w;
      } else {
        above += w;
      }
    }
    const u64 above_l = above;
    const int tie_l = n_tie;
    const u64 wt_l = w_tie;
    above = wave_sum(above);
    n_tie = wave_sum(n_tie);
#pragma unroll
    for (int m = 32; m > 0; m /= 2) {
      const u64 o = __shfl_xor(w_tie, m);
      w_tie = w_tie > o ? w_tie : o;
    }
    __syncthreads();
    if (lane == 0) {
      sums[wave] = above;
      counts[wave] = n_tie;
      hist[wave] = w_tie;
    }
    __syncthreads();
    // every thread the same walk over the stretches
    auto mass = [&](int w, int64_t left) {
      const int64_t n = counts[w] < left ? counts[w] : left;
      return sums[w] + (u64)n * hist[w];
    };
    if (goal < 0.0) {
      int64_t left = ties;
      for (int w = 0; w < kWaves; ++w) {
        all += mass(w, left);
        left -= counts[w] < left ? counts[w] : left;
      }
      goal = (double)a.u[blockIdx.x] * (double)all;
    }
    int pick = -1;
    u64 pick_base = base, run = base;
    int64_t pick_ties = ties, left = ties;
    for (int w = 0; w < kWaves; ++w) {
      const u64 q = mass(w, left);
      if (q > 0) {
        pick = w;
        pick_base = run;
        pick_ties = left;
        if ((double)(run + q) > goal) break;
      }
      run += q;
      left -= counts[w] < left ? counts[w] : left;
    }
    if (pick < 0) pick = 0;
    base = pick_base;
    ties = pick_ties;
    if (step == 64) {
      if (wave == pick) {
        // one token a lane: running sums over the lanes
        int64_t rank = tie_l;
#pragma unroll
        for (int m = 1; m < 64; m *= 2) {
          const int64_t o = __shfl_up(rank, m);
          if (lane >= m) rank += o;
        }
        const u64 mine = tie_l ? (rank <= ties ? wt_l : 0) : above_l;
        u64 sum = mine;
#pragma unroll
        for (int m = 1; m < 64; m *= 2) {
          const u64 o = __shfl_up(sum, m);
          if (lane >= m) sum += o;
        }
        const u64 hit = __ballot(mine > 0 && (double)(base + sum) > goal);
        const u64 some = __ballot(mine > 0);
        const int at = hit ? __ffsll(hit) - 1 : 63 - __clzll(some | 1);
        if (lane == at) {
          const int token = lo + pick * 64 + lane;
          a.tokens[blockIdx.x] = token;
          if (a.logprobs) {
            const float x = logit(row, token);
            const double z = greedy || (double)x == r.top ? 0.0 : ((double)x - r.top) * r.inv_t;
            a.logprobs[blockIdx.x] = greedy ? 0.0f : (float)(z - log((double)all / r.one));
          }
        }
      }
      return;
    }
    const int end = lo + len;
    lo += pick * step;
    len = step < end - lo ? step : end - lo;
    __syncthreads();
  }
}

}  // namespace

hipError_t launch_sample(const SampleArgs& a, hipStream_t s) {
  const dim3 g((unsigned)a.rows), t(kNT);
  switch (a.dtype) {
    case Q8TA_F32: hipLaunchKernelGGL((k_sample_any<float>), g, t, 0, s, a); break;
    case Q8TA_F16: hipLaunchKernelGGL((k_sample_any<Half>), g, t, 0, s, a); break;
    default: hipLaunchKernelGGL((k_sample_any<Bfloat>), g, t, 0, s, a); break;
  }
  return hipGetLastError();
}

}  // namespace q8ta
