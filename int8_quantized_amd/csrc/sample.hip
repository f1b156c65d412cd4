// q8ta_sample: one token a row by temperature, top-k, top-p and min-p from a
// given random number.
//
// The kept tokens are a prefix of the row in the order of falling logits
// (equal ones by index), so they are given by a border, and no sort of the row is
// needed to find it.  Four short launches, the first three with as many
// workgroups a row as fill the card:
//  1. k_sample_max: the largest logit of each group of up to 64 neighbouring
//     loads.  Later readings skip the groups whose largest cannot matter.
//  2. k_sample_gather: where the prefix is short -- top-k up to 1024, or min-p --
//     the few tokens that can be in it: with top-k those at or above a bound that
//     k of the groups reach, with min-p those of about its weight.  With top-p
//     over the whole vocabulary, sums of weights in bins of 1/64 of a power of
//     two; with no filter, sums over stretches of 64 loads.
//  3. k_sample_border (top-p over the whole vocabulary): the bin in which the
//     border lies, its tokens, and the sums over stretches of those above it.
//  4. k_sample_pick, a workgroup a row: the collected tokens are sorted in LDS,
//     cut exactly in that order and drawn from in the order of their indices; with
//     sums over stretches the stretch is found, then the token inside it.
//  * What these do not take (more than 4096 tokens tied or collected, top-k
//    beyond 1024, a border below 2^-32 of the largest weight, infinite logits)
//    goes the slow way:
//    selection digit by digit of the key (the logit's bits in an
//    order-preserving form), on counts (top-k) and on sums of weights (top-p).
//
// Which token a random number meets depends on sums of up to vocab weights,
// and one weight's error can move a border or the token: weights are 64-bit
// (2^x by a polynomial, 4e-14 of the weight), and are added as whole numbers (a
// weight of 1 is 2^shift), which makes every sum exact and independent of the
// order in which lanes and atomics add.
//
// Measured (256 rows x 131072 fp32, each filter): the first reading 25 us (134 MB
// at 5.4 TB/s; a bare read of large buffers runs at 6.9); gathering 5 us greedy, 13
// top-k, 10 min-p, 50 where all weights are summed (21 instructions of 4 cycles a
// weight are 18 us of it), 69 for bins; the border 57; the pick 3 to 12.  24 x 100003
// bf16 by top-p: 4 + 12 + 13 + 16 us; 1 x 32000 with top-k 50: 3 + 9 + 2 + 4 us, a chain
// of latencies.
#include <cmath>

#include "decode.h"
#include "weights.h"

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

// The row's number: below 0 as 0 (no sum is below a negative goal); a NaN stays and
// passes no sum, as numbers from 1 on.
__device__ __forceinline__ double number_of(const SampleArgs& a, int row) {
  const float u = a.u[row];
  return u < 0.0f ? 0.0 : (double)u;
}

struct Row {
  double top, inv_t;   // largest logit, 1 / temperature
  double scale;        // log2(e) / temperature
  double one;          // 2^shift
};
__device__ __forceinline__ Row make_row(float top, float temp, int shift) {
  const double inv = temp > 0.0f ? 1.0 / (double)temp : 1.0;
  return Row{(double)top, inv, inv * 1.4426950408889634, __builtin_ldexp(1.0, shift)};
}

// exp((x - top) / T), 0 for -inf and 1 for the largest itself.
__device__ __forceinline__ double weight(const Row& r, float x) {
  const double y = ((double)x - r.top) * r.scale;
  const double w = exp2_of(y);
  return (double)x == r.top ? 1.0 : (x == -INFINITY ? 0.0 : w);
}
// Rounded to a whole number of 2^-shift: adding 2^52 leaves it in the low bits
// (shift <= 50, so it is below 2^51).
__device__ __forceinline__ u64 units(const Row& r, double w) {
  const double big = 4503599627370496.0;
  return __builtin_bit_cast(u64, __builtin_fma(w, r.one, big)) - __builtin_bit_cast(u64, big);
}

// The weight of a finite logit or -inf as a whole number of 2^-shift, where the
// row's largest logit is finite, in one straight line (a branch an element costs
// more than the weight): 2^shift goes on in the exponent, and y no lower than -8
// leaves 0 in any case.
struct UnitsOf {
  double top, scale, shift;
  __device__ __forceinline__ u64 operator()(float x) const {
    const double magic = 6755399441055744.0;   // 1.5 * 2^52: the sum's low word is the nearest whole number
    double y = __builtin_fma((double)x - top, scale, shift);
    y = __builtin_fmax(y, -8.0);               // (also for the NaN of -inf * 0)
    const double t = y + magic;
    const double f = y - (t - magic);
    const double q = __builtin_fma(exp2_poly(f), f, 1.0);
    const uint32_t n = (uint32_t)__builtin_bit_cast(u64, t);
    const u64 w = __builtin_bit_cast(u64, q) + ((u64)(n << 20) << 32);
    const double big = 4503599627370496.0;     // 2^52 leaves the rounded value in the low bits
    return __builtin_bit_cast(u64, __builtin_bit_cast(double, w) + big) - __builtin_bit_cast(u64, big);
  }
};
__device__ __forceinline__ UnitsOf units_of(const Row& r, int shift) {
  return UnitsOf{r.top, r.scale, (double)shift};
}

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

struct Shared {
  u64 hist[256];
  u64 sums[kWaves];
  int counts[kWaves];
  float tops[kWaves];
  uint32_t digit;
  u64 before;
};

// The slow way: any settings, any ties.  mx: the row's largest logit (not
// -inf).
template <class T>
__device__ void sample_any(const SampleArgs& a, Shared& sh, float mx) {
  u64(&hist)[256] = sh.hist;
  u64(&sums)[kWaves] = sh.sums;
  int(&counts)[kWaves] = sh.counts;
  uint32_t& sh_digit = sh.digit;
  u64& sh_before = sh.before;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int V = a.vocab;
  const T* row = (const T*)a.logits + (int64_t)blockIdx.x * a.row_stride;
  const float temp = a.temperature[blockIdx.x];
  const int k = a.top_k ? a.top_k[blockIdx.x] : 0;
  const float given_p = a.top_p ? a.top_p[blockIdx.x] : 1.0f;
  const float p = given_p > 0.0f ? given_p : 0.0f;   // (a NaN keeps the first token alone, as 0 does)
  const float mp = a.min_p ? a.min_p[blockIdx.x] : 0.0f;
  const bool greedy = !(temp > 0.0f);
  const uint32_t top_key = key_of(mx);
  const Row r = make_row(mx, temp, a.shift);

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
      goal = number_of(a, blockIdx.x) * (double)all;
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

// Largest of a block's values, in every thread.
template <int NW>
__device__ __forceinline__ float block_max(float v, float (&tops)[kWaves]) {
#pragma unroll
  for (int m = 32; m > 0; m /= 2) v = __builtin_fmaxf(v, __shfl_xor(v, m));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = v;
  __syncthreads();
  v = tops[0];
#pragma unroll
  for (int w = 1; w < NW; ++w) v = __builtin_fmaxf(v, tops[w]);
  return v;
}

// Sum of v over the threads before this one, and over all.
template <int NW>
__device__ __forceinline__ u64 block_scan(u64 v, u64 (&sums)[kWaves], u64& all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  u64 sum = v;
#pragma unroll
  for (int m = 1; m < 64; m *= 2) {
    const u64 o = __shfl_up(sum, m);
    if (lane >= m) sum += o;
  }
  __syncthreads();
  if (lane == 63) sums[wave] = sum;
  __syncthreads();
  u64 before = 0;
  all = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    before += w < wave ? sums[w] : 0;
    all += sums[w];
  }
  return before + sum - v;
}

constexpr int kCand = 4096;     // tokens that can be collected
constexpr int kBins = 2048;     // weight bins, 64 to a power of two
constexpr int kGroups = 4096;   // groups of loads, at most
constexpr int kCoarse = 64;     // sums of 32 neighbouring bins each
constexpr int kSlot = kBins + kCoarse;   // what a part leaves of them
constexpr int kSteps = 1024;    // steps between the groups' largest logits
constexpr int kBT = 256;        // threads of a part of a row
constexpr int kParts = 32;      // parts of a row, at most

// One 16-byte load of neighbouring elements, the load `at` of the row.  The
// row's last one ends with it: what it shares with the one before, and every
// element of a load that is not wanted, is -inf.
template <class T>
struct Vec {
  static constexpr int N = 16 / sizeof(T);
  typedef uint32_t raw_t __attribute__((ext_vector_type(4)));
  raw_t raw;
  int first;   // token of x[0]
  float x[N];
  // unconditional, so that several are in flight
  __device__ __forceinline__ void fetch(const T* row, int at, bool wanted, int V) {
    first = wanted ? at * N : 0;
    first = first < V - N ? first : V - N;
    if (first < 0) {   // V < N, every lane alike
      first = 0;
      raw = raw_t{0, 0, 0, 0};
#pragma unroll
      for (int e = 0; e < N; ++e) {
        if (e >= V) break;
        if constexpr (sizeof(T) == 4) raw[e] = __builtin_bit_cast(uint32_t, to_float(row[e]));
        else raw[e / 2] |= (uint32_t)row[e].bits << (16 * (e % 2));
      }
    } else {
      __builtin_memcpy(&raw, row + first, 16);   // rows start anywhere
    }
  }
  __device__ __forceinline__ void finish(int at, bool wanted, int V) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const uint32_t w = raw[e * sizeof(T) / 4];
      float y;
      if constexpr (sizeof(T) == 4) y = __builtin_bit_cast(float, w);
      else y = to_float(T{(uint16_t)(w >> (16 * (e % 2)))});
      x[e] = wanted && first + e >= at * N && first + e < V && y == y ? y : -INFINITY;
    }
  }
};

// How a row is divided, and its share of the workspace.
struct Plan {
  int loads;       // 16-byte loads of a row
  int group_log;   // log2 of the loads of a group
  int groups;
  int per, parts;  // loads of a thread of a part; parts of a row
  int stretches;   // of 64 loads
  // bytes from a row's share to ...
  int at_max, at_sums, at_bins, at_cand, row_bytes;
  char* ws;
};
struct State {
  int first;       // the first token of the largest logit
  int n_cand;      // tokens collected
  int cut_bin;
  float mx;
  u64 base;        // weight above the cut bin
  double goal;     // top-p's share of all weights
  u64 totals[kParts];
};
// Workgroup (x, part): all rows' first parts before the second ones, since some
// rows need fewer; the rows go round with the parts, so that a period of 8
// among the rows' settings does not leave them to one XCD.
__device__ __forceinline__ int row_of(int rows) {
  return (int)((blockIdx.x + blockIdx.y) % (unsigned)rows);
}
template <class P>
__device__ __forceinline__ P* share(const Plan& p, int row, int at) {
  return (P*)(p.ws + (int64_t)row * p.row_bytes + at);
}

enum Mode { kFirst, kFewK, kMinP, kTopP, kAll, kSlow };
struct Settings {
  float temp, p, mp;
  int k;
  Mode mode;
  bool cut_p, cut_m;
};
__device__ __forceinline__ Settings settings_of(const SampleArgs& a, int row) {
  Settings s;
  s.temp = a.temperature[row];
  s.k = a.top_k ? a.top_k[row] : 0;
  s.p = a.top_p ? a.top_p[row] : 1.0f;
  s.mp = a.min_p ? a.min_p[row] : 0.0f;
  s.cut_p = s.p < 1.0f;
  s.cut_m = s.mp > 0.0f;
  if (!(s.temp > 0.0f) || !(1.0f >= s.mp) || s.k == 1 || !(s.p > 0.0f)) s.mode = kFirst;
  else if (s.k > 0 && s.k < a.vocab) s.mode = s.k <= kSteps ? kFewK : kSlow;
  else s.mode = s.cut_m ? kMinP : (s.cut_p ? kTopP : kAll);
  return s;
}

__device__ __forceinline__ u64 place_of(float x, int token) {   // falls as the definition's order goes on
  return (u64)key_of(x) << 32 | (uint32_t)~(uint32_t)token;
}
__device__ __forceinline__ float value_of(u64 place) {
  const uint32_t key = (uint32_t)(place >> 32);
  return __builtin_bit_cast(float, key & 0x80000000u ? key & 0x7fffffffu : ~key);
}
__device__ __forceinline__ int token_of(u64 place) { return (int)~(uint32_t)place; }   // its low word

struct BinOf {
  float mx, per_bin;
  __device__ __forceinline__ int operator()(float x) const {
    const float at = (mx - x) * per_bin;   // inf * 0 and inf - inf: NaN, the last bin
    return x == mx ? 0 : (at < (float)(kBins - 1) ? (int)at : kBins - 1);
  }
};
__device__ __forceinline__ BinOf bins_of(const Row& r, float mx) {
  return BinOf{mx, (float)(r.scale * (kBins / 32))};
}

// f(load of the row, its values) for n loads, load_at(i) the i-th of this thread
// (-1: none, values of -inf), four in flight; every lane takes part in every one.
template <class T, class L, class F>
__device__ __forceinline__ void each_of(const SampleArgs& a, const T* row, int n, L&& load_at, F&& f) {
  for (int i = 0; i < n; i += 4) {
    Vec<T> v[4];
    int at[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      at[u] = i + u < n ? load_at(i + u) : -1;
      v[u].fetch(row, at[u], at[u] >= 0, a.vocab);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      v[u].finish(at[u], at[u] >= 0, a.vocab);
      if (i + u < n) f(at[u], v[u]);
    }
  }
}
// All loads of a part, in the row's order; the first of a wave's is a multiple of 64.
template <class T, class F>
__device__ __forceinline__ void each_load(const SampleArgs& a, const Plan& p, const T* row, F&& f) {
  const int first = blockIdx.y * p.per * kBT + threadIdx.x;
  each_of(a, row, p.per, [&](int i) { return first + i * kBT < p.loads ? first + i * kBT : -1; }, f);
}
// The loads of the listed groups, in any order.
template <class T, class F>
__device__ __forceinline__ void each_listed(const SampleArgs& a, const Plan& p, const T* row, const uint16_t* list,
                                            int n, F&& f) {
  const int all = n << p.group_log;
  each_of(a, row, (all + kBT - 1) / kBT,
          [&](int i) {
            const int q = i * kBT + (int)threadIdx.x;
            if (q >= all) return -1;
            const int at = ((int)list[q >> p.group_log] << p.group_log) + (q & ((1 << p.group_log) - 1));
            return at < p.loads ? at : -1;
          },
          f);
}

template <class T>
__global__ __launch_bounds__(kBT) void k_sample_max(SampleArgs a, Plan p) {
  const int row = row_of(a.rows);
  if (blockIdx.y == 0 && threadIdx.x == 0) {
    State* st = share<State>(p, row, 0);
    st->first = a.vocab;
    st->n_cand = 0;
    st->cut_bin = -1;
    st->mx = -INFINITY;
  }
  float* tops = share<float>(p, row, p.at_max);
  const int g = 1 << p.group_log;
  each_load(a, p, (const T*)a.logits + (int64_t)row * a.row_stride, [&](int at, const Vec<T>& v) {
    float m = v.x[0];
#pragma unroll
    for (int e = 1; e < Vec<T>::N; ++e) m = __builtin_fmaxf(m, v.x[e]);
    for (int x = 1; x < g; x *= 2) m = __builtin_fmaxf(m, __shfl_xor(m, x));
    if (at >= 0 && at % g == 0) tops[at >> p.group_log] = m;
  });
}

// Tokens that a part of a row collects: the first kLocal are handed on at once,
// any more one by one.  (More than kCand in all: the slow way.)
constexpr int kLocal = 1024;
struct Collected {
  u64 place[kLocal];
  int n, base;
};
__device__ __forceinline__ void append(Collected& c, State* st, u64* cand, float x, int token) {
  const int to = atomicAdd(&c.n, 1);
  if (to < kLocal) {
    c.place[to] = place_of(x, token);
  } else {
    const int at = atomicAdd(&st->n_cand, 1);
    if (at < kCand) cand[at] = place_of(x, token);
  }
}
__device__ __forceinline__ void hand_on(Collected& c, State* st, u64* cand) {
  __syncthreads();
  const int n = c.n < kLocal ? c.n : kLocal;
  if (n == 0) return;
  if (threadIdx.x == 0) c.base = atomicAdd(&st->n_cand, n);
  __syncthreads();
  const int base = c.base;
  for (int i = threadIdx.x; i < n; i += kBT)
    if (base + i < kCand) cand[base + i] = c.place[i];
}

template <class T>
__global__ __launch_bounds__(kBT) void k_sample_gather(SampleArgs a, Plan p) {
  constexpr int N = Vec<T>::N, NW = kBT / 64;
  __shared__ union {
    Collected c;
    u64 bins[kBins];
  } sh;
  __shared__ int steps[kSteps];
  __shared__ uint16_t list[kGroups];
  __shared__ int n_list;
  __shared__ u64 sums[kWaves];
  __shared__ float tops[kWaves];
  __shared__ int sh_last;
  const int tid = threadIdx.x, lane = tid & 63, row = row_of(a.rows), part = blockIdx.y;
  // where groups are picked out, as many parts as have something to do
  const Settings s = settings_of(a, row);
  const bool picks = s.mode == kFirst || s.mode == kFewK || (s.mode == kMinP && !s.cut_p);
  int parts = p.parts;
  if (picks) {
    const int some = s.mode == kFirst ? 1 : (s.mode == kFewK ? 1 + s.k / 128 : 4);
    parts = some < parts ? some : parts;
  }
  if (part >= parts) return;
  const T* logits = (const T*)a.logits + (int64_t)row * a.row_stride;
  const float* group = share<float>(p, row, p.at_max);
  State* st = share<State>(p, row, 0);
  u64* cand = share<u64>(p, row, p.at_cand);
  float g[kGroups / kBT], mine = -INFINITY;
#pragma unroll
  for (int i = 0; i < kGroups / kBT; ++i) {
    const int at = tid + i * kBT;
    g[i] = at < p.groups ? group[at] : -INFINITY;
    mine = __builtin_fmaxf(mine, g[i]);
  }
  if (tid == 0) {
    sh.c.n = 0;
    n_list = 0;
  }
  const float mx = block_max<NW>(mine, tops);
  if (part == 0 && tid == 0) st->mx = mx;
  if (mx == -INFINITY || s.mode == kSlow || (mx == INFINITY && s.mode != kFirst)) return;
  const Row r = make_row(mx, s.temp, a.shift);
  const UnitsOf un = units_of(r, a.shift);
  // the groups of this part's share whose largest logit passes, listed
  const int g0 = part * p.groups / parts, g1 = (part + 1) * p.groups / parts;
  auto list_groups = [&](auto&& passes) {
#pragma unroll
    for (int i = 0; i < kGroups / kBT; ++i) {
      const int at = tid + i * kBT;
      if (at >= g0 && at < g1 && passes(g[i])) list[atomicAdd(&n_list, 1)] = (uint16_t)at;
    }
    __syncthreads();
    return n_list;
  };

  if (s.mode == kFirst) {
    const int n = list_groups([&](float x) { return x == mx; });
    each_listed(a, p, logits, list, n, [&](int, const Vec<T>& v) {
      int first = a.vocab;
#pragma unroll
      for (int e = N - 1; e >= 0; --e) first = v.x[e] == mx ? v.first + e : first;
      if (first < a.vocab) atomicMin(&st->first, first);
    });
  } else if (s.mode == kFewK) {
    // a bound that k groups' largest logits reach: their places between the
    // smallest finite one and the row's, in steps
#pragma unroll
    for (int i = 0; i < kSteps / kBT; ++i) steps[tid + i * kBT] = 0;
    if (tid == 0) sh_last = -1;
    float least = INFINITY;
#pragma unroll
    for (int i = 0; i < kGroups / kBT; ++i) least = __builtin_fminf(least, g[i] == -INFINITY ? INFINITY : g[i]);
    const float low = -block_max<NW>(-least, tops);
    const float unit = mx > low ? (float)(kSteps - 1) / (mx - low) : 0.0f;
    auto step_of = [&](float x) {   // (fmax: 0 for the NaN of infinite logits)
      return (int)__builtin_fminf(__builtin_fmaxf((mx - x) * unit, 0.0f), (float)(kSteps - 1));
    };
#pragma unroll
    for (int i = 0; i < kGroups / kBT; ++i)
      if (g[i] != -INFINITY) atomicAdd(&steps[step_of(g[i])], 1);
    __syncthreads();
    constexpr int C = kSteps / kBT;
    int n[C], sum = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      n[c] = steps[C * tid + c];
      sum += n[c];
    }
    u64 all;
    int before = (int)block_scan<NW>((u64)sum, sums, all);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (before < s.k && before + n[c] >= s.k) sh_last = C * tid + c;
      before += n[c];
    }
    __syncthreads();
    const int last = sh_last;   // -1: fewer than k groups have a finite logit
    auto in = [&](float x) { return x != -INFINITY && (last < 0 || (x >= low && step_of(x) <= last)); };
    const int n_groups = list_groups(in);
    each_listed(a, p, logits, list, n_groups, [&](int, const Vec<T>& v) {
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (in(v.x[e])) append(sh.c, st, cand, v.x[e], v.first + e);
    });
    hand_on(sh.c, st, cand);
  } else if (s.mode == kMinP) {
    // a margin of 0.1 % for the 32-bit test; the weights decide later
    const float far = (float)(log((double)s.mp) / r.inv_t) * 1.001f - 1e-30f;
    auto in = [&](float x) { return x != -INFINITY && (x - mx >= far || x == mx); };
    u64 sum = 0;   // of all weights, where top-p needs it
    if (s.cut_p) {
      each_load(a, p, logits, [&](int, const Vec<T>& v) {
#pragma unroll
        for (int e = 0; e < N; ++e) sum += un(v.x[e]);
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (in(v.x[e])) append(sh.c, st, cand, v.x[e], v.first + e);
      });
    } else {
      const int n = list_groups(in);
      each_listed(a, p, logits, list, n, [&](int, const Vec<T>& v) {
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (in(v.x[e])) append(sh.c, st, cand, v.x[e], v.first + e);
      });
    }
    u64 all;
    block_scan<NW>(sum, sums, all);
    if (tid == 0) st->totals[part] = all;
    hand_on(sh.c, st, cand);
  } else if (s.mode == kTopP) {
    __syncthreads();
    for (int i = tid; i < kBins; i += kBT) sh.bins[i] = 0;
    __syncthreads();
    const BinOf bin = bins_of(r, mx);
    each_load(a, p, logits, [&](int, const Vec<T>& v) {
      u64 w[N];
#pragma unroll
      for (int e = 0; e < N; ++e) w[e] = un(v.x[e]);
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (w[e] > 0) atomicAdd(&sh.bins[bin(v.x[e])], w[e]);
    });
    __syncthreads();
    u64* out = share<u64>(p, row, p.at_bins) + part * kSlot;
    for (int i = tid; i < kBins; i += kBT) out[i] = sh.bins[i];
    u64 sum = 0;
#pragma unroll
    for (int i = 0; i < kBins / kBT; ++i) sum += sh.bins[kBins / kBT * tid + i];
    static_assert(kBT == 4 * kCoarse, "four threads a coarse sum");
    sum += __shfl_xor(sum, 1);
    sum += __shfl_xor(sum, 2);
    if (tid % 4 == 0) out[kBins + tid / 4] = sum;
  } else {
    u64* out = share<u64>(p, row, p.at_sums);
    each_load(a, p, logits, [&](int at, const Vec<T>& v) {
      u64 sum = 0;
#pragma unroll
      for (int e = 0; e < N; ++e) sum += un(v.x[e]);
      sum = wave_sum(sum);
      if (lane == 0 && at >= 0) out[at / 64] = sum;
    });
  }
}

template <class T>
__global__ __launch_bounds__(kBT) void k_sample_border(SampleArgs a, Plan p) {
  constexpr int N = Vec<T>::N;
  __shared__ Collected c;
  __shared__ u64 split[kBT];
  __shared__ int sh_bin;
  __shared__ u64 sh_base;
  __shared__ double sh_goal;
  const int tid = threadIdx.x, lane = tid & 63, row = row_of(a.rows), part = blockIdx.y;
  const Settings s = settings_of(a, row);
  State* st = share<State>(p, row, 0);
  const float mx = st->mx;
  if (s.mode != kTopP || !(__builtin_fabsf(mx) < INFINITY)) return;
  const Row r = make_row(mx, s.temp, a.shift);
  const UnitsOf un = units_of(r, a.shift);
  const u64* bins = share<u64>(p, row, p.at_bins);
  // sums over the parts of `of` neighbouring sums from `from` on, one a lane of
  // the first wave
  auto over_parts = [&](int from, int of) {
    const int i = tid & (of - 1);
    u64 n = 0;
#pragma unroll 4
    for (int q = tid / of; q < p.parts; q += kBT / of) n += bins[q * kSlot + from + i];
    __syncthreads();
    split[tid] = n;
    __syncthreads();
    n = 0;
    if (tid < of)
      for (int q = tid; q < kBT; q += of) n += split[q];
    return n;
  };
  // the sum in which the running one reaches the goal
  auto find = [&](u64 n, u64 base, bool known) {
    u64 upto = n;
#pragma unroll
    for (int m = 1; m < 64; m *= 2) {
      const u64 o = __shfl_up(upto, m);
      if (lane >= m) upto += o;
    }
    if (!known && lane == 63) sh_goal = (double)s.p * (double)upto;
    __builtin_amdgcn_wave_barrier();
    const double goal = known ? sh_goal : (double)s.p * (double)__shfl(upto, 63);
    upto += base;
    if (n > 0 && (double)(upto - n) < goal && !((double)upto < goal)) {
      sh_bin = lane;
      sh_base = upto - n;
    }
  };
  if (tid == 0) c.n = 0;
  const u64 coarse = over_parts(kBins, kCoarse);
  if (tid < 64) find(coarse, 0, false);
  __syncthreads();
  const int from = sh_bin * (kBins / kCoarse);
  const u64 fine = over_parts(from, kBins / kCoarse);
  if (tid < 64) find(fine, sh_base, true);
  __syncthreads();
  const int cut = from + sh_bin;
  if (part == 0 && tid == 0) {
    st->cut_bin = cut;
    st->base = sh_base;
    st->goal = sh_goal;
  }
  if (cut >= kBins - 1) return;
  const BinOf bin = bins_of(r, mx);
  u64* out = share<u64>(p, row, p.at_sums);
  u64* cand = share<u64>(p, row, p.at_cand);
  each_load(a, p, (const T*)a.logits + (int64_t)row * a.row_stride, [&](int at, const Vec<T>& v) {
    u64 w = 0;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const int b = v.x[e] == -INFINITY ? kBins : bin(v.x[e]);
      const u64 u = un(v.x[e]);
      w += b < cut ? u : 0;
      if (b == cut) append(c, st, cand, v.x[e], v.first + e);
    }
    w = wave_sum(w);
    if (lane == 0 && at >= 0) out[at / 64] = w;
  });
  hand_on(c, st, cand);
}

// Falling order of n different places.
__device__ __forceinline__ void sort_down(u64* place, int n) {
  if (n <= kNT) {   // each one's rank, counted by as many threads as there are to a place
    int share_log = 0;
    while (share_log < 5 && n << (share_log + 1) <= kNT) ++share_log;
    const int per = 1 << share_log;
    __syncthreads();
    const int i = threadIdx.x >> share_log;
    const u64 mine = i < n ? place[i] : 0;
    int rank = 0;
    if (i < n) {
#pragma unroll 4
      for (int j = threadIdx.x & (per - 1); j < n; j += per) rank += place[j] > mine;
    }
    for (int x = 1; x < per; x *= 2) rank += __shfl_xor(rank, x);
    __syncthreads();
    if (i < n && (threadIdx.x & (per - 1)) == 0) place[rank] = mine;
    __syncthreads();
    return;
  }
  int size = 64;
  while (size < n) size *= 2;
  __syncthreads();
  for (int i = n + threadIdx.x; i < size; i += kNT) place[i] = 0;
  for (int run = 2; run <= size; run *= 2)
    for (int step = run / 2; step > 0; step /= 2) {
      __syncthreads();
      for (int i = threadIdx.x; i < size / 2; i += kNT) {
        const int at = 2 * i - (i & (step - 1)), to = at + step;
        const u64 x = place[at], y = place[to];
        if ((x < y) == ((at & run) == 0)) {
          place[at] = y;
          place[to] = x;
        }
      }
    }
  __syncthreads();
}

template <class T>
__global__ __launch_bounds__(kNT) void k_sample_pick(SampleArgs a, Plan p) {
  constexpr int N = Vec<T>::N;
  __shared__ Shared sh;
  __shared__ u64 cand[kCand];
  __shared__ u64 wts[kCand];   // weights of the collected, or sums of the stretches
  __shared__ int sh_first;
  __shared__ u64 sh_base;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, row = blockIdx.x;
  const T* logits = (const T*)a.logits + (int64_t)row * a.row_stride;
  const State* st = share<State>(p, row, 0);
  const Settings s = settings_of(a, row);
  const float mx = st->mx;
  const int n_cand = st->n_cand;
  const double u = number_of(a, row);
  auto put = [&](int token, float logprob) {
    a.tokens[row] = token;
    if (a.logprobs) a.logprobs[row] = logprob;
  };
  if (mx == -INFINITY) {
    if (tid == 0) put(-1, -INFINITY);
    return;
  }
  if (s.mode == kFirst) {
    if (tid == 0) put(st->first, 0.0f);
    return;
  }
  if (s.mode == kSlow || mx == INFINITY || n_cand > kCand || (s.mode == kTopP && st->cut_bin >= kBins - 1)) {
    sample_any<T>(a, sh, mx);
    return;
  }
  const Row r = make_row(mx, s.temp, a.shift);
  const UnitsOf un = units_of(r, a.shift);
  auto log_prob = [&](float x, u64 all) {
    const double z = (double)x == r.top ? 0.0 : ((double)x - r.top) * r.inv_t;
    return (float)(z - log((double)all / r.one));
  };
  constexpr int C = kCand / kNT;
  u64 w[C], sum = 0, all;
  int n = n_cand;
  if (s.mode != kAll) {
    const u64* from = share<u64>(p, row, p.at_cand);
    for (int i = tid; i < n; i += kNT) cand[i] = from[i];
    sort_down(cand, n);
  }

  if (s.mode == kFewK || s.mode == kMinP) {
    u64 total = 0;   // of all weights, where top-k does not bound them
    if (s.mode == kFewK) n = n < s.k ? n : s.k;
    else if (s.cut_p) for (int i = 0; i < p.parts; ++i) total += st->totals[i];
    if (n <= 64) {   // a lane each
      if (wave != 0) return;
      const u64 mine = lane < n ? cand[lane] : 0;
      const double wd = lane < n ? weight(r, value_of(mine)) : 0.0;
      const u64 w1 = lane < n ? un(value_of(mine)) : 0;
      u64 upto = w1;
#pragma unroll
      for (int m = 1; m < 64; m *= 2) {
        const u64 o = __shfl_up(upto, m);
        if (lane >= m) upto += o;
      }
      const double goal = (double)s.p * (double)(s.mode == kFewK ? __shfl(upto, 63) : total);
      const bool in = lane < n && (lane == 0 || ((!s.cut_p || (double)(upto - w1) < goal) &&
                                                 (!s.cut_m || wd >= (double)s.mp)));
      const int m = __popcll(__ballot(in));
      all = __shfl(upto, m - 1);
      const double reach = u * (double)all;
      // in the order of the indices: the sum of the kept ones of no larger index
      const uint32_t low = (uint32_t)mine;
      wts[lane] = w1;
      __builtin_amdgcn_wave_barrier();
      u64 run = 0;
      for (int j = 0; j < m; ++j) run += (uint32_t)cand[j] >= low ? wts[j] : 0;
      if (in && w1 > 0 && ((double)run > reach ? !((double)(run - w1) > reach) : run == all))
        put(token_of(mine), log_prob(value_of(mine), all));
      return;
    }
    // weights in that order, four neighbours a thread; the prefix that stays
    double wd[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = C * tid + c;
      wd[c] = j < n ? weight(r, value_of(cand[j])) : 0.0;
      w[c] = j < n ? un(value_of(cand[j])) : 0;
      sum += w[c];
    }
    u64 before = block_scan<kWaves>(sum, sh.sums, all);
    const double goal = (double)s.p * (double)(s.mode == kFewK ? all : total);
    u64 kept = 0;   // kept tokens
    sum = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = C * tid + c;
      const bool in = j < n && (j == 0 || ((!s.cut_p || (double)before < goal) && (!s.cut_m || wd[c] >= (double)s.mp)));
      before += w[c];
      kept += in;
      if (in) sum += w[c];
      wts[j] = w[c];
    }
    u64 n_kept;
    block_scan<kWaves>(kept, sh.sums, n_kept);
    block_scan<kWaves>(sum, sh.sums, all);
    const int m = (int)n_kept;
    const double reach = u * (double)all;
    // In the order of the indices, the first whose running sum passes u * all,
    // else the last with a weight.
    if (m > 1024) {
      // sorted by index (low words fall as the index grows), places riding along
      u64 by_index[C];
#pragma unroll
      for (int c = 0; c < C; ++c) by_index[c] = C * tid + c < m ? cand[C * tid + c] << 32 | (uint32_t)(C * tid + c) : 0;
      __syncthreads();
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (C * tid + c < m) cand[C * tid + c] = by_index[c];
      sort_down(cand, m);
      sum = 0;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        w[c] = C * tid + c < m ? wts[(uint32_t)cand[C * tid + c]] : 0;
        sum += w[c];
      }
      u64 upto = block_scan<kWaves>(sum, sh.sums, all);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        upto += w[c];
        if (w[c] > 0 && ((double)upto > reach ? !((double)(upto - w[c]) > reach) : upto == all)) {
          const int token = token_of(cand[C * tid + c] >> 32);
          const float x = to_float(logits[token]);
          put(token, log_prob(x, all));
        }
      }
      return;
    }
    // by its running sum, which is that of the kept tokens of no larger index
    for (int i0 = 0; i0 < m; i0 += kNT / 2) {
      const int i = i0 + tid / 2;
      const uint32_t low = i < m ? (uint32_t)cand[i] : 0;
      u64 upto = 0;
      if (i < m)
        for (int j = tid % 2; j < m; j += 2) upto += (uint32_t)cand[j] >= low ? wts[j] : 0;
      upto += __shfl_xor(upto, 1);
      const u64 mine = i < m ? wts[i] : 0;
      if (tid % 2 == 0 && mine > 0 &&
          ((double)upto > reach ? !((double)(upto - mine) > reach) : upto == all))
        put(token_of(cand[i]), log_prob(value_of(cand[i]), all));
    }
    return;
  }

  // Sums over the stretches, in the vocabulary's order.
  u64 border = 0;   // tokens of the cut bin at or before this place are kept
  const int cut = s.mode == kTopP ? st->cut_bin : kBins;
  int n_kept = 0;
  if (s.mode == kTopP) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = C * tid + c;
      w[c] = j < n ? un(value_of(cand[j])) : 0;
      sum += w[c];
    }
    u64 in_bin;
    u64 at = st->base + block_scan<kWaves>(sum, sh.sums, in_bin);
    const double goal = st->goal;
    u64 kept = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      kept += C * tid + c < n && (double)at < goal;
      at += w[c];
    }
    u64 some;
    block_scan<kWaves>(kept, sh.sums, some);
    n_kept = (int)some;   // at least one: the running sum before the bin is below the goal
    border = cand[n_kept - 1];
  }
  const u64* from = share<u64>(p, row, p.at_sums);
  for (int i = tid; i < kCand; i += kNT) wts[i] = i < p.stretches ? from[i] : 0;
  __syncthreads();
  if (s.mode == kTopP) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = C * tid + c;
      if (j < n_kept && w[c] > 0) atomicAdd(&wts[token_of(cand[j]) / (64 * N)], w[c]);
    }
    __syncthreads();
  }
  sum = 0;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    w[c] = wts[C * tid + c];
    sum += w[c];
  }
  u64 before = block_scan<kWaves>(sum, sh.sums, all);
  const double reach = u * (double)all;
  if (tid == 0) sh_first = -1;
  __syncthreads();
  int hit = -1, some = -1;
  u64 upto = before;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    upto += w[c];
    if (w[c] > 0) {
      some = C * tid + c;
      if (hit < 0 && (double)upto > reach) hit = C * tid + c;
    }
  }
  // the first hit, else the last with a weight
  if (hit >= 0) atomicMax(&sh_first, 0x40000000 + (kCand - hit));
  else if (some >= 0) atomicMax(&sh_first, some);
  __syncthreads();
  const int found = sh_first;
  const int seg = found >= 0x40000000 ? kCand - (found - 0x40000000) : found;
  if (seg / C == tid) {
    u64 b = before;
#pragma unroll
    for (int c = 0; c < C; ++c) b += C * tid + c < seg ? w[c] : 0;
    sh_base = b;
  }
  __syncthreads();
  if (wave != 0) return;
  // one stretch: 64 loads, a lane each
  const BinOf bin = bins_of(r, mx);
  auto kept = [&](float x, int i) {
    if (x == -INFINITY) return false;
    if (s.mode == kAll) return true;
    const int b = bin(x);
    return b < cut || (b == cut && place_of(x, i) >= border);
  };
  Vec<T> v;
  const int load = seg * 64 + lane;
  v.fetch(logits, load, load < p.loads, a.vocab);
  v.finish(load, load < p.loads, a.vocab);
  const int at = v.first;
  u64 mass[N], lanes = 0;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    mass[e] = kept(v.x[e], at + e) ? un(v.x[e]) : 0;
    lanes += mass[e];
  }
  u64 run = lanes;
#pragma unroll
  for (int m = 1; m < 64; m *= 2) {
    const u64 o = __shfl_up(run, m);
    if (lane >= m) run += o;
  }
  run += sh_base - lanes;
  int token = -1, last = -1;
  float x = 0.0f, x_last = 0.0f;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    run += mass[e];
    if (mass[e] > 0) {
      last = at + e;
      x_last = v.x[e];
      if (token < 0 && (double)run > reach) {
        token = at + e;
        x = v.x[e];
      }
    }
  }
  const u64 hits = __ballot(token >= 0), somes = __ballot(last >= 0);
  const int who = hits ? __ffsll(hits) - 1 : 63 - __clzll(somes | 1);
  if (lane == who) put(hits ? token : last, log_prob(hits ? x : x_last, all));
}

// Vocabularies beyond the groups.
template <class T>
__global__ __launch_bounds__(kNT) void k_sample_long(SampleArgs a) {
  __shared__ Shared sh;
  const T* row = (const T*)a.logits + (int64_t)blockIdx.x * a.row_stride;
  float mx = -INFINITY;
  for (int i = threadIdx.x; i < a.vocab; i += kNT) mx = __builtin_fmaxf(mx, logit(row, i));
  mx = block_max<kWaves>(mx, sh.tops);
  if (mx == -INFINITY) {
    if (threadIdx.x == 0) {
      a.tokens[blockIdx.x] = -1;
      if (a.logprobs) a.logprobs[blockIdx.x] = -INFINITY;
    }
    return;
  }
  sample_any<T>(a, sh, mx);
}

constexpr int kBatch = 1024;   // rows of a launch, and bytes of its workspace (110 MB in whole MiB), at most
constexpr int kWorkspace = 104 << 20;

template <class T>
hipError_t launch_type(const SampleArgs& all, hipStream_t s) {
  constexpr int N = Vec<T>::N;
  Plan p{};
  p.loads = (all.vocab + N - 1) / N;
  while (((p.loads - 1) >> p.group_log) + 1 > kGroups) ++p.group_log;
  const bool is_long = p.group_log > 6;
  int batch = all.rows < kBatch ? all.rows : kBatch;
  void* ws = nullptr;
  if (!is_long) {
    p.groups = ((p.loads - 1) >> p.group_log) + 1;
    p.stretches = (p.loads + 63) / 64;
    // eight workgroups a CU (256 rows x 131072: 65 us, 71 with four, 99 with
    // two; 24 x 100003: 41 us with any)
    int parts = (2048 + batch - 1) / batch;
    parts = parts < kParts ? parts : kParts;
    p.per = (p.loads + kBT * parts - 1) / (kBT * parts);
    p.parts = (p.loads + kBT * p.per - 1) / (kBT * p.per);
    auto up = [](int bytes) { return (bytes + 255) / 256 * 256; };
    p.at_max = up((int)sizeof(State));
    p.at_sums = p.at_max + up(p.groups * 4);
    p.at_bins = p.at_sums + up(p.stretches * 8);
    p.at_cand = p.at_bins + p.parts * kSlot * 8;
    p.row_bytes = p.at_cand + kCand * 8;
    batch = batch < kWorkspace / p.row_bytes ? batch : kWorkspace / p.row_bytes;
    const hipError_t e = workspace_acquire(&ws, (size_t)batch * p.row_bytes, s);
    if (e != hipSuccess) return e;
    p.ws = (char*)ws;
  }
  hipError_t e = hipSuccess;
  for (int r0 = 0; r0 < all.rows && e == hipSuccess; r0 += batch) {
    SampleArgs a = all;
    a.rows = all.rows - r0 < batch ? all.rows - r0 : batch;
    a.logits = (const T*)all.logits + r0 * all.row_stride;
    a.temperature += r0;
    a.u += r0;
    a.tokens += r0;
    if (a.top_k) a.top_k += r0;
    if (a.top_p) a.top_p += r0;
    if (a.min_p) a.min_p += r0;
    if (a.logprobs) a.logprobs += r0;
    const dim3 rows((unsigned)a.rows), parts((unsigned)a.rows, (unsigned)p.parts), t(kNT), bt(kBT);
    if (is_long) {
      hipLaunchKernelGGL((k_sample_long<T>), rows, t, 0, s, a);
    } else {
      hipLaunchKernelGGL((k_sample_max<T>), parts, bt, 0, s, a, p);
      hipLaunchKernelGGL((k_sample_gather<T>), parts, bt, 0, s, a, p);
      if (a.top_p) hipLaunchKernelGGL((k_sample_border<T>), parts, bt, 0, s, a, p);
      hipLaunchKernelGGL((k_sample_pick<T>), rows, t, 0, s, a, p);
    }
    e = hipGetLastError();
  }
  if (ws) {
    const hipError_t f = workspace_release(ws, s);
    if (e == hipSuccess) e = f;
  }
  return e;
}

}  // namespace

hipError_t launch_sample(const SampleArgs& a, hipStream_t s) {
  switch (a.dtype) {
    case Q8TA_F32: return launch_type<float>(a, s);
    case Q8TA_F16: return launch_type<Half>(a, s);
    default: return launch_type<Bfloat>(a, s);
  }
}

}  // namespace q8ta
