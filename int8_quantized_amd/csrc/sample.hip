// q8ta_sample: one token a row by temperature, top-k, top-p and min-p from a
// given random number.
//
// The kept tokens are a prefix of the row in the order of falling logits
// (equal ones by index), so they are given by a border, and no sort of the row is
// needed to find it.  One workgroup of 16 waves a row:
//  * The largest logit, and each thread's own (first reading of the row).
//  * Where the prefix is short -- top-k up to 1024, or min-p -- the few tokens that
//    can be in it are collected (second reading): with top-k those at or above
//    a bound that k of the threads' own largest logits reach, with min-p those
//    of about its weight.  They are sorted in LDS, cut exactly in that order,
//    sorted by index and drawn from.
//  * Top-p over the whole vocabulary sums weights into bins of 1/64 of a
//    power of two, finds the bin in which the border lies, and collects, sorts
//    and cuts the tokens of that bin alone.
//  * There the token is found in the vocabulary's order by sums over stretches
//    of 64 lanes' elements (third reading), then inside one stretch.
//  * What these do not take (more than 4096 tokens tied or collected, top-k
//    beyond 1024, a border below 2^-32 of the largest weight) goes the slow way:
//    selection digit by digit of the key (the logit's bits in an
//    order-preserving form), on counts (top-k) and on sums of weights (top-p).
//
// Which token a random number meets depends on sums of up to vocab weights,
// and one weight's error can move a border or the token: weights are 64-bit
// (2^x by a polynomial, 4e-14 of the weight), and are added as whole numbers (a
// weight of 1 is 2^shift), which makes every sum exact and independent of the
// order in which lanes and atomics add.
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
  double scale;        // log2(e) / temperature
  double one;          // 2^shift
};
__device__ __forceinline__ Row make_row(float top, float temp, int shift) {
  const double inv = temp > 0.0f ? 1.0 / (double)temp : 1.0;
  return Row{(double)top, inv, inv * 1.4426950408889634, __builtin_ldexp(1.0, shift)};
}

// 2^y for y <= 0: 2^n times a polynomial in the rest f of [-1/2, 1/2], 1 + f * q(f)
// with q of degree 8 through (2^f - 1) / f at nine Chebyshev points (off by
// 4e-14 at most; exactly 1 for y = 0).
__device__ __forceinline__ double exp2_of(double y) {
  y = __builtin_fmax(y, -1100.0);
  const double n = __builtin_rint(y);
  const double f = y - n;
  double q = 0x1.b63880f16b7cap-24;
  q = __builtin_fma(q, f, 0x1.63d1363459636p-20);
  q = __builtin_fma(q, f, 0x1.ffcb95155d9ebp-17);
  q = __builtin_fma(q, f, 0x1.4308ac85ac57dp-13);
  q = __builtin_fma(q, f, 0x1.5d87fe86fe9e8p-10);
  q = __builtin_fma(q, f, 0x1.3b2ab7181b748p-7);
  q = __builtin_fma(q, f, 0x1.c6b08d7047e52p-5);
  q = __builtin_fma(q, f, 0x1.ebfbdff823cedp-3);
  q = __builtin_fma(q, f, 0x1.62e42fefa39efp-1);
  return __builtin_ldexp(__builtin_fma(q, f, 1.0), (int)n);
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

// Largest logit of a block's values, in every thread.
__device__ __forceinline__ float block_max(float v, Shared& sh) {
#pragma unroll
  for (int m = 32; m > 0; m /= 2) v = __builtin_fmaxf(v, __shfl_xor(v, m));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sh.tops[threadIdx.x >> 6] = v;
  __syncthreads();
  v = sh.tops[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) v = __builtin_fmaxf(v, sh.tops[w]);
  return v;
}

// Sum of v over the threads before this one, and over all.
__device__ __forceinline__ u64 block_scan(u64 v, Shared& sh, u64& all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  u64 sum = v;
#pragma unroll
  for (int m = 1; m < 64; m *= 2) {
    const u64 o = __shfl_up(sum, m);
    if (lane >= m) sum += o;
  }
  __syncthreads();
  if (lane == 63) sh.sums[wave] = sum;
  __syncthreads();
  u64 before = 0;
  all = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    before += w < wave ? sh.sums[w] : 0;
    all += sh.sums[w];
  }
  return before + sum - v;
}

// Falling order of n keys (a power of two of them, zeros behind the real ones).
__device__ __forceinline__ void sort_down(u64* key, int n) {
  for (int size = 2; size <= n; size *= 2)
    for (int step = size / 2; step > 0; step /= 2) {
      __syncthreads();
      for (int i = threadIdx.x; i < n / 2; i += kNT) {
        const int at = 2 * i - (i & (step - 1)), to = at + step;
        const u64 x = key[at], y = key[to];
        if ((x < y) == ((at & size) == 0)) {
          key[at] = y;
          key[to] = x;
        }
      }
    }
  __syncthreads();
}

constexpr int kCand = 4096;       // tokens that can be collected
constexpr int kBins = 2048;       // weight bins, 64 to a power of two
constexpr int kMaxRounds = 128;   // rounds of 1024 16-byte loads (vocab up to 2^19 fp32, 2^20 16-bit)

// One 16-byte load of elements, or fewer at the row's end (-inf behind it).
template <class T>
struct Vec {
  static constexpr int N = 16 / sizeof(T);
  float x[N];
  __device__ __forceinline__ void load(const T* row, int64_t at, int V) {
    typedef uint32_t raw_t __attribute__((ext_vector_type(4)));
    raw_t raw;
    if (at + N <= V) {
      __builtin_memcpy(&raw, row + at, 16);   // rows start anywhere
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const uint32_t w = raw[e * sizeof(T) / 4];
        if constexpr (sizeof(T) == 4) x[e] = __builtin_bit_cast(float, w);
        else x[e] = to_float(T{(uint16_t)(w >> (16 * (e % 2)))});
      }
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) x[e] = at + e < V ? to_float(row[at + e]) : -INFINITY;
    }
#pragma unroll
    for (int e = 0; e < N; ++e) x[e] = x[e] != x[e] ? -INFINITY : x[e];
  }
};

template <class T>
__global__ __launch_bounds__(kNT) void k_sample(SampleArgs a) {
  constexpr int N = Vec<T>::N;
  __shared__ Shared sh;
  __shared__ u64 cand[kCand];     // key << 32 | ~index, falling: the order of the definition
  __shared__ u64 wts[kCand];      // their weights; before that, the bins
  __shared__ int n_cand, sh_bin, sh_first;
  __shared__ u64 sh_base;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int V = a.vocab;
  const T* row = (const T*)a.logits + (int64_t)blockIdx.x * a.row_stride;
  const int rounds = (V + kNT * N - 1) / (kNT * N);
  // f(first element of the load, its N values, round) for every load of the
  // row, four in flight; every lane takes part in every one
  auto each = [&](auto&& f) {
    for (int i = 0; i < rounds; i += 4) {
      Vec<T> v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u].load(row, ((int64_t)(i + u) * kNT + tid) * N, V);
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (i + u < rounds) f(((i + u) * kNT + tid) * N, v[u], i + u);
    }
  };

  const float temp = a.temperature[blockIdx.x];
  const int k = a.top_k ? a.top_k[blockIdx.x] : 0;
  const float p = a.top_p ? a.top_p[blockIdx.x] : 1.0f;
  const float mp = a.min_p ? a.min_p[blockIdx.x] : 0.0f;
  const double u = (double)a.u[blockIdx.x];
  if (tid == 0) {
    n_cand = 0;
    sh_first = V;
  }
  float mine = -INFINITY;
  each([&](int, const Vec<T>& v, int) {
#pragma unroll
    for (int e = 0; e < N; ++e) mine = __builtin_fmaxf(mine, v.x[e]);
  });
  const float mx = block_max(mine, sh);
  auto put = [&](int token, float logprob) {
    a.tokens[blockIdx.x] = token;
    if (a.logprobs) a.logprobs[blockIdx.x] = logprob;
  };
  if (mx == -INFINITY) {
    if (tid == 0) put(-1, -INFINITY);
    return;
  }
  if (!(temp > 0.0f) || !(1.0f >= mp) || k == 1 || !(p > 0.0f)) {
    // the first token alone
    each([&](int at, const Vec<T>& v, int) {
      int first = V;
#pragma unroll
      for (int e = N - 1; e >= 0; --e) first = v.x[e] == mx ? at + e : first;
      if (first < V) atomicMin(&sh_first, first);
    });
    __syncthreads();
    if (tid == 0) put(sh_first, 0.0f);
    return;
  }
  const Row r = make_row(mx, temp, a.shift);
  const bool few_k = k > 0 && k < V && k <= 1024, all_k = k <= 0 || k >= V;
  const bool cut_p = p < 1.0f, cut_m = mp > 0.0f;
  if (!few_k && !all_k) {
    sample_any<T>(a, sh, mx);
    return;
  }
  auto log_prob = [&](float x, u64 all) {
    const double z = (double)x == r.top ? 0.0 : ((double)x - r.top) * r.inv_t;
    return (float)(z - log((double)all / r.one));
  };
  auto value_of = [](uint32_t key) {
    return __builtin_bit_cast(float, key & 0x80000000u ? key & 0x7fffffffu : ~key);
  };
  // Collects the tokens for which in(x) holds; false where they are too many.
  auto collect = [&](auto&& in) {
    each([&](int at, const Vec<T>& v, int) {
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (in(v.x[e])) {
          const int to = atomicAdd(&n_cand, 1);
          if (to < kCand) cand[to] = (u64)key_of(v.x[e]) << 32 | (uint32_t)~(uint32_t)(at + e);
        }
    });
    __syncthreads();
    return n_cand <= kCand;
  };
  auto pad_and_sort = [&](int n) {
    int size = 64;
    while (size < n) size *= 2;
    for (int i = n + tid; i < size; i += kNT) cand[i] = 0;
    sort_down(cand, size);
  };

  if (few_k || cut_m) {
    u64 total = 0;   // of all weights, where top-p needs it and top-k does not bound it
    bool ok;
    if (few_k) {
      // a bound that k threads' own largest logits reach: their places between
      // the smallest finite one and the row's, in 1024 steps
      int* steps = reinterpret_cast<int*>(wts);
      steps[tid] = 0;
      if (tid == 0) sh_bin = -1;
      const float low = -block_max(mine == -INFINITY ? -INFINITY : -mine, sh);
      const float unit = mx > low ? 1023.0f / (mx - low) : 0.0f;
      auto step_of = [&](float x) {   // (fmax: 0 for the NaN of infinite logits)
        return (int)__builtin_fminf(__builtin_fmaxf((mx - x) * unit, 0.0f), 1023.0f);
      };
      if (mine != -INFINITY) atomicAdd(&steps[step_of(mine)], 1);
      __syncthreads();
      u64 all;
      const u64 before = block_scan((u64)steps[tid], sh, all);
      if (before < (u64)k && before + steps[tid] >= (u64)k) sh_bin = tid;
      __syncthreads();
      const int last = sh_bin;   // -1: fewer than k threads have a finite logit
      __syncthreads();
      ok = collect([&](float x) {
        return x != -INFINITY && (last < 0 || (x >= low && step_of(x) <= last));
      });
    } else {
      if (cut_p) {
        u64 sum = 0;
        each([&](int, const Vec<T>& v, int) {
#pragma unroll
          for (int e = 0; e < N; ++e) sum += units(r, weight(r, v.x[e]));
        });
        block_scan(sum, sh, total);
      }
      // a margin of 0.1 % for the 32-bit test; the weights decide below
      const float far = (float)(log((double)mp) / r.inv_t) * 1.001f - 1e-30f;
      ok = collect([&](float x) { return x - mx >= far || x == mx; });
    }
    if (!ok) {
      sample_any<T>(a, sh, mx);
      return;
    }
    int n = n_cand;
    pad_and_sort(n);
    if (few_k && n > k) n = k;
    // weights in that order, four neighbours a thread; the prefix that stays
    constexpr int C = kCand / kNT;
    u64 w[C], sum = 0;
    double wd[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = C * tid + c;
      wd[c] = j < n ? weight(r, value_of((uint32_t)(cand[j] >> 32))) : 0.0;
      w[c] = units(r, wd[c]);
      sum += w[c];
    }
    u64 all;
    u64 before = block_scan(sum, sh, all);
    const double goal = (double)p * (double)(few_k ? all : total);
    int kept = 0;
    sum = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = C * tid + c;
      const bool in = j < n && (j == 0 || ((!cut_p || (double)before < goal) && (!cut_m || wd[c] >= (double)mp)));
      before += w[c];
      kept += in;
      if (in) sum += w[c];
      if (j < kCand) wts[j] = w[c];
    }
    u64 n_kept, kept_sum;
    block_scan((u64)kept, sh, n_kept);
    block_scan(sum, sh, kept_sum);
    // by index: ~index falls as the index grows; the place in the order above
    // rides along
    const int m = (int)n_kept;
    u64 by_index[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = C * tid + c;
      by_index[c] = j < m ? (cand[j] << 32) | (uint32_t)j : 0;
    }
    // the keys of the kept, before their places are overwritten
    __syncthreads();
    uint32_t keys[C];
#pragma unroll
    for (int c = 0; c < C; ++c) keys[c] = C * tid + c < m ? (uint32_t)(cand[C * tid + c] >> 32) : 0;
    __syncthreads();
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (C * tid + c < m) cand[C * tid + c] = by_index[c];
    pad_and_sort(m);
    sum = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = C * tid + c;
      w[c] = j < m ? wts[(uint32_t)cand[j]] : 0;
      sum += w[c];
    }
    before = block_scan(sum, sh, all);
    const double reach = u * (double)all;
    // the first whose running sum passes u * all, else the last with a weight
    if (tid == 0) sh_first = -1;
    __syncthreads();
    int hit = -1, some = -1;
#pragma unroll
    for (int c = C - 1; c >= 0; --c) {
      u64 upto = before;
#pragma unroll
      for (int d = 0; d <= c; ++d) upto += w[d];
      if (w[c] > 0) {
        some = some < 0 ? C * tid + c : some;
        if ((double)upto > reach) hit = C * tid + c;
      }
    }
    // smallest hit: hits are kept as ~place so that the maximum is the first
    if (hit >= 0) atomicMax(&sh_first, 0x40000000 + (kCand - hit));
    else if (some >= 0) atomicMax(&sh_first, some);
    __syncthreads();
    const int found = sh_first;
    const int place = found >= 0x40000000 ? kCand - (found - 0x40000000) : found;
    const u64 chosen = cand[place];
    const int j = (int)(uint32_t)chosen;
    if (j / C == tid)
      put((int)~(uint32_t)(chosen >> 32), log_prob(value_of(keys[j % C]), all));
    return;
  }

  // The whole vocabulary, cut by top-p at most.
  int cut_bin = kBins;             // bins below it are kept
  u64 border = 0;                  // of the cut bin: tokens of at least this key << 32 | ~index
  const float per_bin = (float)(r.scale * 64.0);
  auto bin_of = [&](float x) {
    const float at = (mx - x) * per_bin;   // inf * 0 and inf - inf: NaN, the last bin
    return x == mx ? 0 : (at < (float)(kBins - 1) ? (int)at : kBins - 1);
  };
  if (cut_p) {
    u64* bins = wts;
    for (int i = tid; i < kBins; i += kNT) bins[i] = 0;
    __syncthreads();
    each([&](int, const Vec<T>& v, int) {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const u64 w = units(r, weight(r, v.x[e]));
        if (w > 0) atomicAdd(&bins[bin_of(v.x[e])], w);
      }
    });
    __syncthreads();
    const u64 b0 = bins[2 * tid], b1 = bins[2 * tid + 1];
    u64 all;
    const u64 before = block_scan(b0 + b1, sh, all);
    const double goal = (double)p * (double)all;
    // the bin in which the running sum reaches the goal
    if (b0 > 0 && (double)before < goal && !((double)(before + b0) < goal)) {
      sh_bin = 2 * tid;
      sh_base = before;
    }
    if (b1 > 0 && (double)(before + b0) < goal && !((double)(before + b0 + b1) < goal)) {
      sh_bin = 2 * tid + 1;
      sh_base = before + b0;
    }
    __syncthreads();
    cut_bin = sh_bin;
    const u64 base = sh_base;
    if (cut_bin >= kBins - 1 || !collect([&](float x) { return x != -INFINITY && bin_of(x) == cut_bin; })) {
      sample_any<T>(a, sh, mx);
      return;
    }
    const int n = n_cand;
    pad_and_sort(n);
    constexpr int C = kCand / kNT;
    u64 w[C], sum = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = C * tid + c;
      w[c] = j < n ? units(r, weight(r, value_of((uint32_t)(cand[j] >> 32)))) : 0;
      sum += w[c];
    }
    u64 in_bin;
    u64 at = base + block_scan(sum, sh, in_bin);
    int kept = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      kept += C * tid + c < n && (double)at < goal;
      at += w[c];
    }
    u64 n_kept;
    block_scan((u64)kept, sh, n_kept);
    // at least one: the running sum before the bin is below the goal
    border = cand[(int)n_kept - 1];
    __syncthreads();
  }
  auto kept = [&](float x, int i) {
    if (!cut_p) return x != -INFINITY;
    const int b = bin_of(x);
    return x != -INFINITY &&
           (b < cut_bin || (b == cut_bin && ((u64)key_of(x) << 32 | (uint32_t)~(uint32_t)i) >= border));
  };
  // sums of the stretches (a wave's loads of one round), in the vocabulary's order
  u64* segs = wts;
  for (int i = tid; i < kMaxRounds * kWaves; i += kNT) segs[i] = 0;
  __syncthreads();
  each([&](int at, const Vec<T>& v, int round) {
    u64 s = 0;
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (kept(v.x[e], at + e)) s += units(r, weight(r, v.x[e]));
    s = wave_sum(s);
    if (lane == 0) segs[round * kWaves + wave] = s;
  });
  __syncthreads();
  constexpr int C = kMaxRounds * kWaves / kNT;
  u64 w[C], sum = 0, all;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    w[c] = segs[C * tid + c];
    sum += w[c];
  }
  u64 before = block_scan(sum, sh, all);
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
  if (hit >= 0) atomicMax(&sh_first, 0x40000000 + (kMaxRounds * kWaves - hit));
  else if (some >= 0) atomicMax(&sh_first, some);
  __syncthreads();
  const int found = sh_first;
  const int seg = found >= 0x40000000 ? kMaxRounds * kWaves - (found - 0x40000000) : found;
  if (seg / C == tid) {
    u64 b = before;
#pragma unroll
    for (int c = 0; c < C; ++c) b += C * tid + c < seg ? w[c] : 0;
    sh_base = b;
  }
  __syncthreads();
  if (wave != 0) return;
  // one stretch: 64 loads, a lane each
  Vec<T> v;
  const int at = (seg / kWaves * kNT + seg % kWaves * 64 + lane) * N;
  v.load(row, at, V);
  u64 mass[N], lanes = 0;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    mass[e] = kept(v.x[e], at + e) ? units(r, weight(r, v.x[e])) : 0;
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

// Vocabularies beyond k_sample's stretches.
template <class T>
__global__ __launch_bounds__(kNT) void k_sample_long(SampleArgs a) {
  __shared__ Shared sh;
  const T* row = (const T*)a.logits + (int64_t)blockIdx.x * a.row_stride;
  float mx = -INFINITY;
  for (int i = threadIdx.x; i < a.vocab; i += kNT) mx = __builtin_fmaxf(mx, logit(row, i));
  mx = block_max(mx, sh);
  if (mx == -INFINITY) {
    if (threadIdx.x == 0) {
      a.tokens[blockIdx.x] = -1;
      if (a.logprobs) a.logprobs[blockIdx.x] = -INFINITY;
    }
    return;
  }
  sample_any<T>(a, sh, mx);
}

template <class T>
hipError_t launch_type(const SampleArgs& a, hipStream_t s) {
  const dim3 g((unsigned)a.rows), t(kNT);
  if (a.vocab <= kMaxRounds * kNT * Vec<T>::N) hipLaunchKernelGGL((k_sample<T>), g, t, 0, s, a);
  else hipLaunchKernelGGL((k_sample_long<T>), g, t, 0, s, a);
  return hipGetLastError();
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
