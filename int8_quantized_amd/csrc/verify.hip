// q8ta_verify_drafts: which drafted tokens the target keeps, and the token that
// follows them.
//
//   p = softmax(logits / T) of each node; at the current node, children in order:
//   deterministic drafts:  c is kept if u_c * left < p(c); else p(c) leaves `left`
//   drafts drawn from q:   c is kept if u_c * q(c) < p(c); else what is left is
//                          max(p - q, 0)
//   the next token: the first index where the running sum of what is left at the
//   last kept node passes u_0 times its total
//
// Three launches:
//  1. k_verify_stats: every node's logits once (and the drafter's), in chunks of
//     4096: largest value, its first index, sum of weights relative to it.  All nodes,
//     since which are reached is not known before.
//  2. k_verify_walk: a workgroup for each chunk of the last node's row: the walk
//     first, each for itself (a lane holds a node; all that it may need is loaded
//     at once), then the chunk's sum of what is left.
//  3. k_verify_pick: a workgroup a request finds the chunk, then the token in it.
//
// The weights that the next token is drawn from, and each drafted token's own, are 64-bit
// (2^x by a polynomial, 4e-14 of the weight).  The sums that these are divided by, of
// which every node has one, take the weights below a quarter of their chunk's largest in
// 32 bits, sixteen of them added in 32.  Such a weight is off by 2^-23 of itself and by
// 0.7 * 2^-23 for each power of two that it is below the largest, of which a chunk of 4096 has
// at most twelve on average, and equal logits are off the same way: a sum by up to 2^-19
// of itself (131072 logits of two values: 3e-7 measured), and by some 1e-8 where its logits are
// spread.  The shares p, q and what is left of 1 after rejected brothers take that over,
// p - q too: a random number that falls between the two borders, at worst once in 5e5 tests,
// decides otherwise.  (64-bit weights throughout took 41 us in place of 30, below.)
// All is added in one fixed order, so that a result does not depend on what else is
// in the batch.
//
// Measured: 16 trees of 24 nodes over 131072 bf16 logits, 28 + 9.5 + 7 us.  The first
// launch reads 101 MB at 3.6 TB/s; the vector instructions bound it (18 for a logit, busy
// nine tenths of the time; all weights in 64 bits took 41 us, a loop without the
// question for large weights, taken by waves that have none, 30 in place of 32).  A chain
// of 5 over 32000 fp32 logits with its drafter's, 4 + 10 + 6.7 us: latencies, of which the
// launches are a third.
#include <cmath>

#include "decode.h"
#include "weights.h"

namespace q8ta {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

constexpr int kChunk = 4096;
// of a chunk, in the statistics: 16 a thread, for the loads; in the sums of what is left 8,
// for the time that 64-bit weights take (the last two launches: a chain of 5 with drafter's
// rows of 32000 16.8 us, 16 a thread 19.3, 4 a thread 18.5; 16 trees of 24 16.7, 17.2, 23)
constexpr int kPer = 16, kNT = kChunk / kPer, kWaves = kNT / 64;
constexpr int kFew = 8, kMany = kChunk / kFew, kManyWaves = kMany / 64;
constexpr int kParts = 4;   // waves that share a node's chunks in the walk
constexpr float kLarge = -2.0f;   // log2 of the weight from which one is formed in 64 bits

struct Stat {
  float top;     // largest logit of the chunk, -inf where there is none
  int32_t at;    // its first index in the row
  double sum;    // of weights relative to it
};
// The last node of a request and what is left there.
struct Last {
  int32_t node, mode, rejected;   // mode: kDone, kWhole, kLess or kResidual
  float top, draft_top;
  double z, draft_z;              // sums of weights, relative to the tops
  int32_t ids[64];                // kLess: the rejected tokens
};
enum { kDone, kWhole, kLess, kResidual };

struct Plan {
  VerifyArgs v;
  int chunks, rows;               // chunks of a row; rows of a request: tokens, then tokens - 1 drafter's
  int b0;                         // first request of this launch
  Stat* stats;                    // [requests of the launch, rows, chunks]
  double* sums;                   // [requests, chunks]
  Last* last;                     // [requests]
};

template <class T>
__device__ __forceinline__ const T* row_of(const VerifyArgs& v, int b, int row) {
  return row < v.tokens ? (const T*)v.logits + b * v.bs + row * v.ts
                        : (const T*)v.draft + b * v.dbs + (row - v.tokens) * v.dts;
}
__device__ __forceinline__ float no_nan(float x) { return x != x ? -INFINITY : x; }

// This thread's P neighbouring logits of a chunk, -inf past the vocabulary.
template <bool VEC, int P>
__device__ __forceinline__ void load(const float* row, int i0, int vocab, float (&x)[P]) {
  if (VEC && i0 + P <= vocab) {
#pragma unroll
    for (int j = 0; j < P / 4; ++j) {
      const v4f v = *reinterpret_cast<const v4f*>(row + i0 + 4 * j);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[4 * j + i] = v[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < P; ++i) x[i] = i0 + i < vocab ? row[i0 + i] : -INFINITY;
  }
}
template <bool VEC, int P, class T>
__device__ __forceinline__ void load(const T* row, int i0, int vocab, float (&x)[P]) {
  typedef uint32_t V __attribute__((ext_vector_type(P < 8 ? P / 2 : 4)));
  constexpr int E = P < 8 ? P : 8;
  if (VEC && i0 + P <= vocab) {
#pragma unroll
    for (int j = 0; j < P / E; ++j) {
      const V v = *reinterpret_cast<const V*>(row + i0 + E * j);
#pragma unroll
      for (int i = 0; i < E; ++i) x[E * j + i] = to_float(T{(uint16_t)(v[i / 2] >> (16 * (i % 2)))});
    }
  } else {
#pragma unroll
    for (int i = 0; i < P; ++i) x[i] = i0 + i < vocab ? to_float(row[i0 + i]) : -INFINITY;
  }
}
// -inf for NaN, where a wave has any.
template <int P>
__device__ __forceinline__ void clean(float (&x)[P]) {
  bool any = false;
#pragma unroll
  for (int i = 0; i < P; i += 2) any |= __builtin_isunordered(x[i], x[i + 1]);
  if (!__any(any)) return;
#pragma unroll
  for (int i = 0; i < P; ++i) x[i] = no_nan(x[i]);
}

__device__ __forceinline__ int count_of(const VerifyArgs& v, int b) {
  const int c = v.counts ? v.counts[b] : v.tokens;
  return c < 0 ? 0 : (c < v.tokens ? c : v.tokens);
}
__device__ __forceinline__ float heat_of(const VerifyArgs& v, int b, bool draft) {
  return draft && v.draft_temperature ? v.draft_temperature[b] : v.temperature[b];
}

// Over the 64 lanes of a wave (all active), the same in every lane.
template <int CTRL>
__device__ __forceinline__ float move(float v) {
  return __builtin_bit_cast(float, row_move<CTRL>(__builtin_bit_cast(int32_t, v)));
}
template <int CTRL>
__device__ __forceinline__ double move(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)row_move<CTRL>((int32_t)(uint32_t)b);
  const uint32_t hi = (uint32_t)row_move<CTRL>((int32_t)(uint32_t)(b >> 32));
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ float lane_of(float v, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int32_t, v), lane));
}
__device__ __forceinline__ double lane_of(double v, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int32_t)(uint32_t)b, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int32_t)(uint32_t)(b >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
template <class V, class F>
__device__ __forceinline__ V over_wave(V v, F&& f) {
  v = f(v, move<kDppMirror16>(v));
  v = f(v, move<kDppMirror8>(v));
  v = f(v, move<kDppRev4>(v));
  v = f(v, move<kDppSwap1>(v));
  return f(f(lane_of(v, 0), lane_of(v, 16)), f(lane_of(v, 32), lane_of(v, 48)));
}
__device__ __forceinline__ double wave_sum(double v) {
  return over_wave(v, [](double a, double b) { return a + b; });
}
__device__ __forceinline__ float wave_max(float v) {
  return over_wave(v, [](float a, float b) { return __builtin_fmaxf(a, b); });
}
__device__ __forceinline__ int wave_min(int v) {
#pragma unroll
  for (int m = 32; m > 0; m /= 2) {
    const int o = __shfl_xor(v, m);
    v = o < v ? o : v;
  }
  return v;
}

template <class T, bool VEC>
__global__ __launch_bounds__(kNT) void k_verify_stats(Plan p) {
  __shared__ float tops[kWaves];
  __shared__ int firsts[kWaves];
  __shared__ double sums[kWaves];
  const VerifyArgs& v = p.v;
  const int tid = threadIdx.x, wave = tid / 64;
  const int chunk = blockIdx.x % p.chunks;
  const int at = blockIdx.x / p.chunks;
  const int lb = at / p.rows, row = at - lb * p.rows;
  const int b = p.b0 + lb;
  const bool draft = row >= v.tokens;
  const int node = draft ? row - v.tokens : row;
  const float heat = heat_of(v, b, draft);
  const bool greedy = !(v.temperature[b] > 0.0f);
  // a drafter's row serves the node after it
  if (node + draft >= count_of(v, b) || (greedy && draft)) return;
  const int i0 = chunk * kChunk + tid * kPer;
  float x[kPer];
  load<VEC, kPer>(row_of<T>(v, b, row), i0, v.vocab, x);
  clean(x);
  float top = x[0];
#pragma unroll
  for (int i = 1; i < kPer; ++i) top = __builtin_fmaxf(top, x[i]);
  const float wave_top = wave_max(top);
  if (tid % 64 == 0) tops[wave] = wave_top;
  __syncthreads();
  top = __builtin_fmaxf(__builtin_fmaxf(tops[0], tops[1]), __builtin_fmaxf(tops[2], tops[3]));
  int first = INT32_MAX;
  double sum = 0.0;
  if (greedy || !(heat > 0.0f)) {
#pragma unroll
    for (int i = kPer - 1; i >= 0; --i) first = x[i] == top ? i0 + i : first;
    first = wave_min(first);
    if (tid % 64 == 0) firsts[wave] = first;
  } else if (top == INFINITY) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) sum += x[i] == top ? 1.0 : 0.0;
  } else if (top > -INFINITY) {
    const Heat h = make_heat(top, heat);
    const Near near = make_near(h);
    float four[4] = {};
    if (!near_scale(h)) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) sum += weight(h, x[i]);
    } else if (near_log2(near, wave_top) > kLarge) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const float y = near_log2(near, x[i]);
        const bool is = y > kLarge;
        four[i % 4] += is ? 0.0f : __builtin_amdgcn_exp2f(y);
        if (__any(is)) sum += is ? weight(h, x[i]) : 0.0;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) four[i % 4] += __builtin_amdgcn_exp2f(near_log2(near, x[i]));
    }
    sum += ((double)four[0] + (double)four[1]) + ((double)four[2] + (double)four[3]);
  }
  sum = wave_sum(sum);
  if (tid % 64 == 0) sums[wave] = sum;
  __syncthreads();
  if (tid == 0) {
    Stat s{top, 0, ((sums[0] + sums[1]) + sums[2]) + sums[3]};
    if (greedy || !(heat > 0.0f)) {
      s.at = firsts[0];
      for (int w = 1; w < kWaves; ++w) s.at = firsts[w] < s.at ? firsts[w] : s.at;
    }
    p.stats[(int64_t)at * p.chunks + chunk] = s;
  }
}

// A row's largest logit, its first index and its sum of weights.
struct Row {
  float top;
  int at;
  double z;
};
// Disjoint parts of a row as one; `scale` is that of its weights.
template <int N>
__device__ __forceinline__ Row join(const Row (&part)[N], double scale) {
  Row r = part[0];
#pragma unroll
  for (int i = 1; i < N; ++i) {
    const bool over = part[i].top > r.top || (part[i].top == r.top && part[i].at < r.at);
    r.top = over ? part[i].top : r.top;
    r.at = over ? part[i].at : r.at;
  }
  r.z = 0.0;
#pragma unroll
  for (int i = 0; i < N; ++i) r.z += part[i].z * weight(Heat{(double)r.top, scale}, part[i].top);
  return r;
}
// Every kParts-th chunk of a row, from `first` on, four of them loaded at once.
__device__ __forceinline__ Row part_of(const Plan& p, const Stat* st, int first, double scale) {
  Row r{-INFINITY, INT32_MAX, 0.0};
  for (int c = first; c < p.chunks; c += kParts * 4) {
    Row part[5];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = c + kParts * i;
      const Stat x = st[at < p.chunks ? at : first];
      const bool some = at < p.chunks && x.top > -INFINITY;
      part[i] = Row{some ? x.top : -INFINITY, some ? x.at : INT32_MAX, some ? x.sum : 0.0};
    }
    part[4] = r;
    r = join(part, scale);
  }
  return r;
}

// Lane i of each wave holds token i; every value that the walk needs is
// loaded beforehand, for all tokens at once.
template <class T>
__device__ __forceinline__ void walk(const Plan& p, int lb, bool writes, Row (&rows)[2][kParts][64], Last& out) {
  const VerifyArgs& v = p.v;
  const int lane = threadIdx.x & 63, wave = threadIdx.x / 64, b = p.b0 + lb;
  const int count = count_of(v, b);
  const float heat = heat_of(v, b, false), dheat = heat_of(v, b, true);
  const bool greedy = !(heat > 0.0f), dgreedy = !(dheat > 0.0f);
  const int64_t at = (int64_t)b * v.tokens + lane;
  const bool in = lane < count;
  const bool drawn = v.draft && !greedy && in && lane > 0;   // from the drafter's row of the token before
  const double scale = make_heat(0.0f, greedy ? 1.0f : heat).scale;
  const double dscale = make_heat(0.0f, dgreedy ? 1.0f : dheat).scale;
  // (what depends on loads in two steps comes first)
  const bool walks = in && wave == 0;
  const int id = walks ? v.ids[at] : -1;
  const bool is_id = id >= 0 && id < v.vocab;
  float u = walks ? v.u[at] : 0.0f;
  if (u < 0.0f) u = 0.0f;
  int parent = lane - 1;   // (-1: none)
  if (v.mask && walks) {
    const uint64_t above = (uint64_t)v.mask[at] & ((1ull << lane) - 1);
    parent = above ? 63 - __builtin_clzll(above) : -1;
  }
  const bool child = walks && parent >= 0 && is_id;
  const float x = child ? no_nan(to_float(row_of<T>(v, b, parent)[id])) : -INFINITY;
  const float y = drawn && is_id ? no_nan(to_float(row_of<T>(v, b, v.tokens + lane - 1)[id])) : -INFINITY;
  const Stat* stats = p.stats + (int64_t)lb * p.rows * p.chunks;
  const int part = wave % kParts, which = wave / kParts;   // (which 1: the drafter's rows)
  if (which == 0 ? in : which == 1 && drawn)
    rows[which][part][lane] = part_of(
        p, stats + (int64_t)(which ? v.tokens + lane - 1 : lane) * p.chunks, part, which ? dscale : scale);
  __syncthreads();
  if (wave > 0) return;
  Row row{-INFINITY, INT32_MAX, 0.0}, drow = row;
  if (in) row = join<kParts>({rows[0][0][lane], rows[0][1][lane], rows[0][2][lane], rows[0][3][lane]}, scale);
  if (drawn) drow = join<kParts>({rows[1][0][lane], rows[1][1][lane], rows[1][2][lane], rows[1][3][lane]}, dscale);
  const bool some = row.top > -INFINITY;
  // this token's weight among its parent's, and its share of the drafter's
  const float ptop = __shfl(row.top, parent & 63);
  const double pz = __shfl(row.z, parent & 63);
  const int pat = __shfl(row.at, parent & 63);
  const double mine = greedy ? 0.0 : weight(Heat{(double)ptop, scale}, x);
  double q = 0.0;
  if (drawn && drow.top > -INFINITY)
    q = dgreedy ? (id == drow.at ? 1.0 : 0.0) : weight(Heat{(double)drow.top, dscale}, y) / drow.z;
  const uint64_t hits = __ballot(child && id == pat);                        // greedy
  const uint64_t kept_by_q = __ballot(child && (double)u * q < mine / pz);   // chains
  const uint64_t filled = __ballot(in && some);
  int node = 0, kept = 0, path = -1, mode = kWhole, rejected = 0;
  while (count > 0) {
    if (lane == kept) path = node;
    ++kept;
    mode = kWhole;
    rejected = 0;
    if (!((filled >> node) & 1)) break;
    uint64_t children = __ballot(in && parent == node && lane > node);
    int next = -1;
    if (greedy || v.draft) {
      const uint64_t good = children & (greedy ? hits : kept_by_q);
      if (good) next = __builtin_ctzll(good);
      else if (!greedy && children) mode = kResidual;
    } else {
      double left = __shfl(row.z, node);
      while (children) {
        const int c = __builtin_ctzll(children);
        children &= children - 1;
        const double wc = __shfl(mine, c);
        const int idc = __builtin_amdgcn_readlane(id, c);
        bool again = false;   // rejected before: nothing left
        for (int k = 0; k < rejected; ++k) again |= out.ids[k] == idc;
        if (again || !(wc > 0.0)) continue;
        if ((double)__shfl(u, c) * left < wc) {
          next = c;
          break;
        }
        left -= wc;
        out.ids[rejected++] = idc;   // (every lane the same)
        mode = kLess;
      }
    }
    if (next < 0) break;
    node = next;
  }
  const float top = __shfl(row.top, node);
  const int first = __shfl(row.at, node);
  const bool none = count <= 0 || !(top > -INFINITY);   // nothing to take a token from
  const int drafted = node + 1 < 64 ? node + 1 : 63;    // the drafter's row of this node is its child's
  const int datum = __shfl(drow.top > -INFINITY ? drow.at : -1, drafted);
  if (mode == kResidual) out.ids[0] = datum;
  const double z = __shfl(row.z, node), draft_z = __shfl(drow.z, drafted);
  const float draft_top = __shfl(drow.top, drafted);
  if (lane == 0) {
    out.node = node;
    out.mode = none || greedy ? kDone : mode;
    out.rejected = rejected;
    out.top = top;
    out.z = z;
    out.draft_top = draft_top;
    out.draft_z = draft_z;
  }
  if (writes) {
    if (lane < v.tokens) v.path[at] = path;
    if (lane == 0) {
      v.accepted[b] = kept;
      v.next[b] = none || !greedy ? -1 : first;
    }
  }
}

__device__ __forceinline__ double of_waves(const double* sums) {
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < kManyWaves; ++w) s += sums[w];
  return s;
}

// What is left of a thread's tokens.
template <class T, bool VEC>
__device__ __forceinline__ void left_of(const VerifyArgs& v, int b, const Last& l, int mode, int i0,
                                       double (&r)[kFew]) {
  float x[kFew];
  load<VEC, kFew>(row_of<T>(v, b, l.node), i0, v.vocab, x);
  clean(x);
  const Heat h = make_heat(l.top, heat_of(v, b, false));
#pragma unroll
  for (int i = 0; i < kFew; ++i) r[i] = weight(h, x[i]);
  if (mode == kResidual) {
    float y[kFew];
    load<VEC, kFew>(row_of<T>(v, b, v.tokens + l.node), i0, v.vocab, y);
    clean(y);
    const float dheat = heat_of(v, b, true);
    const Heat d = make_heat(l.draft_top, dheat);
    const double pz = 1.0 / l.z, qz = l.draft_top > -INFINITY ? 1.0 / l.draft_z : 0.0;
    int first = INT32_MAX;
    if (!(dheat > 0.0f)) first = l.ids[0];
#pragma unroll
    for (int i = 0; i < kFew; ++i) {
      double q;
      if (dheat > 0.0f) q = weight(d, y[i]) * qz;
      else q = i0 + i == first ? 1.0 : 0.0;
      r[i] = __builtin_fmax(r[i] * pz - q, 0.0);
    }
  } else if (mode == kLess) {
    for (int k = 0; k < l.rejected; ++k) {
      const int e = l.ids[k] - i0;
#pragma unroll
      for (int i = 0; i < kFew; ++i) r[i] = i == e ? 0.0 : r[i];
    }
  }
}

template <class T, bool VEC>
__global__ __launch_bounds__(kMany) void k_verify_walk(Plan p) {
  __shared__ Last l;
  __shared__ Row rows[2][kParts][64];
  __shared__ double sums[kManyWaves];
  const int tid = threadIdx.x;
  const int lb = blockIdx.x / p.chunks, chunk = blockIdx.x - lb * p.chunks;
  walk<T>(p, lb, chunk == 0, rows, l);
  __syncthreads();
  if (chunk == 0) {   // for the last launch
    constexpr int kWords = sizeof(Last) / 4;
    if (tid < kWords) ((int32_t*)&p.last[lb])[tid] = ((const int32_t*)&l)[tid];
  }
  if (l.mode == kDone) return;
  double r[kFew], sum = 0.0;
  left_of<T, VEC>(p.v, p.b0 + lb, l, l.mode, chunk * kChunk + tid * kFew, r);
#pragma unroll
  for (int i = 0; i < kFew; ++i) sum += r[i];
  sum = wave_sum(sum);
  if (tid % 64 == 0) sums[tid / 64] = sum;
  __syncthreads();
  if (tid == 0) p.sums[(int64_t)lb * p.chunks + chunk] = of_waves(sums);
}

// Of `mine`, one value a thread: the first thread at which the running sum from
// `before` on passes `goal`, else the last one with a value above 0; -1 where there
// is none.  `below`: the running sum before it.  The same in every thread.
struct Find {
  double sums[kManyWaves];
  int hit[kManyWaves], any[kManyWaves];
  double below[kMany];
};
__device__ __forceinline__ int find(Find& f, double mine, double before, double goal, double& below) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid / 64;
  double run = mine;
#pragma unroll
  for (int m = 1; m < 64; m *= 2) {
    const double o = __shfl_up(run, m);
    if (lane >= m) run += o;
  }
  __syncthreads();
  if (lane == 63) f.sums[wave] = run;
  __syncthreads();
  double base = before;
  for (int w = 0; w < wave; ++w) base += f.sums[w];
  f.below[tid] = base + (run - mine);
  const uint64_t over = __ballot(base + run > goal && mine > 0.0), some = __ballot(mine > 0.0);
  if (lane == 0) {
    f.hit[wave] = over ? 64 * wave + __builtin_ctzll(over) : -1;
    f.any[wave] = some ? 64 * wave + 63 - __builtin_clzll(some) : -1;
  }
  __syncthreads();
  int at = -1;
  for (int w = kManyWaves - 1; w >= 0; --w) at = f.hit[w] >= 0 ? f.hit[w] : at;
  if (at < 0)
    for (int w = 0; w < kManyWaves; ++w) at = f.any[w] >= 0 ? f.any[w] : at;
  below = at >= 0 ? f.below[at] : before;
  return at;
}

// The running total of what is left in the chunks, each thread's own `each` neighbouring ones in
// `mine`.
__device__ __forceinline__ double total_of(const Plan& p, const double* sums, int each, double* sh, double& mine) {
  const int tid = threadIdx.x;
  mine = 0.0;
  for (int c = tid * each; c < tid * each + each && c < p.chunks; ++c) mine += sums[c];
  const double part = wave_sum(mine);
  __syncthreads();
  if (tid % 64 == 0) sh[tid / 64] = part;
  __syncthreads();
  return of_waves(sh);
}

template <class T, bool VEC>
__global__ __launch_bounds__(kMany) void k_verify_pick(Plan p) {
  __shared__ Find f;
  __shared__ double sh[kManyWaves];
  const VerifyArgs& v = p.v;
  const int tid = threadIdx.x, lb = blockIdx.x, b = p.b0 + lb;
  const Last& l = p.last[lb];
  double* sums = p.sums + (int64_t)lb * p.chunks;
  const int each = (p.chunks + kMany - 1) / kMany;
  const float given = v.u[(int64_t)b * v.tokens];
  const double u = given < 0.0f ? 0.0 : (double)given;
  int mode = l.mode;
  if (mode == kDone) return;
  double mine;
  double total = total_of(p, sums, each, sh, mine);
  if (!(total > 0.0) && mode != kWhole) {
    // nothing left, as for a u of 1 (or but by rounding): the row itself
    mode = kWhole;
    for (int c = 0; c < p.chunks; ++c) {
      double r[kFew], part = 0.0;
      left_of<T, VEC>(v, b, l, mode, c * kChunk + tid * kFew, r);
#pragma unroll
      for (int i = 0; i < kFew; ++i) part += r[i];
      part = wave_sum(part);
      __syncthreads();
      if (tid % 64 == 0) sh[tid / 64] = part;
      __syncthreads();
      if (tid == 0) sums[c] = of_waves(sh);
    }
    __syncthreads();
    total = total_of(p, sums, each, sh, mine);
  }
  const double goal = u * total;
  double below;
  const int run = find(f, mine, 0.0, goal, below);
  if (run < 0) return;   // (no weight at all: next stays -1)
  // of the run's chunks the one that passes, else its last with a weight
  int chunk = -1;
  double sum = below, at_chunk = below;
  for (int c = run * each; c < run * each + each && c < p.chunks; ++c) {
    const double s = sums[c];
    if (s > 0.0) {
      chunk = c;
      at_chunk = sum;
      if (sum + s > goal) break;
    }
    sum += s;
  }
  double r[kFew], part = 0.0;
  const int i0 = chunk * kChunk + tid * kFew;
  left_of<T, VEC>(v, b, l, mode, i0, r);
#pragma unroll
  for (int i = 0; i < kFew; ++i) part += r[i];
  const int who = find(f, part, at_chunk, goal, below);
  if (tid != who) return;
  int token = -1;
  for (int i = 0; i < kFew; ++i) {
    if (!(r[i] > 0.0)) continue;
    token = i0 + i;
    below += r[i];
    if (below > goal) break;
  }
  v.next[b] = token;
}

template <class T, bool VEC>
hipError_t launch_parts(const VerifyArgs& v, hipStream_t s) {
  Plan p{};
  p.v = v;
  p.chunks = (v.vocab + kChunk - 1) / kChunk;
  p.rows = v.tokens + (v.draft ? v.tokens - 1 : 0);
  // requests of a launch: up to 2^20 workgroups and 33 MB (one takes 8.4 MB at most)
  const int64_t blocks = (int64_t)p.rows * p.chunks;
  const int64_t each = blocks * (int64_t)sizeof(Stat) + p.chunks * (int64_t)sizeof(double) + (int64_t)sizeof(Last);
  int64_t part = ((int64_t)1 << 20) / blocks;
  part = part < 33000000 / each ? part : 33000000 / each;
  part = part < 1 ? 1 : (part < v.batch ? part : v.batch);
  const size_t stats = (size_t)part * blocks * sizeof(Stat);
  const size_t sums = (size_t)part * p.chunks * sizeof(double);
  void* ws = nullptr;
  hipError_t e = workspace_acquire(&ws, (size_t)(part * each), s);
  if (e != hipSuccess) return e;
  p.stats = (Stat*)ws;
  p.sums = (double*)((char*)ws + stats);
  p.last = (Last*)((char*)ws + stats + sums);
  for (int64_t b0 = 0; b0 < v.batch && e == hipSuccess; b0 += part) {
    const int64_t n = v.batch - b0 < part ? v.batch - b0 : part;
    p.b0 = (int)b0;
    hipLaunchKernelGGL((k_verify_stats<T, VEC>), dim3((unsigned)(n * blocks)), dim3(kNT), 0, s, p);
    hipLaunchKernelGGL((k_verify_walk<T, VEC>), dim3((unsigned)(n * p.chunks)), dim3(kMany), 0, s, p);
    hipLaunchKernelGGL((k_verify_pick<T, VEC>), dim3((unsigned)n), dim3(kMany), 0, s, p);
    e = hipGetLastError();
  }
  const hipError_t f = workspace_release(ws, s);
  return e != hipSuccess ? e : f;
}

template <class T>
hipError_t launch_type(const VerifyArgs& v, hipStream_t s) {
  const uintptr_t bytes = ((uintptr_t)v.logits | (uintptr_t)v.draft |
                           sizeof(T) * (uintptr_t)(v.bs | v.ts | (v.draft ? v.dbs | v.dts : 0)));
  return bytes % 16 == 0 ? launch_parts<T, true>(v, s) : launch_parts<T, false>(v, s);
}

}  // namespace

hipError_t launch_verify_drafts(const VerifyArgs& v, hipStream_t s) {
  switch (v.dtype) {
    case Q8TA_F32: return launch_type<float>(v, s);
    case Q8TA_F16: return launch_type<Half>(v, s);
    default: return launch_type<Bfloat>(v, s);
  }
}

}  // namespace q8ta
