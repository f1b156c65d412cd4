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
//     first, each for itself (a chain of short loads, one node after the
//     other; a lane holds a node), then the chunk's sum of what is left.  Where
//     nothing was rejected the first launch has that sum already.
//  3. k_verify_pick: a workgroup a request finds the chunk, then the token in it.
//
// Weights are 64-bit (2^x by a polynomial, 4e-14 of the weight) and added in one
// fixed order, so that a result does not depend on what else is in the batch.
#include <cmath>

#include "decode.h"
#include "weights.h"

namespace q8ta {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

constexpr int kNT = 256, kPer = 16, kChunk = kNT * kPer;
constexpr int kWaves = kNT / 64;

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

// This thread's 16 neighbouring logits of a chunk, -inf past the vocabulary.
template <bool VEC>
__device__ __forceinline__ void load16(const float* row, int i0, int vocab, float (&x)[kPer]) {
  if (VEC && i0 + kPer <= vocab) {
#pragma unroll
    for (int j = 0; j < kPer / 4; ++j) {
      const v4f v = *reinterpret_cast<const v4f*>(row + i0 + 4 * j);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[4 * j + i] = no_nan(v[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) x[i] = i0 + i < vocab ? no_nan(row[i0 + i]) : -INFINITY;
  }
}
template <bool VEC, class T>
__device__ __forceinline__ void load16(const T* row, int i0, int vocab, float (&x)[kPer]) {
  if (VEC && i0 + kPer <= vocab) {
#pragma unroll
    for (int j = 0; j < kPer / 8; ++j) {
      const v4u v = *reinterpret_cast<const v4u*>(row + i0 + 8 * j);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[8 * j + i] = no_nan(to_float(T{(uint16_t)(v[i / 2] >> (16 * (i % 2)))}));
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) x[i] = i0 + i < vocab ? no_nan(to_float(row[i0 + i])) : -INFINITY;
  }
}

__device__ __forceinline__ int count_of(const VerifyArgs& v, int b) {
  const int c = v.counts ? v.counts[b] : v.tokens;
  return c < 0 ? 0 : (c < v.tokens ? c : v.tokens);
}
__device__ __forceinline__ float heat_of(const VerifyArgs& v, int b, bool draft) {
  return draft && v.draft_temperature ? v.draft_temperature[b] : v.temperature[b];
}

template <class V>
__device__ __forceinline__ V wave_sum(V v) {
#pragma unroll
  for (int m = 32; m > 0; m /= 2) v += __shfl_xor(v, m);
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int m = 32; m > 0; m /= 2) v = __builtin_fmaxf(v, __shfl_xor(v, m));
  return v;
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
  load16<VEC>(row_of<T>(v, b, row), i0, v.vocab, x);
  float top = x[0];
#pragma unroll
  for (int i = 1; i < kPer; ++i) top = __builtin_fmaxf(top, x[i]);
  top = wave_max(top);
  if (tid % 64 == 0) tops[wave] = top;
  __syncthreads();
  top = __builtin_fmaxf(__builtin_fmaxf(tops[0], tops[1]), __builtin_fmaxf(tops[2], tops[3]));
  int first = INT32_MAX;
  double sum = 0.0;
  if (greedy || !(heat > 0.0f)) {
#pragma unroll
    for (int i = kPer - 1; i >= 0; --i) first = x[i] == top ? i0 + i : first;
    first = wave_min(first);
    if (tid % 64 == 0) firsts[wave] = first;
  } else if (top > -INFINITY) {
    const Heat h = make_heat(top, heat);
#pragma unroll
    for (int i = 0; i < kPer; ++i) sum += weight(h, x[i]);
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

// A row's largest logit, its first index and its sum of weights, from its
// chunks (every lane of a wave active).
struct Row {
  float top;
  int at;
  double z;
};
__device__ __forceinline__ Row row_stat(const Plan& p, const Stat* st, int lane, float heat) {
  Row r{-INFINITY, INT32_MAX, 0.0};
  for (int c = lane; c < p.chunks; c += 64) r.top = __builtin_fmaxf(r.top, st[c].top);
  r.top = wave_max(r.top);
  const Heat h = make_heat(r.top, heat);
  for (int c = lane; c < p.chunks; c += 64) {
    const Stat s = st[c];
    if (s.top == r.top && s.at < r.at) r.at = s.at;
    if (s.top > -INFINITY) r.z += s.sum * weight(h, s.top);
  }
  r.at = wave_min(r.at);
  r.z = wave_sum(r.z);
  return r;
}

template <class T>
__device__ __forceinline__ void walk(const Plan& p, int lb, bool writes, Last& out) {
  const VerifyArgs& v = p.v;
  const int lane = threadIdx.x & 63, b = p.b0 + lb;
  const int count = count_of(v, b);
  const float heat = heat_of(v, b, false), dheat = heat_of(v, b, true);
  const bool greedy = !(heat > 0.0f);
  const int64_t at = (int64_t)b * v.tokens + lane;
  const bool in = lane < count;
  const int id = in ? v.ids[at] : -1;
  float u = in ? v.u[at] : 0.0f;
  if (u < 0.0f) u = 0.0f;
  int parent = lane - 1;   // (-1: none)
  if (v.mask && in) {
    const uint64_t above = (uint64_t)v.mask[at] & ((1ull << lane) - 1);
    parent = above ? 63 - __builtin_clzll(above) : -1;
  }
  const Stat* stats = p.stats + (int64_t)lb * p.rows * p.chunks;
  int node = 0, kept = 0, path = -1;
  int mode = kWhole, rejected = 0;
  Row row{-INFINITY, 0, 0.0}, drow{-INFINITY, 0, 0.0};
  while (count > 0) {
    if (lane == kept) path = node;
    ++kept;
    mode = kWhole;
    rejected = 0;
    row = row_stat(p, stats + (int64_t)node * p.chunks, lane, greedy ? 1.0f : heat);
    uint64_t children = __ballot(in && lane > 0 && parent == node && lane > node);
    if (!(row.top > -INFINITY)) break;
    int next = -1;
    if (greedy) {
      const uint64_t hit = __ballot(id == row.at) & children;
      if (hit) next = __builtin_ctzll(hit);
    } else if (children) {
      const bool mine = (children >> lane) & 1 && id >= 0 && id < v.vocab;
      const float x = mine ? no_nan(to_float(row_of<T>(v, b, node)[id])) : -INFINITY;
      const double w = weight(make_heat(row.top, heat), x);
      if (v.draft) {
        // a chain: one child
        double q = 0.0;
        if (dheat > 0.0f) {
          const float y = mine ? no_nan(to_float(row_of<T>(v, b, v.tokens + node)[id])) : -INFINITY;
          drow = row_stat(p, stats + (int64_t)(v.tokens + node) * p.chunks, lane, dheat);
          if (drow.top > -INFINITY) q = weight(make_heat(drow.top, dheat), y) / drow.z;
        } else {   // a greedy drafter: all on its largest
          drow = row_stat(p, stats + (int64_t)(v.tokens + node) * p.chunks, lane, 1.0f);
          drow.z = 1.0;
          if (!(drow.top > -INFINITY)) drow.at = -1;
          q = id == drow.at ? 1.0 : 0.0;
          out.ids[0] = drow.at;
        }
        const uint64_t good = __ballot((double)u * q < w / row.z) & children;
        if (good) next = __builtin_ctzll(good);
        else mode = kResidual;
      } else {
        double left = row.z;
        while (children) {
          const int c = __builtin_ctzll(children);
          children &= children - 1;
          const double wc = __shfl(w, c);
          const int idc = __builtin_amdgcn_readlane(id, c);
          bool again = false;   // rejected before: nothing left
          for (int k = 0; k < rejected; ++k) again |= out.ids[k] == idc;
          if (!again && (double)__shfl(u, c) * left < wc) {
            next = c;
            break;
          }
          if (!again && wc > 0.0) {
            left -= wc;
            out.ids[rejected++] = idc;   // (every lane the same)
            mode = kLess;
          }
        }
      }
    }
    if (next < 0) break;
    node = next;
  }
  const bool none = !(row.top > -INFINITY);   // nothing to take a token from
  if (lane == 0) {
    out.node = node;
    out.mode = none || greedy ? kDone : mode;
    out.rejected = rejected;
    out.top = row.top;
    out.z = row.z;
    out.draft_top = drow.top;
    out.draft_z = drow.z;
  }
  if (writes) {
    if (lane < v.tokens) v.path[at] = path;
    if (lane == 0) {
      v.accepted[b] = kept;
      v.next[b] = none || !greedy ? -1 : row.at;
    }
  }
}

// What is left of a thread's 16 tokens.
template <class T, bool VEC>
__device__ __forceinline__ void left16(const VerifyArgs& v, int b, const Last& l, int mode, int i0,
                                       double (&r)[kPer]) {
  float x[kPer];
  load16<VEC>(row_of<T>(v, b, l.node), i0, v.vocab, x);
  const Heat h = make_heat(l.top, heat_of(v, b, false));
#pragma unroll
  for (int i = 0; i < kPer; ++i) r[i] = weight(h, x[i]);
  if (mode == kResidual) {
    float y[kPer];
    load16<VEC>(row_of<T>(v, b, v.tokens + l.node), i0, v.vocab, y);
    const float dheat = heat_of(v, b, true);
    const Heat d = make_heat(l.draft_top, dheat);
    const double pz = 1.0 / l.z, qz = l.draft_top > -INFINITY ? 1.0 / l.draft_z : 0.0;
    int first = INT32_MAX;
    if (!(dheat > 0.0f)) first = l.ids[0];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      double q;
      if (dheat > 0.0f) q = weight(d, y[i]) * qz;
      else q = i0 + i == first ? 1.0 : 0.0;
      r[i] = __builtin_fmax(r[i] * pz - q, 0.0);
    }
  } else if (mode == kLess) {
    for (int k = 0; k < l.rejected; ++k) {
      const int e = l.ids[k] - i0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) r[i] = i == e ? 0.0 : r[i];
    }
  }
}

template <class T, bool VEC>
__global__ __launch_bounds__(kNT) void k_verify_walk(Plan p) {
  __shared__ Last l;
  __shared__ double sums[kWaves];
  const int tid = threadIdx.x;
  const int lb = blockIdx.x / p.chunks, chunk = blockIdx.x - lb * p.chunks;
  if (tid < 64) walk<T>(p, lb, chunk == 0, l);
  __syncthreads();
  if (chunk == 0) {   // for the last launch
    constexpr int kWords = sizeof(Last) / 4;
    if (tid < kWords) ((int32_t*)&p.last[lb])[tid] = ((const int32_t*)&l)[tid];
  }
  if (l.mode == kDone || l.mode == kWhole) return;
  double r[kPer], sum = 0.0;
  left16<T, VEC>(p.v, p.b0 + lb, l, l.mode, chunk * kChunk + tid * kPer, r);
#pragma unroll
  for (int i = 0; i < kPer; ++i) sum += r[i];
  sum = wave_sum(sum);
  if (tid % 64 == 0) sums[tid / 64] = sum;
  __syncthreads();
  if (tid == 0) p.sums[(int64_t)lb * p.chunks + chunk] = ((sums[0] + sums[1]) + sums[2]) + sums[3];
}

// Of `mine`, one value a thread: the first thread at which the running sum from
// `before` on passes `goal`, else the last one with a value above 0; -1 where there
// is none.  `below`: the running sum before it.  The same in every thread.
struct Find {
  double sums[kWaves];
  int hit[kWaves], any[kWaves];
  double below[kNT];
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
  for (int w = kWaves - 1; w >= 0; --w) at = f.hit[w] >= 0 ? f.hit[w] : at;
  if (at < 0)
    for (int w = 0; w < kWaves; ++w) at = f.any[w] >= 0 ? f.any[w] : at;
  below = at >= 0 ? f.below[at] : before;
  return at;
}

template <class T, bool VEC>
__global__ __launch_bounds__(kNT) void k_verify_pick(Plan p) {
  __shared__ Find f;
  __shared__ double totals[kWaves];
  const VerifyArgs& v = p.v;
  const int tid = threadIdx.x, lb = blockIdx.x, b = p.b0 + lb;
  const Last& l = p.last[lb];
  if (l.mode == kDone) return;
  int mode = l.mode;
  const float given = v.u[(int64_t)b * v.tokens];
  const double u = given < 0.0f ? 0.0 : (double)given;
  const Stat* st = p.stats + ((int64_t)lb * p.rows + l.node) * p.chunks;
  const Heat h = make_heat(l.top, heat_of(v, b, false));
  auto chunk_sum = [&](int c) {
    if (c >= p.chunks) return 0.0;
    if (mode != kWhole) return p.sums[(int64_t)lb * p.chunks + c];
    return st[c].top > -INFINITY ? st[c].sum * weight(h, st[c].top) : 0.0;
  };
  // each thread a run of neighbouring chunks
  const int each = (p.chunks + kNT - 1) / kNT;
  double mine, total;
  while (true) {
    mine = 0.0;
    for (int c = tid * each; c < tid * each + each; ++c) mine += chunk_sum(c);
    total = wave_sum(mine);
    __syncthreads();
    if (tid % 64 == 0) totals[tid / 64] = total;
    __syncthreads();
    total = ((totals[0] + totals[1]) + totals[2]) + totals[3];
    if (total > 0.0 || mode == kWhole) break;
    mode = kWhole;   // nothing left but by rounding: the row itself
  }
  const double goal = u * total;
  double below;
  const int run = find(f, mine, 0.0, goal, below);
  if (run < 0) return;   // (no weight at all: next stays -1)
  // of the run's chunks the one that passes, else its last with a weight
  int chunk = -1;
  double sum = below, at_chunk = below;
  for (int c = run * each; c < run * each + each; ++c) {
    const double s = chunk_sum(c);
    if (s > 0.0) {
      chunk = c;
      at_chunk = sum;
      if (sum + s > goal) break;
    }
    sum += s;
  }
  double r[kPer], part = 0.0;
  const int i0 = chunk * kChunk + tid * kPer;
  left16<T, VEC>(v, b, l, mode, i0, r);
#pragma unroll
  for (int i = 0; i < kPer; ++i) part += r[i];
  const int who = find(f, part, at_chunk, goal, below);
  if (tid != who) return;
  int token = -1;
  for (int i = 0; i < kPer; ++i) {
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
  // requests of a launch: up to 2^20 workgroups and as many chunks' sums
  const int64_t blocks = (int64_t)p.rows * p.chunks;
  int64_t part = ((int64_t)1 << 20) / blocks;
  part = part < 1 ? 1 : (part < v.batch ? part : v.batch);
  const size_t stats = (size_t)part * blocks * sizeof(Stat);
  const size_t sums = (size_t)part * p.chunks * sizeof(double);
  void* ws = nullptr;
  hipError_t e = workspace_acquire(&ws, stats + sums + (size_t)part * sizeof(Last), s);
  if (e != hipSuccess) return e;
  p.stats = (Stat*)ws;
  p.sums = (double*)((char*)ws + stats);
  p.last = (Last*)((char*)ws + stats + sums);
  for (int64_t b0 = 0; b0 < v.batch && e == hipSuccess; b0 += part) {
    const int64_t n = v.batch - b0 < part ? v.batch - b0 : part;
    p.b0 = (int)b0;
    hipLaunchKernelGGL((k_verify_stats<T, VEC>), dim3((unsigned)(n * blocks)), dim3(kNT), 0, s, p);
    hipLaunchKernelGGL((k_verify_walk<T, VEC>), dim3((unsigned)(n * p.chunks)), dim3(kNT), 0, s, p);
    hipLaunchKernelGGL((k_verify_pick<T, VEC>), dim3((unsigned)n), dim3(kNT), 0, s, p);
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
