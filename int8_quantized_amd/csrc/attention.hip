// q8ta_tree_attention: single tokens, or a tree of drafted tokens, over the
// paged int8 cache.
//
//   s_ij = softmax_scale * kscale_j * sum_d q_i[d] kcode_j[d]
//   out_i = sum_j softmax_j(s_ij) vscale_j vcode_j,   lse_i = log sum_j exp s_ij
//
// j runs over the keys row i sees: the request's context and, of its drafted
// tokens (the cache's next rows), those whose bit is set in the token's mask.
//
// One pass over the keys with the running maximum and sum of the softmax, on
// the 16x16x32 fp16 matrix instruction.  A wave takes 16 * TL keys per step for
// up to 16 * QT rows of one key head; the waves of a workgroup take every
// WAVES-th step and join their sums in LDS at the end; the keys of all requests
// are dealt out evenly over the workgroups, and k_attn_join joins what was cut.
// No wave waits for another inside the loop: with few rows the step is as long
// as its loads, and with many every wave widens the codes for itself.
//  * Codes are whole numbers of [-128, 127] and exact in fp16.  A key's byte b ^
//    0x80 under the exponent byte 0x64 is 1024 + 128 + code, less 1152; a value's
//    under a zero byte is the subnormal (128 + code) * 2^-24, less 128 * 2^-24,
//    since there the permute has two keys' bytes to fetch and none to spare for
//    a constant (fp16's subnormals are exact in the adder and the matrix unit;
//    the outputs are scaled back).  Five operations for four codes.  (Leaving
//    the 128 in and taking it off the sums saves two of the five, but cancels
//    128 against outputs that are means over the context and come out near
//    zero: off by 1 % of such an output at 700 keys.)
//  * Queries: fp16 as they are; bf16 scaled by a power of two that puts the
//    row's largest element in [2^14, 2^15), where fp16 holds every element
//    exactly but those more than 2^28 below it.  So a score is a sum
//    of exact products in 32 bits.
//  * The keys are the A operand: lane l gets the scores of query l % 16 for
//    keys 16t + 4(l / 16) + r, which is also where the B operand of the second
//    product wants the probabilities if its K slots are numbered to match
//    (slot 8g + j = key 4g + j of the first 16-key tile for j < 4, key 4g + j - 4
//    of the second beyond), so they never leave their registers, and a
//    query's maximum, sum and rescaling are its lanes' own.
//  * Values: lane (i, g) loads VB = DP / 16 bytes of each of four neighbouring keys
//    and transposes them with the byte permutes that widen them.
//  * Probabilities go into the second product as fp16: with bf16 outputs
//    rounded to it (half a step is 2^-12 of each, against 2^-9 of the output's own
//    rounding), with fp16 outputs as two parts that hold 22 bits (rounded to
//    one, the errors of the outputs against 64 bits are 1.42 to 1.47 times those of
//    their own rounding, with two 1.00; 24-token trees x 16 x 4k 90.6 us against
//    86.2, and nothing where the cache's bytes bound it).  The sum that divides them
//    stays 32-bit.  The value's scale goes onto its
//    probability, divided by a power of two near the largest scale so far and
//    times 2^10: products up to 2^15 leave fp16's range below for weights down
//    to 2^-34 of the largest, whatever the scales are.
//  * 2^(s - m) is taken straight from the products; the maximum m is renewed
//    only when one passes 2^4, the values' power of two when a scale passes
//    twice it: most steps need no exchange between lanes and no rescaling.
//  * What bounds it: single tokens over long contexts, the cache's bytes (32
//    requests x up to 24k keys x 8 heads x 128: 1.22 GB in 228 us with the join,
//    5.3 TB/s; a bare read of as much takes 176, a copy runs at 4.9 TB/s).  Trees, the
//    vector instructions that widen codes and form the
//    softmax beside the matrix instructions, about three to one, at the two
//    waves a SIMD that the registers leave: 24 tokens x 4 heads of a group x 16
//    requests x 4k (fp16) in 85 us and 11 for the join, 64 x 8 x 4 x 16k (bf16) in 102 and
//    8 (four row tiles a wave, which halve the widening, spill and take 98).  One
//    token over 700 keys is a chain of latencies (page table, keys, joins): 13 us.
//  * A step's registers are loaded again for the next one as soon as it has
//    used them (keys after the first product, values after the second), so
//    loads are in flight through all of a step.
#include <cmath>
#include <type_traits>

#include "decode.h"

namespace q8ta {
namespace {

typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kMargin = 4.0f;      // a score may pass the running maximum by 2^4
constexpr float kMaxWeight = 16.0f;  // 2^kMargin
constexpr int kLift = 10;            // weights are held times 2^kLift
constexpr float kUp = 16777216.0f;   // 2^24

union Frag {
  v8h h;
  uint32_t u[4];
};

__device__ __forceinline__ uint32_t add_half(uint32_t x, uint32_t c) {
  const v2h y = __builtin_bit_cast(v2h, x) + __builtin_bit_cast(v2h, c);
  return __builtin_bit_cast(uint32_t, y);
}

// Eight codes of a key (two words in byte order, flipped already).
__device__ __forceinline__ v8h widen8(uint32_t w0, uint32_t w1) {
  const uint32_t k = 0x64646464u, less = 0xe480e480u;   // -1152
  Frag f;
  f.u[0] = add_half(__builtin_amdgcn_perm(w0, k, 0x00050004u), less);
  f.u[1] = add_half(__builtin_amdgcn_perm(w0, k, 0x00070006u), less);
  f.u[2] = add_half(__builtin_amdgcn_perm(w1, k, 0x00050004u), less);
  f.u[3] = add_half(__builtin_amdgcn_perm(w1, k, 0x00070006u), less);
  return f.h;
}

// Byte `byte` of words a and b (two values' same element, flipped already),
// times 2^-24.
__device__ __forceinline__ uint32_t widen_pair(uint32_t a, uint32_t b, int byte) {
  const uint32_t less = 0x80808080u;   // -128 * 2^-24
  return add_half(__builtin_amdgcn_perm(b, a, 0x0c000c00u | (uint32_t)(4 + byte) << 16 | (uint32_t)byte), less);
}

__device__ __forceinline__ uint32_t pack_half(float a, float b) {
  const v2h v = v2h{(_Float16)a, (_Float16)b};
  return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ float pow2f(int e) {   // 2^e, -126 <= e <= 127
  return __builtin_bit_cast(float, (uint32_t)(e + 127) << 23);
}
// |x|, 0 where x is not finite.
__device__ __forceinline__ float finite_size(float x) {
  const float y = __builtin_fabsf(x);
  return y < __builtin_inff() ? y : 0.0f;
}
// Exponent of a finite x >= 0 (-127 for 0), and kept in [-110, 110].
__device__ __forceinline__ int exponent_of(float x) {
  return (int)(__builtin_bit_cast(uint32_t, x) >> 23) - 127;
}
__device__ __forceinline__ int unit_exponent(float x) {
  const int e = exponent_of(x);
  return e < -110 ? -110 : (e > 110 ? 110 : e);
}

// What of the request this launch's rows see.
struct Span {
  int ctx, count, total;   // context keys, drafted tokens in use, keys in all
};
__device__ __forceinline__ Span span_of(const AttnArgs& a, int b) {
  const int64_t cap = (int64_t)a.table_pages * a.page;
  Span s;
  const int len = a.lens[b];
  s.ctx = len < 0 ? 0 : (len < cap ? len : (int)cap);
  int c = a.counts ? a.counts[b] : a.tokens;
  s.count = c < 0 ? 0 : (c < a.tokens ? c : a.tokens);
  const int64_t all = (int64_t)s.ctx + s.count;
  s.total = (int)(all < cap ? all : cap);
  return s;
}

// Drafted tokens that token t sees, as bits; none for a token not in use.
__device__ __forceinline__ uint64_t seen_bits(const AttnArgs& a, const Span& s, int b, int t) {
  if (t >= s.count) return 0;
  const uint64_t used = s.count >= 64 ? ~0ull : (1ull << s.count) - 1;
  const uint64_t chain = t >= 63 ? ~0ull : (2ull << t) - 1;
  return (a.mask ? (uint64_t)a.mask[(int64_t)b * a.tokens + t] : chain) & used;
}

// Eight elements from p on: one load where every row is 16-byte aligned.
template <class T>
__device__ __forceinline__ v4u load8(const T* p, bool aligned) {
  v4u r;
  if (aligned) {
    r = *reinterpret_cast<const v4u*>(p);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = (uint32_t)p[2 * e].bits | (uint32_t)p[2 * e + 1].bits << 16;
  }
  return r;
}

template <int VB>
struct Bytes {
  uint32_t w[VB / 4];
};
template <int VB>
__device__ __forceinline__ Bytes<VB> load_bytes(const int8_t* p) {
  Bytes<VB> r;
  if constexpr (VB == 4) {
    r.w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (VB == 8) {
    const v2u v = *reinterpret_cast<const v2u*>(p);
    r.w[0] = v[0];
    r.w[1] = v[1];
  } else {
    const v4u v = *reinterpret_cast<const v4u*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) r.w[i] = v[i];
  }
  return r;
}

// Result row of (request, row of the key head): its place among all rows.
__device__ __forceinline__ int64_t row_at(const AttnArgs& a, int b, int kvh, int row) {
  const int t = (int)fast_div((uint32_t)row, a.group_div);
  return ((int64_t)b * a.tokens + t) * a.heads + kvh * a.group + (row - t * a.group);
}

// How the work is dealt out.  A unit is a row block of one key head of one
// request; its keys come in grains of a.grain keys (at least one, so that every
// row is written).  All grains of all units in order are cut into a.groups equal
// runs, one a workgroup, whatever the requests' lengths are: as many
// workgroups as are resident at once finish together, and none is started for
// keys that are not there.  A unit that lies within one run is finished by its
// workgroup; of the others each run holds a last part of the first and a first
// part of the last, whose sums go to slots 2i and 2i + 1 of workgroup i, for
// k_attn_join.
__device__ __forceinline__ int grains_of(const AttnArgs& a, int b) {
  const int total = span_of(a, b).total;
  return total < 1 ? 1 : (int)fast_div((uint32_t)(total - 1), a.grain_div) + 1;
}
// Running sums over the lanes of a wave (every lane active): within rows of 16
// lanes, then each row's last sum onto the rows after it.
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);   // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);   // row_shr:2
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);   // row_shr:4
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);   // row_shr:8
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);   // row_bcast:15 into rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);   // row_bcast:31 into rows 2 and 3
  return v;
}
// The grains of the batch, 64 requests at a time: `scan` the running sums of the
// requests from `b0` on, on top of `before`.  Batches of up to 64 (one round)
// are read once.
struct Grains {
  int b0, before, scan;
  __device__ __forceinline__ void at(const AttnArgs& a, int lane, int from, int sum) {
    b0 = from;
    before = sum;
    scan = wave_scan(b0 + lane < a.batch ? grains_of(a, b0 + lane) : 0);
  }
  __device__ __forceinline__ int end() const { return before + __builtin_amdgcn_readlane(scan, 63); }
  // Moves to the round that holds request b, or grain x where b < 0.
  __device__ __forceinline__ void seek(const AttnArgs& a, int lane, int b, int x) {
    if (b < 0 ? x < before : b < b0) at(a, lane, 0, 0);
    while (b < 0 ? x >= end() : b >= b0 + 64) at(a, lane, b0 + 64, end());
  }
  // Request of grain x of the batch; first: the first grain of request b, n its grains.
  __device__ __forceinline__ int find(const AttnArgs& a, int lane, int x) {
    seek(a, lane, -1, x);
    return b0 + __builtin_ctzll(__ballot(before + scan > x));
  }
  __device__ __forceinline__ void of(const AttnArgs& a, int lane, int b, int& first, int& n) {
    seek(a, lane, b, 0);
    const int at = b - b0;
    first = before + (at > 0 ? __builtin_amdgcn_readlane(scan, at - 1) : 0);
    n = before + __builtin_amdgcn_readlane(scan, at) - first;
  }
};
// Runs: the first `more` have each + 1 grains, the others `each`.
struct Runs {
  int each, more;
};
__device__ __forceinline__ Runs runs_of(const AttnArgs& a, int lane, Grains& g) {
  g.at(a, lane, 0, 0);
  while (g.b0 + 64 < a.batch) g.at(a, lane, g.b0 + 64, g.end());
  const int all = g.end() * a.kv_heads * a.row_blocks;
  const int each = (int)fast_div((uint32_t)all, a.groups_div);
  return Runs{each, all - each * a.groups};
}
__device__ __forceinline__ int run_start(const Runs& r, int i) { return i * r.each + (i < r.more ? i : r.more); }
__device__ __forceinline__ int run_of(const Runs& r, int x) {
  const int big = r.more * (r.each + 1);
  return x < big ? x / (r.each + 1) : r.more + (x - big) / r.each;
}

// Up to 16 * QT query rows of one key head and a stretch of the keys.  DP: dim
// rounded up to 64, 128 or 256.
template <class T, int DP, int WAVES, int QT, int TL>
__global__ __launch_bounds__(64 * WAVES, DP == 256 ? 1 : 2) void k_attn(AttnArgs a) {
  constexpr int U = DP / 64, VB = DP / 16, R = 16 * QT, kStep = 16 * TL;
  constexpr bool kBf = std::is_same<T, Bfloat>::value;
  constexpr int kParts = kBf ? 1 : 2;   // of a probability
  __shared__ __attribute__((aligned(16))) float merge[WAVES][R][DP];
  __shared__ float2 stats[WAVES][R];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int rows = a.tokens * a.group;
  const int D = a.dim;
  // workgroups go round the 8 XCDs: renumbered so that an XCD's run together,
  // and the row blocks of a key head, which read the same keys, share its L2
  int run = blockIdx.x;
  if (a.groups % 8 == 0) run = run % 8 * (a.groups / 8) + run / 8;
  Grains grains;
  const Runs runs = runs_of(a, lane, grains);
  const int heads_blocks = a.kv_heads * a.row_blocks;
  int x = run_start(runs, run);
  const int x_end = run_start(runs, run + 1);
  while (x < x_end) {
  // request b's units follow one another, of_b grains each
  const int b = grains.find(a, lane, (int)fast_div((uint32_t)x, a.heads_blocks_div));
  int first, of_b;
  grains.of(a, lane, b, first, of_b);
  const int in_b = x - first * heads_blocks;
  const int unit_at = in_b / of_b, g0 = in_b - unit_at * of_b;
  const int g1 = of_b - g0 < x_end - x ? of_b : g0 + (x_end - x);
  x += g1 - g0;
  const int kvh = unit_at / a.row_blocks, row0 = (unit_at - kvh * a.row_blocks) * R;
  const Span sp = span_of(a, b);
  const int k_begin = g0 * a.grain;
  const int k_end = grains_end(sp.total, of_b, a.grain, g1);
  const bool whole = g0 == 0 && g1 == of_b;
  const int64_t slot = 2 * run + (g0 == 0 ? 1 : 0);

  // A 16-key tile lies in one page.  No load is conditional (a branch around
  // one would end in a wait for it): a tile past the last reads the table's
  // last entry, one without a page the first page's rows, elements past dim the
  // row's first; such keys' scales are replaced by zeros, and elements past dim
  // meet zero queries or go to outputs that are not stored.
  const int64_t part = (int64_t)a.kv_heads * a.page;   // rows from a page's keys to its values
  const int32_t* table = a.table + (int64_t)b * a.table_pages;
  v4u k_raw[TL][U];
  Bytes<VB> v_raw[TL][4];
  v4f ks[TL], vs[TL];
  int64_t prow[TL];    // cache row of each 16-key tile's first key
  uint32_t ok = 0;     // bit t: tile t's page is one
  auto find = [&](int step) {
    const int first = (int)fast_div((uint32_t)step, a.page_div);
    if (a.page % kStep == 0) {   // (a step starts on a multiple of kStep)
      int64_t pg = table[first];
      const bool in = pg >= 0 && pg < a.pages;
      ok = in ? ~0u >> (32 - TL) : 0;
      if (!in) pg = 0;
      prow[0] = (pg * 2 * a.kv_heads + kvh) * a.page + (step - first * a.page);
#pragma unroll
      for (int t = 1; t < TL; ++t) prow[t] = prow[0] + 16 * t;
      return;
    }
    ok = 0;
#pragma unroll
    for (int t = 0; t < TL; ++t) {
      const int key = step + 16 * t;
      int idx = (int)fast_div((uint32_t)key, a.page_div);
      const int within = key - idx * a.page;
      idx = idx < a.table_pages ? idx : a.table_pages - 1;
      int64_t pg = table[idx];
      const bool in = pg >= 0 && pg < a.pages;
      ok |= (uint32_t)in << t;
      if (!in) pg = 0;
      prow[t] = (pg * 2 * a.kv_heads + kvh) * a.page + within;
    }
  };
  // a lane's place among a tile's rows, as unsigned offsets to uniform bases
  uint32_t k_off[U], v_off[4];
#pragma unroll
  for (int u = 0; u < U; ++u) k_off[u] = (uint32_t)(n * D + (16 * (4 * u + g) < D ? 16 * (4 * u + g) : 0));
#pragma unroll
  for (int r = 0; r < 4; ++r) v_off[r] = (uint32_t)((4 * g + r) * D + (VB * n < D ? VB * n : 0));
  const uint32_t s_off = 16 * (uint32_t)g;
  auto load_k = [&] {
#pragma unroll
    for (int t = 0; t < TL; ++t) {
      const int8_t* base = a.cache + prow[t] * D;
#pragma unroll
      for (int u = 0; u < U; ++u) k_raw[t][u] = *reinterpret_cast<const v4u*>(base + k_off[u]);
      ks[t] = *reinterpret_cast<const v4f*>((const int8_t*)(a.scales + prow[t]) + s_off);
    }
  };
  auto load_v = [&] {
#pragma unroll
    for (int t = 0; t < TL; ++t) {
      const int8_t* base = a.cache + (prow[t] + part) * D;
#pragma unroll
      for (int r = 0; r < 4; ++r) v_raw[t][r] = load_bytes<VB>(base + v_off[r]);
      vs[t] = *reinterpret_cast<const v4f*>((const int8_t*)(a.scales + prow[t] + part) + s_off);
    }
  };
  // Queries as B operands: element e of operand k holds d = 16 * (4 * (k / 2) +
  // g) + 8 * (k % 2) + e, the order in which load_k's 16 bytes a lane come.  fac
  // turns a product of codes into a score in powers of two.
  // (loaded ahead of the first keys, so that they are there when those are.)
  int step = k_begin + kStep * wave;
  v8h q[QT][DP / 32];
  uint64_t bits[QT];
  float fac = a.scale * kLog2e;   // the first row tile's
  int less[QT] = {};              // log2 of tile i - 1's factor over tile i's
  uint32_t ok_now;
  {
    v4u raw[QT][DP / 32];
    int last = 0;
#pragma unroll
    for (int i = 0; i < QT; ++i) {
      const int row = row0 + 16 * i + n;
      const bool live = row < rows;
      const int tok = live ? (int)fast_div((uint32_t)row, a.group_div) : 0;
      bits[i] = live ? seen_bits(a, sp, b, tok) : 0;
      const T* src = (const T*)a.q + b * a.q_bs + tok * a.q_ts +
                     (int64_t)(kvh * a.group + (row - tok * a.group)) * a.q_hs;
#pragma unroll
      for (int k = 0; k < DP / 32; ++k) {
        const int d = 16 * (4 * (k / 2) + g) + 8 * (k % 2);
        raw[i][k] = v4u{0, 0, 0, 0};
        if (live && d < D) raw[i][k] = load8(src + d, a.q_aligned);
      }
    }
    if (step < k_end) {
      find(step);
      load_k();
      load_v();
    }
    ok_now = ok;
#pragma unroll
    for (int i = 0; i < QT; ++i) {
      float up = 1.0f;
      if constexpr (kBf) {
        float top = 0.0f;
#pragma unroll
        for (int k = 0; k < DP / 32; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t w = raw[i][k][e];
            top = __builtin_fmaxf(top, finite_size(__builtin_bit_cast(float, w << 16)));
            top = __builtin_fmaxf(top, finite_size(__builtin_bit_cast(float, w & 0xffff0000u)));
          }
        top = __builtin_fmaxf(top, __shfl_xor(top, 16));
        top = __builtin_fmaxf(top, __shfl_xor(top, 32));
        // (rows below 2^-40, whose scores are none, by as much as that)
        const int e = exponent_of(top), sh = 14 - (e < -40 ? -40 : e);
        up = pow2f(sh);
        less[i] = sh - last;
        last = sh;
        if (i == 0) fac = fac * pow2f(-sh);
      }
#pragma unroll
      for (int k = 0; k < DP / 32; ++k) {
        Frag f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t w = raw[i][k][e];
          if constexpr (kBf)
            f.u[e] = pack_half(__builtin_bit_cast(float, w << 16) * up,
                               __builtin_bit_cast(float, w & 0xffff0000u) * up);
          else
            f.u[e] = w;
        }
        q[i][k] = f.h;
      }
    }
  }

  const float none = -INFINITY;
  float m[QT], l[QT];
  v4f o[QT][VB];
#pragma unroll
  for (int i = 0; i < QT; ++i) {
    m[i] = none;
    l[i] = 0.0f;
#pragma unroll
    for (int w = 0; w < VB; ++w) o[i][w] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  }
  // the values' power of two (unit also undoes the values' 2^-24)
  float unit = kUp, inv_unit = 1.0f, limit = 0.0f;

  for (; step < k_end; step += kStep * WAVES) {
    const bool more = step + kStep * WAVES < k_end;
    if (more) find(step + kStep * WAVES);
    // products of keys 16t + 4g + r
    v4f s[QT][TL];
#pragma unroll
    for (int t = 0; t < TL; ++t) {
#pragma unroll
      for (int i = 0; i < QT; ++i) s[i][t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const v4u x = k_raw[t][u] ^ 0x80808080u;
        const v8h k0 = widen8(x[0], x[1]), k1 = widen8(x[2], x[3]);
#pragma unroll
        for (int i = 0; i < QT; ++i) {
          s[i][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k0, q[i][2 * u], s[i][t], 0, 0, 0);
          s[i][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k1, q[i][2 * u + 1], s[i][t], 0, 0, 0);
        }
      }
    }
    v4f kf[TL];
#pragma unroll
    for (int t = 0; t < TL; ++t) kf[t] = ks[t] * fac;
    if (more) load_k();
    // past the context, and where a page is none: keys a row may not see
    // (their scales may hold anything, so they are replaced, not multiplied away)
    const bool masked = step + kStep > sp.ctx || step + kStep > k_end || ok_now != (1u << TL) - 1;
    uint32_t real = ~0u;   // bit 4t + r: this lane's key 16t + 4g + r is one that some row sees
    if (masked) {
      real = 0;
      uint64_t any_bits = bits[0];
#pragma unroll
      for (int i = 1; i < QT; ++i) any_bits |= bits[i];
#pragma unroll
      for (int x = 1; x < 16; x *= 2) any_bits |= __shfl_xor(any_bits, x);
#pragma unroll
      for (int t = 0; t < TL; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int at = step + 16 * t + 4 * g + r - sp.ctx;
          const bool in = ((ok_now >> t) & 1) && at < k_end - sp.ctx && (at < 0 || ((any_bits >> (at & 63)) & 1));
          real |= (uint32_t)in << (4 * t + r);
          vs[t][r] = in ? vs[t][r] : 0.0f;
        }
    }
    float vtop = 0.0f;
#pragma unroll
    for (int t = 0; t < TL; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) vtop = __builtin_fmaxf(vtop, __builtin_fabsf(vs[t][r]));
    if (__any(vtop > limit)) {
      // (a scale that is not finite spoils the rows that see it, not the unit)
      vtop = 0.0f;
#pragma unroll
      for (int t = 0; t < TL; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) vtop = __builtin_fmaxf(vtop, finite_size(vs[t][r]));
#pragma unroll
      for (int x = 1; x < 64; x *= 2) vtop = __builtin_fmaxf(vtop, __shfl_xor(vtop, x));
      if (vtop > limit) {
        const int e = unit_exponent(vtop);
        inv_unit = pow2f(kLift - e);
        const float f = unit / kUp * inv_unit;
#pragma unroll
        for (int i = 0; i < QT; ++i)
#pragma unroll
          for (int w = 0; w < VB; ++w) o[i][w] *= f;
        unit = pow2f(e - kLift + 24);
        limit = pow2f(e + 1);
      }
    }
#pragma unroll
    for (int t = 0; t < TL; ++t) vs[t] = vs[t] * inv_unit;
    Frag p[QT][TL / 2][kParts];
#pragma unroll
    for (int i = 0; i < QT; ++i) {
      // e = 2^(s - m)
      float e[TL][4], top = 0.0f;
      const float base = m[i] == none ? 0.0f : m[i];
      if (kBf && i > 0) {   // from one row's factor to the next
#pragma unroll
        for (int t = 0; t < TL; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r) kf[t][r] = __builtin_ldexpf(kf[t][r], -less[i]);
      }
#pragma unroll
      for (int t = 0; t < TL; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          e[t][r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i][t][r], kf[t][r], -base));
          top = __builtin_fmaxf(top, e[t][r]);
        }
      uint32_t seen = ~0u;
      if (masked || __any(m[i] == none || top > kMaxWeight)) {
        if (masked) {
          seen = 0;
#pragma unroll
          for (int t = 0; t < TL; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int at = step + 16 * t + 4 * g + r - sp.ctx;
              const bool in = ((real >> (4 * t + r)) & 1) && (at < 0 || ((bits[i] >> (at & 63)) & 1));
              seen |= (uint32_t)in << (4 * t + r);
            }
        }
        top = none;
#pragma unroll
        for (int t = 0; t < TL; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            e[t][r] = (seen >> (4 * t + r)) & 1 ? s[i][t][r] * kf[t][r] : none;
            top = __builtin_fmaxf(top, e[t][r]);
          }
        if (__any(top > m[i] + kMargin)) {
          top = __builtin_fmaxf(top, __shfl_xor(top, 16));
          top = __builtin_fmaxf(top, __shfl_xor(top, 32));
          const float next = __builtin_fmaxf(m[i], top);
          const float c = next == none ? 1.0f : __builtin_amdgcn_exp2f(m[i] - next);
          m[i] = next;
          l[i] *= c;
#pragma unroll
          for (int w = 0; w < VB; ++w) o[i][w] *= c;
        }
        const float now = m[i] == none ? 0.0f : m[i];
#pragma unroll
        for (int t = 0; t < TL; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r) e[t][r] = __builtin_amdgcn_exp2f(e[t][r] - now);
      }
#pragma unroll
      for (int t = 0; t < TL; ++t) {
        float x[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          l[i] += e[t][r];
          x[r] = e[t][r] * vs[t][r];
        }
        if (masked) {   // a scale that only another row sees may not be finite
#pragma unroll
          for (int r = 0; r < 4; ++r) x[r] = (seen >> (4 * t + r)) & 1 ? x[r] : 0.0f;
        }
#pragma unroll
        for (int h = 0; h < kParts; ++h) {   // each the rounding of what is left
          const uint32_t p01 = pack_half(x[0], x[1]), p23 = pack_half(x[2], x[3]);
          p[i][t / 2][h].u[2 * (t % 2)] = p01;
          p[i][t / 2][h].u[2 * (t % 2) + 1] = p23;
          if (h + 1 < kParts) {
            const v2h h01 = __builtin_bit_cast(v2h, p01), h23 = __builtin_bit_cast(v2h, p23);
            x[0] -= (float)h01[0];
            x[1] -= (float)h01[1];
            x[2] -= (float)h23[0];
            x[3] -= (float)h23[1];
          }
        }
      }
    }
#pragma unroll
    for (int t = 0; t < TL; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int x = 0; x < VB / 4; ++x) v_raw[t][r].w[x] ^= 0x80808080u;
#pragma unroll
    for (int w = 0; w < VB; ++w) {
#pragma unroll
      for (int h = 0; h < TL / 2; ++h) {
        Frag f;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const Bytes<VB>(&v)[4] = v_raw[2 * h + t];
          f.u[2 * t] = widen_pair(v[0].w[w / 4], v[1].w[w / 4], w % 4);
          f.u[2 * t + 1] = widen_pair(v[2].w[w / 4], v[3].w[w / 4], w % 4);
        }
#pragma unroll
        for (int i = 0; i < QT; ++i)
#pragma unroll
          for (int part = 0; part < kParts; ++part)
            o[i][w] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f.h, p[i][h][part].h, o[i][w], 0, 0, 0);
      }
    }
    if (more) {
      load_v();
      ok_now = ok;
    }
  }

  // o[i][w][r]: query n of tile i, d = VB * (4g + r) + w
#pragma unroll
  for (int i = 0; i < QT; ++i) {
    l[i] += __shfl_xor(l[i], 16);
    l[i] += __shfl_xor(l[i], 32);
    if (g == 0) stats[wave][16 * i + n] = float2{m[i], l[i]};
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int w = 0; w < VB; ++w)
        merge[wave][16 * i + n][VB * (4 * g + r) + w] = o[i][w][r] * unit;
  }
  __syncthreads();
  // each row by kPer threads, four elements at a time
  constexpr int kPer = 64 * WAVES / R, kQuads = DP / 4;
  const int mr = tid / kPer, mi = tid % kPer;
  const int r_at = row0 + mr;
  if (r_at < rows) {
    // a token not in use sees nothing, its row's context sums notwithstanding
    const bool used = (int)fast_div((uint32_t)r_at, a.group_div) < sp.count;
    float2 st[WAVES];
    v4f sum[(kQuads + kPer - 1) / kPer], part4[(kQuads + kPer - 1) / kPer][WAVES];
#pragma unroll
    for (int w = 0; w < WAVES; ++w) st[w] = stats[w][mr];
#pragma unroll
    for (int j = 0; j < (kQuads + kPer - 1) / kPer; ++j)
#pragma unroll
      for (int w = 0; w < WAVES; ++w)
        part4[j][w] = *reinterpret_cast<const v4f*>(&merge[w][mr][4 * ((mi + kPer * j) % kQuads)]);
    float M = none;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) M = __builtin_fmaxf(M, used ? st[w].x : none);
    float L = 0.0f, f[WAVES];
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      f[w] = M == none ? 0.0f : __builtin_amdgcn_exp2f(st[w].x - M);
      if (used) L += st[w].y * f[w];   // (an unused row's sum may not be finite)
    }
#pragma unroll
    for (int j = 0; j < (kQuads + kPer - 1) / kPer; ++j) {
      sum[j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
      if (used) {
#pragma unroll
        for (int w = 0; w < WAVES; ++w) sum[j] += part4[j][w] * f[w];
      }
    }
    const int64_t at = row_at(a, b, kvh, r_at);
    const float inv = L != 0.0f ? 1.0f / L : 0.0f;
#pragma unroll
    for (int j = 0; j < (kQuads + kPer - 1) / kPer; ++j) {
      const int d = 4 * (mi + kPer * j);
      if (d < D) {
        if (whole) {
          T* dst = (T*)a.out + at * D + d;
#pragma unroll
          for (int e = 0; e < 4; ++e) dst[e] = from_float<T>(sum[j][e] * inv);
        } else {
          *reinterpret_cast<v4f*>(a.part_o + (slot * R + mr) * D + d) = sum[j];
        }
      }
    }
    if (mi == 0) {
      if (!whole) a.part_ml[slot * R + mr] = float2{M, L};
      else if (a.lse) a.lse[at] = L != 0.0f ? (M + __builtin_log2f(L)) * kLn2 : none;
    }
  }
  if (x < x_end) __syncthreads();   // merge and stats are written again
  }
}

// Joins the parts of the rows whose unit was cut: one wave per row, lane l
// elements l, l + 64, ..; up to 64 parts' maxima and sums at once, one a lane.
template <class T, int DP, int R>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a) {
  constexpr int E = DP / 64;
  const int lane = threadIdx.x & 63;
  const int64_t rows = (int64_t)a.batch * a.tokens * a.heads;
  for (int64_t at = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
       at < rows; at += (int64_t)gridDim.x * 4) {
  const int b = (int)(at / ((int64_t)a.tokens * a.heads));
  const int within = (int)(at - (int64_t)b * a.tokens * a.heads);
  const int tok = within / a.heads, head = within % a.heads;
  const int kvh = head / a.group, r = tok * a.group + head % a.group;
  Grains grains;
  const Runs runs = runs_of(a, lane, grains);
  int before, of_b;
  grains.of(a, lane, b, before, of_b);
  const int x0 = before * a.kv_heads * a.row_blocks + (kvh * a.row_blocks + r / R) * of_b;
  const int first = run_of(runs, x0), last = run_of(runs, x0 + of_b - 1);
  if (first == last) continue;   // finished where it was computed
  const int n = last - first + 1, mr = r % R;
  // part i: the first run's last slot, then the others' first
  auto slot_of = [&](int i) { return (int64_t)(2 * (first + i) + (i == 0 ? 1 : 0)) * R + mr; };
  float M = -INFINITY, L = 0.0f, x[E] = {};
  for (int s0 = 0; s0 < n; s0 += 64) {
    const float2 ml = s0 + lane < n ? a.part_ml[slot_of(s0 + lane)] : float2{-INFINITY, 0.0f};
    float top = ml.x;
#pragma unroll
    for (int m = 1; m < 64; m *= 2) top = __builtin_fmaxf(top, __shfl_xor(top, m));
    const float next = __builtin_fmaxf(M, top);
    const float old = M == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(M - next);
    const float f = ml.x == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(ml.x - next);
    float sum = ml.y * f;
#pragma unroll
    for (int m = 1; m < 64; m *= 2) sum += __shfl_xor(sum, m);
    L = L * old + sum;
    M = next;
#pragma unroll
    for (int j = 0; j < E; ++j) x[j] *= old;
    const int c = n - s0 < 64 ? n - s0 : 64;
    constexpr int B = 4;   // parts whose sums are in flight at once
    for (int i = 0; i < c; i += B) {
      float v[B][E];
#pragma unroll
      for (int u = 0; u < B; ++u) {
        const float* src = a.part_o + slot_of(i + u < c ? s0 + i + u : s0) * a.dim;
#pragma unroll
        for (int j = 0; j < E; ++j) v[u][j] = lane + 64 * j < a.dim ? src[lane + 64 * j] : 0.0f;
      }
#pragma unroll
      for (int u = 0; u < B; ++u) {
        const float w = __shfl(f, (i + u) & 63);
#pragma unroll
        for (int j = 0; j < E; ++j) x[j] += i + u < c ? v[u][j] * w : 0.0f;
      }
    }
  }
  const float inv = L != 0.0f ? 1.0f / L : 0.0f;
#pragma unroll
  for (int j = 0; j < E; ++j)
    if (lane + 64 * j < a.dim) ((T*)a.out)[at * a.dim + lane + 64 * j] = from_float<T>(x[j] * inv);
  if (lane == 0 && a.lse) a.lse[at] = L != 0.0f ? (M + __builtin_log2f(L)) * kLn2 : -INFINITY;
  }
}

// `resident`: workgroups of this shape that run at once; 0: no unit is cut
// (one launch, for caches of few keys).
template <class T, int DP, int WAVES, int QT, int TL>
hipError_t launch_shape(AttnArgs a, int resident, hipStream_t s) {
  constexpr int R = 16 * QT;
  const int64_t keys = (int64_t)a.table_pages * a.page;
  a.row_blocks = (a.tokens * a.group + R - 1) / R;
  const int64_t units = (int64_t)a.batch * a.kv_heads * a.row_blocks;
  int64_t grain = resident ? 16 * TL * WAVES : keys;
  while (units * ((keys + grain - 1) / grain) >= (int64_t)1 << 30) grain = 2 * grain < keys ? 2 * grain : keys;
  const int64_t most = units * ((keys + grain - 1) / grain);
  a.grain = (int)grain;
  // (the one-launch form: a workgroup a unit, within a launch's 2^32 threads)
  const int64_t cap = resident ? resident : 65536;
  a.groups = (int)(most < cap ? most : cap);
  a.grain_div = make_fastdiv((uint32_t)a.grain);
  a.groups_div = make_fastdiv((uint32_t)a.groups);
  a.heads_blocks_div = make_fastdiv((uint32_t)(a.kv_heads * a.row_blocks));
  const bool cut = grain < keys;
  const int64_t all = (int64_t)a.batch * a.tokens * a.heads;
  void* ws = nullptr;
  if (cut) {
    const size_t slots = (size_t)a.groups * 2 * R;
    hipError_t e = workspace_acquire(&ws, slots * (a.dim * 4 + 8), s);
    if (e != hipSuccess) return e;
    a.part_o = (float*)ws;
    a.part_ml = (float2*)((char*)ws + slots * a.dim * 4);
  }
  hipLaunchKernelGGL((k_attn<T, DP, WAVES, QT, TL>), dim3((unsigned)a.groups), dim3(64 * WAVES), 0, s, a);
  hipError_t e = hipGetLastError();
  if (cut) {
    if (e == hipSuccess) {
      hipLaunchKernelGGL((k_attn_join<T, DP, R>), dim3((unsigned)(all < (int64_t)1 << 20 ? (all + 3) / 4 : 1 << 18)), dim3(256), 0, s, a);
      e = hipGetLastError();
    }
    const hipError_t f = workspace_release(ws, s);
    if (e == hipSuccess) e = f;
  }
  return e;
}

template <class T, int DP>
hipError_t launch_dim(const AttnArgs& a, hipStream_t s) {
  const int rows = a.tokens * a.group;
  const int64_t keys = (int64_t)a.table_pages * a.page;
  constexpr int SW = DP == 256 ? 4 : 8;   // waves of the one-launch form
  constexpr int kTwo = DP == 256 ? 256 : 512;   // workgroups of four waves at once on 256 CUs
  // 32 keys a step: 64 fit fewer registers beside the loads in flight (32
  // requests x 24k keys 227 against 244 us, 1 x 700 15.0 against 15.8); two row
  // tiles a wave where there are more than 16 rows (probabilities of one part,
  // 24-token trees x 16 x 4k 80 us against 113 with one tile, 64-token trees x 4 x
  // 16k 102 against 141)
  if (rows <= 16) {
    // One workgroup of more waves a unit and no joining launch, where a few steps a
    // wave cost less than that: 8 heads, 1 request: 250 keys 10.7 us against 12.7,
    // 500 12.5 and 12.7, 700 14.7 and 13.1; 8 requests: 700 14.7 and 16.3; 64: 1000
    // 35 and 40.  Up to 128 keys four waves do without the join too (64 requests
    // x 100: 10.9 us against 16.2 with eight).
    const int64_t units = (int64_t)a.batch * a.kv_heads;
    if (keys > 128 && keys <= (units < 64 ? 64 : 128) * SW) return launch_shape<T, DP, SW, 1, 2>(a, 0, s);
    return launch_shape<T, DP, 4, 1, 2>(a, kTwo, s);
  }
  if constexpr (DP == 256) return launch_shape<T, DP, 4, 1, 2>(a, kTwo, s);
  else return launch_shape<T, DP, 4, 2, 2>(a, kTwo, s);
}

template <class T>
hipError_t launch_type(const AttnArgs& a, hipStream_t s) {
  if (a.dim <= 64) return launch_dim<T, 64>(a, s);
  if (a.dim <= 128) return launch_dim<T, 128>(a, s);
  return launch_dim<T, 256>(a, s);
}

}  // namespace

hipError_t launch_tree_attention(AttnArgs a, hipStream_t s) {
  a.group = a.heads / a.kv_heads;
  a.q_aligned = (((uintptr_t)a.q | (uintptr_t)(2 * (a.q_bs | a.q_ts | a.q_hs))) & 15) == 0;
  a.page_div = make_fastdiv((uint32_t)a.page);
  a.group_div = make_fastdiv((uint32_t)a.group);
  return a.dtype == Q8TA_F16 ? launch_type<Half>(a, s) : launch_type<Bfloat>(a, s);
}

}  // namespace q8ta
