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
// the 16x16x32 fp16 matrix instruction:
//  * Codes are whole numbers of [-128, 127] and exact in fp16: byte b ^ 0x80
//    under the exponent byte 0x64 is 1024 + 128 + code, less 1152.  Two
//    operations for two elements, no table and no 32-bit detour.
//  * Queries: fp16 as they are; bf16 rows scaled by a power of two that puts
//    their largest element in [2^14, 2^15) (undone on the scores), where fp16
//    holds every element exactly but those more than 2^28 below the
//    largest.  So a score is a sum of exact products in 32 bits.
//  * The keys are the A operand: lane l gets the scores of query l % 16 for
//    keys 16t + 4(l / 16) + r, which is also where the B operand of the second
//    product wants the probabilities if its K slots are numbered to match
//    (slot 8g + j = key 4g + j of the first 16-key tile for j < 4, key 4g + j - 4
//    of the second beyond), so they never leave their registers, and a
//    query's maximum, sum and rescaling are its lanes' own.
//  * Values: lane (i, g) loads VB = DP / 16 bytes of each of four neighbouring keys
//    and transposes them with byte permutes while it widens them to fp16.
//  * Probabilities are rounded to fp16 for the second product (half a step is
//    2^-12 of each, against 2^-9 or 2^-12 of the output's own rounding; the sum
//    that divides them stays 32-bit).  The value's scale goes onto its
//    probability, divided by a power of two near the largest scale so far and
//    times 2^10: products up to 2^15 leave fp16's range below for weights down
//    to 2^-34 of the largest, whatever the scales are.
//  * The maximum is renewed only when a score passes it by 2^4, the values'
//    power of two when a scale passes twice it: most steps need no exchange
//    between lanes and no rescaling.
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

constexpr int kWaves = 4;
constexpr int kStep = 64;       // keys a wave takes per step
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kMargin = 4.0f;   // a score may pass the running maximum by 2^4
constexpr int kLift = 10;         // weights are held times 2^kLift

union Frag {
  v8h h;
  uint32_t u[4];
};

__device__ __forceinline__ uint32_t less1152(uint32_t x) {
  const v2h c = v2h{(_Float16)-1152.0f, (_Float16)-1152.0f};
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(v2h, x) + c);
}

// Eight codes (two words, byte order) as fp16.
__device__ __forceinline__ v8h widen8(uint32_t w0, uint32_t w1) {
  const uint32_t k = 0x64646464u;
  Frag f;
  w0 ^= 0x80808080u;
  w1 ^= 0x80808080u;
  f.u[0] = less1152(__builtin_amdgcn_perm(w0, k, 0x00050004u));
  f.u[1] = less1152(__builtin_amdgcn_perm(w0, k, 0x00070006u));
  f.u[2] = less1152(__builtin_amdgcn_perm(w1, k, 0x00050004u));
  f.u[3] = less1152(__builtin_amdgcn_perm(w1, k, 0x00070006u));
  return f.h;
}

// Byte B of words a and b (two keys, one element) as a pair of fp16.
template <int B>
__device__ __forceinline__ uint32_t widen_pair(uint32_t a, uint32_t b) {
  constexpr uint32_t sel = 0x0c000c00u | (uint32_t)(4 + B) << 16 | (uint32_t)B;
  return less1152(__builtin_amdgcn_perm(b, a, sel) ^ 0x64806480u);
}
__device__ __forceinline__ uint32_t widen_pair(uint32_t a, uint32_t b, int byte) {
  switch (byte) {
    case 0: return widen_pair<0>(a, b);
    case 1: return widen_pair<1>(a, b);
    case 2: return widen_pair<2>(a, b);
    default: return widen_pair<3>(a, b);
  }
}

__device__ __forceinline__ uint32_t pack_half(float a, float b) {
  const v2h v = v2h{(_Float16)a, (_Float16)b};
  return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ float pow2f(int e) {   // 2^e, -126 <= e <= 127
  return __builtin_bit_cast(float, (uint32_t)(e + 127) << 23);
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

// The queries of one 16-row tile as B operands: element e of operand k holds
// d = 16 * (4 * (k / 2) + g) + 8 * (k % 2) + e.  `fac` turns a product of codes
// into a score in powers of two (softmax scale and log2 e included).
template <class T, int DP>
__device__ __forceinline__ void load_queries(const AttnArgs& a, const T* src, bool live, int g,
                                             v8h (&q)[DP / 32], float& fac) {
  constexpr bool kBf = std::is_same<T, Bfloat>::value;
  fac = a.scale * kLog2e;
  float top = 0.0f;
  v4u raw[DP / 32];
#pragma unroll
  for (int k = 0; k < DP / 32; ++k) {
    const int d = 16 * (4 * (k / 2) + g) + 8 * (k % 2);
    raw[k] = v4u{0, 0, 0, 0};
    if (live && d < a.dim) {
      // rows start on element boundaries only (any strides)
      const T* p = src + d;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        raw[k][e] = (uint32_t)p[2 * e].bits | (uint32_t)p[2 * e + 1].bits << 16;
    }
  }
  if constexpr (!kBf) {
#pragma unroll
    for (int k = 0; k < DP / 32; ++k) q[k] = __builtin_bit_cast(v8h, raw[k]);
  } else {
#pragma unroll
    for (int k = 0; k < DP / 32; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        top = __builtin_fmaxf(top, __builtin_fabsf(__builtin_bit_cast(float, raw[k][e] << 16)));
        top = __builtin_fmaxf(top, __builtin_fabsf(__builtin_bit_cast(float, raw[k][e] & 0xffff0000u)));
      }
    top = __builtin_fmaxf(top, __shfl_xor(top, 16));
    top = __builtin_fmaxf(top, __shfl_xor(top, 32));
    int sh = 14 - ((int)(__builtin_bit_cast(uint32_t, top) >> 23) - 127);
    sh = sh < -112 ? -112 : (sh > 112 ? 112 : sh);
    const float up = pow2f(sh);
    fac = fac * pow2f(-sh);
#pragma unroll
    for (int k = 0; k < DP / 32; ++k) {
      Frag f;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        f.u[e] = pack_half(__builtin_bit_cast(float, raw[k][e] << 16) * up,
                           __builtin_bit_cast(float, raw[k][e] & 0xffff0000u) * up);
      q[k] = f.h;
    }
  }
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

// Up to 16 query rows of one key head and a stretch of the keys, the waves of
// the workgroup each taking every kWaves-th step of 64 keys straight from
// memory into operands; their sums meet in LDS at the end.  DP: dim rounded up
// to 64, 128 or 256.
template <class T, int DP>
__global__ __launch_bounds__(64 * kWaves) void k_attn_rows16(AttnArgs a) {
  constexpr int U = DP / 64, VB = DP / 16;
  __shared__ __attribute__((aligned(16))) float merge[kWaves][16][DP];
  __shared__ float2 stats[kWaves][16];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int b = blockIdx.z;
  const int kvh = blockIdx.y % a.kv_heads, row0 = blockIdx.y / a.kv_heads * 16;
  const int split = blockIdx.x;
  const int rows = a.tokens * a.group;
  const int D = a.dim;
  const Span sp = span_of(a, b);
  const int k_begin = split * a.chunk;
  const int k_end = sp.total - k_begin < a.chunk ? sp.total : k_begin + a.chunk;
  if (k_begin >= k_end && a.splits > 1) return;   // the joining pass knows which splits wrote

  const int row = row0 + n;
  const bool live = row < rows;
  const int tok = live ? (int)fast_div((uint32_t)row, a.group_div) : 0;
  const uint64_t bits = live ? seen_bits(a, sp, b, tok) : 0;
  v8h q[DP / 32];
  float fac;
  load_queries<T, DP>(a, (const T*)a.q + b * a.q_bs + tok * a.q_ts +
                             (int64_t)(kvh * a.group + (row - tok * a.group)) * a.q_hs,
                      live, g, q, fac);

  const int64_t part = (int64_t)a.kv_heads * a.page;   // rows from a page's keys to its values
  uint32_t k_raw[4][U][4];
  Bytes<VB> v_raw[4][4];
  v4f ks[4], vs[4];
  int64_t prow[4];   // cache row of each 16-key tile's first key
  bool bad = false;  // a tile whose page is not one
  auto find = [&](int step) {
    bad = false;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int key = step + 16 * t;
      int idx = (int)fast_div((uint32_t)key, a.page_div);
      const int within = key - idx * a.page;
      idx = idx < a.table_pages ? idx : a.table_pages - 1;
      int64_t pg = a.table[(int64_t)b * a.table_pages + idx];
      const bool ok = pg >= 0 && pg < a.pages;
      if (!ok && key < sp.total) bad = true;
      if (!ok) pg = 0;
      prow[t] = (pg * 2 * a.kv_heads + kvh) * a.page + within;
    }
  };
  auto load_k = [&] {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int8_t* base = a.cache + prow[t] * D;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = 16 * (4 * u + g);
        v4u v = v4u{0, 0, 0, 0};
        if (c < D) v = *reinterpret_cast<const v4u*>(base + (n * D + c));
#pragma unroll
        for (int i = 0; i < 4; ++i) k_raw[t][u][i] = v[i];
      }
      ks[t] = *reinterpret_cast<const v4f*>(a.scales + prow[t] + 4 * g);
      vs[t] = *reinterpret_cast<const v4f*>(a.scales + prow[t] + part + 4 * g);
    }
  };
  auto load_v = [&] {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int8_t* base = a.cache + (prow[t] + part) * D;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (VB * n < D) {
          v_raw[t][r] = load_bytes<VB>(base + ((4 * g + r) * D + VB * n));
        } else {
#pragma unroll
          for (int i = 0; i < VB / 4; ++i) v_raw[t][r].w[i] = 0;
        }
      }
    }
  };

  float m = -INFINITY, l = 0.0f;
  v4f o[VB];
#pragma unroll
  for (int w = 0; w < VB; ++w) o[w] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  float unit = 1.0f, inv_unit = 1.0f, limit = 0.0f;   // the values' power of two

  for (int step = k_begin + kStep * wave; step < k_end; step += kStep * kWaves) {
    find(step);
    load_k();
    load_v();
    // scores of keys 16t + 4g + r, in powers of two
    float s[4][4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      v4f acc = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int u = 0; u < U; ++u) {
        acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(widen8(k_raw[t][u][0], k_raw[t][u][1]),
                                                     q[2 * u], acc, 0, 0, 0);
        acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(widen8(k_raw[t][u][2], k_raw[t][u][3]),
                                                     q[2 * u + 1], acc, 0, 0, 0);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) s[t][r] = acc[r] * (ks[t][r] * fac);
    }
    // past the context: keys this row does not see (their scales may hold
    // anything, so both are replaced rather than multiplied away)
    if (step + kStep > sp.ctx || step + kStep > k_end || bad) {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        int idx = (int)fast_div((uint32_t)(step + 16 * t), a.page_div);
        idx = idx < a.table_pages ? idx : a.table_pages - 1;
        const int pg = a.table[(int64_t)b * a.table_pages + idx];
        const bool ok = pg >= 0 && pg < a.pages;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int key = step + 16 * t + 4 * g + r;
          const int at = key - sp.ctx;
          const bool seen = ok && key < k_end && (at < 0 || ((bits >> (at & 63)) & 1));
          s[t][r] = seen ? s[t][r] : -INFINITY;
          vs[t][r] = seen ? vs[t][r] : 0.0f;
        }
      }
    }
    float top = s[0][0], vtop = 0.0f;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        top = __builtin_fmaxf(top, s[t][r]);
        vtop = __builtin_fmaxf(vtop, __builtin_fabsf(vs[t][r]));
      }
    if (__any(vtop > limit)) {
#pragma unroll
      for (int x = 1; x < 64; x *= 2) vtop = __builtin_fmaxf(vtop, __shfl_xor(vtop, x));
      int e = (int)(__builtin_bit_cast(uint32_t, vtop) >> 23) - 127;
      e = e < -110 ? -110 : (e > 110 ? 110 : e);
      const float next = pow2f(e - kLift);
      inv_unit = pow2f(kLift - e);
      const float f = unit * inv_unit;
#pragma unroll
      for (int w = 0; w < VB; ++w) o[w] *= f;
      unit = next;
      limit = pow2f(e + 1);
    }
    if (__any(top > m + kMargin)) {
      top = __builtin_fmaxf(top, __shfl_xor(top, 16));
      top = __builtin_fmaxf(top, __shfl_xor(top, 32));
      const float next = __builtin_fmaxf(m, top);
      const float f = next == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - next);
      m = next;
      l *= f;
#pragma unroll
      for (int w = 0; w < VB; ++w) o[w] *= f;
    }
    const float base = m == -INFINITY ? 0.0f : m;
    Frag p[2];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      float x[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float e = __builtin_amdgcn_exp2f(s[t][r] - base);
        l += e;
        x[r] = e * (vs[t][r] * inv_unit);
      }
      p[t / 2].u[2 * (t % 2)] = pack_half(x[0], x[1]);
      p[t / 2].u[2 * (t % 2) + 1] = pack_half(x[2], x[3]);
    }
#pragma unroll
    for (int w = 0; w < VB; ++w) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        Frag f;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const Bytes<VB>(&v)[4] = v_raw[2 * h + t];
          f.u[2 * t] = widen_pair(v[0].w[w / 4], v[1].w[w / 4], w % 4);
          f.u[2 * t + 1] = widen_pair(v[2].w[w / 4], v[3].w[w / 4], w % 4);
        }
        o[w] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f.h, p[h].h, o[w], 0, 0, 0);
      }
    }
  }

  // o[w][r]: query n, d = VB * (4g + r) + w
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  if (g == 0) stats[wave][n] = float2{m, l};
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int w = 0; w < VB; ++w) merge[wave][n][VB * (4 * g + r) + w] = o[w][r] * unit;
  __syncthreads();
  // each row by 16 threads, DP / 16 elements apart
  const int mr = tid / 16, mi = tid % 16;
  const int r_at = row0 + mr;
  if (r_at >= rows) return;
  // a token not in use sees nothing, its row's context sums notwithstanding
  const bool used = (int)fast_div((uint32_t)r_at, a.group_div) < sp.count;
  float M = -INFINITY;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) M = __builtin_fmaxf(M, used ? stats[w][mr].x : -INFINITY);
  float L = 0.0f, f[kWaves];
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    f[w] = M == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(stats[w][mr].x - M);
    L += stats[w][mr].y * f[w];
  }
  const int64_t at = row_at(a, b, kvh, r_at);
  const float inv = a.splits > 1 ? 1.0f : (L != 0.0f ? 1.0f / L : 0.0f);
#pragma unroll
  for (int j = 0; j < DP / 16; ++j) {
    const int d = mi + 16 * j;
    float x = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) x += merge[w][mr][d] * f[w];
    if (d < D) {
      if (a.splits > 1)
        a.part_o[((int64_t)split * a.batch * a.tokens * a.heads + at) * D + d] = x;
      else
        ((T*)a.out)[at * D + d] = from_float<T>(x * inv);
    }
  }
  if (mi == 0) {
    if (a.splits > 1)
      a.part_ml[(int64_t)split * a.batch * a.tokens * a.heads + at] = float2{M, L};
    else if (a.lse)
      a.lse[at] = L != 0.0f ? (M + __builtin_log2f(L)) * kLn2 : -INFINITY;
  }
}

// Joins the splits of each row: one wave per row, lane l elements l, l + 64, ..
template <class T>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t rows = (int64_t)a.batch * a.tokens * a.heads;
  const int64_t at = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (at >= rows) return;
  const int b = (int)(at / ((int64_t)a.tokens * a.heads));
  const Span sp = span_of(a, b);
  const int n = (sp.total + a.chunk - 1) / a.chunk;
  float M = -INFINITY;
  for (int s = 0; s < n; ++s) M = __builtin_fmaxf(M, a.part_ml[s * rows + at].x);
  float L = 0.0f, x[4] = {};
  for (int s = 0; s < n; ++s) {
    const float2 ml = a.part_ml[s * rows + at];
    const float f = M == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(ml.x - M);
    L += ml.y * f;
    const float* src = a.part_o + (s * rows + at) * a.dim;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (lane + 64 * j < a.dim) x[j] += src[lane + 64 * j] * f;
  }
  const float inv = L != 0.0f ? 1.0f / L : 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (lane + 64 * j < a.dim) ((T*)a.out)[at * a.dim + lane + 64 * j] = from_float<T>(x[j] * inv);
  if (lane == 0 && a.lse) a.lse[at] = L != 0.0f ? (M + __builtin_log2f(L)) * kLn2 : -INFINITY;
}

template <class T>
hipError_t launch_type(AttnArgs a, hipStream_t s) {
  const int rows = a.tokens * a.group;
  const int tiles = (rows + 15) / 16;
  const int64_t base = (int64_t)a.batch * a.kv_heads * tiles;
  const int64_t keys = (int64_t)a.table_pages * a.page;
  constexpr int kGrain = kStep * kWaves;
  int64_t splits = (2048 + base - 1) / base;
  int64_t chunk = (keys + splits - 1) / splits;
  chunk = (chunk + kGrain - 1) / kGrain * kGrain;
  splits = (keys + chunk - 1) / chunk;
  a.chunk = (int)chunk;
  a.splits = (int)splits;
  const int64_t all = (int64_t)a.batch * a.tokens * a.heads;
  void* ws = nullptr;
  if (splits > 1) {
    const size_t o_bytes = (size_t)splits * all * a.dim * 4;
    hipError_t e = workspace_acquire(&ws, o_bytes + (size_t)splits * all * 8, s);
    if (e != hipSuccess) return e;
    a.part_o = (float*)ws;
    a.part_ml = (float2*)((char*)ws + o_bytes);
  }
  const dim3 grid((unsigned)splits, (unsigned)(a.kv_heads * tiles), (unsigned)a.batch);
  if (a.dim <= 64)
    hipLaunchKernelGGL((k_attn_rows16<T, 64>), grid, dim3(64 * kWaves), 0, s, a);
  else if (a.dim <= 128)
    hipLaunchKernelGGL((k_attn_rows16<T, 128>), grid, dim3(64 * kWaves), 0, s, a);
  else
    hipLaunchKernelGGL((k_attn_rows16<T, 256>), grid, dim3(64 * kWaves), 0, s, a);
  hipError_t e = hipGetLastError();
  if (splits > 1) {
    if (e == hipSuccess) {
      hipLaunchKernelGGL((k_attn_join<T>), dim3((unsigned)((all + 3) / 4)), dim3(256), 0, s, a);
      e = hipGetLastError();
    }
    const hipError_t f = workspace_release(ws, s);
    if (e == hipSuccess) e = f;
  }
  return e;
}

}  // namespace

hipError_t launch_tree_attention(AttnArgs a, hipStream_t s) {
  a.group = a.heads / a.kv_heads;
  a.page_div = make_fastdiv((uint32_t)a.page);
  a.group_div = make_fastdiv((uint32_t)a.group);
  return a.dtype == Q8TA_F16 ? launch_type<Half>(a, s) : launch_type<Bfloat>(a, s);
}

}  // namespace q8ta
