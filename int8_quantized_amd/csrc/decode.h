// Arguments and launchers of the decode-step operators: rotary positions with
// the int8 cache append, tree attention over that cache, the linear with
// low-rank adapters, and token sampling.
#pragma once

#include "../../include/q8ta.h"

#include "q8ta_internal.h"

namespace q8ta {

// Records the message of a failed call (q8ta_last_error) and returns st.
q8ta_status report(q8ta_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));

// Unsigned division of n < 2^31 by a fixed d in [1, 2^31): with
// l = ceil(log2 d) and m = floor(2^(31+l) / d) + 1 (< 2^32), n * m / 2^(31+l)
// exceeds n / d by n * (m * d - 2^(31+l)) / (d * 2^(31+l)), where
// 0 < m * d - 2^(31+l) <= d <= 2^l: by at most n / (d * 2^31) < 1 / d, so the
// floor is the quotient's.
struct FastDiv {
  uint32_t mul = 0, d = 1;
  int shift = 31;
};
inline FastDiv make_fastdiv(uint32_t d) {
  int l = 0;
  while (((uint64_t)1 << l) < d) ++l;
  FastDiv f;
  f.d = d;
  f.shift = 31 + l;
  f.mul = (uint32_t)((((uint64_t)1 << (31 + l)) / d) + 1);
  return f;
}
__host__ __device__ __forceinline__ uint32_t fast_div(uint32_t n, const FastDiv& f) {
  return (uint32_t)(((uint64_t)n * f.mul) >> f.shift);
}

// Where the keys of a request's grains up to g1 (not included) end: `total` keys
// in `grains` grains of `grain`.  (The last grain's end may pass 2^31.)
__host__ __device__ __forceinline__ int grains_end(int total, int grains, int grain, int g1) {
  return g1 == grains ? total : g1 * grain;
}

// 16-bit floating-point values by their bits.
struct Half {
  uint16_t bits;
};
struct Bfloat {
  uint16_t bits;
};
__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(Half x) { return (float)__builtin_bit_cast(_Float16, x.bits); }
__device__ __forceinline__ float to_float(Bfloat x) {
  return __builtin_bit_cast(float, (uint32_t)x.bits << 16);
}
// One rounding to nearest even; NaN stays NaN.
template <class T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ Half from_float<Half>(float x) {
  return Half{__builtin_bit_cast(uint16_t, (_Float16)x)};
}
template <>
__device__ __forceinline__ Bfloat from_float<Bfloat>(float x) {
  return Bfloat{__builtin_bit_cast(uint16_t, (__bf16)x)};
}

struct RopeArgs {
  const void *q, *k, *v;                         // [tokens, heads, dim] views, unit inner stride
  int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs;   // token and head strides in elements
  int dtype;
  int64_t tokens;
  int heads, kv_heads, dim, rot;
  const int32_t* positions;
  const int64_t* slots;
  const double* inv_freq;
  double factor;
  bool interleaved;
  void* q_out;
  int8_t* cache;
  float* scales;
  int64_t pages, page;
};
hipError_t launch_rope_append(const RopeArgs& a, hipStream_t s);

struct AttnArgs {
  const void* q;            // [batch, tokens, heads, dim] view, unit inner stride
  int64_t q_bs, q_ts, q_hs;
  bool q_aligned;           // every row starts on 16 bytes
  int dtype;
  int batch, tokens, heads, kv_heads, group, dim;   // group = heads / kv_heads
  const int8_t* cache;      // [pages, 2, kv_heads, page, dim]
  const float* scales;      // [pages, 2, kv_heads, page]
  int64_t pages;
  int page;
  FastDiv page_div, group_div;
  const int32_t* table;     // [batch, table_pages]
  int table_pages;
  const int32_t* lens;      // [batch]
  const int32_t* counts;    // [batch] or NULL
  const int64_t* mask;      // [batch, tokens] or NULL
  float scale;              // softmax scale
  void* out;                // [batch, tokens, heads, dim]
  float* lse;               // [batch, tokens, heads] or NULL
  // Row blocks of a key head; keys of a grain; workgroups; and where a cut
  // unit's sums go: part_o [slots, rows of a block, dim] and part_ml [slots,
  // rows of a block] (running maximum in powers of two, sum), two slots a
  // workgroup (see grains_of in attention.hip).
  int row_blocks, grain, groups;
  FastDiv grain_div, groups_div, heads_blocks_div;
  float* part_o;
  float2* part_ml;
};
hipError_t launch_tree_attention(AttnArgs a, hipStream_t s);

struct SampleArgs {
  const void* logits;       // [rows, vocab], row stride in elements
  int64_t row_stride;
  int dtype;
  int rows, vocab;
  int shift;                // a weight of 1 is 2^shift in whole numbers
  const float* temperature;
  const int32_t* top_k;     // NULL: off
  const float* top_p;       // NULL: off
  const float* min_p;       // NULL: off
  const float* u;
  int32_t* tokens;
  float* logprobs;          // NULL: not wanted
};
hipError_t launch_sample(const SampleArgs& a, hipStream_t s);

constexpr int kLoraParts = 3;   // 3 x 8 bits and their signs hold fp32's 24

// The linear with low-rank adapters: lin holds x, w, the scales, bias, sizes
// and the input zero point (lin.rq.s_in the input scale); row m adds
// adapter_scale * B (A (x - zp) s_in) of adapter ids[m].
struct LoraArgs {
  LinearArgs lin;
  const void *a, *b;        // [adapters, rank, K], [adapters, N, rank]
  int ad_type;
  int adapters, rank;
  int rank_pad;             // rank rounded up to 16
  const float* ad_scales;   // NULL: 1
  const int32_t* ranks;     // NULL: rank each
  const int32_t* ids;
  bool relu;
  void* y;
  int y_type;
  int64_t n0 = 0;           // first channel of a launch of the row kernel
  // t[m, r] = adapter_scale * s_in * sum_k A[r, k] (x[m, k] - zp) of the row's
  // adapter (0 past its rank), [M, rank_pad]; rows without one are not written.
  // With in_parts, as kLoraParts bf16 values whose sum it is, [kLoraParts, M,
  // rank_pad], instead.
  float* t = nullptr;
  uint16_t* tp = nullptr;
  bool in_parts = false;
};
// The adapter of row m, -1 for none (any id outside [0, adapters)).
__device__ __forceinline__ int adapter_of(const LoraArgs& a, int64_t m) {
  const int id = a.ids[m];
  return id >= 0 && id < a.adapters ? id : -1;
}
__device__ __forceinline__ int rank_of(const LoraArgs& a, int id) {
  if (!a.ranks) return a.rank;
  const int r = a.ranks[id];
  return r < 0 ? 0 : (r < a.rank ? r : a.rank);
}
hipError_t launch_linear_lora(LoraArgs a, hipStream_t s);
// The large GEMMs with the adapters' epilogue (t formed before): K and
// alignment as for launch_gemm_w8 / launch_gemm_mx.
hipError_t launch_gemm_w8_lora(const LoraArgs& a, hipStream_t s);
hipError_t launch_gemm_mx_lora(const LoraArgs& a, hipStream_t s);

}  // namespace q8ta
