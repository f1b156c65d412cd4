// C entry points of the decode-step operators: argument checks, then the
// launch.  Every check runs before any HIP call.
#include <cmath>
#include <cstring>

#include "decode.h"

using namespace q8ta;

namespace {

constexpr int64_t kMaxElems = (int64_t)1 << 40;

q8ta_status hip_status(hipError_t e, const char* what) {
  if (e == hipSuccess) return Q8TA_OK;
  return report(Q8TA_ERR_HIP, "%s: HIP error %d (%s)", what, (int)e, hipGetErrorString(e));
}

bool dtype_ok(int d) { return d == Q8TA_F32 || d == Q8TA_F16 || d == Q8TA_BF16; }

// a * b * .. <= 2^40 for factors >= 1.
bool fits(std::initializer_list<int64_t> f) {
  int64_t left = kMaxElems;
  for (int64_t x : f) {
    if (x > left) return false;
    left /= x;
  }
  return true;
}

}  // namespace

extern "C" {

q8ta_status q8ta_rope_append(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                             const void* k, int64_t k_token_stride, int64_t k_head_stride,
                             const void* v, int64_t v_token_stride, int64_t v_head_stride,
                             q8ta_dtype dtype, int64_t tokens, int64_t heads, int64_t kv_heads,
                             int64_t dim, const int32_t* positions, const int64_t* slots,
                             const double* inv_freq, int64_t rot, double factor,
                             int64_t interleaved, void* q_out, int8_t* cache, float* cache_scales,
                             int64_t pages, int64_t page_size, hipStream_t stream) {
  const char* op = "q8ta_rope_append";
  if (!dtype_ok(dtype)) return report(Q8TA_ERR_UNSUPPORTED, "%s: unknown dtype %d", op, (int)dtype);
  if (tokens < 0 || tokens >= ((int64_t)1 << 31))
    return report(Q8TA_ERR_SHAPE, "%s: tokens out of range (%lld)", op, (long long)tokens);
  if (heads < 1 || kv_heads < 1 || heads > 65535 || kv_heads > 65535 || heads + 2 * kv_heads > 65535)
    return report(Q8TA_ERR_SHAPE, "%s: heads and kv_heads must be >= 1 and heads + 2 * kv_heads <= "
                  "65535 (got %lld, %lld)", op, (long long)heads, (long long)kv_heads);
  if (dim < 1 || dim > 65536)
    return report(Q8TA_ERR_SHAPE, "%s: dim must be in [1, 65536] (got %lld)", op, (long long)dim);
  if (rot < 0 || rot > dim || rot % 2 != 0)
    return report(Q8TA_ERR_SHAPE, "%s: rot must be even and in [0, dim] (got %lld of %lld)", op,
                  (long long)rot, (long long)dim);
  if (pages < 1 || page_size < 1 || !fits({pages, page_size, kv_heads, dim, 2}))
    return report(Q8TA_ERR_SHAPE, "%s: pages and page_size must be >= 1 and the cache at most 2^40 "
                  "elements (got %lld, %lld)", op, (long long)pages, (long long)page_size);
  if (tokens > 0 && !fits({tokens, heads, dim}))
    return report(Q8TA_ERR_SHAPE, "%s: sizes too large", op);
  for (int64_t st : {q_token_stride, q_head_stride, k_token_stride, k_head_stride, v_token_stride,
                     v_head_stride})
    if (st < 0 || st > kMaxElems)
      return report(Q8TA_ERR_SHAPE, "%s: strides must be in [0, 2^40] (got %lld)", op, (long long)st);
  if (!std::isfinite(factor))
    return report(Q8TA_ERR_QPARAM, "%s: factor must be finite (got %g)", op, factor);
  if (interleaved != 0 && interleaved != 1)
    return report(Q8TA_ERR_UNSUPPORTED, "%s: interleaved must be 0 or 1 (got %lld)", op,
                  (long long)interleaved);
  if (tokens == 0) return Q8TA_OK;
  if (!q || !k || !v || !positions || !slots || !q_out || !cache || !cache_scales ||
      (rot > 0 && !inv_freq))
    return report(Q8TA_ERR_NULL, "%s: a required pointer is NULL", op);
  RopeArgs a{};
  a.q = q; a.k = k; a.v = v;
  a.q_ts = q_token_stride; a.q_hs = q_head_stride; a.k_ts = k_token_stride;
  a.k_hs = k_head_stride; a.v_ts = v_token_stride; a.v_hs = v_head_stride;
  a.dtype = dtype; a.tokens = tokens; a.heads = (int)heads; a.kv_heads = (int)kv_heads;
  a.dim = (int)dim; a.rot = (int)rot; a.positions = positions; a.slots = slots;
  a.inv_freq = inv_freq; a.factor = factor; a.interleaved = interleaved != 0; a.q_out = q_out;
  a.cache = cache; a.scales = cache_scales; a.pages = pages; a.page = page_size;
  return hip_status(launch_rope_append(a, stream), op);
}

q8ta_status q8ta_tree_attention(const void* q, int64_t q_batch_stride, int64_t q_token_stride,
                                int64_t q_head_stride, q8ta_dtype dtype, int64_t batch,
                                int64_t tokens, int64_t heads, int64_t kv_heads, int64_t dim,
                                const int8_t* cache, const float* cache_scales, int64_t pages,
                                int64_t page_size, const int32_t* table, int64_t table_pages,
                                const int32_t* lens, const int32_t* counts, const int64_t* mask,
                                double softmax_scale, void* out, float* lse, hipStream_t stream) {
  const char* op = "q8ta_tree_attention";
  if (dtype != Q8TA_F16 && dtype != Q8TA_BF16)
    return report(Q8TA_ERR_UNSUPPORTED, "%s: dtype must be fp16 or bf16 (got %d)", op, (int)dtype);
  if (batch < 0 || batch > 65535)
    return report(Q8TA_ERR_SHAPE, "%s: batch must be in [0, 65535] (got %lld)", op, (long long)batch);
  if (tokens < 1 || tokens > 64)
    return report(Q8TA_ERR_SHAPE, "%s: tokens must be in [1, 64] (got %lld)", op, (long long)tokens);
  if (heads < 1 || kv_heads < 1 || heads > 65535 || heads % kv_heads != 0)
    return report(Q8TA_ERR_SHAPE, "%s: heads must be a multiple of kv_heads and at most 65535 (got "
                  "%lld, %lld)", op, (long long)heads, (long long)kv_heads);
  // rows of a key head in tiles of 16, times the key heads
  const int64_t blocks = kv_heads * ((tokens * (heads / kv_heads) + 15) / 16);
  if (blocks > 65535)
    return report(Q8TA_ERR_SHAPE, "%s: too many heads (%lld) for %lld tokens", op, (long long)heads,
                  (long long)tokens);
  if (batch * blocks > (int64_t)1 << 29)
    return report(Q8TA_ERR_SHAPE, "%s: batch (%lld) times row tiles of 16 (%lld) must be at most 2^29",
                  op, (long long)batch, (long long)blocks);
  if (dim < 1) return report(Q8TA_ERR_SHAPE, "%s: dim must be >= 1 (got %lld)", op, (long long)dim);
  if (dim % 16 != 0 || dim > 256)
    return report(Q8TA_ERR_UNSUPPORTED, "%s: dim must be a multiple of 16 up to 256 (got %lld)", op,
                  (long long)dim);
  if (pages < 1 || page_size < 1 || table_pages < 1 || page_size >= ((int64_t)1 << 31) ||
      !fits({pages, page_size, kv_heads, dim, 2}))
    return report(Q8TA_ERR_SHAPE, "%s: pages, page_size and table_pages must be >= 1 and the cache at "
                  "most 2^40 elements (got %lld, %lld, %lld)", op, (long long)pages,
                  (long long)page_size, (long long)table_pages);
  if (table_pages > (((int64_t)1 << 31) - 1024) / page_size)
    return report(Q8TA_ERR_SHAPE, "%s: table_pages * page_size must be at most 2^31 - 1024", op);
  if (page_size % 16 != 0)
    return report(Q8TA_ERR_UNSUPPORTED, "%s: page_size must be a multiple of 16 (got %lld)", op,
                  (long long)page_size);
  for (int64_t st : {q_batch_stride, q_token_stride, q_head_stride})
    if (st < 0 || st > kMaxElems)
      return report(Q8TA_ERR_SHAPE, "%s: strides must be in [0, 2^40] (got %lld)", op, (long long)st);
  if (!std::isfinite(softmax_scale) || !(softmax_scale > 0.0) || !std::isfinite((float)softmax_scale) ||
      (float)softmax_scale == 0.0f)
    return report(Q8TA_ERR_QPARAM, "%s: softmax_scale must be finite and > 0 (got %g)", op, softmax_scale);
  if (batch == 0) return Q8TA_OK;
  if (!q || !cache || !cache_scales || !table || !lens || !out)
    return report(Q8TA_ERR_NULL, "%s: a required pointer is NULL", op);
  if (((uintptr_t)cache | (uintptr_t)cache_scales) & 15)
    return report(Q8TA_ERR_UNSUPPORTED, "%s: cache and cache_scales must be 16-byte aligned", op);
  AttnArgs a{};
  a.q = q; a.q_bs = q_batch_stride; a.q_ts = q_token_stride; a.q_hs = q_head_stride;
  a.dtype = dtype; a.batch = (int)batch; a.tokens = (int)tokens; a.heads = (int)heads;
  a.kv_heads = (int)kv_heads; a.dim = (int)dim; a.cache = cache; a.scales = cache_scales;
  a.pages = pages; a.page = (int)page_size; a.table = table; a.table_pages = (int)table_pages;
  a.lens = lens; a.counts = counts; a.mask = mask; a.scale = (float)softmax_scale; a.out = out;
  a.lse = lse;
  return hip_status(launch_tree_attention(a, stream), op);
}

q8ta_status q8ta_sample(const void* logits, int64_t row_stride, q8ta_dtype dtype, int64_t rows,
                        int64_t vocab, const float* temperature, const int32_t* top_k,
                        const float* top_p, const float* min_p, const float* u, int32_t* tokens,
                        float* logprobs, hipStream_t stream) {
  const char* op = "q8ta_sample";
  if (!dtype_ok(dtype)) return report(Q8TA_ERR_UNSUPPORTED, "%s: unknown dtype %d", op, (int)dtype);
  if (rows < 0 || rows >= ((int64_t)1 << 31))
    return report(Q8TA_ERR_SHAPE, "%s: rows out of range (%lld)", op, (long long)rows);
  if (vocab < 1 || vocab > ((int64_t)1 << 24))
    return report(Q8TA_ERR_SHAPE, "%s: vocab must be in [1, 2^24] (got %lld)", op, (long long)vocab);
  if (rows > 1 && (row_stride < vocab || row_stride > kMaxElems / rows))
    return report(Q8TA_ERR_SHAPE, "%s: row_stride must be >= vocab and rows * row_stride <= 2^40 (got "
                  "%lld)", op, (long long)row_stride);
  if (rows == 0) return Q8TA_OK;
  if (!logits || !temperature || !u || !tokens)
    return report(Q8TA_ERR_NULL, "%s: logits, temperature, u and tokens must not be NULL", op);
  SampleArgs a{};
  a.logits = logits; a.row_stride = row_stride; a.dtype = dtype; a.rows = (int)rows;
  a.vocab = (int)vocab; a.temperature = temperature; a.top_k = top_k; a.top_p = top_p;
  a.min_p = min_p; a.u = u; a.tokens = tokens; a.logprobs = logprobs;
  int bits = 0;
  while (((int64_t)1 << bits) < vocab) ++bits;
  a.shift = 62 - bits < 50 ? 62 - bits : 50;
  return hip_status(launch_sample(a, stream), op);
}

q8ta_status q8ta_linear_lora(const int8_t* x, int64_t M, int64_t K, double input_scale,
                             int64_t input_zero_point, const int8_t* weight, int64_t N,
                             const float* weight_scales, const float* bias, const void* lora_a,
                             const void* lora_b, q8ta_dtype adapter_dtype, int64_t adapters,
                             int64_t rank, const float* adapter_scales, const int32_t* ranks,
                             const int32_t* adapter_ids, const char* activation, void* out,
                             q8ta_dtype out_dtype, hipStream_t stream) {
  const char* op = "q8ta_linear_lora";
  if (!x || !weight || !weight_scales || !lora_a || !lora_b || !adapter_ids || !out)
    return report(Q8TA_ERR_NULL, "%s: a required pointer is NULL", op);
  if (M < 1 || K < 1 || N < 1)
    return report(Q8TA_ERR_SHAPE, "%s: M, K, N must be >= 1 (got %lld, %lld, %lld)", op, (long long)M,
                  (long long)K, (long long)N);
  if (rank < 1 || rank > 512 || adapters < 1 || adapters > ((int64_t)1 << 24))
    return report(Q8TA_ERR_SHAPE, "%s: rank must be in [1, 512] and adapters in [1, 2^24] (got %lld, "
                  "%lld)", op, (long long)rank, (long long)adapters);
  const int64_t lim = (int64_t)1 << 30;
  if (M > ((int64_t)1 << 21) || N > lim || K > lim || !fits({M, K}) || !fits({N, K}) || !fits({M, N}) ||
      !fits({adapters, rank, K}) || !fits({adapters, rank, N}))
    return report(Q8TA_ERR_SHAPE, "%s: sizes too large", op);
  if (!std::isfinite(input_scale) || !(input_scale > 0.0))
    return report(Q8TA_ERR_QPARAM, "%s: scale must be finite and > 0 (got %g)", op, input_scale);
  if (input_zero_point < -128 || input_zero_point > 127)
    return report(Q8TA_ERR_QPARAM, "%s: zero_point must be in [-128, 127] (got %lld)", op,
                  (long long)input_zero_point);
  if (adapter_dtype != Q8TA_F16 && adapter_dtype != Q8TA_BF16)
    return report(Q8TA_ERR_UNSUPPORTED, "%s: adapter dtype must be fp16 or bf16 (got %d)", op,
                  (int)adapter_dtype);
  if (!dtype_ok(out_dtype))
    return report(Q8TA_ERR_UNSUPPORTED, "%s: unknown output dtype %d", op, (int)out_dtype);
  if (!activation || (strcmp(activation, "none") != 0 && strcmp(activation, "relu") != 0))
    return report(Q8TA_ERR_UNSUPPORTED, "%s: activation \"%.64s\" is not supported (\"none\" or "
                  "\"relu\")", op, activation ? activation : "NULL");
  LoraArgs a{};
  a.lin.x = x; a.lin.w = weight; a.lin.wscale = weight_scales; a.lin.bias = bias;
  a.lin.M = M; a.lin.K = K; a.lin.N = N; a.lin.izp = (int32_t)input_zero_point;
  a.lin.rq.s_in = (float)input_scale;
  a.a = lora_a; a.b = lora_b; a.ad_type = adapter_dtype; a.adapters = (int)adapters;
  a.rank = (int)rank; a.rank_pad = (int)((rank + 15) / 16 * 16); a.ad_scales = adapter_scales;
  a.ranks = ranks; a.ids = adapter_ids; a.relu = strcmp(activation, "relu") == 0; a.y = out;
  a.y_type = out_dtype;
  return hip_status(launch_linear_lora(a, stream), op);
}

}  // extern "C"
