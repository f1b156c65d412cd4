// C entry points of what follows a step with drafted tokens: their verification
// and the pages of the cache.  Every check runs before any HIP call.
#include "api_checks.h"

using namespace q8ta;

namespace {

// The checks of the calls on block tables.
q8ta_status table_ok(const char* op, const PagesArgs& a) {
  if (a.requests < 0 || a.requests > ((int64_t)1 << 24) || a.table_pages < 1 || a.page < 1 ||
      a.page >= ((int64_t)1 << 31) || a.table_pages > (((int64_t)1 << 31) - 1) / a.page ||
      (a.requests > 0 && !fits({a.requests, a.table_pages})))
    return report(Q8TA_ERR_SHAPE, "%s: requests must be in [0, 2^24], page_size and table_pages >= 1 and "
                  "table_pages * page_size < 2^31 (got %lld, %lld, %lld)", op, (long long)a.requests,
                  (long long)a.page, (long long)a.table_pages);
  if (a.pages < 1 || a.pages >= ((int64_t)1 << 31))
    return report(Q8TA_ERR_SHAPE, "%s: pages must be in [1, 2^31) (got %lld)", op, (long long)a.pages);
  if (a.n < 0 || a.n > ((int64_t)1 << 24))
    return report(Q8TA_ERR_SHAPE, "%s: n must be in [0, 2^24] (got %lld)", op, (long long)a.n);
  return Q8TA_OK;
}

// The checks of the calls that move rows.
q8ta_status cache_ok(const char* op, const CacheArgs& a, int64_t kv_heads, int64_t dim) {
  if (a.pages < 1 || a.pages >= ((int64_t)1 << 31) || a.page < 1 || a.page >= ((int64_t)1 << 31) ||
      kv_heads < 1 || kv_heads > 32767 || dim < 1 || dim > 65536 || !fits({a.pages, a.page, kv_heads, dim, 2}))
    return report(Q8TA_ERR_SHAPE, "%s: pages, page_size, kv_heads (<= 32767) and dim (<= 65536) must be >= 1 "
                  "and the cache at most 2^40 elements (got %lld, %lld, %lld, %lld)", op, (long long)a.pages,
                  (long long)a.page, (long long)kv_heads, (long long)dim);
  return Q8TA_OK;
}

}  // namespace

extern "C" {

q8ta_status q8ta_verify_drafts(const void* logits, int64_t batch_stride, int64_t token_stride,
                               const void* draft_logits, int64_t draft_batch_stride,
                               int64_t draft_token_stride, q8ta_dtype dtype, int64_t batch, int64_t tokens,
                               int64_t vocab, const int32_t* ids, const int32_t* counts, const int64_t* mask,
                               const float* temperature, const float* draft_temperature, const float* u,
                               int32_t* path, int32_t* accepted, int32_t* next, hipStream_t stream) {
  const char* op = "q8ta_verify_drafts";
  if (!dtype_ok(dtype)) return report(Q8TA_ERR_UNSUPPORTED, "%s: unknown dtype %d", op, (int)dtype);
  if (batch < 0 || batch > 65535)
    return report(Q8TA_ERR_SHAPE, "%s: batch must be in [0, 65535] (got %lld)", op, (long long)batch);
  if (tokens < 1 || tokens > 64)
    return report(Q8TA_ERR_SHAPE, "%s: tokens must be in [1, 64] (got %lld)", op, (long long)tokens);
  if (vocab < 1 || vocab > ((int64_t)1 << 24))
    return report(Q8TA_ERR_SHAPE, "%s: vocab must be in [1, 2^24] (got %lld)", op, (long long)vocab);
  if (!draft_logits) draft_batch_stride = draft_token_stride = 0;
  for (int64_t st : {batch_stride, token_stride, draft_batch_stride, draft_token_stride})
    if (st < 0 || st > kMaxElems)
      return report(Q8TA_ERR_SHAPE, "%s: strides must be in [0, 2^40] (got %lld)", op, (long long)st);
  if (draft_logits && mask)
    return report(Q8TA_ERR_UNSUPPORTED, "%s: drafts drawn from draft_logits are chains (mask must be NULL)", op);
  if (batch == 0) return Q8TA_OK;
  if (!logits || !ids || !temperature || !u || !path || !accepted || !next)
    return report(Q8TA_ERR_NULL, "%s: a required pointer is NULL", op);
  VerifyArgs a{};
  a.logits = logits; a.bs = batch_stride; a.ts = token_stride; a.draft = draft_logits;
  a.dbs = draft_batch_stride; a.dts = draft_token_stride; a.dtype = dtype; a.batch = (int)batch;
  a.tokens = (int)tokens; a.vocab = (int)vocab; a.ids = ids; a.counts = counts; a.mask = mask;
  a.temperature = temperature; a.draft_temperature = draft_temperature; a.u = u; a.path = path;
  a.accepted = accepted; a.next = next;
  return hip_status(launch_verify_drafts(a, stream), op);
}

q8ta_status q8ta_pages_take(int32_t* table, int64_t requests, int64_t table_pages, int64_t page_size,
                            const int32_t* lens, const int32_t* more, int32_t* refs, int64_t pages,
                            int32_t* granted, hipStream_t stream) {
  const char* op = "q8ta_pages_take";
  PagesArgs a{};
  a.table = table; a.requests = requests; a.table_pages = table_pages; a.page = page_size;
  a.lens = const_cast<int32_t*>(lens);   // (not written)
  a.a = more; a.refs = refs; a.pages = pages; a.granted = granted;
  if (const q8ta_status st = table_ok(op, a)) return st;
  if (requests == 0) return Q8TA_OK;
  if (!table || !lens || !more || !refs || !granted)
    return report(Q8TA_ERR_NULL, "%s: a required pointer is NULL", op);
  return hip_status(launch_pages_take(a, stream), op);
}

q8ta_status q8ta_pages_fork(int32_t* table, int64_t requests, int64_t table_pages, int64_t page_size,
                            int32_t* lens, const int32_t* src, const int32_t* dst, int64_t n, int32_t* refs,
                            int64_t pages, int32_t* granted, int32_t* copy_src, int32_t* copy_dst,
                            int32_t* copy_rows, hipStream_t stream) {
  const char* op = "q8ta_pages_fork";
  PagesArgs a{};
  a.table = table; a.requests = requests; a.table_pages = table_pages; a.page = page_size; a.lens = lens;
  a.a = src; a.b = dst; a.n = n; a.refs = refs; a.pages = pages; a.granted = granted;
  a.copy_src = copy_src; a.copy_dst = copy_dst; a.copy_rows = copy_rows;
  if (const q8ta_status st = table_ok(op, a)) return st;
  if (n == 0) return Q8TA_OK;
  if (!table || !lens || !src || !dst || !refs || !granted || !copy_src || !copy_dst || !copy_rows)
    return report(Q8TA_ERR_NULL, "%s: a required pointer is NULL", op);
  return hip_status(launch_pages_fork(a, stream), op);
}

q8ta_status q8ta_pages_release(int32_t* table, int64_t requests, int64_t table_pages, int64_t page_size,
                               int32_t* lens, const int32_t* rows, const int32_t* keep, int64_t n,
                               int32_t* refs, int64_t pages, hipStream_t stream) {
  const char* op = "q8ta_pages_release";
  PagesArgs a{};
  a.table = table; a.requests = requests; a.table_pages = table_pages; a.page = page_size; a.lens = lens;
  a.a = rows; a.b = keep; a.n = n; a.refs = refs; a.pages = pages;
  if (const q8ta_status st = table_ok(op, a)) return st;
  if (!rows && n != requests)
    return report(Q8TA_ERR_SHAPE, "%s: without rows n must be the number of requests (got %lld, %lld)", op,
                  (long long)n, (long long)requests);
  if (n == 0) return Q8TA_OK;
  if (!table || !lens || !refs) return report(Q8TA_ERR_NULL, "%s: a required pointer is NULL", op);
  return hip_status(launch_pages_release(a, stream), op);
}

q8ta_status q8ta_pages_copy(int8_t* cache, float* cache_scales, int64_t pages, int64_t page_size,
                            int64_t kv_heads, int64_t dim, const int32_t* src, const int32_t* dst,
                            const int32_t* rows, int64_t n, hipStream_t stream) {
  const char* op = "q8ta_pages_copy";
  CacheArgs a{};
  a.cache = cache; a.scales = cache_scales; a.pages = pages; a.page = page_size; a.kv_heads = (int)kv_heads;
  a.dim = (int)dim; a.src = src; a.dst = dst; a.rows = rows; a.n = n;
  if (const q8ta_status st = cache_ok(op, a, kv_heads, dim)) return st;
  if (n < 0 || n >= ((int64_t)1 << 31))
    return report(Q8TA_ERR_SHAPE, "%s: n must be in [0, 2^31) (got %lld)", op, (long long)n);
  if (n == 0) return Q8TA_OK;
  if (!cache || !cache_scales || !src || !dst) return report(Q8TA_ERR_NULL, "%s: a required pointer is NULL", op);
  return hip_status(launch_pages_copy(a, stream), op);
}

q8ta_status q8ta_cache_compact(int8_t* cache, float* cache_scales, int64_t pages, int64_t page_size,
                               int64_t kv_heads, int64_t dim, const int32_t* table, int64_t batch,
                               int64_t table_pages, const int32_t* base, const int32_t* path, int64_t n,
                               const int32_t* counts, hipStream_t stream) {
  const char* op = "q8ta_cache_compact";
  CacheArgs a{};
  a.cache = cache; a.scales = cache_scales; a.pages = pages; a.page = page_size; a.kv_heads = (int)kv_heads;
  a.dim = (int)dim; a.n = n; a.table = table; a.batch = batch; a.table_pages = table_pages; a.base = base;
  a.path = path; a.counts = counts;
  if (const q8ta_status st = cache_ok(op, a, kv_heads, dim)) return st;
  if (batch < 0 || batch > ((int64_t)1 << 24) || n < 0 || n >= ((int64_t)1 << 31) || table_pages < 1 ||
      table_pages > (((int64_t)1 << 31) - 1) / page_size || (batch > 0 && !fits({batch, table_pages})) ||
      (batch > 0 && n > 0 && !fits({batch, n})))
    return report(Q8TA_ERR_SHAPE, "%s: batch must be in [0, 2^24], n in [0, 2^31), table_pages >= 1, table_pages "
                  "* page_size < 2^31 and batch * n <= 2^40 (got %lld, %lld, %lld)", op, (long long)batch,
                  (long long)n, (long long)table_pages);
  if (batch == 0 || n == 0) return Q8TA_OK;
  if (!cache || !cache_scales || !table || !base || !path || !counts)
    return report(Q8TA_ERR_NULL, "%s: a required pointer is NULL", op);
  return hip_status(launch_cache_compact(a, stream), op);
}

}  // extern "C"
