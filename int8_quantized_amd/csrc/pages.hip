// The pages of the int8 cache: q8ta_pages_take, q8ta_pages_fork and
// q8ta_pages_release keep the block tables and each page's number of holders on
// the device, q8ta_pages_copy and q8ta_cache_compact move rows.
//
// A page is free where refs[page] <= 0.  There is no list of free pages that could
// disagree with that: releasing is a subtraction, in any order, and the k-th page
// that a call asks for is the k-th free one by its number, so that results do not
// depend on the order in which anything ran.  A shared page in part is given to nobody
// (a fork's last page is its own); what a caller who cuts a request back into one, or compacts one, has
// to see to stands in the header.  Three launches for it: free pages are
// counted in chunks of 4096 (and what each entry asks for, beside it), the counts
// are summed, and each chunk hands out its free pages to whom they belong.  Up to 65536
// pages and 4096 entries one workgroup does all of it (64 forks 4.6 us, 64 requests
// that take pages 8.5; the three launches 12.5): latencies of a few dependent
// loads and scans.  Of the three, the second is one workgroup, 1.6 us for each 1024 entries (65536
// requests that take pages 105 us, 2^20 1.6 ms; the other two 9 and 15).
//
// Rows move in 16-byte chunks where the cache allows it, a workgroup a stretch of
// rows of one head, all of its loads before its stores; memory bounds it.  Measured (8
// heads of 128): 8 windows of 6001 rows moved up, 203 MB read and written
// in 42 to 48 us, 4.2 to 4.8 TB/s (a copy of as much reaches 5.6); 64 trees' rows 5.4 us, 64 pages'
// parts copied 3.6, both the latency of table, path and row one after the other.  Where rows move among
// places that others leave, one workgroup takes a (head, request)'s stretches in turn: 16384 rows that lose
// 64 behind the first four, 218 us for one request and 1.13 ms for eight (0.3 and 0.5 TB/s).
#include "decode.h"

namespace q8ta {
namespace {

typedef uint32_t v4u __attribute__((ext_vector_type(4)));

constexpr int kNT = 256;
constexpr int kChunk = 4096;    // pages whose holders a workgroup looks through
constexpr int kPer = kChunk / kNT;

// Workspace of a call that hands out pages.
struct Hand {
  PagesArgs p;
  bool fork;
  int64_t entries;    // requests of a take, pairs of a fork
  int chunks;
  int32_t* need;      // [entries]: pages that each asks for
  int32_t* first;     // [entries]: place in the table of the first
  int64_t* before;    // [entries + 1]: sums of need
  int64_t* free_before;   // [chunks + 1]: sums of free pages
};

__device__ __forceinline__ int64_t rows_of(const PagesArgs& p, int64_t request) {
  const int64_t n = p.lens[request], cap = p.table_pages * p.page;
  return n < 0 ? 0 : (n < cap ? n : cap);
}
__device__ __forceinline__ bool is_request(const PagesArgs& p, int64_t r) { return r >= 0 && r < p.requests; }
__device__ __forceinline__ bool is_pair(const PagesArgs& p, int64_t i) {
  return is_request(p, p.a[i]) && is_request(p, p.b[i]) && p.a[i] != p.b[i];
}

__device__ __forceinline__ int wave_sum(int v) {
#pragma unroll
  for (int m = 32; m > 0; m /= 2) v += __shfl_xor(v, m);
  return v;
}

// Free pages of this thread's part of a chunk, as bits.
__device__ __forceinline__ uint32_t free_bits(const PagesArgs& p, int64_t p0) {
  uint32_t bits = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (p0 + i < p.pages && p.refs[p0 + i] <= 0) bits |= 1u << i;
  return bits;
}

// Pages that entry i asks for, and the place in its table of the first; -1 where
// the table cannot hold them.
__device__ __forceinline__ int need_of(const Hand& h, int64_t i, int& first) {
  const PagesArgs& p = h.p;
  first = 0;
  if (h.fork) return is_pair(p, i) && rows_of(p, p.a[i]) % p.page != 0 ? 1 : 0;
  const int64_t rows = rows_of(p, i), more = p.a[i];
  if (more <= 0) return 0;
  const int64_t end = (rows + more + p.page - 1) / p.page;
  if (end > p.table_pages) return -1;
  // its pages are the entries before the first below 0; those of its rows are there
  int64_t lo = rows / p.page, hi = end;
  while (lo < hi) {
    const int64_t mid = (lo + hi) / 2;
    if (p.table[i * p.table_pages + mid] < 0) hi = mid;
    else lo = mid + 1;
  }
  first = (int)lo;
  return (int)(end - lo);
}

// What entry i gets, with `before` pages asked for before it and `free` in all, beside
// the pages themselves.
__device__ __forceinline__ void answer(const Hand& h, int64_t i, int need, int64_t before, int64_t free) {
  const PagesArgs& p = h.p;
  const bool good = need == 0 || (need > 0 && before + need <= free);
  if (!h.fork) {
    p.granted[i] = good;
    return;
  }
  const bool pair = is_pair(p, i), copies = pair && good && need > 0;
  const int64_t rows = pair ? rows_of(p, p.a[i]) : 0;
  p.granted[i] = pair && good;
  p.copy_src[i] = copies ? p.table[p.a[i] * p.table_pages + rows / p.page] : -1;
  p.copy_rows[i] = copies ? (int32_t)(rows % p.page) : 0;
  if (!copies) p.copy_dst[i] = -1;
}

// Free page of rank `rank` to the entry it belongs to: the last one with at most that many
// asked for before it (which asks for some itself), if all that it asks for is there.
template <class B>
__device__ __forceinline__ void give(const Hand& h, int64_t rank, int64_t page, int64_t free, const B* before,
                                     const int32_t* first) {
  int64_t lo = 0, hi = h.entries;
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) / 2;
    if ((int64_t)before[mid] <= rank) lo = mid;
    else hi = mid;
  }
  if ((int64_t)before[lo + 1] > free) return;
  h.p.refs[page] = 1;
  if (h.fork) h.p.copy_dst[lo] = (int32_t)page;
  else h.p.table[lo * h.p.table_pages + first[lo] + (rank - (int64_t)before[lo])] = (int32_t)page;
}

__global__ __launch_bounds__(kNT) void k_pages_count(Hand h) {
  __shared__ int sums[kNT / 64];
  const PagesArgs& p = h.p;
  const int tid = threadIdx.x, lane = tid & 63;
  if ((int)blockIdx.x < h.chunks) {
    const int n = wave_sum(__builtin_popcount(free_bits(p, (int64_t)blockIdx.x * kChunk + tid * kPer)));
    if (lane == 0) sums[tid / 64] = n;
    __syncthreads();
    if (tid == 0) h.free_before[blockIdx.x] = sums[0] + sums[1] + sums[2] + sums[3];
    return;
  }
  const int64_t i = (int64_t)(blockIdx.x - h.chunks) * kNT + tid;
  if (i >= h.entries) return;
  int first;
  h.need[i] = need_of(h, i, first);
  h.first[i] = first;
}

// Sums before each of n values (and behind the last), by one workgroup of 1024, on top
// of `base`; the last sum in every thread.
template <class F, class G>
__device__ __forceinline__ int64_t scan(int64_t n, int64_t* sh, int64_t base, F&& value, G&& put) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid / 64;
  for (int64_t i0 = 0; i0 < n; i0 += 1024) {
    const int64_t i = i0 + tid;
    const int64_t mine = i < n ? value(i) : 0;
    int64_t run = mine;
#pragma unroll
    for (int m = 1; m < 64; m *= 2) {
      const int64_t o = __shfl_up(run, m);
      if (lane >= m) run += o;
    }
    __syncthreads();
    if (lane == 63) sh[wave] = run;
    __syncthreads();
    int64_t before = base, all = base;
    for (int w = 0; w < 16; ++w) {
      if (w < wave) before += sh[w];
      all += sh[w];
    }
    if (i < n) put(i, before + run - mine);
    base = all;
  }
  return base;
}

__global__ __launch_bounds__(1024) void k_pages_sum(Hand h) {
  __shared__ int64_t sh[16];
  const int64_t free = scan(h.chunks, sh, 0, [&](int64_t i) { return h.free_before[i]; },
                            [&](int64_t i, int64_t s) { h.free_before[i] = s; });
  const int64_t all = scan(h.entries, sh, 0, [&](int64_t i) { return (int64_t)(h.need[i] > 0 ? h.need[i] : 0); },
                           [&](int64_t i, int64_t s) {
                             h.before[i] = s;
                             answer(h, i, h.need[i], s, free);
                           });
  if (threadIdx.x == 0) {
    h.free_before[h.chunks] = free;
    h.before[h.entries] = all;
  }
}

__global__ __launch_bounds__(kNT) void k_pages_give(Hand h) {
  __shared__ int sums[kNT / 64];
  const PagesArgs& p = h.p;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid / 64;
  const int64_t wanted = h.before[h.entries], from = h.free_before[blockIdx.x];
  if (from >= wanted || from == h.free_before[blockIdx.x + 1]) return;
  const int64_t p0 = (int64_t)blockIdx.x * kChunk + tid * kPer;
  uint32_t bits = free_bits(p, p0);
  const int mine = __builtin_popcount(bits);
  int run = mine;
#pragma unroll
  for (int m = 1; m < 64; m *= 2) {
    const int o = __shfl_up(run, m);
    if (lane >= m) run += o;
  }
  if (lane == 63) sums[wave] = run;
  __syncthreads();
  int64_t rank = from + run - mine;
  for (int w = 0; w < wave; ++w) rank += sums[w];
  for (; bits && rank < wanted; ++rank, bits &= bits - 1)
    give(h, rank, p0 + __builtin_ctz(bits), h.free_before[h.chunks], h.before, h.first);
}

// All of it by one workgroup, where there are few entries and pages: one launch of a few
// microseconds instead of three.
constexpr int kFewEntries = 4096, kFewPages = 65536, kRound = 1024 * kPer;
__global__ __launch_bounds__(1024) void k_pages_few(Hand h) {
  __shared__ int64_t sh[16];
  __shared__ int32_t need[kFewEntries], first[kFewEntries];
  __shared__ int64_t before[kFewEntries + 1];
  const PagesArgs& p = h.p;
  const int tid = threadIdx.x;
  const int64_t wanted = scan(h.entries, sh, 0,
                              [&](int64_t i) {
                                int at;
                                need[i] = need_of(h, i, at);
                                first[i] = at;
                                return (int64_t)(need[i] > 0 ? need[i] : 0);
                              },
                              [&](int64_t i, int64_t s) { before[i] = s; });
  if (tid == 0) before[h.entries] = wanted;
  // free pages, as far as they are asked for
  int64_t free = 0;
  uint32_t bits = free_bits(p, tid * kPer);   // of the first round
  for (int64_t p0 = 0; p0 < p.pages && free < wanted; p0 += kRound) {
    const int n = wave_sum(__builtin_popcount(p0 ? free_bits(p, p0 + tid * kPer) : bits));
    __syncthreads();
    if ((tid & 63) == 0) sh[tid / 64] = n;
    __syncthreads();
    for (int w = 0; w < 16; ++w) free += sh[w];
  }
  __syncthreads();
  for (int64_t i = tid; i < h.entries; i += 1024) answer(h, i, need[i], before[i], free);
  int64_t rank = 0;
  for (int64_t p0 = 0; p0 < p.pages && rank < wanted; p0 += kRound) {
    if (p0) bits = free_bits(p, p0 + tid * kPer);
    rank = scan(1024, sh, rank, [&](int64_t) { return (int64_t)__builtin_popcount(bits); },
                [&](int64_t, int64_t s) {
                  for (; bits && s < wanted; ++s, bits &= bits - 1)
                    give(h, s, p0 + tid * kPer + __builtin_ctz(bits), free, before, first);
                });
  }
}

// The forked request's table: whole pages shared, then its own page, then none.
__global__ __launch_bounds__(kNT) void k_pages_share(PagesArgs p) {
  for (int64_t i = blockIdx.x; i < p.n; i += gridDim.x) {
    if (!p.granted[i]) continue;
    const int32_t* from = p.table + p.a[i] * p.table_pages;
    int32_t* to = p.table + p.b[i] * p.table_pages;
    const int64_t rows = rows_of(p, p.a[i]), full = rows / p.page;
    for (int64_t j = threadIdx.x; j < p.table_pages; j += kNT) {
      int32_t page = -1;
      if (j < full) {
        page = from[j];
        if (page >= 0 && page < p.pages) atomicAdd(&p.refs[page], 1);
      } else if (j == full) {
        page = p.copy_dst[i];
      }
      to[j] = page;
    }
    if (threadIdx.x == 0) p.lens[p.b[i]] = (int32_t)rows;
  }
}

__global__ __launch_bounds__(kNT) void k_pages_release(PagesArgs p) {
  const int64_t entries = p.a ? p.n : p.requests;
  for (int64_t i = blockIdx.x; i < entries; i += gridDim.x) {
    const int64_t r = p.a ? p.a[i] : i;
    if (!is_request(p, r)) continue;
    const int64_t given = p.b ? p.b[i] : 0, keep = given < 0 ? 0 : given;
    for (int64_t j = (keep + p.page - 1) / p.page + threadIdx.x; j < p.table_pages; j += kNT) {
      int32_t* at = p.table + r * p.table_pages + j;
      if (*at < 0) continue;
      // (taken out before it is counted: a request that stands twice gives up its pages once)
      const int32_t page = atomicExch(at, -1);
      if (page >= 0 && page < p.pages) atomicSub(&p.refs[page], 1);
    }
    if (threadIdx.x == 0) atomicMin(&p.lens[r], (int32_t)keep);
  }
}

hipError_t hand_out(const PagesArgs& p, bool fork, hipStream_t s) {
  Hand h{};
  h.p = p;
  h.fork = fork;
  h.entries = fork ? p.n : p.requests;
  h.chunks = (int)((p.pages + kChunk - 1) / kChunk);
  if (h.entries <= kFewEntries && p.pages <= kFewPages) {
    hipLaunchKernelGGL(k_pages_few, dim3(1), dim3(1024), 0, s, h);
    if (fork) hipLaunchKernelGGL(k_pages_share, dim3((unsigned)p.n), dim3(kNT), 0, s, p);
    return hipGetLastError();
  }
  const size_t sums = (size_t)(h.entries + 1 + h.chunks + 1) * 8;
  void* ws = nullptr;
  hipError_t e = workspace_acquire(&ws, sums + (size_t)h.entries * 8, s);
  if (e != hipSuccess) return e;
  h.before = (int64_t*)ws;
  h.free_before = h.before + h.entries + 1;
  h.need = (int32_t*)((char*)ws + sums);
  h.first = h.need + h.entries;
  const unsigned entry_blocks = (unsigned)((h.entries + kNT - 1) / kNT);
  hipLaunchKernelGGL(k_pages_count, dim3((unsigned)h.chunks + entry_blocks), dim3(kNT), 0, s, h);
  hipLaunchKernelGGL(k_pages_sum, dim3(1), dim3(1024), 0, s, h);
  hipLaunchKernelGGL(k_pages_give, dim3((unsigned)h.chunks), dim3(kNT), 0, s, h);
  if (fork)
    hipLaunchKernelGGL(k_pages_share, dim3((unsigned)(p.n < 65536 ? p.n : 65536)), dim3(kNT), 0, s, p);
  e = hipGetLastError();
  const hipError_t f = workspace_release(ws, s);
  return e != hipSuccess ? e : f;
}

// ------------------------------------------------------------------ rows
// First cache row of (page, segment): segment = part * kv_heads + head.
__device__ __forceinline__ int64_t segment_at(const CacheArgs& c, int64_t page, int seg) {
  return (page * 2 * c.kv_heads + seg) * c.page;
}

// A wave a segment of a page (four neighbouring ones a workgroup), a unit a lane
// and step.
template <class U>
__global__ __launch_bounds__(kNT) void k_pages_copy(CacheArgs c) {
  constexpr int kAhead = 4;   // steps whose loads are in flight
  const int lane = threadIdx.x & 63;
  const int seg = blockIdx.y * (kNT / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  if (seg >= 2 * c.kv_heads) return;
  for (int64_t pair = blockIdx.x; pair < c.n; pair += gridDim.x) {
    const int64_t from = c.src[pair], to = c.dst[pair];
    int64_t rows = c.rows ? c.rows[pair] : c.page;
    rows = rows < 0 ? 0 : (rows < c.page ? rows : c.page);
    if (from < 0 || from >= c.pages || to < 0 || to >= c.pages || from == to) continue;
    const int64_t a = segment_at(c, from, seg), b = segment_at(c, to, seg);
    const U* src = reinterpret_cast<const U*>(c.cache + a * c.dim);
    U* dst = reinterpret_cast<U*>(c.cache + b * c.dim);
    const int64_t n = rows * c.dim / (int)sizeof(U);
    const float sc = lane < rows ? c.scales[a + lane] : 0.0f;
    int64_t e = lane;
    for (; e + 64 * (kAhead - 1) < n; e += 64 * kAhead) {
      U v[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) v[u] = src[e + 64 * u];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) dst[e + 64 * u] = v[u];
    }
    for (; e < n; e += 64) dst[e] = src[e];
    if (lane < rows) c.scales[b + lane] = sc;
    for (int64_t r = lane + 64; r < rows; r += 64) c.scales[b + r] = c.scales[a + r];
  }
}

constexpr int kMostRows = 512;   // of a stretch

// A stretch of up to `stretch` rows of one request's path, `width` bytes of each
// row of one segment.  Row i comes from path[i] >= i, so nothing that a later stretch
// reads is written by an earlier one, nor by the same one where all its loads come first.
// Stretches of one request run at the same time where every row that moves
// comes from behind all that are kept; otherwise one workgroup takes them in turn.
// F: units a thread holds.
template <class U, int F>
__global__ __launch_bounds__(kNT) void k_cache_compact(CacheArgs c, int stretch, int width, int slices,
                                                       FastDiv per_div) {
  __shared__ int64_t from[kMostRows], to[kMostRows];   // cache rows, from < 0: none
  constexpr int V = sizeof(U);
  const int tid = threadIdx.x, seg = blockIdx.y;
  const int slice = blockIdx.x % slices;
  const int at = slice * width, w = c.dim - at < width ? c.dim - at : width;
  const int per = width / V;   // units of a row (the last slice's may be fewer)
  const int64_t parts = (c.n + stretch - 1) / stretch;
  for (int64_t b = blockIdx.z; b < c.batch; b += gridDim.z) {
    const int32_t* path = c.path + b * c.n;
    const int64_t base = c.base[b];
    int64_t count = c.counts[b];
    count = count < 0 ? 0 : (count < c.n ? count : c.n);
    // the first row that moves: path[i] - i never falls (64 places at a time, each
    // wave for itself)
    int64_t lo = 0, hi = count;
    while (lo < hi) {
      const int64_t step = hi - lo <= 64 ? 1 : (hi - lo + 63) / 64, x = lo + (tid & 63) * step;
      const uint64_t moved = __ballot(x < hi && path[x] > x);
      if (moved) {
        const int f = __builtin_ctzll(moved);
        hi = lo + f * step;
        lo = f > 0 ? hi - step + 1 : hi;
      } else {
        lo = step == 1 ? hi : lo + (hi - lo - 1) / step * step + 1;
      }
    }
    if (lo >= count) continue;
    // apart: this workgroup's stretches among all workgroups'; else the first one's are all
    const bool apart = path[lo] >= count;
    const int64_t first = blockIdx.x / slices, next = apart ? gridDim.x / slices : 1;
    if (!apart && first > 0) continue;
    for (int64_t part = first; part < parts && part * stretch < count; part += next) {
      const int64_t i0 = part * stretch;
      if (i0 + stretch <= lo) continue;
      __syncthreads();
      for (int r = tid; r < stretch; r += kNT) {
        const int64_t i = i0 + r;
        int64_t f = -1, t = -1;
        const int64_t off = i < count ? path[i] : 0;
        if (i < count && off > i && base >= 0 && base + off < c.table_pages * c.page) {
          const uint32_t src = (uint32_t)(base + off), dst = (uint32_t)(base + i);   // (both below 2^31)
          const uint32_t page = (uint32_t)c.page, sp0 = src / page, dp0 = dst / page;
          const int64_t sp = c.table[b * c.table_pages + sp0], dp = c.table[b * c.table_pages + dp0];
          if (sp >= 0 && sp < c.pages && dp >= 0 && dp < c.pages) {
            f = segment_at(c, sp, seg) + (src - sp0 * page);
            t = segment_at(c, dp, seg) + (dst - dp0 * page);
          }
        }
        from[r] = f;
        to[r] = t;
      }
      __syncthreads();
      const int n = stretch * per;
      U v[F];
      float sc[kMostRows / kNT];
      // (a unit past the stretch, or of a row that stays, loads the cache's first bytes)
#pragma unroll
      for (int u = 0; u < F; ++u) {
        const int e = tid + u * kNT, r = (int)fast_div((uint32_t)(e < n ? e : 0), per_div);
        const int64_t f = from[r];
        const int in = (e - r * per) * V;
        v[u] = *reinterpret_cast<const U*>(c.cache + (e < n && in < w && f >= 0 ? f * c.dim + at + in : 0));
      }
#pragma unroll
      for (int u = 0; u < kMostRows / kNT; ++u) {
        const int r = tid + u * kNT;
        const int64_t f = r < stretch ? from[r] : -1;
        sc[u] = c.scales[f >= 0 ? f : 0];
      }
      __builtin_amdgcn_s_waitcnt(0);   // every load has arrived
      __syncthreads();
#pragma unroll
      for (int u = 0; u < F; ++u) {
        const int e = tid + u * kNT, r = (int)fast_div((uint32_t)(e < n ? e : 0), per_div);
        const int in = (e - r * per) * V;
        if (e < n && in < w && from[r] >= 0) *reinterpret_cast<U*>(c.cache + to[r] * c.dim + at + in) = v[u];
      }
#pragma unroll
      for (int u = 0; u < kMostRows / kNT; ++u) {
        const int r = tid + u * kNT;
        if (slice == 0 && r < stretch && from[r] >= 0) c.scales[to[r]] = sc[u];
      }
    }
    __syncthreads();
  }
}

// Bytes that every row's start and length are multiples of.
int unit_of(const CacheArgs& c) {
  const uintptr_t x = (uintptr_t)c.cache | (uintptr_t)c.dim;
  return x % 16 == 0 ? 16 : (x % 4 == 0 ? 4 : 1);
}

template <class U>
hipError_t launch_copy(const CacheArgs& c, hipStream_t s) {
  const dim3 g((unsigned)(c.n < 1 << 22 ? c.n : 1 << 22), (unsigned)((2 * c.kv_heads + 3) / 4));
  hipLaunchKernelGGL((k_pages_copy<U>), g, dim3(kNT), 0, s, c);
  return hipGetLastError();
}

template <class U, int F>
hipError_t launch_compact(const CacheArgs& c, hipStream_t s) {
  constexpr int V = sizeof(U), kMost = F * kNT;   // units of a stretch
  const int width = c.dim / V < kMost ? c.dim : kMost * V;
  const int slices = (c.dim + width - 1) / width;
  int64_t stretch = kMost / (width / V);
  stretch = stretch < kMostRows ? stretch : kMostRows;
  stretch = stretch < c.n ? stretch : c.n;
  int64_t parts = (c.n + stretch - 1) / stretch;
  if (parts > (int64_t)1 << 18) parts = (int64_t)1 << 18;   // (the kernel goes round)
  const dim3 g((unsigned)(parts * slices), (unsigned)(2 * c.kv_heads), (unsigned)(c.batch < 65535 ? c.batch : 65535));
  hipLaunchKernelGGL((k_cache_compact<U, F>), g, dim3(kNT), 0, s, c, (int)stretch, width, slices,
                     make_fastdiv((uint32_t)(width / V)));
  return hipGetLastError();
}

}  // namespace

hipError_t launch_pages_take(const PagesArgs& p, hipStream_t s) { return hand_out(p, false, s); }
hipError_t launch_pages_fork(const PagesArgs& p, hipStream_t s) { return hand_out(p, true, s); }

hipError_t launch_pages_release(const PagesArgs& p, hipStream_t s) {
  const int64_t n = p.a ? p.n : p.requests;
  hipLaunchKernelGGL(k_pages_release, dim3((unsigned)(n < 65536 ? n : 65536)), dim3(kNT), 0, s, p);
  return hipGetLastError();
}

hipError_t launch_pages_copy(const CacheArgs& c, hipStream_t s) {
  const int v = unit_of(c);
  return v == 16 ? launch_copy<v4u>(c, s) : (v == 4 ? launch_copy<uint32_t>(c, s) : launch_copy<uint8_t>(c, s));
}

hipError_t launch_cache_compact(const CacheArgs& c, hipStream_t s) {
  const int v = unit_of(c);
  // (a tree's rows: 64 of 128 bytes and less)
  if (v == 16 && c.n * c.dim <= 2 * kNT * 16) return launch_compact<v4u, 2>(c, s);
  return v == 16 ? launch_compact<v4u, 8>(c, s) : (v == 4 ? launch_compact<uint32_t, 8>(c, s) : launch_compact<uint8_t, 8>(c, s));
}

}  // namespace q8ta
