// The pages of the int8 cache: q8ta_pages_take, q8ta_pages_fork and
// q8ta_pages_release keep the block tables and each page's number of holders on
// the device, q8ta_pages_copy and q8ta_cache_compact move rows.
//
// A page is free where refs[page] <= 0.  There is no list of free pages that could
// disagree with that: releasing is a subtraction, in any order, and the k-th page
// that a call asks for is the k-th free one by its number, so that results do not
// depend on the order in which anything ran.  Three launches for it: free pages are
// counted in chunks of 4096 (and what each entry asks for, beside it), the counts
// are summed, and each chunk hands out its free pages to whom they belong.
//
// Rows move in 16-byte chunks where the cache allows it, a workgroup a stretch of
// rows of one head, all of its loads before its stores.
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
  // a wave an entry
  const int64_t i = (int64_t)(blockIdx.x - h.chunks) * (kNT / 64) + tid / 64;
  if (i >= h.entries) return;
  if (h.fork) {
    if (lane == 0) {
      h.need[i] = is_pair(p, i) && rows_of(p, p.a[i]) % p.page != 0;
      h.first[i] = 0;
    }
    return;
  }
  const int64_t rows = rows_of(p, i), more = p.a[i];
  int64_t end = more > 0 ? (rows + more + p.page - 1) / p.page : 0;
  // a request whose table cannot hold the rows gets none
  const bool fits = end <= p.table_pages;
  // its pages are the entries before the first below 0; those of its rows are there
  int64_t first = end;
  for (int64_t j0 = rows / p.page; fits && j0 < end; j0 += 64) {
    const int64_t j = j0 + lane;
    const uint64_t open = __ballot(j < end && p.table[i * p.table_pages + j] < 0);
    if (open) {
      first = j0 + __builtin_ctzll(open);
      break;
    }
  }
  if (lane == 0) {
    h.need[i] = fits ? (int32_t)(end - first) : -1;
    h.first[i] = (int32_t)first;
  }
}

// Sums before each of n values (and behind the last), by one workgroup of 1024.
template <class F, class G>
__device__ __forceinline__ void scan(int64_t n, int64_t* sh, F&& value, G&& put) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid / 64;
  int64_t base = 0;
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
  if (tid == 0) put(n, base);
}

__global__ __launch_bounds__(1024) void k_pages_sum(Hand h) {
  __shared__ int64_t sh[16];
  const PagesArgs& p = h.p;
  scan(h.chunks, sh, [&](int64_t i) { return h.free_before[i]; },
       [&](int64_t i, int64_t s) { h.free_before[i] = s; });
  __syncthreads();
  const int64_t free = h.free_before[h.chunks];
  scan(h.entries, sh, [&](int64_t i) { return (int64_t)(h.need[i] > 0 ? h.need[i] : 0); },
       [&](int64_t i, int64_t s) {
         h.before[i] = s;
         if (i >= h.entries) return;
         const int64_t need = h.need[i];
         const bool good = need == 0 || (need > 0 && s + need <= free);
         if (!h.fork) {
           p.granted[i] = good;
           return;
         }
         const bool pair = is_pair(p, i), copies = pair && good && need > 0;
         const int64_t rows = pair ? rows_of(p, p.a[i]) : 0;
         p.granted[i] = pair && good;
         p.copy_src[i] = copies ? p.table[p.a[i] * p.table_pages + rows / p.page] : -1;
         p.copy_rows[i] = copies ? (int32_t)(rows % p.page) : 0;
         p.copy_dst[i] = -1;
       });
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
  for (; bits && rank < wanted; ++rank, bits &= bits - 1) {
    const int64_t page = p0 + __builtin_ctz(bits);
    // the last entry whose sum before it is at most the rank, which has need > 0
    int64_t lo = 0, hi = h.entries;
    while (hi - lo > 1) {
      const int64_t mid = (lo + hi) / 2;
      if (h.before[mid] <= rank) lo = mid;
      else hi = mid;
    }
    if (!p.granted[lo]) continue;
    p.refs[page] = 1;
    if (h.fork) p.copy_dst[lo] = (int32_t)page;
    else p.table[lo * p.table_pages + h.first[lo] + (rank - h.before[lo])] = (int32_t)page;
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
  const size_t sums = (size_t)(h.entries + 1 + h.chunks + 1) * 8;
  void* ws = nullptr;
  hipError_t e = workspace_acquire(&ws, sums + (size_t)h.entries * 8, s);
  if (e != hipSuccess) return e;
  h.before = (int64_t*)ws;
  h.free_before = h.before + h.entries + 1;
  h.need = (int32_t*)((char*)ws + sums);
  h.first = h.need + h.entries;
  constexpr int kEach = kNT / 64;
  const unsigned entry_blocks = (unsigned)((h.entries + kEach - 1) / kEach);
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
template <int V>
struct Bytes {
  v4u v;
};
template <>
struct Bytes<4> {
  uint32_t v;
};
template <>
struct Bytes<1> {
  uint8_t v;
};

// First cache row of (page, segment): segment = part * kv_heads + head.
__device__ __forceinline__ int64_t segment_at(const CacheArgs& c, int64_t page, int seg) {
  return (page * 2 * c.kv_heads + seg) * c.page;
}

// A wave a segment of a page, V bytes a lane and step.
template <int V>
__global__ __launch_bounds__(kNT) void k_pages_copy(CacheArgs c) {
  constexpr int U = 4;
  const int lane = threadIdx.x & 63;
  const int segs = 2 * c.kv_heads;
  const int64_t all = c.n * segs;
  for (int64_t i = (int64_t)blockIdx.x * (kNT / 64) + threadIdx.x / 64; i < all; i += (int64_t)gridDim.x * (kNT / 64)) {
    const int64_t pair = i / segs;
    const int seg = (int)(i - pair * segs);
    const int64_t from = c.src[pair], to = c.dst[pair];
    int64_t rows = c.rows ? c.rows[pair] : c.page;
    rows = rows < 0 ? 0 : (rows < c.page ? rows : c.page);
    if (from < 0 || from >= c.pages || to < 0 || to >= c.pages || from == to) continue;
    const int64_t a = segment_at(c, from, seg), b = segment_at(c, to, seg);
    const Bytes<V>* src = reinterpret_cast<const Bytes<V>*>(c.cache + a * c.dim);
    Bytes<V>* dst = reinterpret_cast<Bytes<V>*>(c.cache + b * c.dim);
    const int64_t n = rows * c.dim / V;
    for (int64_t e = lane; e < n; e += 64 * U) {
      Bytes<V> v[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (e + 64 * u < n) v[u] = src[e + 64 * u];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (e + 64 * u < n) dst[e + 64 * u] = v[u];
    }
    for (int64_t e = lane; e < rows; e += 64) c.scales[b + e] = c.scales[a + e];
  }
}

constexpr int kMostRows = 512, kInFlight = 16;   // rows of a stretch; chunks a thread holds

// A stretch of up to `stretch` rows of one request's path, `width` bytes of each
// row of one segment.  Row i comes from path[i] >= i, so nothing that a later stretch
// reads is written by an earlier one, nor by the same one where all its loads come first.
// Stretches of one request run at the same time where every row that moves
// comes from behind all that are kept; otherwise one workgroup takes them in turn.
template <int V>
__global__ __launch_bounds__(kNT) void k_cache_compact(CacheArgs c, int stretch, int width, int slices) {
  __shared__ int64_t from[kMostRows], to[kMostRows];   // cache rows, from < 0: none
  const int tid = threadIdx.x, segs = 2 * c.kv_heads;
  const int64_t stretches = (c.n + stretch - 1) / stretch, all = c.batch * segs * slices * stretches;
  for (int64_t id = blockIdx.x; id < all; id += gridDim.x) {
    int64_t left = id;
    const int64_t part = left % stretches;
    left /= stretches;
    const int slice = (int)(left % slices);
    left /= slices;
    const int seg = (int)(left % segs);
    const int64_t b = left / segs;
    const int32_t* path = c.path + b * c.n;
    int64_t count = c.counts[b];
    count = count < 0 ? 0 : (count < c.n ? count : c.n);
    // the first row that moves: path[i] - i never falls
    // (64 places at a time, each wave for itself)
    int64_t lo = 0, hi = count;
    while (lo < hi) {
      const int64_t step = (hi - lo + 63) / 64, at = lo + (tid & 63) * step;
      const uint64_t moved = __ballot(at < hi && path[at] > at);
      const int64_t f = moved ? __builtin_ctzll(moved) : (hi - lo + step - 1) / step;
      const int64_t top = lo + f * step;
      hi = top < hi ? top : hi;
      lo = f > 0 ? top - step + 1 : lo;
    }
    if (lo >= count) continue;
    const bool apart = path[lo] >= count;
    if (!apart && part > 0) continue;
    const int64_t i_end = apart ? (part + 1) * stretch : count;
    int64_t i0 = part * stretch;
    if (i0 < lo / stretch * stretch) {
      if (apart) continue;
      i0 = lo / stretch * stretch;
    }
    const int at = slice * width, w = c.dim - at < width ? c.dim - at : width;
    const int per = w / V;   // chunks of a row
    for (; i0 < i_end && i0 < count; i0 += stretch) {
      __syncthreads();
      for (int r = tid; r < stretch; r += kNT) {
        const int64_t i = i0 + r;
        int64_t f = -1, t = -1;
        if (i < count && path[i] > i) {
          const int64_t base = c.base[b], src = base + path[i], dst = base + i;
          const int64_t cap = c.table_pages * c.page;
          if (base >= 0 && src < cap) {
            const int64_t sp = c.table[b * c.table_pages + src / c.page];
            const int64_t dp = c.table[b * c.table_pages + dst / c.page];
            if (sp >= 0 && sp < c.pages && dp >= 0 && dp < c.pages) {
              f = segment_at(c, sp, seg) + src % c.page;
              t = segment_at(c, dp, seg) + dst % c.page;
            }
          }
        }
        from[r] = f;
        to[r] = t;
      }
      __syncthreads();
      Bytes<V> v[kInFlight];
      float sc[kMostRows / kNT];
      const int n = stretch * per;
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) {
        const int e = tid + u * kNT;
        if (e < n) {
          const int r = e / per;
          if (from[r] >= 0) v[u] = *reinterpret_cast<const Bytes<V>*>(c.cache + from[r] * c.dim + at + (e - r * per) * V);
        }
      }
#pragma unroll
      for (int u = 0; u < kMostRows / kNT; ++u) {
        const int r = tid + u * kNT;
        if (slice == 0 && r < stretch && from[r] >= 0) sc[u] = c.scales[from[r]];
      }
      __builtin_amdgcn_s_waitcnt(0);   // every load has arrived
      __syncthreads();
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) {
        const int e = tid + u * kNT;
        if (e < n) {
          const int r = e / per;
          if (from[r] >= 0) *reinterpret_cast<Bytes<V>*>(c.cache + to[r] * c.dim + at + (e - r * per) * V) = v[u];
        }
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

template <int V>
hipError_t launch_copy(const CacheArgs& c, hipStream_t s) {
  const int64_t blocks = (c.n * 2 * c.kv_heads + kNT / 64 - 1) / (kNT / 64);
  hipLaunchKernelGGL((k_pages_copy<V>), dim3((unsigned)(blocks < 1 << 20 ? blocks : 1 << 20)), dim3(kNT), 0, s, c);
  return hipGetLastError();
}

template <int V>
hipError_t launch_compact(const CacheArgs& c, hipStream_t s) {
  constexpr int kMost = kInFlight * kNT;   // chunks of a stretch
  const int width = c.dim / V < kMost ? c.dim : kMost * V;
  const int slices = (c.dim + width - 1) / width;
  int64_t stretch = kMost / (width / V);
  stretch = stretch < kMostRows ? stretch : kMostRows;
  stretch = stretch < c.n ? stretch : c.n;
  const int64_t all = c.batch * 2 * c.kv_heads * slices * ((c.n + stretch - 1) / stretch);
  hipLaunchKernelGGL((k_cache_compact<V>), dim3((unsigned)(all < 1 << 20 ? all : 1 << 20)), dim3(kNT), 0, s, c,
                     (int)stretch, width, slices);
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
  return v == 16 ? launch_copy<16>(c, s) : (v == 4 ? launch_copy<4>(c, s) : launch_copy<1>(c, s));
}

hipError_t launch_cache_compact(const CacheArgs& c, hipStream_t s) {
  const int v = unit_of(c);
  return v == 16 ? launch_compact<16>(c, s) : (v == 4 ? launch_compact<4>(c, s) : launch_compact<1>(c, s));
}

}  // namespace q8ta
