// skv_cache_pages.cu -- page operations of a paged KV cache: reserve, fork,
// free, compact, copy.
//
// The counts (refs) are the only record of which pages are free, so the k-th
// lowest free page is a prefix sum over them: each block of k_count counts the
// free pages of 4096 consecutive counts, k_free_list adds up the blocks before
// its own and writes its pages to their places in a list, and the third kernel
// hands them out by index.  No atomics decide an order, so the same cache gives
// the same pages on every run.
#include "skv_cache.cuh"

namespace skv {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 16;                     // counts per thread
constexpr int kChunk = kThreads * kPer;      // counts per block
constexpr int kCheckSplit = 8;               // blocks that check one request
constexpr int kUnit = 2048;                  // bytes a warp copies at a time
constexpr size_t kWsAlign = 256;

size_t up(size_t v) { return (v + kWsAlign - 1) / kWsAlign * kWsAlign; }

__device__ __forceinline__ uint64_t block_sum(uint64_t v) {
  __shared__ uint64_t s[kThreads / 32];
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  uint64_t t = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) t += s[i];
  __syncthreads();
  return t;
}

// Exclusive prefix of v over the block's threads.
__device__ __forceinline__ uint32_t block_prefix(uint32_t v) {
  __shared__ uint32_t s[kThreads / 32];
  const int lane = threadIdx.x & 31;
  uint32_t x = v;
  for (int o = 1; o < 32; o <<= 1) {
    uint32_t y = __shfl_up_sync(~0u, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s[threadIdx.x >> 5] = x;
  __syncthreads();
  uint32_t before = 0;
  for (int i = 0; i < (int)(threadIdx.x >> 5); ++i) before += s[i];
  __syncthreads();
  return before + x - v;
}

__device__ __forceinline__ uint64_t sum_of(const uint32_t *v, int64_t n) {
  uint64_t t = 0;
  for (int64_t i = threadIdx.x; i < n; i += kThreads) t += v[i];
  return block_sum(t);
}

__device__ __forceinline__ uint64_t sum_of(const uint64_t *v, int64_t n) {
  uint64_t t = 0;
  for (int64_t i = threadIdx.x; i < n; i += kThreads) t += v[i];
  return block_sum(t);
}

// A request for pages: fork (parents given) or reserve.
struct Request {
  const int32_t *parents;   // fork only
  const int32_t *slots;     // children, or the slots to extend
  const int32_t *from;      // fork: tokens kept; reserve: tokens there already
  const int32_t *to;        // reserve only
  int32_t n;
};

struct Item {
  bool ok;
  int32_t parent, slot, from;
  int32_t full;    // fork: blocks shared
  int32_t tail;    // fork: tokens in the block that is copied
  int32_t b0, nb;  // blocks b0 .. b0 + nb - 1 get a page
};

__device__ __forceinline__ Item item_of(const CacheView &c, const Request &q, int i) {
  Item t;
  const int64_t most = (int64_t)c.blocks * c.Tb;
  t.slot = q.slots[i];
  t.from = q.from[i];
  t.ok = t.slot >= 0 && t.slot < c.seqs && t.from >= 0 && t.from <= most;
  t.parent = -1;
  t.full = t.from / c.Tb;
  t.tail = t.from - t.full * c.Tb;
  if (q.parents) {
    t.parent = q.parents[i];
    t.ok = t.ok && t.parent >= 0 && t.parent < c.seqs;
    t.b0 = t.full;
    t.nb = t.tail ? 1 : 0;
  } else {
    const int32_t to = q.to[i];
    t.ok = t.ok && to >= t.from && to <= most;
    t.b0 = t.full + (t.tail ? 1 : 0);
    t.nb = (int32_t)(((int64_t)to + c.Tb - 1) / c.Tb) - t.b0;
    if (t.nb < 0) t.nb = 0;
  }
  if (!t.ok) t.nb = 0;
  return t;
}

// Blocks 0 .. n*kCheckSplit-1 check the requests, the others count free pages.
// bad[i*kCheckSplit + s] is set or cleared by one block each; need[i] too.
__global__ void __launch_bounds__(kThreads) k_count(CacheView c, Request q, uint64_t *need,
                                                    uint32_t *bad, uint32_t *counts) {
  const int64_t nb = (int64_t)q.n * kCheckSplit;
  if ((int64_t)blockIdx.x >= nb) {
    const uint64_t chunk = blockIdx.x - nb;
    const uint64_t p0 = chunk * kChunk;
    uint32_t f = 0;
    for (int i = 0; i < kPer; ++i) {
      const uint64_t p = p0 + (uint64_t)i * kThreads + threadIdx.x;
      if (p < c.pages && c.refs[p] == 0) ++f;
    }
    const uint64_t t = block_sum(f);
    if (threadIdx.x == 0) counts[chunk] = (uint32_t)t;
    return;
  }
  const int i = blockIdx.x / kCheckSplit, part = blockIdx.x % kCheckSplit;
  const Item t = item_of(c, q, i);
  bool wrong = !t.ok;
  // named twice, or as a parent as well
  for (int j = part * kThreads + threadIdx.x; j < q.n; j += kCheckSplit * kThreads) {
    if (j != i && q.slots[j] == t.slot) wrong = true;
    if (q.parents && q.parents[j] == t.slot) wrong = true;
  }
  if (t.ok) {
    // fork: the parent's blocks have pages, the child has none; reserve: the
    // blocks to fill are empty
    const int32_t lo = q.parents ? 0 : t.b0;
    const int32_t width = q.parents ? c.blocks : t.nb;
    const int32_t used = t.full + t.nb;
    const uint32_t total = (uint32_t)c.rows * (uint32_t)width;
    const uint32_t *own = c.table + (int64_t)t.slot * c.rows * c.blocks;
    const uint32_t *par = c.table + (int64_t)(q.parents ? t.parent : 0) * c.rows * c.blocks;
#pragma unroll 4
    for (uint32_t k = part * kThreads + threadIdx.x; k < total; k += kCheckSplit * kThreads) {
      const int64_t r = k / (uint32_t)width;
      const int32_t b = lo + (int32_t)(k - (uint32_t)r * (uint32_t)width);
      if (own[r * c.blocks + b] != kNoPage) wrong = true;
      if (q.parents && b < used && par[r * c.blocks + b] >= c.pages) wrong = true;
    }
  }
  const int any = __syncthreads_or(wrong);
  if (threadIdx.x == 0) {
    bad[blockIdx.x] = any ? 1u : 0u;
    if (part == 0) need[i] = (uint64_t)c.rows * (uint64_t)t.nb;
  }
}

// What k_free_list found: go != 0 where the request goes through, and the first
// list index of each item (base).
struct Go {
  uint32_t *go;
  uint32_t *base;
};

// Whether the request goes through: every check passed and there are pages enough.
__device__ __forceinline__ uint32_t verdict(const Request &q, const uint64_t *need,
                                            const uint32_t *bad, const uint32_t *counts,
                                            int64_t nchunks, uint64_t *want) {
  if (sum_of(bad, (int64_t)q.n * kCheckSplit)) return kCacheArg;
  *want = sum_of(need, q.n);
  if (*want == 0) return 0;
  return sum_of(counts, nchunks) < *want ? kCacheCapacity : 0;
}

__global__ void __launch_bounds__(kThreads) k_free_list(CacheView c, Request q,
                                                        const uint64_t *need, const uint32_t *bad,
                                                        const uint32_t *counts, int64_t nchunks,
                                                        Go go, uint32_t *list) {
  uint64_t want = 0;
  const uint32_t v = verdict(q, need, bad, counts, nchunks, &want);
  if (blockIdx.x == 0) {
    if (threadIdx.x == 0) {
      *go.go = v ? 0u : 1u;
      if (v) atomicOr(c.status, v);
    }
    // the items' first list indices (below 2^32: want pages are free)
    uint32_t sum = 0;
    for (int i0 = 0; !v && i0 < q.n; i0 += kThreads) {
      const int i = i0 + threadIdx.x;
      const uint32_t x = i < q.n ? (uint32_t)need[i] : 0u;
      const uint32_t before = block_prefix(x);
      if (i < q.n) go.base[i] = sum + before;
      sum += (uint32_t)block_sum(x);
    }
  }
  if (v) return;
  if (!want) return;
  const uint64_t before = sum_of(counts, blockIdx.x);
  if (before >= want) return;
  const uint64_t p0 = (uint64_t)blockIdx.x * kChunk + (uint64_t)threadIdx.x * kPer;
  uint32_t mask = 0;
  for (int i = 0; i < kPer; ++i)
    if (p0 + i < c.pages && c.refs[p0 + i] == 0) mask |= 1u << i;
  uint64_t k = before + block_prefix(__popc(mask));
  for (int i = 0; i < kPer; ++i)
    if (mask >> i & 1) {
      if (k < want) list[k] = (uint32_t)(p0 + i);
      ++k;
    }
}

// Hands out the pages: table entries and counts (reserve).
__global__ void __launch_bounds__(kThreads) k_reserve(CacheView c, Request q, Go go,
                                                      const uint32_t *list) {
  if (!*go.go) return;
  const int i = blockIdx.y;
  const Item t = item_of(c, q, i);
  if (!t.nb) return;
  const uint32_t *mine = list + go.base[i];
  uint32_t *own = c.table + (int64_t)t.slot * c.rows * c.blocks;
  const uint32_t total = (uint32_t)c.rows * (uint32_t)t.nb;
  for (uint32_t k = blockIdx.x * kThreads + threadIdx.x; k < total; k += gridDim.x * kThreads) {
    const uint32_t r = k / (uint32_t)t.nb;
    const uint32_t p = mine[k];
    own[(int64_t)r * c.blocks + t.b0 + (k - r * t.nb)] = p;
    c.refs[p] = 1;
  }
}

// One block per (row, child): the shared entries and their counts, and the copy
// of the partly filled block.  Children of a row are neighbours in the grid, so
// a parent's page comes from HBM once and from L2 for its other children.
__global__ void __launch_bounds__(kThreads) k_fork(CacheView c, Request q, Go go,
                                                   const uint32_t *list) {
  if (!*go.go) return;
  const uint32_t r = blockIdx.x / (uint32_t)q.n;
  const int i = (int)(blockIdx.x - r * (uint32_t)q.n);
  const Item t = item_of(c, q, i);
  const uint32_t *par = c.table + ((int64_t)t.parent * c.rows + r) * c.blocks;
  uint32_t *own = c.table + ((int64_t)t.slot * c.rows + r) * c.blocks;
  for (int b = threadIdx.x; b < t.full; b += kThreads) {
    const uint32_t p = par[b];
    own[b] = p;
    atomicAdd(c.refs + p, 1u);
  }
  if (!t.tail) return;
  const uint32_t p = list[go.base[i] + r];
  if (threadIdx.x == 0) {
    own[t.full] = p;
    c.refs[p] = 1;
  }
  const uint8_t *src = c.pool + (uint64_t)par[t.full] * c.page_bytes;
  uint8_t *dst = c.pool + (uint64_t)p * c.page_bytes;
  const uint32_t bytes = (uint32_t)t.tail * c.row_bytes;
  constexpr uint32_t kStep = kThreads * 16;
  for (uint32_t o = threadIdx.x * 16; o < bytes; o += 4 * kStep) {
    uint4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (o + u * kStep < bytes) v[u] = *reinterpret_cast<const uint4 *>(src + o + u * kStep);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (o + u * kStep < bytes) st_stream(dst + o + u * kStep, v[u]);
  }
}

// One thread per table entry of the slots given.
__global__ void __launch_bounds__(kThreads) k_free(CacheView c, const int32_t *slots) {
  const int32_t slot = slots[blockIdx.y];
  if (slot < 0 || slot >= c.seqs) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(c.status, kCacheArg);
    return;
  }
  const int64_t total = c.rows * c.blocks;
  uint32_t *own = c.table + (int64_t)slot * total;
  for (int64_t k = (int64_t)blockIdx.x * kThreads + threadIdx.x; k < total;
       k += (int64_t)gridDim.x * kThreads) {
    if (own[k] == kNoPage) continue;
    const uint32_t p = atomicExch(own + k, kNoPage);  // a slot named twice gives its pages back once
    if (p == kNoPage) continue;
    if (p >= c.pages) {
      atomicOr(c.status, kCacheArg);
    } else if (atomicSub(c.refs + p, 1u) == 0) {
      atomicAdd(c.refs + p, 1u);
      atomicOr(c.status, kCacheArg);
    }
  }
}

// ---- compaction ----
// With n pages in use, hole h (the h-th lowest free page below n) takes the
// h-th highest page in use: a page p >= n in use has live rank n - 1 - h with
// h its rank from the top, so both sides are prefix sums and need not know how
// many holes there are.

__global__ void __launch_bounds__(kThreads) k_compact_list(CacheView c, const uint32_t *counts,
                                                           int64_t nchunks, uint32_t *holes,
                                                           uint32_t *tops, uint32_t *rank,
                                                           uint32_t *top_refs, uint64_t *moves) {
  const uint64_t n = c.pages - sum_of(counts, nchunks);  // pages in use
  const uint64_t free_before = sum_of(counts, blockIdx.x);
  const uint64_t p0 = (uint64_t)blockIdx.x * kChunk + (uint64_t)threadIdx.x * kPer;
  uint32_t v[kPer];
  uint32_t f = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    v[i] = p0 + i < c.pages ? c.refs[p0 + i] : 1u;
    f += v[i] == 0;
  }
  uint64_t k = free_before + block_prefix(f);  // free pages below this thread's first
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const uint64_t p = p0 + i;
    // the number of holes: the free pages below n
    if (p == n || (p + 1 == c.pages && n == c.pages)) *moves = p == n ? k : k + (v[i] == 0);
    if (p < c.pages) {
      uint32_t r = kNoPage;
      if (p < n) {
        if (v[i] == 0) {
          r = (uint32_t)k;
          holes[k] = (uint32_t)p;
        }
      } else if (v[i]) {
        r = (uint32_t)(n - 1 - (p - k));  // p - k pages in use lie below p
        tops[r] = (uint32_t)p;
        top_refs[r] = v[i];
      }
      rank[p] = r;
    }
    k += v[i] == 0;
  }
}

// Copies `units` pieces of kUnit bytes, one per warp at a time; piece u belongs
// to move u / per_page.  src/dst lists may name pages out of range (reported).
struct Copy {
  const uint8_t *src_pool;
  uint8_t *dst_pool;
  const uint32_t *src, *dst;
  uint64_t src_pages, dst_pages;
  uint32_t page_bytes;
  uint32_t *status;
};

__device__ __forceinline__ void copy_units(const Copy &c, uint64_t moves, uint64_t warp,
                                           uint64_t warps) {
  const uint32_t per_page = (c.page_bytes + kUnit - 1) / kUnit;
  const uint64_t units = moves * per_page;
  const int lane = threadIdx.x & 31;
  for (uint64_t u = warp; u < units; u += warps) {
    const uint64_t m = u / per_page;
    const uint32_t o = (uint32_t)(u - m * per_page) * kUnit + lane * 16;
    const uint32_t s = c.src[m], d = c.dst[m];
    if (s >= c.src_pages || d >= c.dst_pages) {
      if (lane == 0) atomicOr(c.status, kCacheArg);
      continue;
    }
    const uint8_t *src = c.src_pool + (uint64_t)s * c.page_bytes;
    uint8_t *dst = c.dst_pool + (uint64_t)d * c.page_bytes;
    uint4 v[kUnit / 512];
#pragma unroll
    for (int i = 0; i < kUnit / 512; ++i)
      if (o + i * 512 < c.page_bytes) v[i] = ld_stream(src + o + i * 512);
#pragma unroll
    for (int i = 0; i < kUnit / 512; ++i)
      if (o + i * 512 < c.page_bytes) st_stream(dst + o + i * 512, v[i]);
  }
}

__global__ void __launch_bounds__(kThreads) k_copy(Copy c, int64_t n) {
  copy_units(c, (uint64_t)n, ((uint64_t)blockIdx.x * kThreads + threadIdx.x) >> 5,
             (uint64_t)gridDim.x * kThreads / 32);
}

// Moves the pages and rewrites counts and tables.  In place each thread reads
// only the entries it writes: a moved page's count comes from top_refs.
__global__ void __launch_bounds__(kThreads) k_compact(CacheView c, const uint32_t *counts,
                                                      int64_t nchunks, const uint32_t *holes,
                                                      const uint32_t *tops, const uint32_t *rank,
                                                      const uint32_t *top_refs,
                                                      const uint64_t *moves, uint32_t *table_out,
                                                      uint32_t *refs_out) {
  const uint64_t n = c.pages - sum_of(counts, nchunks);
  const uint64_t tid = (uint64_t)blockIdx.x * kThreads + threadIdx.x;
  const uint64_t threads = (uint64_t)gridDim.x * kThreads;
  for (uint64_t p = tid; p < c.pages; p += threads) {
    const uint32_t r = rank[p];
    uint32_t v = c.refs[p];
    if (p >= n) v = 0;
    else if (r != kNoPage) v = top_refs[r];
    if (refs_out != c.refs || p >= n || r != kNoPage) refs_out[p] = v;
  }
  const uint64_t entries = (uint64_t)c.seqs * c.rows * c.blocks;
  for (uint64_t k = tid; k < entries; k += threads) {
    uint32_t e = c.table[k];
    if (e != kNoPage) {
      const uint32_t r = e < c.pages ? rank[e] : kNoPage;
      // a free page: below n it has a rank, at n and above it has none
      if (e >= c.pages || (e < n) == (r != kNoPage)) atomicOr(c.status, kCacheArg);
      else if (e >= n) e = holes[r];
    }
    table_out[k] = e;
  }
  const Copy m{c.pool, c.pool, tops, holes, c.pages, c.pages, c.page_bytes, c.status};
  copy_units(m, *moves, tid >> 5, threads >> 5);
}

int copy_grid(uint64_t units) {
  // 152 SMs x 8 blocks: 2048 threads each, 64 warps x 2 KB in flight
  const uint64_t most = 152 * 8, want = (units + kThreads / 32 - 1) / (kThreads / 32);
  return (int)(want < 1 ? 1 : want < most ? want : most);
}

int64_t chunks_of(const CacheView &c) { return (int64_t)((c.pages + kChunk - 1) / kChunk); }

}  // namespace

PagesWs pages_ws(uint64_t pages, int64_t n) {
  PagesWs w;
  size_t o = 0;
  w.need = o;  // also the number of moves of a compaction
  o = up(o + sizeof(uint64_t) * (size_t)(n > 0 ? n : 1));
  w.base = o;
  o = up(o + sizeof(uint32_t) * (size_t)(n + 1));
  w.bad = o;
  o = up(o + sizeof(uint32_t) * (size_t)n * kCheckSplit);
  w.counts = o;
  o = up(o + sizeof(uint32_t) * (size_t)((pages + kChunk - 1) / kChunk));
  // the free list; or a compaction's holes and tops, which are at most half of the pages each
  w.list = o;
  o = up(o + sizeof(uint32_t) * 2 * (size_t)(pages / 2 + 1));
  w.rank = o;
  o = up(o + sizeof(uint32_t) * (size_t)pages);
  w.top_refs = o;
  o = up(o + sizeof(uint32_t) * (size_t)(pages / 2 + 1));
  w.total = o;
  return w;
}

namespace {
cudaError_t run_request(const CacheView &c, const Request &q, uint8_t *ws, cudaStream_t st) {
  const PagesWs w = pages_ws(c.pages, q.n);
  uint64_t *need = reinterpret_cast<uint64_t *>(ws + w.need);
  uint32_t *bad = reinterpret_cast<uint32_t *>(ws + w.bad);
  uint32_t *counts = reinterpret_cast<uint32_t *>(ws + w.counts);
  uint32_t *list = reinterpret_cast<uint32_t *>(ws + w.list);
  const Go go{reinterpret_cast<uint32_t *>(ws + w.base) + q.n,
              reinterpret_cast<uint32_t *>(ws + w.base)};
  const int64_t nc = chunks_of(c);
  k_count<<<(unsigned)(nc + (int64_t)q.n * kCheckSplit), kThreads, 0, st>>>(c, q, need, bad, counts);
  k_free_list<<<(unsigned)nc, kThreads, 0, st>>>(c, q, need, bad, counts, nc, go, list);
  if (q.parents) {
    k_fork<<<(unsigned)(c.rows * q.n), kThreads, 0, st>>>(c, q, go, list);
  } else {
    const int64_t most = (c.rows * c.blocks + kThreads - 1) / kThreads;
    k_reserve<<<dim3((unsigned)(most < 16 ? most : 16), (unsigned)q.n), kThreads, 0, st>>>(
        c, q, go, list);
  }
  return cudaGetLastError();
}
}  // namespace

cudaError_t launch_reserve(const CacheView &c, const int32_t *slots, const int32_t *old_len,
                           const int32_t *new_len, int32_t n, uint8_t *ws, cudaStream_t st) {
  return run_request(c, Request{nullptr, slots, old_len, new_len, n}, ws, st);
}

cudaError_t launch_fork(const CacheView &c, const int32_t *parents, const int32_t *children,
                        const int32_t *lens, int32_t n, uint8_t *ws, cudaStream_t st) {
  return run_request(c, Request{parents, children, lens, nullptr, n}, ws, st);
}

cudaError_t launch_free(const CacheView &c, const int32_t *slots, int32_t n, cudaStream_t st) {
  const int64_t most = (c.rows * c.blocks + kThreads - 1) / kThreads;
  k_free<<<dim3((unsigned)(most < 128 ? most : 128), (unsigned)n), kThreads, 0, st>>>(c, slots);
  return cudaGetLastError();
}

cudaError_t launch_compact(const CacheView &c, uint32_t *table_out, uint32_t *refs_out,
                           uint8_t *ws, cudaStream_t st) {
  const PagesWs w = pages_ws(c.pages, 0);
  uint64_t *moves = reinterpret_cast<uint64_t *>(ws + w.need);
  uint32_t *counts = reinterpret_cast<uint32_t *>(ws + w.counts);
  uint32_t *holes = reinterpret_cast<uint32_t *>(ws + w.list);
  uint32_t *tops = holes + (c.pages / 2 + 1);
  uint32_t *rank = reinterpret_cast<uint32_t *>(ws + w.rank);
  uint32_t *top_refs = reinterpret_cast<uint32_t *>(ws + w.top_refs);
  const int64_t nc = chunks_of(c);
  const Request none{nullptr, nullptr, nullptr, nullptr, 0};
  k_count<<<(unsigned)nc, kThreads, 0, st>>>(c, none, nullptr, nullptr, counts);
  k_compact_list<<<(unsigned)nc, kThreads, 0, st>>>(c, counts, nc, holes, tops, rank, top_refs,
                                                    moves);
  const uint64_t most = (c.pages / 2 + 1) * ((c.page_bytes + kUnit - 1) / kUnit);
  k_compact<<<copy_grid(most), kThreads, 0, st>>>(c, counts, nc, holes, tops, rank, top_refs,
                                                  moves, table_out, refs_out);
  return cudaGetLastError();
}

cudaError_t launch_copy_pages(const CacheView &c, const uint8_t *src_pool, uint64_t src_pages,
                              const uint32_t *src, uint8_t *dst_pool, uint64_t dst_pages,
                              const uint32_t *dst, int64_t n, cudaStream_t st) {
  const Copy m{src_pool, dst_pool, src, dst, src_pages, dst_pages, c.page_bytes, c.status};
  const uint64_t units = (uint64_t)n * ((c.page_bytes + kUnit - 1) / kUnit);
  k_copy<<<copy_grid(units), kThreads, 0, st>>>(m, n);
  return cudaGetLastError();
}

}  // namespace skv
