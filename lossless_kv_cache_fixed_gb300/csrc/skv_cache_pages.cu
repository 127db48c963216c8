// skv_cache_pages.cu -- page operations of a paged KV cache: reserve, fork,
// free, compact, copy.
//
// The counts (refs) are the only record of which pages are free, so the k-th
// lowest free page is a prefix sum over them.  k_check counts the free pages of each
// kChunk consecutive counts and checks the request; in k_free_list each block adds up
// the blocks before its own and writes its pages to their places in a list; the third
// kernel hands them out by index.  No atomics decide an order, so the same cache gives
// the same pages on every run.  Each of the first two is one round of loads and one
// barrier deep: they are bound by latency.
#include "skv_cache.cuh"

namespace skv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPer = 16;                     // counts per thread
constexpr int kChunk = kThreads * kPer;      // counts per block
constexpr int kPart = 2048;                  // table entries a block of k_check takes at once
constexpr int kMostParts = 2048;             // blocks that check, in all (or one per sequence)
constexpr int kUnit = 2048;                  // bytes a warp copies at a time
constexpr size_t kWsAlign = 256;

size_t up(size_t v) { return (v + kWsAlign - 1) / kWsAlign * kWsAlign; }

// Inclusive prefix over a warp.
__device__ __forceinline__ uint32_t warp_prefix(uint32_t v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(~0u, v, o);
    if (lane >= o) v += y;
  }
  return v;
}

// This thread's kPer counts from p on, 1 where there is none.
__device__ __forceinline__ void counts_at(const CacheView &c, uint64_t p, uint32_t *v) {
  if (p + kPer <= c.pages) {
#pragma unroll
    for (int i = 0; i < kPer / 4; ++i) {
      const uint4 x = reinterpret_cast<const uint4 *>(c.refs + p)[i];
      v[4 * i] = x.x;
      v[4 * i + 1] = x.y;
      v[4 * i + 2] = x.z;
      v[4 * i + 3] = x.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = p + i < c.pages ? c.refs[p + i] : 1u;
  }
}
__device__ __forceinline__ uint32_t zeros(const uint32_t *v) {
  uint32_t f = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) f += v[i] == 0;
  return f;
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

// What k_free_list found: *go != 0 where the request goes through, the first list index of
// each item (base) and how many pages it was counted for (need).  The kernel that hands
// them out reads the items again, so it keeps to that many: lengths that are overwritten
// meanwhile must not lead out of the list.
struct Go {
  uint32_t *go;
  uint32_t *base;
  uint32_t *need;
};

// Where k_check leaves what it found: need[i] pages for item i, bad[i*parts + part], free
// pages of each chunk.
struct Found {
  uint32_t *need, *bad, *counts;
  int parts;
  int64_t chunks;
};

// Blocks 0 .. chunks-1 count, block chunks + i*parts + part checks a part of item i: a
// fork's parent has pages for the tokens and its child none, the entries that reserve
// fills are empty, no slot is named twice.
__global__ void __launch_bounds__(kThreads) k_check(CacheView c, Request q, Found f) {
  begin();
  if (blockIdx.x < f.chunks) {
    __shared__ uint32_t s_f[kWarps];
    uint32_t v[kPer];
    counts_at(c, (uint64_t)blockIdx.x * kChunk + (uint64_t)threadIdx.x * kPer, v);
    const uint32_t w = __reduce_add_sync(~0u, zeros(v));
    if ((threadIdx.x & 31) == 0) s_f[threadIdx.x >> 5] = w;
    __syncthreads();
    if (threadIdx.x == 0) {
      uint32_t t = 0;
      for (int i = 0; i < kWarps; ++i) t += s_f[i];
      f.counts[blockIdx.x] = t;
    }
    return;
  }
  const uint32_t x = blockIdx.x - (uint32_t)f.chunks;
  const int i = x / f.parts, part = x - i * f.parts;
  const Item t = item_of(c, q, i);
  bool wrong = !t.ok;
  for (int j = part * kThreads + threadIdx.x; j < q.n; j += f.parts * kThreads) {
    if (j != i && q.slots[j] == t.slot) wrong = true;
    if (q.parents && q.parents[j] == t.slot) wrong = true;
  }
  const uint32_t entries = (uint32_t)c.rows * (uint32_t)c.blocks, blocks = c.blocks;
  if (t.ok) {
    const uint32_t *own = c.table + (int64_t)t.slot * entries;
    if (!q.parents) {
      for (uint32_t r = part * kThreads + threadIdx.x; r < (uint32_t)c.rows;
           r += f.parts * kThreads)
        for (int b = 0; b < t.nb; ++b) wrong |= own[(int64_t)r * blocks + t.b0 + b] != kNoPage;
    } else {
      const uint32_t *par = c.table + (int64_t)t.parent * entries;
      const uint32_t used = t.full + t.nb;
      if (entries % 4 == 0) {
        for (uint64_t k = (uint64_t)part * kPart; k < entries; k += (uint64_t)f.parts * kPart) {
          uint4 o[kPart / kThreads / 4], p[kPart / kThreads / 4];
#pragma unroll
          for (int y = 0; y < kPart / kThreads / 4; ++y) {
            const uint64_t e = k + y * kThreads * 4 + threadIdx.x * 4;
            if (e < entries) {
              o[y] = *reinterpret_cast<const uint4 *>(own + e);
              p[y] = *reinterpret_cast<const uint4 *>(par + e);
            }
          }
#pragma unroll
          for (int y = 0; y < kPart / kThreads / 4; ++y) {
            const uint64_t e = k + y * kThreads * 4 + threadIdx.x * 4;
            if (e >= entries) continue;
            wrong |= (o[y].x & o[y].y & o[y].z & o[y].w) != kNoPage;
            uint32_t b = (uint32_t)e % blocks;
            const uint32_t w[4] = {p[y].x, p[y].y, p[y].z, p[y].w};
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              wrong |= b < used && w[z] >= c.pages;
              if (++b == blocks) b = 0;
            }
          }
        }
      } else {
        for (uint64_t e = (uint64_t)part * kThreads + threadIdx.x; e < entries;
             e += (uint64_t)f.parts * kThreads) {
          wrong |= own[e] != kNoPage;
          wrong |= (uint32_t)e % blocks < used && par[e] >= c.pages;
        }
      }
    }
  }
  const int any = __syncthreads_or(wrong);
  if (threadIdx.x == 0) {
    f.bad[x] = any ? 1u : 0u;
    if (part == 0) f.need[i] = (uint32_t)c.rows * (uint32_t)t.nb;  // below 2^31
  }
}

// Blocks 0 .. chunks-1 list their free pages, the last block writes go, base and status.
__global__ void __launch_bounds__(kThreads) k_free_list(CacheView c, Request q, Found f, Go go,
                                                        uint32_t *list) {
  __shared__ uint32_t s[6][kWarps];
  begin();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t p0 = (uint64_t)blockIdx.x * kChunk + (uint64_t)threadIdx.x * kPer;
  uint32_t v[kPer];
  counts_at(c, p0, v);
  // sums of need in two halves of 16 bits, each below 2^32 for 4096 items
  uint32_t bad = 0, lo = 0, hi = 0, before = 0, all = 0;
#pragma unroll 4
  for (int i = threadIdx.x; i < q.n * f.parts; i += kThreads) bad |= f.bad[i];
#pragma unroll 4
  for (int i = threadIdx.x; i < q.n; i += kThreads) {
    lo += f.need[i] & 0xffff;
    hi += f.need[i] >> 16;
  }
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < f.chunks; i += kThreads) {
    const uint32_t x = f.counts[i];
    all += x;
    if (i < blockIdx.x) before += x;
  }
  const uint32_t mine = zeros(v), upto = warp_prefix(mine);
  const uint32_t sums[5] = {__reduce_or_sync(~0u, bad), __reduce_add_sync(~0u, lo),
                            __reduce_add_sync(~0u, hi), __reduce_add_sync(~0u, before),
                            __reduce_add_sync(~0u, all)};
  if (lane == 31) {
#pragma unroll
    for (int k = 0; k < 5; ++k) s[k][warp] = sums[k];
    s[5][warp] = upto;
  }
  __syncthreads();
  bad = lo = hi = before = all = 0;
  uint32_t within = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    bad |= s[0][w];
    lo += s[1][w];
    hi += s[2][w];
    before += s[3][w];
    all += s[4][w];
    if (w < warp) within += s[5][w];
  }
  const uint64_t want = lo + ((uint64_t)hi << 16);
  const uint32_t verdict = bad ? kCacheArg : want > all ? kCacheCapacity : 0;
  if (blockIdx.x < f.chunks) {
    if (verdict) return;
    uint64_t k = (uint64_t)before + within + upto - mine;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (v[i] == 0) {
        if (k < want) list[k] = (uint32_t)(p0 + i);
        ++k;
      }
    return;
  }
  if (threadIdx.x == 0) {
    *go.go = verdict ? 0u : 1u;
    if (verdict) atomicOr(c.status, verdict);
  }
  if (verdict) return;
  uint32_t sum = 0;  // want is below 2^32
  for (int i0 = 0; i0 < q.n; i0 += kThreads) {
    const int i = i0 + threadIdx.x;
    const uint32_t x = i < q.n ? f.need[i] : 0u, y = warp_prefix(x);
    __syncthreads();
    if (lane == 31) s[5][warp] = y;
    __syncthreads();
    uint32_t b = sum;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) b += s[5][w];
      sum += s[5][w];
    }
    if (i < q.n) go.base[i] = b + y - x;
  }
}

// k_check and k_free_list in one block, for pools of up to kSmallPages and requests over
// up to kSmallEntries table entries.  Free, fork and reserve of 8 children over 4 K, 8 K,
// 16 K and 28 K entries take 12.7, 14.4, 18.3 and 32.8 us of the GPU with it and 14.8,
// 15.9, 17.3 and 29.6 us without, and 23 against 28 us of the host.
constexpr int kSmallThreads = 1024;
constexpr uint64_t kSmallPages = (uint64_t)kSmallThreads * kPer;
constexpr int64_t kSmallEntries = 1 << 14;
constexpr int64_t kSmallRows = 2 * kSmallThreads;
__global__ void __launch_bounds__(kSmallThreads) k_small_list(CacheView c, Request q, Go go,
                                                              uint32_t *list) {
  __shared__ uint32_t s[2][32];
  begin();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t v[kPer], free_mask = 0;
  counts_at(c, (uint64_t)threadIdx.x * kPer, v);
#pragma unroll
  for (int i = 0; i < kPer; ++i) free_mask |= (uint32_t)(v[i] == 0) << i;
  // the checks of k_check; a thread's first item is also the one whose pages it counts
  bool wrong = false;
  uint32_t need = 0;
  if ((int)threadIdx.x < q.n) {
    const Item t = item_of(c, q, threadIdx.x);
    wrong = !t.ok;
    need = (uint32_t)c.rows * (uint32_t)t.nb;
    for (int j = 0; j < q.n; ++j) {
      if (j != (int)threadIdx.x && q.slots[j] == t.slot) wrong = true;
      if (q.parents && q.parents[j] == t.slot) wrong = true;
    }
  }
  const uint32_t rows = (uint32_t)c.rows, blocks = c.blocks, entries = rows * blocks;
  if (!q.parents) {
    for (uint32_t x = threadIdx.x; x < rows * q.n; x += kSmallThreads) {
      const uint32_t i = x / rows, r = x - i * rows;
      const Item t = item_of(c, q, i);
      const uint32_t *own = c.table + (int64_t)t.slot * entries + r * blocks + t.b0;
#pragma unroll 4
      for (int b = 0; b < t.nb; ++b) wrong |= own[b] != kNoPage;  // nb is 0 where not ok
    }
  } else {
    const uint32_t step = entries % 4 == 0 ? 4 : 1, per = entries / step;
#pragma unroll 4
    for (uint32_t x = threadIdx.x; x < per * q.n; x += kSmallThreads) {
      const uint32_t i = x / per, e = (x - i * per) * step;
      const Item t = item_of(c, q, i);
      if (!t.ok) continue;
      const uint32_t *own = c.table + (int64_t)t.slot * entries + e;
      const uint32_t *par = c.table + (int64_t)t.parent * entries + e;
      const uint32_t used = t.full + t.nb;
      uint32_t b = e % blocks;
      if (step == 4) {
        const uint4 o = *reinterpret_cast<const uint4 *>(own);
        const uint4 p = *reinterpret_cast<const uint4 *>(par);
        wrong |= (o.x & o.y & o.z & o.w) != kNoPage;
        const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          wrong |= b < used && w[z] >= c.pages;
          if (++b == blocks) b = 0;
        }
      } else {
        wrong |= *own != kNoPage;
        wrong |= b < used && *par >= c.pages;
      }
    }
  }
  // prefixes of need (at most 4 kSmallEntries) and of the free pages
  const uint32_t mine = __popc(free_mask);
  const uint32_t upto_need = warp_prefix(need), upto_free = warp_prefix(mine);
  if (lane == 31) {
    s[0][warp] = upto_need;
    s[1][warp] = upto_free;
  }
  const int any = __syncthreads_or(wrong);
  const uint32_t a = s[0][lane], b = s[1][lane];
  const uint32_t want = __reduce_add_sync(~0u, a), all = __reduce_add_sync(~0u, b);
  const uint32_t need0 = __reduce_add_sync(~0u, lane < warp ? a : 0);
  const uint32_t free0 = __reduce_add_sync(~0u, lane < warp ? b : 0);
  const uint32_t verdict = any ? kCacheArg : want > all ? kCacheCapacity : 0;
  if (threadIdx.x == 0) {
    *go.go = verdict ? 0u : 1u;
    if (verdict) atomicOr(c.status, verdict);
  }
  if (verdict) return;
  if ((int)threadIdx.x < q.n) {
    go.base[threadIdx.x] = need0 + upto_need - need;
    go.need[threadIdx.x] = need;
  }
  uint32_t k = free0 + upto_free - mine;
  for (uint32_t m = free_mask; m && k < want; m &= m - 1)
    list[k++] = threadIdx.x * kPer + (__ffs(m) - 1);
}

// Hands out the pages: table entries and counts (reserve).
__global__ void __launch_bounds__(kThreads) k_reserve(CacheView c, Request q, Go go,
                                                      const uint32_t *list) {
  begin();
  if (!*go.go) return;
  const int i = blockIdx.y;
  const Item t = item_of(c, q, i);
  if (!t.nb) return;
  const uint32_t *mine = list + go.base[i];
  uint32_t *own = c.table + (int64_t)t.slot * c.rows * c.blocks;
  const uint32_t total = min((uint32_t)c.rows * (uint32_t)t.nb, go.need[i]);
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
  begin();
  if (!*go.go) return;
  const uint32_t r = blockIdx.x / (uint32_t)q.n;
  const int i = (int)(blockIdx.x - r * (uint32_t)q.n);
  const Item t = item_of(c, q, i);
  if (!t.ok) return;
  const uint32_t *par = c.table + ((int64_t)t.parent * c.rows + r) * c.blocks;
  uint32_t *own = c.table + ((int64_t)t.slot * c.rows + r) * c.blocks;
  for (int b = threadIdx.x; b < t.full; b += kThreads) {
    const uint32_t p = par[b];
    if (p >= c.pages) continue;  // checked, unless the table is being overwritten
    own[b] = p;
    atomicAdd(c.refs + p, 1u);
  }
  if (!t.tail || r >= go.need[i]) return;
  const uint32_t p = list[go.base[i] + r];
  if (threadIdx.x == 0) {
    own[t.full] = p;
    c.refs[p] = 1;
  }
  const uint32_t from = par[t.full];
  if (from >= c.pages) return;
  const uint8_t *src = c.pool + (uint64_t)from * c.page_bytes;
  uint8_t *dst = c.pool + (uint64_t)p * c.page_bytes;
  const uint32_t bytes = (uint32_t)t.tail * c.row_bytes;
  constexpr uint32_t kRow = kThreads * 16;
  for (uint32_t o = threadIdx.x * 16; o < bytes; o += 4 * kRow) {
    uint4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (o + u * kRow < bytes) v[u] = *reinterpret_cast<const uint4 *>(src + o + u * kRow);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (o + u * kRow < bytes) st_stream(dst + o + u * kRow, v[u]);
  }
}

// One thread per table entry of the slots given.
__global__ void __launch_bounds__(kThreads) k_free(CacheView c, const int32_t *slots) {
  begin();
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
    } else if ((int32_t)atomicSub(c.refs + p, 1u) <= 0) {  // a free page, maybe named often
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

struct CompactPlan {
  uint64_t used, moves;
};

__global__ void __launch_bounds__(kThreads) k_compact_list(CacheView c, const uint32_t *counts,
                                                           int64_t chunks, uint32_t *holes,
                                                           uint32_t *tops, uint32_t *rank,
                                                           uint32_t *top_refs, CompactPlan *plan) {
  __shared__ uint32_t s[3][kWarps];
  begin();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t p0 = (uint64_t)blockIdx.x * kChunk + (uint64_t)threadIdx.x * kPer;
  uint32_t v[kPer];
  counts_at(c, p0, v);
  uint32_t before = 0, all = 0;
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < chunks; i += kThreads) {
    const uint32_t x = counts[i];
    all += x;
    if (i < blockIdx.x) before += x;
  }
  const uint32_t mine = zeros(v), upto = warp_prefix(mine);
  const uint32_t sb = __reduce_add_sync(~0u, before), sa = __reduce_add_sync(~0u, all);
  if (lane == 31) {
    s[0][warp] = sb;
    s[1][warp] = sa;
    s[2][warp] = upto;
  }
  __syncthreads();
  before = all = 0;
  uint32_t within = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    before += s[0][w];
    all += s[1][w];
    if (w < warp) within += s[2][w];
  }
  const uint64_t n = c.pages - all;                  // pages in use
  uint64_t k = (uint64_t)before + within + upto - mine;  // free pages below this thread's first
  if (p0 == 0) {
    plan->used = n;
    if (n == c.pages) plan->moves = 0;
  }
  uint32_t r[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const uint64_t p = p0 + i;
    r[i] = kNoPage;
    if (p >= c.pages) continue;
    if (p == n) plan->moves = k;  // the holes: the free pages below n
    if (p < n) {
      if (v[i] == 0) {
        r[i] = (uint32_t)k;
        holes[k] = (uint32_t)p;
      }
    } else if (v[i]) {
      r[i] = (uint32_t)(n - 1 - (p - k));  // p - k pages in use lie below p
      tops[r[i]] = (uint32_t)p;
      top_refs[r[i]] = v[i];
    }
    k += v[i] == 0;
  }
  if (p0 + kPer <= c.pages) {
#pragma unroll
    for (int i = 0; i < kPer / 4; ++i)
      reinterpret_cast<uint4 *>(rank + p0)[i] =
          make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (p0 + i < c.pages) rank[p0 + i] = r[i];
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
  begin();
  copy_units(c, (uint64_t)n, ((uint64_t)blockIdx.x * kThreads + threadIdx.x) >> 5,
             (uint64_t)gridDim.x * kThreads / 32);
}

// Moves the pages and rewrites counts and tables.  In place each thread reads
// only the entries it writes: a moved page's count comes from top_refs.
__global__ void __launch_bounds__(kThreads) k_compact(CacheView c, const uint32_t *holes,
                                                      const uint32_t *tops, const uint32_t *rank,
                                                      const uint32_t *top_refs,
                                                      const CompactPlan *plan,
                                                      uint32_t *table_out, uint32_t *refs_out) {
  begin();
  const uint64_t n = plan->used, moves = plan->moves;
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
  copy_units(m, moves, tid >> 5, threads >> 5);
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
  w.go = o;  // also a compaction's plan
  o = up(o + 64);
  w.base = o;
  o = up(o + sizeof(uint32_t) * (size_t)n);
  w.need = o;
  o = up(o + sizeof(uint32_t) * (size_t)n);
  w.bad = o;
  o = up(o + sizeof(uint32_t) * (size_t)(n ? (n > kMostParts ? n : kMostParts) : 0));
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
  auto at = [&](size_t o) { return reinterpret_cast<uint32_t *>(ws + o); };
  const Go go{at(w.go), at(w.base), at(w.need)};
  uint32_t *list = at(w.list);
  cudaError_t e;
  // one block where it has little to read: all entries of the slots for a fork; for reserve
  // only those that it fills, mostly few
  const int64_t entries = c.rows * c.blocks * q.n;
  const bool little = q.parents ? entries <= kSmallEntries
                                : c.rows * q.n <= kSmallRows && entries <= 4 * kSmallEntries;
  if (c.pages <= kSmallPages && q.n <= kSmallThreads && little) {
    e = launch(k_small_list, dim3(1), kSmallThreads, 0, st, c, q, go, list);
  } else {
    Found f{at(w.need), at(w.bad), at(w.counts), 1, chunks_of(c)};
    // a block for each kPart entries (fork) or kThreads rows (reserve), kMostParts in all
    const int64_t whole = q.parents ? (c.rows * c.blocks + kPart - 1) / kPart
                                    : (c.rows + kThreads - 1) / kThreads;
    const int64_t most = kMostParts / q.n > 1 ? kMostParts / q.n : 1;
    f.parts = (int)(whole < most ? whole : most);
    e = launch(k_check, dim3((unsigned)(f.chunks + (int64_t)q.n * f.parts)), kThreads, 0, st, c, q,
               f);
    if (e != cudaSuccess) return e;
    e = launch(k_free_list, dim3((unsigned)(f.chunks + 1)), kThreads, 0, st, c, q, f, go, list);
  }
  if (e != cudaSuccess) return e;
  if (q.parents)
    return launch(k_fork, dim3((unsigned)(c.rows * q.n)), kThreads, 0, st, c, q, go, list);
  const int64_t blocks = (c.rows * c.blocks + kThreads - 1) / kThreads;
  return launch(k_reserve, dim3((unsigned)(blocks < 16 ? blocks : 16), (unsigned)q.n), kThreads, 0,
                st, c, q, go, list);
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
  return launch(k_free, dim3((unsigned)(most < 128 ? most : 128), (unsigned)n), kThreads, 0, st, c, slots);
}

cudaError_t launch_compact(const CacheView &c, uint32_t *table_out, uint32_t *refs_out,
                           uint8_t *ws, cudaStream_t st) {
  const PagesWs w = pages_ws(c.pages, 0);
  CompactPlan *plan = reinterpret_cast<CompactPlan *>(ws + w.go);
  uint32_t *holes = reinterpret_cast<uint32_t *>(ws + w.list);
  uint32_t *tops = holes + (c.pages / 2 + 1);
  uint32_t *rank = reinterpret_cast<uint32_t *>(ws + w.rank);
  uint32_t *top_refs = reinterpret_cast<uint32_t *>(ws + w.top_refs);
  uint32_t *counts = reinterpret_cast<uint32_t *>(ws + w.counts);
  const Request none{nullptr, nullptr, nullptr, nullptr, 0};
  const Found f{nullptr, nullptr, counts, 1, chunks_of(c)};
  cudaError_t e = launch(k_check, dim3((unsigned)f.chunks), kThreads, 0, st, c, none, f);
  if (e != cudaSuccess) return e;
  e = launch(k_compact_list, dim3((unsigned)f.chunks), kThreads, 0, st, c, counts, f.chunks, holes, tops, rank,
             top_refs, plan);
  if (e != cudaSuccess) return e;
  const uint64_t most = (c.pages / 2 + 1) * ((c.page_bytes + kUnit - 1) / kUnit);
  return launch(k_compact, dim3((unsigned)copy_grid(most)), kThreads, 0, st, c, holes, tops, rank, top_refs,
                plan, table_out, refs_out);
}

cudaError_t launch_copy_pages(const CacheView &c, const uint8_t *src_pool, uint64_t src_pages,
                              const uint32_t *src, uint8_t *dst_pool, uint64_t dst_pages,
                              const uint32_t *dst, int64_t n, cudaStream_t st) {
  const Copy m{src_pool, dst_pool, src, dst, src_pages, dst_pages, c.page_bytes, c.status};
  const uint64_t units = (uint64_t)n * ((c.page_bytes + kUnit - 1) / kUnit);
  return launch(k_copy, dim3((unsigned)copy_grid(units)), kThreads, 0, st, m, n);
}

}  // namespace skv
