// skv_cache_chunk.cu -- attention of the new tokens of each sequence over a paged KV
// cache, plain and differential.
//
// o_h = sum_t p_t v_t / sum_t p_t with p_t = 2^(x_t - m), x_t = log2(e) * scale * q_h.k_t, m at a
// distance from the running maximum (softmax in one pass: when m grows to m', the sums so far
// are multiplied by 2^(m - m')).  Differential attention runs the halves of q and k as two such
// maps over the same values and subtracts lambda times the second result.
//
// The new tokens of a sequence times the query heads of one kv head are packed rows (token
// major).  An item is the packed rows of one or two tiles of 128 with one kv head; its keys and
// values go by in blocks of 128 (up to 128 channels) or 64 tokens:
//   S = Q K^T   tcgen05.mma, both operands in shared memory, S in tensor memory;
//   P = 2^(S f - m), one thread per row, written over S as 16-bit numbers;
//   O += P V    tcgen05.mma, P in tensor memory, V in shared memory, O in tensor memory.
// The warps of a block have roles: 4 per tile for the softmax (one thread per row), 4 that
// load (cp.async to a ring of slots; e4m3 codes become fp16 on the way), one that issues the
// matrix instructions, one that deals the work.  With two tiles the matrix unit works on one
// tile while the softmax of the other runs; with one (more than 128 channels, whose sums take
// half of the tensor memory), S has two buffers.
//
// Work is dealt as in skv_cache_attend.cu: the blocks of all items in a row, cut evenly over one
// wave of persistent thread blocks whatever the lengths; items that lie in several leave partial
// results, which k_chunk_join adds up in a fixed order.
//
// What a row does not see must not touch it, and 0 * infinity is not 0: rows outside an item's
// range are zeros in shared memory, and in blocks that some rows see only in part the values
// that are not finite become 0, a flag is set, and the rows that see them get them in the end.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "skv_cache.cuh"

namespace skv {
namespace {

constexpr int kMostBlocks = 160;  // thread blocks of a launch
// An item costs a thread block this many blocks of tokens more than it has: queries are
// loaded, results written and the pipeline runs empty in between.
constexpr int kItemCost = 2;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kHoles = 16;       // blocks whose missing tokens are remembered
constexpr uint64_t kPatience = 2000000000;  // ns that a barrier may take before a block gives up

template <int ES, int DP, bool DIFF>
struct Cfg {
  static constexpr int kTiles = DP <= 128 ? 2 : 1;       // tiles of 128 rows
  static constexpr int kN = DP <= 128 ? 128 : 64;        // tokens of a block
  static constexpr int kItem = (DIFF ? 64 : 128) * kTiles;  // packed rows of an item
  static constexpr int kQ = 128 * DP * 2;                // bytes of a tile of queries
  static constexpr int kSlot = kN * DP * 2;              // bytes of a block of keys or values
  static constexpr int kSlots = DP == 64 ? (ES == 2 ? 10 : 8) : (ES == 2 ? 5 : 3);
  static constexpr int kRaw = kN * DP;                   // bytes of a block of codes
  static constexpr int kRaws = ES == 1 ? 4 : 0;
  static constexpr int kSoftmax = 4 * kTiles;            // warps of the softmax
  static constexpr int kThreads = (kSoftmax + 8) * 32;
  // registers per thread of the softmax, the loads and the others; their sum over the threads
  // is within what the block is launched with
  static constexpr int kRegsS = kTiles == 2 ? 200 : 240, kRegsL = kTiles == 2 ? 64 : 120,
                       kRegsM = kTiles == 2 ? 48 : 72;
  static constexpr int kRegs = 32 * (kSoftmax * kRegsS + 4 * kRegsL + 4 * kRegsM);
  static constexpr int kOffSlots = kTiles * kQ;
  static constexpr int kOffRaw = kOffSlots + kSlots * kSlot;
  static constexpr int kOffMisc = kOffRaw + kRaws * kRaw;
  // tensor memory columns
  static constexpr int kS = kN;            // S of a tile (or buffer); P in the first half
  static constexpr int kO = 2 * kN;        // O, DP columns per tile
  // see skv_cache_attend.cu: m is kLift below the running maximum when x - m passes kMost
  static constexpr float kLift = ES == 1 ? 11.f : 0.f, kMost = ES == 1 ? 15.f : 8.f;
};

// What a thread block works on: blocks of tokens of one item.
struct Seg {
  int32_t q0, p0, p1;         // the sequence's first row of q; packed rows
  int32_t base, begin, len;   // the place of the first new token; tokens that any row may see
  int32_t lo, hi, t0;         // tokens that the item sees; the first block's first token
  int32_t nu;                 // blocks; 0: the rows see nothing; -1: the end
  int32_t h, slot, part;      // part: 0 the whole item, 1 and 2: a part, of which slot + 1
  uint32_t fix;               // values that are not finite were left out
};

template <typename C>
struct Misc {
  uint64_t q_full, q_empty, kv_full[C::kSlots], kv_empty[C::kSlots];
  uint64_t s_full[2], p_full[2], o_full[2], seg_full[2], seg_empty[2], pair, last;
  uint32_t tmem, dead;
  Seg seg[2];
  uint4 holes[kHoles];
  uint8_t qe[2][2][128];      // exponents of the rows of q (e4m3)
  float l[2][128];
};

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, const uint4 &v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{.reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p;}"
      : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok;
}
__device__ __forceinline__ uint64_t now() {
  uint64_t t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}
// writes to shared memory become visible to the matrix unit
__device__ __forceinline__ void fence_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// the barrier gets an arrival when all matrix instructions so far of this thread are done
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
               : "memory");
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{.reg .pred p; setp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
      "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{.reg .pred p; setp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;}" ::"r"(d), "r"(a), "l"(b), "r"(idesc),
      "r"((uint32_t)add)
      : "memory");
}
// 32 columns of this thread's row of tensor memory
__device__ __forceinline__ void tm_ld32(float *v, uint32_t a) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
        "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
        "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(a));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tm_st32(uint32_t a, const float *v) {
  uint32_t r[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(v[i]);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(a),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
      "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
      "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tm_st16(uint32_t a, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16};" ::"r"(a), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
      "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tm_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
template <int R>
__device__ __forceinline__ void regs_more() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R>
__device__ __forceinline__ void regs_less() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
template <int ES>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if (ES == 2) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
  }
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ void e4m3x4(uint32_t v, uint32_t &lo, uint32_t &hi) {
  asm("{.reg .b16 a, b; mov.b32 {a, b}, %2; cvt.rn.f16x2.e4m3x2 %0, a; cvt.rn.f16x2.e4m3x2 %1, b;}"
      : "=r"(lo), "=r"(hi)
      : "r"(v));
}

// Tiles in shared memory: blocks of 64 channels, in each a row of 128 bytes per token (or
// packed row), whose 16-byte chunks are permuted by the row (128-byte swizzle).  As an operand
// whose rows are the rows (Q, K) the matrix unit steps 8 rows by 1024 bytes; as one whose rows
// are the channels (V) 8 tokens by 1024 and 64 channels by a block.
__device__ __forceinline__ uint32_t swz(int rows, int row, int ch) {
  return (uint32_t)((ch >> 3) * rows * 128 + row * 128 + (((ch ^ row) & 7) << 4));
}
__device__ __forceinline__ uint64_t desc_of(uint32_t addr, uint32_t lbo) {
  return (uint64_t)((addr & 0x3ffff) >> 4) | ((uint64_t)(lbo >> 4) << 16) |
         ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// A sequence of the batch.
struct Entry {
  int32_t slot, len, begin, q0, n;
  int32_t rows, items;  // packed rows, items per kv head
};
template <typename C>
__device__ __forceinline__ Entry entry_of(const ChunkArgs &a, int group, int b, bool tell) {
  Entry e;
  e.slot = a.slots[b];
  e.len = a.lens[b];
  e.begin = a.begins ? max(a.begins[b], 0) : 0;
  e.q0 = a.starts ? a.starts[b] : b;
  const int32_t q1 = a.starts ? a.starts[b + 1] : b + 1;
  const bool off = e.q0 < 0 || q1 > a.tokens || e.q0 > q1;
  const bool bad = e.slot >= 0 && (e.len < 0 || e.len > a.max_len ||
                                   (int64_t)e.len > (int64_t)a.c.blocks * a.c.Tb || e.slot >= a.c.seqs);
  if ((off || bad) && tell) atomicOr(a.c.status, kCacheArg);
  if (e.slot < 0 || bad) e.len = 0;
  e.n = off ? 0 : q1 - e.q0;
  e.rows = e.n * group;
  e.items = (e.rows + C::kItem - 1) / C::kItem;
  return e;
}
// The tokens [lo, hi) that item i of a sequence sees, in blocks from lo's one on.
struct Span {
  int32_t lo, hi, start, units;
};
template <typename C>
__device__ __forceinline__ Span span_of(const ChunkArgs &a, int group, const Entry &e, int i) {
  Span s;
  const int p0 = i * C::kItem, p1 = min(p0 + C::kItem, e.rows);
  const int base = e.len - e.n;
  s.lo = e.begin;
  if (a.window) s.lo = (int32_t)max((int64_t)s.lo, (int64_t)base + p0 / group - a.window + 1);
  s.hi = a.full ? e.len : min(e.len, base + (p1 - 1) / group + 1);
  if (s.hi < s.lo) s.hi = s.lo;
  s.start = s.lo / C::kN * C::kN;
  s.units = s.hi > s.lo ? (s.hi - s.start + C::kN - 1) / C::kN : 0;
  return s;
}
// How units are dealt: see skv_cache_attend.cu.
__device__ __forceinline__ uint32_t deal(uint32_t W, uint32_t n, uint32_t i) {
  const uint32_t q = W / n;
  return i * q + i * (W - q * n) / n;
}
__device__ __forceinline__ int block_of(uint32_t W, uint32_t n, uint32_t u) {
  return (int)((((uint64_t)u + 1) * n - 1) / W);
}

// What the join has to know of an item that begins in thread block i and ends in another.
struct Cut {
  int32_t q0, p0, p1, h, parts;
};
// Workspace: a Cut per thread block, then for each two partial results.
template <typename C, int DP>
struct Part {
  float o[C::kTiles * 128][DP];
  float m[C::kTiles * 128], l[C::kTiles * 128];
};
constexpr size_t kCutBytes = (sizeof(Cut) * kMostBlocks + 255) / 256 * 256;

__device__ __forceinline__ void store8(float *p, const float *v) {
  *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}

template <int ES, int DP, bool DIFF>
__global__ void __launch_bounds__((Cfg<ES, DP, DIFF>::kThreads), 1) k_chunk(ChunkArgs a, int cut) {
  using C = Cfg<ES, DP, DIFF>;
  constexpr int kTiles = C::kTiles, kN = C::kN;
  extern __shared__ __align__(1024) uint8_t smem[];
  Misc<C> &sh = *reinterpret_cast<Misc<C> *>(smem + C::kOffMisc);
  const uint32_t sm = smem_addr(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const CacheView &c = a.c;
  const int group = a.q_heads / c.heads;
  constexpr int kLoad0 = C::kSoftmax, kMma = C::kSoftmax + 4, kDeal = C::kSoftmax + 5;

  // Waits for a phase of a barrier, with a limit: then the block gives up and says so.
  auto wait1 = [&](uint64_t &bar, uint32_t parity) -> bool {
    const uint32_t b = smem_addr(&bar);
    if (bar_try(b, parity)) return true;
    const uint64_t from = now();
    do {
      if (bar_try(b, parity)) return true;
      if (*reinterpret_cast<volatile uint32_t *>(&sh.dead)) return false;
    } while (now() - from < kPatience);
    *reinterpret_cast<volatile uint32_t *>(&sh.dead) = 1;
    atomicOr(c.status, kCacheStuck);
    return false;
  };
  auto wait = [&](uint64_t &bar, uint32_t parity) -> bool {
    return __all_sync(~0u, wait1(bar, parity));
  };
  auto arrive = [&](uint64_t &bar) {  // one arrival per warp
    __syncwarp();
    if (lane == 0) bar_arrive(smem_addr(&bar));
  };

  if (warp == kMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_addr(&sh.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (threadIdx.x == 0) {
    bar_init(smem_addr(&sh.q_full), 4);
    bar_init(smem_addr(&sh.q_empty), 1);
    for (int i = 0; i < C::kSlots; ++i) {
      bar_init(smem_addr(&sh.kv_full[i]), 4);
      bar_init(smem_addr(&sh.kv_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(smem_addr(&sh.s_full[i]), 1);
      bar_init(smem_addr(&sh.p_full[i]), 4);
      bar_init(smem_addr(&sh.o_full[i]), 1);
      bar_init(smem_addr(&sh.seg_full[i]), 1);
      bar_init(smem_addr(&sh.seg_empty[i]), C::kSoftmax + 5);
    }
    bar_init(smem_addr(&sh.pair), 8);
    bar_init(smem_addr(&sh.last), 1);
    sh.dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async();
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = sh.tmem;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp < C::kSoftmax) {
    // ---------------------------------------------------------------- softmax
    regs_more<C::kRegsS>();
    const int tile = warp >> 2, r = (warp & 3) * 32 + lane;
    // packed row of the item, and the map, of this thread
    const int rr = !DIFF ? tile * 128 + r : kTiles == 2 ? r : (r >> 5) * 16 + (r & 15);
    const int map = !DIFF ? 0 : kTiles == 2 ? tile : (r >> 4) & 1;
    const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);
    const uint32_t tm_o = lanes + C::kO + tile * DP;
    const int maps = DIFF ? 2 : 1;
    uint32_t blocks = 0, mine = 0, ends = 0;  // blocks of all items so far, of this tile; items
    uint32_t pairs = 0;
    auto both = [&]() -> bool {  // the warps of both tiles meet
      arrive(sh.pair);
      return wait(sh.pair, pairs++ & 1);
    };
    for (uint32_t sidx = 0;; ++sidx) {
      Seg &s = sh.seg[sidx & 1];
      if (!wait(sh.seg_full[sidx & 1], (sidx >> 1) & 1)) break;
      const int nu = s.nu;
      if (nu < 0) break;
      const int p = s.p0 + rr;
      const bool on = p < s.p1;
      const int j = p / group, head = s.h * group + (p - j * group);
      const int place = s.base + j;
      int lo = 0, hi = 0x7fffffff;
      if (on) {
        lo = s.begin;
        if (a.window) lo = (int)max((int64_t)lo, (int64_t)place - a.window + 1);
        hi = place < 0 ? 0 : a.full ? s.len : min(s.len, place + 1);
      }
      const bool rows = DIFF || s.p0 + tile * 128 < s.p1;  // the tile has some
      float m = -INFINITY, l = 0.f;
      float unit = 1.f;
      if (ES == 1 && c.scale) unit = c.scale[a.layer * c.heads + s.h];
      if (nu > 0 && rows) {
        float f = a.scale * kLog2e * unit;
        for (int u = 0; u < nu; ++u) {
          const int buf = kTiles == 2 ? tile : (int)(mine & 1);
          const uint32_t phase = kTiles == 2 ? mine & 1 : (mine >> 1) & 1;
          if (!wait(sh.s_full[buf], phase)) break;
          fence_after();
          if (u == 0) {
            if (ES == 1) f *= __uint_as_float((uint32_t)sh.qe[sidx & 1][tile][r] << 23);
            if (f == 0.f) f = 1.17549435e-38f;  // 0 * -infinity is not -infinity
          }
          const uint32_t tm_s = lanes + buf * C::kS;
          float x[kN];
#pragma unroll
          for (int i = 0; i < kN; i += 32) tm_ld32(x + i, tm_s + i);
          tm_wait_ld();
          const int t0 = s.t0 + u * kN;
          const uint4 hole = sh.holes[(blocks + u) % kHoles];
          const bool holes = hole.x | hole.y | hole.z | hole.w;
          const float none = f < 0.f ? INFINITY : -INFINITY;
          if (__any_sync(~0u, lo > t0 || hi < t0 + kN) || holes) {
            const int from = lo - t0, to = hi - t0;
#pragma unroll
            for (int i = 0; i < kN; ++i)
              if (i < from || i >= to) x[i] = none;
            if (holes) {
              const uint32_t w[4] = {hole.x, hole.y, hole.z, hole.w};
#pragma unroll
              for (int i = 0; i < kN; ++i)
                if (w[i / (kN / 4)] >> (i % (kN / 4)) & 1) x[i] = none;
            }
          }
          float top;
          {
            float t[4];
            if (f > 0.f) {
#pragma unroll
              for (int i = 0; i < 4; ++i) t[i] = x[i];
#pragma unroll
              for (int i = 4; i < kN; ++i) t[i & 3] = fmaxf(t[i & 3], x[i]);
              top = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) * f;
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i) t[i] = x[i];
#pragma unroll
              for (int i = 4; i < kN; ++i) t[i & 3] = fminf(t[i & 3], x[i]);
              top = fminf(fminf(t[0], t[1]), fminf(t[2], t[3])) * f;
            }
          }
          if (__any_sync(~0u, top - m > C::kMost)) {
            // only rows that pass it change, so that no row's bits depend on another's
            // (beyond 2^23 a float has no room for kLift)
            const float mn = top - m > C::kMost ? (fabsf(top) < 0x1p23f ? top - C::kLift : top) : m;
            const float by = mn == -INFINITY ? 1.f : ex2(m - mn);
            m = mn;
            l *= by;
            if (u > 0) {
              // With two buffers S may be there before the last product with the values is done
              // (but not before the one before that, so the barrier is one phase ahead at most).
              if (kTiles == 1 && !wait(sh.o_full[0], (mine - 1) & 1)) break;
              fence_after();
#pragma unroll
              for (int d = 0; d < DP; d += 32) {
                float o[32];
                tm_ld32(o, tm_o + d);
                tm_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] *= by;
                tm_st32(tm_o + d, o);
              }
            }
          }
          const float m0 = m == -INFINITY ? 0.f : m;
          // One rounding of the difference where that is exact enough; scores beyond 2^20 are
          // rounded first, as m was, so that their differences are exact.
          const bool far = fabsf(m0) > 0x1p20f;
          if (__any_sync(~0u, far)) {
#pragma unroll
            for (int i = 0; i < kN; ++i)
              x[i] = far ? __fsub_rn(__fmul_rn(x[i], f), m0) : fmaf(x[i], f, -m0);
          } else {
#pragma unroll
            for (int i = 0; i < kN; ++i) x[i] = fmaf(x[i], f, -m0);
          }
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < kN; i += 32) {
            uint32_t w[16];
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              const float p0 = ex2(x[i + k]), p1 = ex2(x[i + k + 1]);
              sum[k & 2] += p0;
              sum[(k & 2) + 1] += p1;
              w[k / 2] = pack2<ES>(p0, p1);
            }
            tm_st16(tm_s + i / 2, w);
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          tm_wait_st();
          fence_before();
          arrive(sh.p_full[buf]);
          ++mine;
        }
        blocks += nu;
        // ---- results
        // (with two buffers o_full[0] counts blocks and o_full[1] items)
        if (!wait(sh.o_full[kTiles == 2 ? tile : 1], ends++ & 1)) break;
        fence_after();
      } else if (nu > 0) {
        blocks += nu;
      }
      const float m0 = m == -INFINITY ? 0.f : m;
      const int64_t oh = ((int64_t)s.q0 + j) * a.q_heads + head;
      // values that are not finite, of partly masked blocks: those that this row sees
      auto mend = [&](float *o, int d0) {
        if (!s.fix || !on) return;
        const int jl = (min(s.p0 + C::kItem, s.p1) - 1) / group;
        const int most = a.window ? (int)max((int64_t)s.begin, (int64_t)s.base + jl - a.window + 1) : s.begin;
        const int least = a.full ? s.len : min(s.len, s.base + s.p0 / group + 1);
        const uint32_t *tab = c.table + ((int64_t)s.slot * c.rows +
                                         ((int64_t)a.layer * 2) * c.heads + s.h) * c.blocks;
        for (int u = 0; u < nu; ++u) {
          const int t0 = s.t0 + u * kN;
          if (t0 >= most && t0 + kN <= least) continue;
          for (int t = max(t0, lo); t < min(t0 + kN, hi); ++t) {
            const uint32_t pk = tab[t / c.Tb], pv = tab[(int64_t)c.heads * c.blocks + t / c.Tb];
            if (pk >= c.pages || pv >= c.pages) continue;
            const uint8_t *row = c.pool + (uint64_t)pv * c.page_bytes + (uint32_t)(t % c.Tb) * c.row_bytes;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              if (d0 + i >= c.D) continue;
              if (ES == 2) {
                const uint16_t w = reinterpret_cast<const uint16_t *>(row)[d0 + i];
                if ((w & 0x7f80) == 0x7f80) o[i] += __uint_as_float((uint32_t)w << 16);
              } else if ((row[d0 + i] & 0x7f) == 0x7f) {
                o[i] = NAN;
              }
            }
          }
        }
      };
      if (nu == 0) {
        if (on && (!DIFF || map == 0)) {
          for (int d = 0; d < c.D; d += 8)
            *reinterpret_cast<uint4 *>(a.out + oh * c.D + d) = make_uint4(0, 0, 0, 0);
          if (a.lse)
            for (int i = 0; i < maps; ++i) a.lse[oh * maps + i] = -INFINITY;
        }
      } else if (s.part && rows) {
        Part<C, DP> &part =
            reinterpret_cast<Part<C, DP> *>(a.ws + kCutBytes)[blockIdx.x * 2 + s.part - 1];
#pragma unroll
        for (int d = 0; d < DP; d += 32) {
          if (d >= c.D) break;
          float o[32];
          tm_ld32(o, tm_o + d);
          tm_wait_ld();
          mend(o, d);
          if (on)
#pragma unroll
            for (int i = 0; i < 32; i += 8) store8(&part.o[tile * 128 + r][d + i], o + i);
        }
        if (on) {
          part.m[tile * 128 + r] = m;
          part.l[tile * 128 + r] = l;
        }
      } else if (!DIFF && rows) {
        const float by = l == 0.f ? 0.f : unit / l;
#pragma unroll
        for (int d = 0; d < DP; d += 32) {
          if (d >= c.D) break;
          float o[32];
          tm_ld32(o, tm_o + d);
          tm_wait_ld();
          mend(o, d);
          if (on)
#pragma unroll
            for (int i = 0; i < 32; i += 8)
              if (d + i < c.D)
                *reinterpret_cast<uint4 *>(a.out + oh * c.D + d + i) =
                    make_uint4(pack2<2>(o[i] * by, o[i + 1] * by), pack2<2>(o[i + 2] * by, o[i + 3] * by),
                               pack2<2>(o[i + 4] * by, o[i + 5] * by), pack2<2>(o[i + 6] * by, o[i + 7] * by));
        }
        if (on && a.lse) a.lse[oh] = (m0 + log2f(l)) * kLn2;
      } else if (DIFF) {
        if (on && a.lse) a.lse[oh * 2 + map] = (m0 + log2f(l)) * kLn2;
        float by = l == 0.f ? 0.f : unit / l;
        if (map && on) by *= a.lambda[head];
        if constexpr (kTiles == 2) {
          // each of the two threads of a row takes half of the channels of both maps
          constexpr int kHalf = DP / 2;
          sh.l[map][r] = by;
          if (!both()) break;
          const float f0 = sh.l[0][r], f1 = sh.l[1][r];
          fence_after();
          float o[kHalf], q = 0.f;
          const int d0 = map * kHalf;
#pragma unroll
          for (int d = 0; d < kHalf; d += 32) {
            float o1[32];
            tm_ld32(o + d, lanes + C::kO + d0 + d);
            tm_ld32(o1, lanes + C::kO + DP + d0 + d);
            tm_wait_ld();
            mend(o + d, d0 + d);
            mend(o1, d0 + d);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              o[d + i] = o[d + i] * f0 - o1[i] * f1;
              if (d0 + d + i < c.D) q = fmaf(o[d + i], o[d + i], q);
            }
          }
          fence_before();
          if (!both()) break;  // (neither tile's sums are overwritten before both are read)
          float n = 1.f;
          if (a.norm) {
            sh.l[map][r] = q;
            if (!both()) break;
            q = sh.l[0][r] + sh.l[1][r];
            n = q == 0.f ? 0.f : rsqrtf(q / c.D + a.eps);
            if (!both()) break;
          }
          if (on)
#pragma unroll
            for (int d = 0; d < kHalf; d += 8) {
              if (d0 + d >= c.D) break;
              uint32_t w[4];
#pragma unroll
              for (int i = 0; i < 8; i += 2) {
                float x0 = o[d + i] * n, x1 = o[d + i + 1] * n;
                if (a.norm) {
                  x0 *= a.norm[d0 + d + i];
                  x1 *= a.norm[d0 + d + i + 1];
                }
                w[i / 2] = pack2<2>(x0, x1);
              }
              *reinterpret_cast<uint4 *>(a.out + oh * c.D + d0 + d) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        } else {
          // lanes i and i + 16 have a row's two maps
          float n = 1.f, q = 0.f;
          for (int pass = a.norm ? 0 : 1; pass < 2; ++pass) {
#pragma unroll
            for (int d = 0; d < DP; d += 32) {
              if (d >= c.D) break;
              float o[32];
              tm_ld32(o, tm_o + d);
              tm_wait_ld();
              mend(o, d);
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float x = o[i] * by, y = __shfl_xor_sync(~0u, x, 16);
                o[i] = map ? y - x : x - y;
                if (pass == 0 && d + i < c.D) q = fmaf(o[i], o[i], q);
              }
              if (pass == 1 && on)
#pragma unroll
                for (int i = 0; i < 32; i += 8) {
                  if (d + i >= c.D || (i >> 4) != map) continue;
                  uint32_t w[4];
#pragma unroll
                  for (int k = 0; k < 8; k += 2) {
                    float x0 = o[i + k] * n, x1 = o[i + k + 1] * n;
                    if (a.norm) {
                      x0 *= a.norm[d + i + k];
                      x1 *= a.norm[d + i + k + 1];
                    }
                    w[k / 2] = pack2<2>(x0, x1);
                  }
                  *reinterpret_cast<uint4 *>(a.out + oh * c.D + d + i) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            if (pass == 0) n = q == 0.f ? 0.f : rsqrtf(q / c.D + a.eps);
          }
        }
      }
      fence_before();
      arrive(sh.seg_empty[sidx & 1]);
    }
  } else if (warp < kMma) {
    // ---------------------------------------------------------------- loads
    regs_less<C::kRegsL>();
    constexpr int kRpw = kN / 4;                     // rows of a block per warp
    constexpr int kCpr = DP / 8;                     // 16-byte chunks of a row of 16-bit numbers
    constexpr int kRpi = 32 / kCpr;                  // rows that a warp copies at once
    const int w = warp - kLoad0, ch = lane % kCpr, sub = lane / kCpr;
    uint32_t tiles = 0, blocks = 0;                  // K and V blocks so far; blocks
    bool alive = true;
    constexpr int kLag = 2;  // copies under way whose arrival is not told yet (bf16)
    for (uint32_t sidx = 0; alive; ++sidx) {
      Seg &s = sh.seg[sidx & 1];
      if (!wait(sh.seg_full[sidx & 1], (sidx >> 1) & 1)) break;
      const int nu = s.nu;
      const int q0 = s.q0, p0 = s.p0, p1 = s.p1, h = s.h, lo = s.lo, hi = s.hi, first = s.t0, slot = s.slot;
      // blocks before `most` or that end after `least` are masked for some rows
      int most = s.begin, least = s.len;
      if (nu > 0) {
        const int jl = (min(p0 + C::kItem, p1) - 1) / group;
        if (a.window) most = (int)max((int64_t)most, (int64_t)s.base + jl - a.window + 1);
        if (!a.full) least = min(least, s.base + p0 / group + 1);
      }
      arrive(sh.seg_empty[sidx & 1]);
      if (nu < 0) break;
      if (nu == 0) continue;
      // ---- queries
      if (!wait(sh.q_empty, (sidx & 1) ^ 1)) break;
#pragma unroll 1
      for (int t = 0; t < kTiles; ++t) {
        const uint32_t dst = sm + t * C::kQ;
        if (ES == 2) {
          // packed row -> (token, head), step by step
          int row = w * 32 + sub;
          const int step = DIFF && kTiles == 1 ? 0 : kRpi;
          int p = p0 + (!DIFF ? t * 128 + row : row);
          int j = p / group, g = p - j * group;
          const int dj = step / group, dg = step - dj * group;
#pragma unroll 1
          for (int i = 0; i < 32 / kRpi; ++i, row += kRpi) {
            int map = t;
            if (DIFF && kTiles == 1) {
              p = p0 + (row >> 5) * 16 + (row & 15);
              map = (row >> 4) & 1;
              j = p / group;
              g = p - j * group;
            }
            bool on = p < p1 && ch * 8 < c.D;
            if (DIFF) {
              // halves end at a multiple of 8 channels
              const int half = c.D / 2;
              if (map == 0 ? ch * 8 >= half : ch * 8 < half) on = false;
            }
            const uint16_t *src = a.q + ((int64_t)q0 + j) * a.qs + (int64_t)(h * group + g) * a.qhs + ch * 8;
            cp_async16(dst + swz(128, row, ch), on ? src : a.q, on);
            p += step;
            j += dj;
            g += dg;
            if (g >= group) {
              g -= group;
              ++j;
            }
          }
        } else {
          // a thread per row: fp16 after a power of two, the largest channel in [1, 2)
          const int row = w * 32 + lane;
          int rr = !DIFF ? t * 128 + row : row, map = t;
          if (DIFF && kTiles == 1) {
            rr = (row >> 5) * 16 + (row & 15);
            map = (row >> 4) & 1;
          }
          const int p = p0 + rr, j = p / group, g = p - j * group;
          const uint16_t *src = a.q + ((int64_t)q0 + j) * a.qs + (int64_t)(h * group + g) * a.qhs;
          int from = 0, to = c.D / 8;
          if (DIFF) (map ? from : to) = c.D / 16;
          if (p >= p1) to = from;
          float mx = 0.f;
          for (int k = from; k < to; ++k) {
            const uint4 v = *reinterpret_cast<const uint4 *>(src + k * 8);
            const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(x[i] << 16)),
                                   fabsf(__uint_as_float(x[i] & 0xffff0000u))));
          }
          uint32_t ex = __float_as_uint(mx) >> 23;
          if (ex < 1 || ex >= 253) ex = 127;  // kept where 1 / 2^(ex - 127) is normal
          const float r = __uint_as_float((254 - ex) << 23);
          for (int k = 0; k < kCpr; ++k) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (k >= from && k < to) {
              v = *reinterpret_cast<const uint4 *>(src + k * 8);
              uint32_t *x = &v.x;
#pragma unroll
              for (int i = 0; i < 4; ++i)
                x[i] = pack2<1>(__uint_as_float(x[i] << 16) * r, __uint_as_float(x[i] & 0xffff0000u) * r);
            }
            sts128(dst + swz(128, row, k), v);
          }
          sh.qe[sidx & 1][t][row] = (uint8_t)ex;
        }
      }
      const uint32_t *tab_k =
          c.table + ((int64_t)slot * c.rows + ((int64_t)a.layer * 2) * c.heads + h) * c.blocks;
      const uint32_t *tab_v = tab_k + (int64_t)c.heads * c.blocks;
      // byte offsets in the pool of this lane's row of a block, ~0 where it has none
      uint64_t bk = ~0ull, bv = ~0ull;
      auto find = [&](int u) {
        const int t = first + u * kN + w * kRpw + lane % kRpw;
        const bool in = t >= lo && t < hi;
        bk = bv = ~0ull;
        if (in) {
          const int blk = t / c.Tb;
          const uint32_t pk = tab_k[blk], pv = tab_v[blk];
          if (pk < c.pages && pv < c.pages) {
            const uint32_t off = (uint32_t)(t - blk * c.Tb) * c.row_bytes;
            bk = (uint64_t)pk * c.page_bytes + off;
            bv = (uint64_t)pv * c.page_bytes + off;
          }
        }
        const uint32_t gone = __ballot_sync(~0u, in && bk == ~0ull && lane < kRpw);
        if (lane == 0) {
          reinterpret_cast<uint32_t *>(&sh.holes[(blocks + u) % kHoles])[w] = gone;
          if (gone) atomicOr(c.status, kCacheArg);
        }
      };
      auto masked = [&](int u) {
        const int t0 = first + u * kN;
        return t0 < most || t0 + kN > least;
      };
      if constexpr (ES == 2) {
        cp_commit();
        // values that are not finite in this thread's chunks of a partly masked block
        auto clean = [&](uint32_t dst) {
          bool any = false;
          for (int i = 0; i < kRpw / kRpi; ++i) {
            const int row = w * kRpw + i * kRpi + sub;
            uint4 v = lds128(dst + swz(kN, row, ch));
            uint32_t *x = &v.x, bad = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t e = __vcmpeq2(x[k] & 0x7f807f80u, 0x7f807f80u);
              x[k] &= ~e;
              bad |= e;
            }
            if (bad) {
              sts128(dst + swz(kN, row, ch), v);
              any = true;
            }
          }
          if (any) s.fix = 1;
        };
        auto tell = [&](int n) {  // n: 0 the queries, 1 + 2u K, 2 + 2u V of block u
          if (n > 0 && !(n & 1) && masked(n / 2 - 1))
            clean(sm + C::kOffSlots + (tiles + n - 1) % C::kSlots * C::kSlot);
          fence_async();
          arrive(n == 0 ? sh.q_full : sh.kv_full[(tiles + n - 1) % C::kSlots]);
        };
        const int copies = 1 + 2 * nu;
        for (int n = 1; n < copies && alive; ++n) {
          const uint32_t i = tiles + n - 1;
          const int u = (n - 1) / 2;
          const bool is_k = n & 1;
          if (is_k) find(u);
          if (!wait(sh.kv_empty[i % C::kSlots], ((i / C::kSlots) & 1) ^ 1)) {
            alive = false;
            break;
          }
          const uint32_t dst = sm + C::kOffSlots + i % C::kSlots * C::kSlot;
          const uint64_t from = is_k ? bk : bv;
#pragma unroll 4
          for (int x = 0; x < kRpw / kRpi; ++x) {
            const int row = x * kRpi + sub;
            const uint64_t b = __shfl_sync(~0u, from, row);
            const bool on = b != ~0ull && ch * 8 < c.D;
            cp_async16(dst + swz(kN, w * kRpw + row, ch), c.pool + (on ? b + ch * 16 : 0), on);
          }
          cp_commit();
          if (n >= kLag) {
            cp_wait<kLag>();
            tell(n - kLag);
          }
        }
        if (alive) {
          // (the next item's queries wait for this item's last block)
          cp_wait<1>();
          tell(copies - 2);
          cp_wait<0>();
          tell(copies - 1);
        }
      } else {
        fence_async();
        arrive(sh.q_full);
        constexpr int kCprRaw = DP / 16, kRpiRaw = 32 / kCprRaw > 0 ? 32 / kCprRaw : 1;
        constexpr int kCopies = kRpw * kCprRaw / 32;  // chunks of 16 codes of a thread per block
        const int chr = lane % kCprRaw, subr = lane / kCprRaw;
        const uint32_t raw = sm + C::kOffRaw + threadIdx.x % 128 * 16;
        const int copies = 2 * nu;
        auto fetch = [&](int n) {
          if (n < copies) {
            if (!(n & 1)) find(n / 2);
            const uint64_t from = n & 1 ? bv : bk;
            const uint32_t dst = raw + (tiles + n) % C::kRaws * C::kRaw;
#pragma unroll
            for (int x = 0; x < kCopies; ++x) {
              const uint64_t b = __shfl_sync(~0u, from, x * kRpiRaw + subr);
              const bool on = b != ~0ull && chr * 16 < c.D;
              cp_async16(dst + x * 2048, c.pool + (on ? b + chr * 16 : 0), on);
            }
          }
          cp_commit();
        };
        for (int n = 0; n < C::kRaws - 1; ++n) fetch(n);
        for (int n = 0; n < copies; ++n) {
          fetch(n + C::kRaws - 1);
          cp_wait<C::kRaws - 1>();
          const uint32_t i = tiles + n;
          if (!wait(sh.kv_empty[i % C::kSlots], ((i / C::kSlots) & 1) ^ 1)) {
            alive = false;
            break;
          }
          const uint32_t src = raw + i % C::kRaws * C::kRaw;
          const uint32_t dst = sm + C::kOffSlots + i % C::kSlots * C::kSlot;
          const bool check = (n & 1) && masked(n / 2);
          bool any = false;
#pragma unroll
          for (int x = 0; x < kCopies; ++x) {
            uint4 v = lds128(src + x * 2048);
            uint32_t *e = &v.x;
            if (check) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t bad = __vcmpeq4(e[k] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                e[k] &= ~bad;
                any = any || bad;
              }
            }
            uint4 y0, y1;
            e4m3x4(v.x, y0.x, y0.y);
            e4m3x4(v.y, y0.z, y0.w);
            e4m3x4(v.z, y1.x, y1.y);
            e4m3x4(v.w, y1.z, y1.w);
            const int row = w * kRpw + x * kRpiRaw + subr;
            sts128(dst + swz(kN, row, 2 * chr), y0);
            sts128(dst + swz(kN, row, 2 * chr + 1), y1);
          }
          if (any) s.fix = 1;
          fence_async();
          arrive(sh.kv_full[i % C::kSlots]);
        }
        cp_wait<0>();
      }
      tiles += 2 * nu;
      blocks += nu;
    }
    cp_wait<0>();
  } else {
    regs_less<C::kRegsM>();
    if (warp == kMma) {
      // -------------------------------------------------------------- products
      if (lane == 0) {
        const uint32_t half = 1u << 4 | (ES == 2 ? 1u << 7 | 1u << 10 : 0) | 8u << 24;
        const uint32_t dn = (c.D + 15) / 16 * 16;
        const uint32_t idesc_s = half | (uint32_t)(kN / 8) << 17;
        const uint32_t idesc_o = half | 1u << 16 | (dn / 8) << 17;
        uint32_t tiles = 0, sbuf = 0, items = 0;
        uint32_t np[2] = {0, 0};  // P of each tile (buffer) so far
        auto slot_wait = [&](uint32_t i) {
          return wait1(sh.kv_full[i % C::kSlots], (i / C::kSlots) & 1);
        };
        auto free_slot = [&](uint32_t i) { mma_commit(smem_addr(&sh.kv_empty[i % C::kSlots])); };
        auto scores = [&](int t, int buf, uint32_t i) {  // S of tile t with the keys in copy i
          const uint32_t q = sm + t * C::kQ, k = sm + C::kOffSlots + i % C::kSlots * C::kSlot;
          int from = 0, to = (c.D + 15) / 16;
          if (DIFF && kTiles == 2) {
            if (t == 0) to = (c.D / 2 + 15) / 16;
            else from = c.D / 2 / 16;
          }
          for (int x = from; x < to; ++x)
            mma_ss(tmem + buf * C::kS, desc_of(q + (x >> 2) * (128 * 128) + (x & 3) * 32, 16),
                   desc_of(k + (x >> 2) * (kN * 128) + (x & 3) * 32, 16), idesc_s, x > from);
          mma_commit(smem_addr(&sh.s_full[buf]));
        };
        auto sums = [&](int t, int buf, uint32_t i, bool add) {  // O of tile t += P V, V in copy i
          const uint32_t v = sm + C::kOffSlots + i % C::kSlots * C::kSlot;
#pragma unroll
          for (int x = 0; x < kN / 16; ++x)
            mma_ts(tmem + C::kO + t * DP, tmem + buf * C::kS + x * 8, desc_of(v + x * 2048, kN * 128),
                   idesc_o, add || x > 0);
        };
        for (uint32_t sidx = 0;; ++sidx) {
          Seg &s = sh.seg[sidx & 1];
          if (!wait1(sh.seg_full[sidx & 1], (sidx >> 1) & 1)) break;
          const int nu = s.nu;
          const bool two = kTiles == 2 && (DIFF || s.p0 + 128 < s.p1);
          bar_arrive(smem_addr(&sh.seg_empty[sidx & 1]));
          if (nu < 0) break;
          if (nu == 0) {
            mma_commit(smem_addr(&sh.q_empty));  // its phases count segments
            continue;
          }
          if (!wait1(sh.q_full, items++ & 1) || !slot_wait(tiles)) break;
          fence_after();
          bool ok = true;
          if constexpr (kTiles == 2) {
            scores(0, 0, tiles);
            if (two) scores(1, 1, tiles);
            free_slot(tiles);
            if (nu == 1) mma_commit(smem_addr(&sh.q_empty));
            for (int u = 0; u < nu && ok; ++u) {
              const uint32_t iv = tiles + 2 * u + 1, ik = iv + 1;
              if (!(ok = slot_wait(iv))) break;
              for (int t = 0; t < (two ? 2 : 1); ++t) {
                if (!(ok = wait1(sh.p_full[t], np[t]++ & 1))) break;
                fence_after();
                sums(t, t, iv, u > 0);
                if (t == (two ? 1 : 0)) free_slot(iv);
                if (u + 1 < nu) {
                  if (t == 0 && !(ok = slot_wait(ik))) break;
                  scores(t, t, ik);
                } else {
                  mma_commit(smem_addr(&sh.o_full[t]));
                }
              }
              if (ok && u + 1 < nu) {
                free_slot(ik);
                if (u + 2 == nu) mma_commit(smem_addr(&sh.q_empty));
              }
            }
          } else {
            scores(0, sbuf & 1, tiles);
            free_slot(tiles);
            if (nu == 1) mma_commit(smem_addr(&sh.q_empty));
            for (int u = 0; u < nu && ok; ++u, ++sbuf) {
              const uint32_t iv = tiles + 2 * u + 1, ik = iv + 1;
              if (u + 1 < nu) {
                if (!(ok = slot_wait(ik))) break;
                scores(0, (sbuf + 1) & 1, ik);
                free_slot(ik);
                if (u + 2 == nu) mma_commit(smem_addr(&sh.q_empty));
              }
              if (!(ok = slot_wait(iv) && wait1(sh.p_full[sbuf & 1], (sbuf >> 1) & 1))) break;
              fence_after();
              sums(0, sbuf & 1, iv, u > 0);
              free_slot(iv);
              mma_commit(smem_addr(&sh.o_full[0]));
              if (u + 1 == nu) mma_commit(smem_addr(&sh.o_full[1]));
            }
          }
          if (!ok) break;
          tiles += 2 * nu;
        }
        // nothing of the matrix unit is in flight when the tensor memory is given back
        mma_commit(smem_addr(&sh.last));
        for (const uint64_t from = now(); !bar_try(smem_addr(&sh.last), 0) && now() - from < kPatience;) {
        }
      }
      __syncwarp();
    } else if (warp == kDeal) {
      // -------------------------------------------------------------- the work
      // Costs of all sequences; every lane owns `per` neighbouring ones.
      const int per = (a.batch + 31) / 32, b0 = lane * per;
      auto cost_of = [&](const Span &sp) -> uint32_t { return cut ? sp.units + kItemCost : 1; };
      auto one_cost = [&](const Entry &e) -> uint64_t {  // of one kv head, this lane alone
        uint64_t x = 0;
        for (int i = 0; i < e.items; ++i) x += cost_of(span_of<C>(a, group, e, i));
        return x;
      };
      auto warp_cost = [&](const Entry &e) -> uint64_t {  // the same, all lanes
        uint64_t x = 0;
        for (int i = lane; i < e.items; i += 32) x += cost_of(span_of<C>(a, group, e, i));
#pragma unroll
        for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
        return x;
      };
      constexpr int kFew = 8;
      uint64_t own = 0;
      for (int k = 0; k < per; ++k) {
        const int b = b0 + k;
        Entry e;
        e.items = 0;
        if (b < a.batch) e = entry_of<C>(a, group, b, blockIdx.x == 0);
        const bool big = e.items > kFew;
        if (!big) own += one_cost(e) * c.heads;
        for (uint32_t todo = __ballot_sync(~0u, big); todo; todo &= todo - 1) {
          const int who = __ffs(todo) - 1;
          const Entry x = entry_of<C>(a, group, who * per + k, false);
          const uint64_t y = warp_cost(x) * c.heads;
          if (lane == who) own += y;
        }
      }
      uint64_t before = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(~0u, before, o);
        if (lane >= o) before += y;
      }
      const uint64_t all = __shfl_sync(~0u, before, 31);
      before -= own;
      uint32_t sidx = 0;
      Seg s;
      s.fix = 0;
      // hands a segment to the other warps (lane 0)
      auto hand = [&]() -> bool {
        if (!wait1(sh.seg_empty[sidx & 1], ((sidx >> 1) & 1) ^ 1)) return false;
        sh.seg[sidx & 1] = s;
        bar_arrive(smem_addr(&sh.seg_full[sidx & 1]));
        ++sidx;
        return true;
      };
      Cut *cuts = reinterpret_cast<Cut *>(a.ws);
      const uint32_t W = (uint32_t)all;
      const bool good = all > 0 && all <= 0x7fffffffull;  // (starts that decrease may add up to more)
      if (all > 0x7fffffffull && lane == 0) atomicOr(c.status, kCacheArg);
      const uint32_t nblk = good ? max(1u, min(cut ? W / 4 : W, gridDim.x)) : 1;
      uint32_t pos = 0, stop = 0;
      if (good && blockIdx.x < nblk) {
        pos = deal(W, nblk, blockIdx.x);
        stop = deal(W, nblk, blockIdx.x + 1);
      }
      if (lane == 0 && cut) cuts[blockIdx.x].parts = 0;
      if (pos < stop) {
        // the sequence b, the kv head h and the item i that unit `pos` lies in
        const int owner = __ffs(__ballot_sync(~0u, pos < before + own)) - 1;
        uint64_t at = __shfl_sync(~0u, before, owner);
        int b = owner * per;
        Entry e = entry_of<C>(a, group, b, false);
        uint64_t x = warp_cost(e);
        while (b + 1 < a.batch && pos >= at + x * c.heads) {
          at += x * c.heads;
          e = entry_of<C>(a, group, ++b, false);
          x = warp_cost(e);
        }
        const int h0 = x ? min((int)((pos - at) / x), c.heads - 1) : 0;
        at += x * h0;
        int i = 0;
        for (;;) {  // 32 items at a time
          const uint32_t mine = i + lane < e.items ? cost_of(span_of<C>(a, group, e, i + lane)) : 0;
          uint32_t y = mine;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const uint32_t z = __shfl_up_sync(~0u, y, o);
            if (lane >= o) y += z;
          }
          const uint32_t hit = __ballot_sync(~0u, pos < at + y);
          if (hit) {
            const int k = __ffs(hit) - 1;
            i += k;
            at += __shfl_sync(~0u, y - mine, k);
            break;
          }
          at += __shfl_sync(~0u, y, 31);
          i += 32;
          if (i >= e.items) break;  // (lengths that changed meanwhile)
        }
        if (lane == 0) {
          int h = h0;
          bool ok = true;
          while (ok && pos < stop && b < a.batch) {
            if (i >= e.items) {
              i = 0;
              if (++h >= c.heads) {
                h = 0;
                if (++b >= a.batch) break;
              }
              e = entry_of<C>(a, group, b, false);
              continue;
            }
            const Span sp = span_of<C>(a, group, e, i);
            const uint32_t cost = cost_of(sp);
            const int c0 = (int)(pos - (uint32_t)at);
            const int c1 = (int)min(cost, (uint32_t)c0 + (stop - pos));
            const int u0 = cut ? max(c0 - kItemCost, 0) : 0;
            const int nu = cut ? c1 - kItemCost - u0 : sp.units;
            if (nu > 0 || (sp.units == 0 && c1 == (int)cost)) {
              s.q0 = e.q0;
              s.p0 = i * C::kItem;
              s.p1 = min(s.p0 + C::kItem, e.rows);
              s.base = e.len - e.n;
              s.begin = e.begin;
              s.len = e.len;
              s.lo = sp.lo;
              s.hi = sp.hi;
              s.t0 = sp.start + u0 * kN;
              s.nu = max(nu, 0);
              s.h = h;
              s.slot = e.slot;
              s.part = nu <= 0 || nu == sp.units ? 0 : u0 == 0 ? 2 : 1;
              if (s.part == 2) {
                Cut k;
                k.q0 = s.q0;
                k.p0 = s.p0;
                k.p1 = s.p1;
                k.h = h;
                k.parts = min(block_of(W, nblk, (uint32_t)at + cost - 1), (int)nblk - 1) - blockIdx.x + 1;
                cuts[blockIdx.x] = k;
              }
              ok = hand();
            }
            pos += c1 - c0;
            if (c1 == (int)cost) {
              at += cost;
              ++i;
            }
          }
        }
      }
      __syncwarp();
      s.nu = -1;
      if (lane == 0) hand();
      __syncwarp();
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == kMma)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// Adds up the parts of the items that lie in several thread blocks, in their order: one warp
// per packed row.  blockIdx.x: the thread block that an item begins in.
constexpr int kJoin = 8;
template <int ES, int DP, bool DIFF>
__global__ void __launch_bounds__(kJoin * 32) k_chunk_join(ChunkArgs a) {
  using C = Cfg<ES, DP, DIFF>;
  constexpr int kVec = DP / 32, kMaps = DIFF ? 2 : 1;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const CacheView &c = a.c;
  const Cut k = reinterpret_cast<const Cut *>(a.ws)[blockIdx.x];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rr = blockIdx.y * kJoin + warp, p = k.p0 + rr;
  const int parts = min(k.parts, (int)gridDim.x - (int)blockIdx.x);
  if (parts <= 0 || p >= k.p1) return;
  const Part<C, DP> *part = reinterpret_cast<const Part<C, DP> *>(a.ws + kCutBytes) + blockIdx.x * 2;
  const int group = a.q_heads / c.heads;
  const int j = p / group, head = k.h * group + (p - j * group);
  const int64_t oh = ((int64_t)k.q0 + j) * a.q_heads + head;
  float unit = 1.f;
  if (ES == 1 && c.scale) unit = c.scale[a.layer * c.heads + k.h];
  float res[kVec];
#pragma unroll
  for (int map = 0; map < kMaps; ++map) {
    const int r = !DIFF ? rr : C::kTiles == 2 ? map * 128 + rr : (rr >> 4) * 32 + map * 16 + (rr & 15);
    float M = -INFINITY;
    for (int i = lane; i < parts; i += 32) M = fmaxf(M, part[2 * i + (i == 0)].m[r]);
#pragma unroll
    for (int s = 16; s; s >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, s));
    const float m0 = M == -INFINITY ? 0.f : M;
    float L = 0.f, o[kVec];
#pragma unroll
    for (int v = 0; v < kVec; ++v) o[v] = 0.f;
#pragma unroll 4
    for (int i = 0; i < parts; ++i) {
      const Part<C, DP> &x = part[2 * i + (i == 0)];
      const float w = ex2(x.m[r] - m0);
      L += w * x.l[r];
#pragma unroll
      for (int v = 0; v < kVec; ++v) o[v] += w * x.o[r][v * 32 + lane];
    }
    float by = L == 0.f ? 0.f : unit / L;
    if (map) by *= a.lambda[head];
#pragma unroll
    for (int v = 0; v < kVec; ++v) res[v] = map ? res[v] - o[v] * by : o[v] * by;
    if (lane == 0 && a.lse) a.lse[oh * kMaps + map] = (m0 + log2f(L)) * kLn2;
  }
  float n = 1.f;
  if (DIFF && a.norm) {
    float q = 0.f;
#pragma unroll
    for (int v = 0; v < kVec; ++v)
      if (v * 32 + lane < c.D) q = fmaf(res[v], res[v], q);
#pragma unroll
    for (int s = 16; s; s >>= 1) q += __shfl_xor_sync(~0u, q, s);
    n = q == 0.f ? 0.f : rsqrtf(q / c.D + a.eps);
  }
#pragma unroll
  for (int v = 0; v < kVec; ++v) {
    const int d = v * 32 + lane;
    if (d < c.D) {
      const __nv_bfloat16 y = __float2bfloat16_rn(res[v] * n * (DIFF && a.norm ? a.norm[d] : 1.f));
      a.out[oh * c.D + d] = *reinterpret_cast<const uint16_t *>(&y);
    }
  }
}

int sm_count() {
  static std::atomic<int> known[64];  // by device; a device's SMs do not change
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed))) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (n > kMostBlocks) n = kMostBlocks;
  if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

template <int ES, int DP, bool DIFF>
cudaError_t run(const ChunkArgs &a, cudaStream_t st) {
  using C = Cfg<ES, DP, DIFF>;
  constexpr size_t smem = C::kOffMisc + sizeof(Misc<C>);
  static_assert(smem <= 227 * 1024, "shared memory of a block");
  const int sms = sm_count();
  if (!sms) return cudaErrorInvalidDevice;
  const int64_t group = a.q_heads / a.c.heads;
  const int64_t items = (a.tokens * group / C::kItem + a.batch) * a.c.heads;
  const int64_t units = a.max_len / C::kN + 2;
  const int cut = units > 4;
  int64_t grid = cut ? items * units : items;
  if (grid > sms) grid = sms;
  auto kern = k_chunk<ES, DP, DIFF>;
  static std::atomic<bool> fits{false};  // the registers that the roles ask for are there
  cudaError_t e = cudaSuccess;
  if (!fits.load(std::memory_order_relaxed)) {
    cudaFuncAttributes at;
    if ((e = cudaFuncGetAttributes(&at, kern)) != cudaSuccess) return e;
    if (at.numRegs * C::kThreads < C::kRegs) return cudaErrorInvalidConfiguration;
    fits.store(true, std::memory_order_relaxed);
  }
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  e = launch(kern, dim3((unsigned)grid), C::kThreads, smem, st, a, cut);
  if (e != cudaSuccess || !cut) return e;
  return launch(k_chunk_join<ES, DP, DIFF>, dim3((unsigned)grid, C::kItem / kJoin), kJoin * 32, 0, st, a);
}

template <int ES, bool DIFF>
cudaError_t run_d(const ChunkArgs &a, cudaStream_t st) {
  if (a.c.D <= 64) return run<ES, 64, DIFF>(a, st);
  if (a.c.D <= 128) return run<ES, 128, DIFF>(a, st);
  return run<ES, 256, DIFF>(a, st);
}

}  // namespace

size_t chunk_ws_bytes(const CacheView &c, int32_t) {
  const int sms = sm_count();
  if (!sms) return 0;
  const size_t rows = c.D <= 128 ? 256 : 128, DP = c.D <= 64 ? 64 : c.D <= 128 ? 128 : 256;
  return kCutBytes + (size_t)sms * 2 * rows * (DP + 2) * sizeof(float);
}

cudaError_t launch_chunk(const ChunkArgs &a, cudaStream_t st) {
  if (a.lambda) return a.c.dtype == 1 ? run_d<1, true>(a, st) : run_d<2, true>(a, st);
  return a.c.dtype == 1 ? run_d<1, false>(a, st) : run_d<2, false>(a, st);
}

}  // namespace skv
