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
// The warps of a block have roles: 4 per tile for the softmax (one thread per row), 4 that load
// (whole boxes of pages by the TMA, else rows by cp.async, to a ring of slots; e4m3 codes, which a
// warp of their own brings, become fp16 on the way), one per tile that issues its matrix
// instructions, one that deals the work.  With two tiles the matrix unit works on one tile while
// the softmax of the other runs: they take turns, since mixed the instructions of both take as long
// as both (2048 tokens on 6144, 64 heads of 128, in the version of that step: 415 us against 367; now
// 376 to 390 by GPU).  With one tile (more than 128
// channels, whose sums take half of the tensor memory) S has two buffers.  Items of up to 128 rows
// let both tiles work on every second block with the same rows (9 tokens on 131071, e4m3: 90 us
// against 110).  bf16 weights round to bf16 (2^-8 of each): in two parts, as with one new token and in
// differential attention, the second product takes twice as long and the weights half as long again
// (a prompt of 4096 tokens 103 us against 85.5, 2048 tokens on 6144 522 against 379).
//
// What bounds it: a tile's chain of scores, weights and sums.  128 x 128 scores take a tile 1350
// clocks (512 of them the rate of the exponentials), its two products 1024, and the barriers
// between them 600; two tiles overlap to 3400 clocks a block where the products need 2048: 1260
// TFLOP/s (64% of the library's product) with 2048 tokens on 6144.  Blocks of 64 tokens with two
// buffers of S per tile took 574 us where this took 358 at the time, 4 slots of keys and values instead
// of 5 with room for the results the same.  A block of threads needs 10 us before its first scores
// (the code itself is fetched) and the join 3 to 10 us.
//
// Work is dealt as in skv_cache_attend.cuh: the blocks of all items in a row, cut evenly over one
// wave of persistent thread blocks whatever the lengths; items that lie in several leave partial
// results, which k_chunk_join adds up in a fixed order.
//
// What a row does not see must not touch it, and 0 * infinity is not 0: rows outside an item's
// range are zeros in shared memory, and in blocks that some rows see only in part the values
// that are not finite become 0, a flag is set, and the rows that see them get them in the end.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "skv_cache.cuh"

namespace skv {
namespace {

constexpr int kMostBlocks = 160;  // thread blocks of a launch
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kHoles = 16;       // blocks whose missing tokens are remembered
// Clocks that a barrier may take before a block gives up (2 s), and as many more as its two long waits may
// take in earnest: for the first work of a batch, every sequence of which is looked at, and for room for
// the next item while one of up to max_len tokens is worked on.
constexpr long long kPatience = 4000000000, kPerSequence = 1 << 13, kPerBlock = 1 << 16;

constexpr uint32_t kDescHigh = 1024 >> 4 | 1u << 14 | 2u << 29;  // see desc_of

template <int ES, int DP, bool DIFF>
struct Cfg {
  static constexpr int kTiles = DP <= 128 ? 2 : 1;       // tiles of 128 rows
  static constexpr int kN = DP <= 128 ? 128 : 64;        // tokens of a block
  static constexpr int kItem = (DIFF ? 64 : 128) * kTiles;  // packed rows of an item
  // An item costs a thread block this many blocks of tokens more than it has: queries are loaded,
  // results written and the pipeline runs empty in between.  us with 2 / 4 / 8, bf16: a prompt of
  // 4096 tokens 83.8 / 82.1 / 86.0, differential 159 / 137 / 147, windows with 256 channels 104.5 /
  // 101.1 / 100.3 (6: 100.1); e4m3: ragged turns 200 / 187 / 182, differential 207 / 195 / 186.  64
  // channels, bf16: a prompt 71.8 / 71.1 / 77.3, differential (weights in one part) 135 / 121 / 130;
  // e4m3: ragged turns 135.5 / 132.2 / 133.9, a prompt 82.6 / 76.5 / 81.5 (4 would do for them).
  static constexpr int kItemCost = ES == 1 ? 8 : DP == 256 ? 6 : 4;
  static constexpr int kQ = 128 * DP * 2;                // bytes of a tile of queries
  static constexpr int kSlot = kN * DP * 2;              // bytes of a block of keys or values
  static constexpr int kSlots = DP == 64 ? (ES == 2 ? 10 : 8) : (ES == 2 ? 4 : 3);
  static constexpr int kRaw = kN * DP;                   // bytes of a block of codes
  static constexpr int kRaws = ES == 2 ? 0 : DP == 64 ? 4 : 3;
  static constexpr int kSoftmax = 4 * kTiles;            // warps of the softmax
  static constexpr int kThreads = (kSoftmax + 8) * 32;
  // registers per thread of the softmax, the loads and the others; their sum over the threads
  // is within what the block is launched with
  static constexpr int kRegsS = kTiles == 2 ? 176 : 240, kRegsL = kTiles == 2 ? 80 : 120,
                       kRegsM = kTiles == 2 ? 80 : 72;
  static constexpr int kRegs = 32 * (kSoftmax * kRegsS + 4 * kRegsL + 4 * kRegsM);
  static constexpr int kOffSlots = kTiles * kQ;
  static constexpr int kOffRaw = kOffSlots + kSlots * kSlot;
  static constexpr int kOffStage = kOffRaw + kRaws * kRaw;  // results on their way out, 2 KB a warp
  static constexpr int kOffMisc = kOffStage + kSoftmax * 2048;
  // tensor memory columns
  static constexpr int kS = kN;            // S of a tile (or buffer); P in the first half, two parts all over it
  static constexpr int kO = 2 * kN;        // O, DP columns per tile
  // A row's m grows, to kLift below its maximum, when a block's weights add up to more than 2^kMost
  // (so no weight is larger; with two parts, when one is larger).  e4m3: weights meet the values as
  // fp16, which ends at 2^16, holds 11 bits down to 2^-14 and nothing below 2^-25; with the largest
  // weight at 2^8 to 2^15, and 128 of them at most 2^15, weights keep 11 bits down to 2^-22 of it and
  // the others are off by 2^-33 of it at most.  bf16 has a float's exponent.
  // Differential attention of bf16 caches: weights meet the values as two bf16 parts (2^-16 in all), since
  // the difference of two maps that attend to the same tokens is small next to either: one token with most
  // of both maps' weight, lambda 0.8, 1.4% off in the worst row with one part, 0.26% with two (the
  // result's rounding), for 176 us in place of 139 (a prompt of 4096 tokens).
  static constexpr int kParts = ES == 2 && DIFF ? 2 : 1;
  static constexpr float kLift = ES == 1 ? 8.f : 0.f;
  static constexpr int kMost = ES == 1 ? 15 : 20;
};

// What a thread block works on: blocks of tokens of one item.
struct Seg {
  int32_t q0, p0, p1;         // the sequence's first row of q; packed rows
  int32_t base, begin, len;   // the place of the first new token; tokens that any row may see
  int32_t lo, hi, t0;         // tokens that the item sees; the first block's first token
  int32_t nu;                 // blocks; 0: the rows see nothing; -1: the end
  int32_t h, slot, part;      // part: 0 the whole item, 1 and 2: a part, of which slot + 1
  int32_t twin;               // both tiles have the same rows and every second block
  uint32_t fix;               // values that are not finite were left out
};

template <typename C>
struct Misc {
  uint64_t q_full, q_empty, kv_full[C::kSlots], kv_empty[C::kSlots];
  uint64_t raw_full[4], raw_empty[4];
  uint64_t s_full[2], p_full[2], o_full[2], seg_full[2], seg_empty[2], turn[2], pair, last;
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
// an arrival that also waits for this many bytes of bulk copies
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// a box of the pool (see map_pages): channel, token of the page, block of 64 channels, page
__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x, int y,
                                         int b, uint32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, "
      "%6}], [%2];" ::"r"(dst), "l"(map), "r"(bar), "r"(x), "r"(y), "r"(b), "r"((int)z)
      : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{.reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p;}"
      : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok;
}
// the same without waiting (try_wait may sleep for a microsecond)
__device__ __forceinline__ bool bar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{.reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p;}"
      : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok;
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
// One lane of a warp, always the same.  What a matrix instruction takes lies in registers of the
// whole warp: all lanes go through the same code with the same values, and one issues.
__device__ __forceinline__ bool elect() {
  uint32_t p;
  asm volatile("{.reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p;}" : "=r"(p));
  return p;
}
// the barrier gets an arrival when all matrix instructions so far of this thread are done
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
               : "memory");
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{.reg .pred p; .reg .b64 a, b; setp.ne.b32 p, %4, 0; mov.b64 a, {%1, %5}; mov.b64 b, {%2, %5};\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;}" ::"r"(d), "r"(a), "r"(b), "r"(idesc),
      "r"((uint32_t)add), "r"(kDescHigh)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{.reg .pred p; .reg .b64 b; setp.ne.b32 p, %4, 0; mov.b64 b, {%2, %5};\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;}" ::"r"(d), "r"(a), "r"(b), "r"(idesc),
      "r"((uint32_t)add), "r"(kDescHigh)
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
// two floats at once
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<unsigned long long &>(d))
      : "l"(reinterpret_cast<const unsigned long long &>(a)),
        "l"(reinterpret_cast<const unsigned long long &>(b)),
        "l"(reinterpret_cast<const unsigned long long &>(c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long &>(d))
      : "l"(reinterpret_cast<const unsigned long long &>(a)),
        "l"(reinterpret_cast<const unsigned long long &>(b)));
  return d;
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

// Two weights as two bf16 parts each: their upper halves, and what these leave.  The rest is kept above 0
// (2^-18 of the weight more), so that no weight above 0 meets an infinite value as 0 times it.  (Single
// multiply-adds, which negate for nothing: 180 us against 194 with pairs.)
__device__ __forceinline__ float rest(float e) {
  return fmaf(e, 1.f + 0x1p-18f, -__uint_as_float(__float_as_uint(e) & 0xffff0000u));
}
__device__ __forceinline__ void two_parts(float2 e, uint32_t &high, uint32_t &low) {
  high = __byte_perm(__float_as_uint(e.x), __float_as_uint(e.y), 0x7632);
  low = pack2<2>(rest(e.x), rest(e.y));
}

// Tiles in shared memory: blocks of 64 channels, in each a row of 128 bytes per token (or
// packed row), whose 16-byte chunks are permuted by the row (128-byte swizzle).  As an operand
// whose rows are the rows (Q, K) the matrix unit steps 8 rows by 1024 bytes; as one whose rows
// are the channels (V) 8 tokens by 1024 and 64 channels by a block.
__device__ __forceinline__ uint32_t swz(int rows, int row, int ch) {
  return (uint32_t)((ch >> 3) * rows * 128 + row * 128 + (((ch ^ row) & 7) << 4));
}
// The low half of an operand's descriptor: address and lbo, both in 16 bytes; the high half is
// the same for all.  Steps along an operand are added to the low half.
__device__ __forceinline__ uint32_t desc_of(uint32_t addr, uint32_t lbo) {
  return (addr & 0x3ffff) >> 4 | (lbo >> 4) << 16;
}

// A place in the ring of slots and the parity of its round.
template <int N>
struct Ring {
  uint32_t at = 0, round = 0;
  __device__ __forceinline__ Ring plus(uint32_t n) const {
    Ring r;
    r.at = (at + n) % N;
    r.round = (round + (at + n) / N) & 1;
    return r;
  }
  __device__ __forceinline__ Ring after() const {
    Ring r;
    r.at = at + 1 == N ? 0 : at + 1;
    r.round = round ^ (at + 1 == N);
    return r;
  }
};

// A sequence of the batch.
struct Entry {
  int32_t slot, len, begin, q0, n;
  int32_t rows, items;  // packed rows, items per kv head
};
template <typename C>
__device__ __noinline__ Entry entry_of(const ChunkArgs &a, int group, int b, bool tell) {
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
__device__ __forceinline__ Entry from_lane(const Entry &e, int who) {
  Entry r;
  r.slot = __shfl_sync(~0u, e.slot, who);
  r.len = __shfl_sync(~0u, e.len, who);
  r.begin = __shfl_sync(~0u, e.begin, who);
  r.q0 = __shfl_sync(~0u, e.q0, who);
  r.n = __shfl_sync(~0u, e.n, who);
  r.rows = __shfl_sync(~0u, e.rows, who);
  r.items = __shfl_sync(~0u, e.items, who);
  return r;
}
// The tokens [lo, hi) that item i of a sequence sees, in blocks from lo's one on.
struct Span {
  int32_t lo, hi, start, units;
};
template <typename C>
__device__ __noinline__ Span span_of(const ChunkArgs &a, int group, const Entry &e, int i) {
  Span s;
  const int p0 = i * C::kItem, p1 = min(p0 + C::kItem, e.rows);
  const int base = e.len - e.n;
  s.lo = e.begin;
  if (a.window) s.lo = (int32_t)max((int64_t)s.lo, (int64_t)base + a.by_group.of(p0) - a.window + 1);
  s.hi = a.full ? e.len : min(e.len, base + a.by_group.of(p1 - 1) + 1);
  if (s.hi < s.lo) s.hi = s.lo;
  s.start = s.lo / C::kN * C::kN;
  s.units = s.hi > s.lo ? (s.hi - s.start + C::kN - 1) / C::kN : 0;
  return s;
}
// How units are dealt: see skv_cache_attend.cuh.
__device__ __forceinline__ uint32_t deal(uint32_t W, uint32_t n, uint32_t i) {
  const uint32_t q = W / n;
  return i * q + i * (W - q * n) / n;
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

// What follows runs rarely and is kept out of the loops' code.
// Scores of a row in tensor memory times f, where mul says so; with edge those of tokens outside
// [from, to) of the block, and the missing ones, become -infinity.
template <int N>
__device__ __noinline__ void settle_scores(uint32_t tm_s, bool mul, float f, bool edge, int from, int to,
                                           const uint32_t *missing) {
#pragma unroll 1
  for (int i = 0; i < N; i += 32) {
    float x[32];
    tm_ld32(x, tm_s + i);
    tm_wait_ld();
    uint32_t out = 0;  // tokens that this row does not see
    if (edge) {
      const int a = min(max(from - i, 0), 32), b = min(max(to - i, 0), 32);
      out = N == 128 ? missing[i / 32] : (missing[i / 16] & 0xffffu) | missing[i / 16 + 1] << 16;
      out |= ~(uint32_t)(((1ull << b) - 1) & ~((1ull << a) - 1));
    }
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      x[k] = mul ? __fmul_rn(x[k], f) : x[k];
      if (out >> k & 1) x[k] = -INFINITY;
    }
    tm_st32(tm_s + i, x);
  }
  tm_wait_st();
}
// The largest of a row's scores in tensor memory times f.
template <int N>
__device__ __noinline__ float top_score(uint32_t tm_s, float f) {
  float top = -INFINITY;
#pragma unroll 1
  for (int i = 0; i < N; i += 32) {
    float x[32];
    tm_ld32(x, tm_s + i);
    tm_wait_ld();
#pragma unroll
    for (int k = 0; k < 32; ++k) top = fmaxf(top, __fmul_rn(x[k], f));
  }
  return top;
}
// A row's sums in tensor memory times f.
template <int N>
__device__ __noinline__ void scale_sums(uint32_t tm_o, float f) {
#pragma unroll 1
  for (int d = 0; d < N; d += 32) {
    float o[32];
    tm_ld32(o, tm_o + d);
    tm_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] *= f;
    tm_st32(tm_o + d, o);
  }
}
// Whether any of a row's scores in tensor memory is NaN (or infinities of both signs are there).
template <int N>
__device__ __noinline__ bool any_nan(uint32_t tm_s) {
  float all = 0.f;
#pragma unroll 1
  for (int i = 0; i < N; i += 32) {
    float x[32];
    tm_ld32(x, tm_s + i);
    tm_wait_ld();
#pragma unroll
    for (int k = 0; k < 32; ++k) all += x[k];
  }
  return all != all;
}
// Sums become 0 where `none` says so.
template <int N>
__device__ __noinline__ void clear_sums(uint32_t tm_o, bool none) {
#pragma unroll 1
  for (int d = 0; d < N; d += 32) {
    float o[32];
    tm_ld32(o, tm_o + d);
    tm_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = none ? 0.f : o[i];
    tm_st32(tm_o + d, o);
  }
  tm_wait_st();
}
// Adds the values that were left out of a row's sums because they are not finite: those of tokens
// [lo, hi) that the row sees in blocks that some row of the item does not see in whole.
template <int ES, int N>
__device__ __noinline__ void add_not_finite(uint32_t tm_o, const CacheView &c, Div by_page, const uint32_t *tab,
                                            bool on, int lo, int hi, int most, int least, int t0, int end,
                                            int step) {
#pragma unroll 1
  for (int d = 0; d < c.D; d += 32) {
    float o[32];
    tm_ld32(o, tm_o + d);
    tm_wait_ld();
#pragma unroll 1
    for (int b = t0; b < end; b += step) {
      if (!on || (b >= most && b + N <= least)) continue;
#pragma unroll 1
      for (int t = max(b, lo); t < min(b + N, hi); ++t) {
        const int blk = by_page.of(t);
        const uint32_t pk = tab[blk], pv = tab[(int64_t)c.heads * c.blocks + blk];
        if (pk >= c.pages || pv >= c.pages) continue;
        const uint8_t *row = c.pool + (uint64_t)pv * c.page_bytes + (uint32_t)(t - blk * c.Tb) * c.row_bytes;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          if (d + i >= c.D) continue;
          if (ES == 2) {
            const uint16_t w = reinterpret_cast<const uint16_t *>(row)[d + i];
            if ((w & 0x7f80) == 0x7f80) o[i] += __uint_as_float((uint32_t)w << 16);
          } else if ((row[d + i] & 0x7f) == 0x7f) {
            o[i] = NAN;
          }
        }
      }
    }
    __syncwarp();
    tm_st32(tm_o + d, o);
  }
  tm_wait_st();
}
// The norm of a row of n channels in tensor memory, whatever power of two they lie at.
__device__ __noinline__ float inverse_norm(uint32_t tm, int n, float eps) {
  Squares all;
#pragma unroll 1
  for (int d = 0; d < n; d += 32) {
    float o[32];
    tm_ld32(o, tm + d);
    tm_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (d + i < n) all.add(o[i]);
  }
  return all.inverse(n, eps);
}
// Scores in tensor memory that are NaN, of the tokens from t0 on: made again of this row's half of the
// channels alone (map), times by.  (Tokens that the row does not see are not NaN by now.)
template <int ES, int N>
__device__ __noinline__ void own_half(uint32_t tm_s, const CacheView &c, bool on, int t0, Div by_page,
                                      const uint32_t *tab, const uint16_t *q, int map, float by) {
#pragma unroll 1
  for (int i = 0; i < N; i += 32) {
    float x[32];
    tm_ld32(x, tm_s + i);
    tm_wait_ld();
    uint32_t bad = 0;
#pragma unroll
    for (int k = 0; k < 32; ++k) bad |= (uint32_t)(x[k] != x[k]) << k;
    if (!on) bad = 0;
#pragma unroll 1
    for (; bad; bad &= bad - 1) {
      const int at = __ffs(bad) - 1, t = t0 + i + at, blk = by_page.of(t);
      const uint32_t pk = tab[blk];
      if (pk >= c.pages) continue;
      const float y = half_score<ES>(
          q, c.pool + (uint64_t)pk * c.page_bytes + (uint32_t)(t - blk * c.Tb) * c.row_bytes + map * (c.row_bytes / 2),
          c.D / 2);
#pragma unroll
      for (int k = 0; k < 32; ++k) x[k] = k == at ? y * by : x[k];
    }
    __syncwarp();
    tm_st32(tm_s + i, x);
  }
  tm_wait_st();
}

template <int ES, int DP, bool DIFF>
__global__ void __launch_bounds__((Cfg<ES, DP, DIFF>::kThreads), 1) k_chunk(
    ChunkArgs a, int cut, int box, const __grid_constant__ CUtensorMap map) {
  using C = Cfg<ES, DP, DIFF>;
  constexpr int kTiles = C::kTiles, kN = C::kN;
  extern __shared__ __align__(1024) uint8_t smem[];
  Misc<C> &sh = *reinterpret_cast<Misc<C> *>(smem + C::kOffMisc);
  const uint32_t sm = smem_addr(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const CacheView &c = a.c;
  const int group = a.q_heads / c.heads;
  // the warps behind those of the softmax: loads, the matrix instructions of the tiles, the work,
  // codes
  constexpr int kLoad0 = C::kSoftmax, kMma = kLoad0 + 4, kDeal = kLoad0 + 5, kFetch = kLoad0 + 6,
                kMma1 = kTiles == 2 ? kLoad0 + 7 : kMma;

  // Waits for a phase of a barrier, with a limit: then the block gives up and says so.
  auto wait1 = [&](uint64_t &bar, uint32_t parity, long long patience = kPatience) -> bool {
    const uint32_t b = smem_addr(&bar);
    if (bar_try(b, parity)) return true;
    // (the device's clock; the global timer takes a microsecond to read)
    const long long from = clock64();
    do {
#pragma unroll 1
      for (int i = 0; i < 32; ++i)
        if (bar_try(b, parity)) return true;
      if (*reinterpret_cast<volatile uint32_t *>(&sh.dead)) return false;
    } while (clock64() - from < patience);
    *reinterpret_cast<volatile uint32_t *>(&sh.dead) = 1;
    atomicOr(c.status, kCacheStuck);
    return false;
  };
  auto wait = [&](uint64_t &bar, uint32_t parity) -> bool {
    const bool ok = wait1(bar, parity);
    return __all_sync(~0u, ok);
  };
  auto wait_work = [&](uint32_t sidx) -> bool {  // for segment sidx
    const bool ok = wait1(sh.seg_full[sidx & 1], (sidx >> 1) & 1, a.patience);
    return __all_sync(~0u, ok);
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
    bar_init(smem_addr(&sh.q_empty), kTiles);
    for (int i = 0; i < C::kSlots; ++i) {
      bar_init(smem_addr(&sh.kv_full[i]), 4);
      bar_init(smem_addr(&sh.kv_empty[i]), kTiles);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(smem_addr(&sh.s_full[i]), 1);
      bar_init(smem_addr(&sh.p_full[i]), 4);
      bar_init(smem_addr(&sh.o_full[i]), 1);
      bar_init(smem_addr(&sh.seg_full[i]), 1);
      bar_init(smem_addr(&sh.turn[i]), 1);
      bar_init(smem_addr(&sh.seg_empty[i]), C::kSoftmax + 4 + kTiles + (ES == 1));
    }
    for (int i = 0; i < C::kRaws; ++i) {
      bar_init(smem_addr(&sh.raw_full[i]), 32);
      bar_init(smem_addr(&sh.raw_empty[i]), 4);
    }
    bar_init(smem_addr(&sh.pair), 8);
    bar_init(smem_addr(&sh.last), kTiles);
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
#pragma unroll 1
    for (uint32_t sidx = 0;; ++sidx) {
      Seg &s = sh.seg[sidx & 1];
      if (!wait_work(sidx)) break;
      const int nu = s.nu;
      if (nu < 0) break;
      const bool twin = s.twin;
      // packed row of the item of this thread
      const int rr = twin ? r : !DIFF ? tile * 128 + r : kTiles == 2 ? r : (r >> 5) * 16 + (r & 15);
      const int p = s.p0 + rr;
      const bool on = p < s.p1;
      const int j = a.by_group.of(p), head = s.h * group + (p - j * group);
      const int place = s.base + j;
      int lo = 0, hi = 0x7fffffff;
      if (on) {
        lo = s.begin;
        if (a.window) lo = (int)max((int64_t)lo, (int64_t)place - a.window + 1);
        hi = place < 0 ? 0 : a.full ? s.len : min(s.len, place + 1);
      }
      const bool rows = DIFF || twin || s.p0 + tile * 128 < s.p1;  // the tile has some
      const int u_from = twin ? tile : 0, u_step = twin ? 2 : 1;    // its blocks
      float m = -INFINITY;
      float l = 0.f;
      bool far = false, some_far = false;  // |m| > 2^20; of a row of the warp
      float unit = 1.f;
      if (ES == 1 && c.scale) unit = c.scale[a.layer * c.heads + s.h];
      if (nu > 0 && rows) {
        float f = a.scale * kLog2e * unit;
        // (of all rows alike: with e4m3 a row's own f may be too small to have a sign)
        const bool negative = f < 0.f;
        // blocks from wlo to whi are seen by all rows of the warp
        const int wlo = __reduce_max_sync(~0u, lo), whi = __reduce_min_sync(~0u, hi), end = s.t0 + nu * kN;
        bool fresh = true;  // the first of the tile's blocks
        // Where a step of 16 channels has some of both halves, or a tile rows of both maps, the zeros of a
        // row's query meet the other half's keys, and 0 * infinity is NaN.
        const bool mixed = DIFF && (kTiles == 1 || c.D % 32);
#pragma unroll 1
        for (int t0 = s.t0 + u_from * kN; t0 < end; t0 += u_step * kN) {
          const int buf = kTiles == 2 ? tile : (int)(mine & 1);
          const uint32_t phase = kTiles == 2 ? mine & 1 : (mine >> 1) & 1;
          if (!wait(sh.s_full[buf], phase)) break;
          fence_after();
          if (ES == 1 && fresh) f *= __uint_as_float((uint32_t)sh.qe[sidx & 1][twin ? 0 : tile][r] << 23);
          const uint32_t tm_s = lanes + buf * C::kS;
          float x[2][32];
          tm_ld32(x[0], tm_s);
          const uint4 &hole_of = sh.holes[(blocks + (t0 - s.t0) / kN) % kHoles];
          const uint4 hole = hole_of;
          const bool holes = hole.x | hole.y | hole.z | hole.w;
          const bool edge = t0 < wlo || t0 + kN > whi || holes;
          float fx = f;  // x = fx * what is in S
          bool product = false;  // S of this row holds x
          // The rare cases put x itself in S: masks, a negative f, and scores beyond 2^20, whose
          // differences from m are exact only when they are rounded before, as m was.  (Row by row:
          // which of its neighbours are such cases does not change a row's bits.)
          auto settle = [&]() {
            const bool mul = !product && (edge || negative || far);
            settle_scores<kN>(tm_s, mul, f, edge, lo - t0, hi - t0, reinterpret_cast<const uint32_t *>(&hole_of));
            product |= mul;
            fx = product ? 1.f : f;
          };
          if (edge || negative || some_far) {
            tm_wait_ld();  // (no load is under way where a function is called)
            settle();
            tm_ld32(x[0], tm_s);
          }
          float total = 0.f;
          bool ok = true;
          // m grows, in some rows, to the largest score
          auto grow = [&](bool more, float top) {
            // (beyond 2^23 a float has no room for kLift)
            const float mn = more ? (fabsf(top) < 0x1p23f ? top - C::kLift : top) : m;
            const float by = mn == -INFINITY ? 1.f : ex2(m - mn);
            m = mn;
            far = on && fabsf(m) > 0x1p20f && m != -INFINITY;
            some_far = __any_sync(~0u, far);
            l *= by;
            if (!fresh) {
              // With two buffers S may be there before the last product with the values is done
              // (but not before the one before that, so the barrier is one phase ahead at most).
              if (kTiles == 1 && !(ok = wait(sh.o_full[0], (mine - 1) & 1))) return;
              fence_after();
              scale_sums<DP>(tm_o, by);
            }
            if (__any_sync(~0u, far && !product)) settle();
          };
          // a NaN may be of the other half's channels: those scores are made again
          auto look = [&]() {
            // (e4m3: S is of q over a power of two)
            const float by = ES == 1 ? 1.f / __uint_as_float((uint32_t)sh.qe[sidx & 1][tile][r] << 23) : 1.f;
            own_half<ES, kN>(
                tm_s, c, on, t0, a.by_page,
                c.table + ((int64_t)s.slot * c.rows + ((int64_t)a.layer * 2) * c.heads + s.h) * c.blocks,
                a.q + ((int64_t)s.q0 + j) * a.qs + (int64_t)head * a.qhs + map * (c.D / 2), map,
                product ? by * f : by);
          };
          if constexpr (C::kParts == 2) {
            // The two parts of 32 tokens lie where their scores were, so m is settled before.
            if (mixed) {
              tm_wait_ld();
              const bool nan = any_nan<kN>(tm_s);  // (all lanes: its loads are the whole warp's)
              if (__any_sync(~0u, on && nan)) look();
              tm_ld32(x[0], tm_s);
            }
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < kN; i += 32) {
              const float *y = x[(i >> 5) & 1];
              tm_wait_ld();
              tm_ld32(x[((i >> 5) & 1) ^ 1], tm_s + (i + 32 < kN ? i + 32 : 0));
#pragma unroll
              for (int k = 0; k < 32; k += 2) top = fmaxf(top, fmaxf(y[k], y[k + 1]));
            }
            top = __fmul_rn(top, fx);
            // only rows that pass it change, so that no row's bits depend on another's
            const bool more = top - m > C::kMost;
            if (__any_sync(~0u, on && more)) {
              tm_wait_ld();
              grow(more, top);
              if (!ok) break;
              tm_ld32(x[0], tm_s);
            }
            const float m0 = m == -INFINITY ? 0.f : m;
            const float2 f2 = make_float2(fx, fx), m2 = make_float2(-m0, -m0);
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            // (rolled up and without a load ahead: 178 us; two or four at a time with one 180 and 185)
#pragma unroll 1
            for (int i = 0; i < kN; i += 32) {
              if (i) tm_ld32(x[0], tm_s + i);
              tm_wait_ld();
              uint32_t w[32];
#pragma unroll
              for (int k = 0; k < 32; k += 2) {
                const float2 z = fma2(make_float2(x[0][k], x[0][k + 1]), f2, m2);
                const float2 e = make_float2(ex2(z.x), ex2(z.y));
                sum[(k >> 1) & 1] = add2(sum[(k >> 1) & 1], e);
                two_parts(e, w[k / 2], w[16 + k / 2]);
              }
              tm_st16(tm_s + i, w);
              tm_st16(tm_s + i + 16, w + 16);
            }
            total = (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
          } else {
            uint32_t w[kN / 2];
            // The weights with the m so far.  Where they add up to more than 2^kMost, or a row has
            // not seen a token yet, m grows and they are made again: S is there until the weights
            // are written over it.
            bool looked = !mixed;
            constexpr float kFull = 1 << C::kMost;
#pragma unroll 1
            for (bool grows = fresh;;) {
              if (grows) {
                tm_wait_ld();
                // only rows that pass it change, so that no row's bits depend on another's
                grow(total > kFull || m == -INFINITY, top_score<kN>(tm_s, fx));
                if (!ok) break;
                tm_ld32(x[0], tm_s);
              }
              const float m0 = m == -INFINITY ? 0.f : m;
              const float2 f2 = make_float2(fx, fx), m2 = make_float2(-m0, -m0);
              float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
              for (int i = 0; i < kN; i += 32) {
                float *y = x[(i >> 5) & 1];
                tm_wait_ld();
                if (i + 32 < kN) tm_ld32(x[((i >> 5) & 1) ^ 1], tm_s + i + 32);
#pragma unroll
                for (int k = 0; k < 32; k += 2) {
                  const float2 z = fma2(make_float2(y[k], y[k + 1]), f2, m2);
                  const float2 e = make_float2(ex2(z.x), ex2(z.y));
                  sum[(k >> 1) & 1] = add2(sum[(k >> 1) & 1], e);
                  w[(i + k) / 2] = pack2<ES>(e.x, e.y);
                }
              }
              total = (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
              // (with two maps NaN too: see below)
              if (!__any_sync(~0u, on && ((DIFF ? !(total <= kFull) : total > kFull) || m == -INFINITY))) break;
              if (DIFF && !looked && __any_sync(~0u, on && total != total)) {
                look();
                looked = true;
                grows = false;
                tm_ld32(x[0], tm_s);
                continue;
              }
              if (grows) break;
              grows = true;
            }
            if (!ok) break;
#pragma unroll
            for (int i = 0; i < kN / 2; i += 16) tm_st16(tm_s + i, w + i);
          }
          l += total;
          tm_wait_st();
          fence_before();
          arrive(sh.p_full[buf]);
          ++mine;
          fresh = false;
        }
        blocks += nu;
        // ---- results
        // (with two buffers o_full[0] counts blocks and o_full[1] items)
        if (!wait(sh.o_full[kTiles == 2 ? tile : 1], ends++ & 1)) break;
        fence_after();
      } else if (nu > 0) {
        blocks += nu;
      }
      const float m0 = m == -INFINITY ? 0.f : m, L = l;
      const int64_t oh = ((int64_t)s.q0 + j) * a.q_heads + head;
      if (nu > 0 && rows && s.fix) {
        // values that are not finite, of partly masked blocks: those that this row sees
        const int jl = a.by_group.of(s.p1 - 1);
        const int most = a.window ? (int)max((int64_t)s.begin, (int64_t)s.base + jl - a.window + 1) : s.begin;
        const int least = a.full ? s.len : min(s.len, s.base + a.by_group.of(s.p0) + 1);
        const uint32_t *tab =
            c.table + ((int64_t)s.slot * c.rows + ((int64_t)a.layer * 2) * c.heads + s.h) * c.blocks;
        add_not_finite<ES, kN>(tm_o, c, a.by_page, tab, on, lo, hi, most, least, s.t0 + u_from * kN,
                               s.t0 + nu * kN, u_step * kN);
      }
      // Sums of rows that see nothing may be 0 times infinity.  They become 0 here, so that below a factor
      // of 0 (a tile's weight next to the other's, lambda, the norm of an infinite row) is a number like
      // others, whose product with an infinity is NaN.
      if (nu > 0 && rows && __any_sync(~0u, l == 0.f)) clear_sums<DP>(tm_o, l == 0.f);
      // Results leave through shared memory, so that 4 lanes write 64 bytes of one row: a lane's
      // own row in 16-byte pieces would be 32 rows per store (10000 clocks a tile, 2000 so).
      const bool emits = on && !(DIFF && kTiles == 1 && lane >= 16);
      uint32_t writes = 0;  // which of the four rows that this lane writes are there
      int64_t to_row[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        to_row[i] = __shfl_sync(~0u, oh, i * 8 + (lane >> 2)) * c.D;
        writes |= (uint32_t)__shfl_sync(~0u, (int)emits, i * 8 + (lane >> 2)) << i;
      }
      const uint32_t stage = sm + C::kOffStage + warp * 2048;
      auto place_of = [&](int row, int piece) { return stage + row * 64 + ((piece ^ (row >> 1)) & 3) * 16; };
      // 32 channels of the warp's rows, times by
      auto emit = [&](int d, const float *o, float by) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float x0 = o[k * 8 + 2 * i] * by, x1 = o[k * 8 + 2 * i + 1] * by;
            if (DIFF && a.norm && d + k * 8 < c.D) {
              x0 *= a.norm[d + k * 8 + 2 * i];
              x1 *= a.norm[d + k * 8 + 2 * i + 1];
            }
            w[i] = pack2<2>(x0, x1);
          }
          sts128(place_of(lane, k), make_uint4(w[0], w[1], w[2], w[3]));
        }
        __syncwarp();
        const int at = d + (lane & 3) * 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 v = lds128(place_of(i * 8 + (lane >> 2), lane & 3));
          if ((writes >> i & 1) && at < c.D) *reinterpret_cast<uint4 *>(a.out + to_row[i] + at) = v;
        }
        __syncwarp();
      };
      // the same of a partial result, fp32
      auto emit_part = [&](float (*to)[DP], int d, const float *o) {
#pragma unroll
        for (int half = 0; half < 32; half += 16) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float *x = o + half + k * 4;
            sts128(place_of(lane, k), make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]),
                                                 __float_as_uint(x[2]), __float_as_uint(x[3])));
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = i * 8 + (lane >> 2);
            const uint4 v = lds128(place_of(row, lane & 3));
            if (__shfl_sync(~0u, (int)on, row))
              *reinterpret_cast<uint4 *>(&to[row][d + half + (lane & 3) * 4]) = v;
          }
          __syncwarp();
        }
      };
      if (nu == 0) {
        if (on && (!DIFF || map == 0)) {
#pragma unroll 1
          for (int d = 0; d < c.D; d += 8)
            *reinterpret_cast<uint4 *>(a.out + oh * c.D + d) = make_uint4(0, 0, 0, 0);
          if (a.lse)
            for (int i = 0; i < maps; ++i) a.lse[oh * maps + i] = -INFINITY;
        }
      } else if (twin) {
        // the sums of both tiles, each of the two threads of a row half of the channels
        auto ml_of = [&](int warp) { return sm + C::kOffStage + warp * 2048 + lane * 8; };
        asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(ml_of(warp)), "f"(m), "f"(L) : "memory");
        fence_before();
        if (!both()) break;
        float om, ol;  // of the other
        asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(om), "=f"(ol) : "r"(ml_of(warp ^ 4)) : "memory");
        if (!both()) break;
        fence_after();
        const float M = fmaxf(m, om) == -INFINITY ? 0.f : fmaxf(m, om);
        float by = ex2(m - M), oby = ex2(om - M);
        const float all = tile ? ol * oby + L * by : L * by + ol * oby;
        if (!s.part) {
          const float scale = all == 0.f ? 0.f : unit / all;
          by *= scale;
          oby *= scale;
        }
        const float f0 = tile ? oby : by, f1 = tile ? by : oby;
        Part<C, DP> &part =
            reinterpret_cast<Part<C, DP> *>(a.ws + kCutBytes)[blockIdx.x * 2 + max(s.part - 1, 0)];
#pragma unroll 1
        for (int d = tile * (DP / 2); d < min(c.D, (tile + 1) * (DP / 2)); d += 32) {
          float o[32], o1[32];
          tm_ld32(o, lanes + C::kO + d);
          tm_ld32(o1, lanes + C::kO + DP + d);
          tm_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __fadd_rn(__fmul_rn(o[i], f0), __fmul_rn(o1[i], f1));
          if (s.part) emit_part(&part.o[r - lane], d, o);
          else emit(d, o, 1.f);
        }
        if (on && tile == 0) {
          const float top = fmaxf(m, om);
          if (s.part) {
            part.m[r] = top;
            part.l[r] = all;
          } else if (a.lse) {
            a.lse[oh] = (M + log2f(all)) * kLn2;
          }
        }
        fence_before();
        if (!both()) break;  // (neither tile's sums are overwritten before both are read)
      } else if (rows && (s.part || !DIFF)) {
        Part<C, DP> &part =
            reinterpret_cast<Part<C, DP> *>(a.ws + kCutBytes)[blockIdx.x * 2 + max(s.part - 1, 0)];
        const float by = L == 0.f ? 0.f : unit / L;
#pragma unroll 1
        for (int d = 0; d < c.D; d += 32) {
          float o[32];
          tm_ld32(o, tm_o + d);
          tm_wait_ld();
          if (s.part) emit_part(&part.o[tile * 128 + r - lane], d, o);
          else emit(d, o, by);
        }
        if (on && s.part) {
          part.m[tile * 128 + r] = m;
          part.l[tile * 128 + r] = L;
        } else if (on && a.lse) {
          a.lse[oh] = (m0 + log2f(L)) * kLn2;
        }
      } else if (DIFF) {
        if (on && a.lse) a.lse[oh * 2 + map] = (m0 + log2f(L)) * kLn2;
        float by = L == 0.f ? 0.f : unit / L;
        if (map && on && L != 0.f) by *= a.lambda[head];
        float n = 1.f, q = 0.f;
        if constexpr (kTiles == 2) {
          // each of the two threads of a row takes half of the channels of both maps
          sh.l[map][r] = by;
          fence_before();
          if (!both()) break;
          const float f0 = sh.l[0][r], f1 = sh.l[1][r];
          fence_after();
#pragma unroll 1
          for (int d = map * (DP / 2); d < min(c.D, (map + 1) * (DP / 2)); d += 32) {
            float o[32], o1[32];
            tm_ld32(o, lanes + C::kO + d);
            tm_ld32(o1, lanes + C::kO + DP + d);
            tm_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              o[i] = __fsub_rn(__fmul_rn(o[i], f0), __fmul_rn(o1[i], f1));
              if (d + i < c.D) q = fmaf(o[i], o[i], q);
            }
            if (a.norm) tm_st32(lanes + C::kO + d, o);
            else emit(d, o, 1.f);
          }
          if (a.norm) {
            tm_wait_st();
            fence_before();
            if (!both()) break;  // (both have read the factors)
            sh.l[map][r] = q;
            if (!both()) break;
            q = sh.l[0][r] + sh.l[1][r];
            n = rsqrtf(q / c.D + a.eps);
            const bool odd = on && !Squares::enough(q, a.eps);
            if (__any_sync(~0u, odd)) {  // (each of a row's threads takes all channels)
              fence_after();
              const float m = inverse_norm(lanes + C::kO, c.D, a.eps);
              if (odd) n = m;
            }
#pragma unroll 1
            for (int d = map * (DP / 2); d < min(c.D, (map + 1) * (DP / 2)); d += 32) {
              float o[32];
              tm_ld32(o, lanes + C::kO + d);
              tm_wait_ld();
              emit(d, o, n);
            }
          }
          fence_before();
          if (!both()) break;  // (neither tile's sums are overwritten before both are read)
        } else {
          // lanes i and i + 16 have a row's two maps
#pragma unroll 1
          for (int pass = a.norm ? 0 : 2; pass < 3; ++pass) {
            Squares all;  // second pass, where a row asks for it
            if (pass == 1 && !__any_sync(~0u, on && !Squares::enough(q, a.eps))) continue;
#pragma unroll 1
            for (int d = 0; d < c.D; d += 32) {
              float o[32];
              tm_ld32(o, tm_o + d);
              tm_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float x = __fmul_rn(o[i], by), y = __shfl_xor_sync(~0u, x, 16);
                o[i] = map ? y - x : x - y;
                if (pass == 0 && d + i < c.D) q = fmaf(o[i], o[i], q);
                if (pass == 1 && d + i < c.D) all.add(o[i]);
              }
              if (pass == 2) emit(d, o, n);
            }
            if (pass == 0) n = rsqrtf(q / c.D + a.eps);
            if (pass == 1 && !Squares::enough(q, a.eps)) n = all.inverse(c.D, a.eps);
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
    Ring<C::kSlots> ring;                            // of the next copy
    Ring<(C::kRaws > 0 ? C::kRaws : 1)> rawr;        // and of its codes
    bool alive = true;
    constexpr int kLag = 2;  // copies under way whose arrival is not told yet (bf16)
#pragma unroll 1
    for (uint32_t sidx = 0; alive; ++sidx) {
      Seg &s = sh.seg[sidx & 1];
      if (!wait_work(sidx)) break;
      const int nu = s.nu;
      const int q0 = s.q0, p0 = s.p0, p1 = s.p1, h = s.h, lo = s.lo, hi = s.hi, first = s.t0, slot = s.slot;
      // blocks before `most` or that end after `least` are masked for some rows
      int most = s.begin, least = s.len;
      if (nu > 0) {
        const int jl = a.by_group.of(p1 - 1);
        if (a.window) most = (int)max((int64_t)most, (int64_t)s.base + jl - a.window + 1);
        if (!a.full) least = min(least, s.base + a.by_group.of(p0) + 1);
      }
      arrive(sh.seg_empty[sidx & 1]);
      if (nu < 0) break;
      if (nu == 0) continue;
      const uint32_t *tab_k =
          c.table + ((int64_t)slot * c.rows + ((int64_t)a.layer * 2) * c.heads + h) * c.blocks;
      const uint32_t *tab_v = tab_k + (int64_t)c.heads * c.blocks;
      auto masked = [&](int u) {
        const int t0 = first + u * kN;
        return t0 < most || t0 + kN > least;
      };
      // Byte offsets in the pool of this lane's row of a block, ~0 where it has none.
      uint64_t bk = ~0ull, bv = ~0ull;
      auto find = [&](int u) {
        const int t = first + u * kN + w * kRpw + lane % kRpw;
        const bool in = t >= lo && t < hi;
        bk = bv = ~0ull;
        if (in) {
          const int blk = a.by_page.of(t);
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
      // A block that all rows see is copied by the TMA in whole boxes: lane i has box i.  Other
      // blocks are copied row by row (zeros where there is nothing).  Nothing that is in memory decides
      // which: the four warps bring a block's bytes together, also when its table entries change
      // between their look-ups.  (The pages of the next such block are looked up meanwhile.)
      uint32_t pk = 0, pv = 0, next_k = 0, next_v = 0;
      int off = 0, at_blk = 0, at_off = 0, at_u = -1;
      const bool has_box = lane * box < kN;
      auto inside = [&](int u) {
        return box && u < nu && !masked(u) && first + u * kN >= lo && first + (u + 1) * kN <= hi;
      };
      auto look = [&](int u) {  // calls come with u that grows
        if (at_u < 0) {
          const int t = first + u * kN + lane * box;
          at_blk = a.by_page.of(t);
          at_off = t - at_blk * c.Tb;
        } else {
          for (at_off += (u - at_u) * kN; at_off >= c.Tb; at_off -= c.Tb) ++at_blk;
        }
        at_u = u;
        if (has_box) {
          next_k = tab_k[at_blk];
          next_v = tab_v[at_blk];
        }
      };
      auto boxes = [&](int u) {
        if (at_u != u) look(u);
        pk = next_k;
        pv = next_v;
        off = at_off;
        if (inside(u + 1)) look(u + 1);
        // a box without a page: behind the pool's last one the TMA finds zeros
        const bool none = has_box && !(pk < c.pages && pv < c.pages);
        if (none) pk = pv = (uint32_t)c.pages;
        const uint32_t lost = __ballot_sync(~0u, none);
        uint32_t gone = 0;  // tokens of this warp's part of the block
        if (lost) gone = __ballot_sync(~0u, lane < kRpw && (lost >> (w * kRpw + lane % kRpw) / box & 1));
        if (lane == 0) {
          reinterpret_cast<uint32_t *>(&sh.holes[(blocks + u) % kHoles])[w] = gone;
          if (gone) atomicOr(c.status, kCacheArg);
        }
      };
      auto queries = [&]() {
#pragma unroll 1
        for (int t = 0; t < kTiles; ++t) {
          const uint32_t dst = sm + t * C::kQ;
          // rows behind the last are left as they are: nothing of them gets out of their lanes
          const int rows = DIFF && kTiles == 1 ? 128 : min(p1 - p0 - (DIFF ? 0 : t * 128), 128);
          if (ES == 2) {
#pragma unroll 1
            for (int row0 = w * kRpi; row0 < rows; row0 += 4 * kRpi) {
              const int row = row0 + sub;
              const int rr = !DIFF ? t * 128 + row : kTiles == 2 ? row : (row >> 5) * 16 + (row & 15);
              const int p = p0 + rr, j = a.by_group.of(p), g = p - j * group;
              bool on = p < p1 && ch * 8 < c.D;
              if (DIFF) {
                // halves end at a multiple of 8 channels
                const bool second = kTiles == 2 ? t : (row >> 4) & 1;
                if (second ? ch * 8 < c.D / 2 : ch * 8 >= c.D / 2) on = false;
              }
              const uint16_t *src = a.q + ((int64_t)q0 + j) * a.qs + (int64_t)(h * group + g) * a.qhs + ch * 8;
              cp_async16(dst + swz(128, row, ch), on ? src : a.q, on);
            }
          } else {
            // a thread per row: fp16 after a power of two, the largest channel in [1, 2)
            const int row = w * 32 + lane;
            if (row >= rows) {
              sh.qe[sidx & 1][t][row] = 127;
              continue;
            }
            int rr = !DIFF ? t * 128 + row : row, of = t;
            if (DIFF && kTiles == 1) {
              rr = (row >> 5) * 16 + (row & 15);
              of = (row >> 4) & 1;
            }
            const int p = p0 + rr, j = a.by_group.of(p), g = p - j * group;
            const uint16_t *src = a.q + ((int64_t)q0 + j) * a.qs + (int64_t)(h * group + g) * a.qhs;
            int from = 0, to = c.D / 8;
            if (DIFF) (of ? from : to) = c.D / 16;
            if (p >= p1) to = from;
            float mx = 0.f;
#pragma unroll 1
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
#pragma unroll 2
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
      };
      if constexpr (ES == 2) {
        // values that are not finite in this thread's chunks of a partly masked block
        auto clean = [&](uint32_t dst) {
          bool any = false;
#pragma unroll 1
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
        // Copies of this item: K0, V0, K1, ...  Those of single rows are told kLag copies later.
        bool bulk = false, bulk_before = true;
        auto tell = [&](int n) {
          const uint32_t i = tiles + n;
          if ((n & 1) && masked(n / 2)) clean(sm + C::kOffSlots + i % C::kSlots * C::kSlot);
          fence_async();
          arrive(sh.kv_full[i % C::kSlots]);
        };
        const int copies = 2 * nu;
        // the queries: at once when the item before has read its own, else after the first block
        bool asked = __all_sync(~0u, bar_test(smem_addr(&sh.q_empty), (sidx & 1) ^ 1));
        if (asked) queries();
#pragma unroll 1
        for (int n = 0; n < copies; ++n) {
          const int u = n / 2;
          const bool is_v = n & 1;
          if (!is_v) {
            bulk_before = n == 0 || bulk;
            bulk = inside(u);
            if (bulk) boxes(u);
            else find(u);
          }
          if (!wait(sh.kv_empty[ring.at], ring.round ^ 1)) {
            alive = false;
            break;
          }
          const uint32_t dst = sm + C::kOffSlots + ring.at * C::kSlot;
          if (bulk) {
            // every warp issues a quarter of the boxes; one arrival brings the bytes
            const uint32_t bar = smem_addr(&sh.kv_full[ring.at]);
            const int wide = (c.D + 63) / 64, per = c.D % 64 == 0 && box == kN ? wide : 1;
            const bool blocked = c.D % 64 == 0;
            if (has_box && (lane & 3) == w)
              for (int x = 0; x < wide; x += per)
                copy_box(dst + x * kN * 128 + lane * box * 128, &map, bar, blocked ? 0 : x * 64, off,
                         blocked ? x : 0, is_v ? pv : pk);
            __syncwarp();
            if (lane == 0) {
              if (w == 0) bar_expect(bar, wide * kN * 128);
              else bar_arrive(bar);
            }
          } else {
            const uint64_t from = is_v ? bv : bk;
#pragma unroll 4
            for (int x = 0; x < kRpw / kRpi; ++x) {
              const int row = x * kRpi + sub;
              const uint64_t b = __shfl_sync(~0u, from, row);
              const bool on = b != ~0ull && ch * 8 < c.D;
              cp_async16(dst + swz(kN, w * kRpw + row, ch), c.pool + (on ? b + ch * 16 : 0), on);
            }
          }
          cp_commit();
          ring = ring.after();
          if (n == 1) {
            if (!asked) {
              if (!wait(sh.q_empty, (sidx & 1) ^ 1)) {
                alive = false;
                break;
              }
              queries();
              cp_commit();
            }
            cp_wait<0>();
            fence_async();
            arrive(sh.q_full);
            if (!bulk) {
              tell(0);
              tell(1);
            }
            bulk = true;  // told
          } else if (n >= kLag + 2 && !bulk_before) {
            cp_wait<kLag>();
            tell(n - kLag);
          }
        }
        if (alive && !bulk) {
          // (the next item's queries wait for this item's last block)
          cp_wait<1>();
          tell(copies - 2);
          cp_wait<0>();
          tell(copies - 1);
        }
      } else {
        // codes, which the warp kFetch brings to the ring of raw blocks, become fp16
        constexpr int kCprRaw = DP / 16, kRpiRaw = 32 / kCprRaw;
        constexpr int kCopies = kRpw * kCprRaw / 32;  // chunks of 16 codes of a thread per block
        const int chr = lane % kCprRaw, subr = lane / kCprRaw;
        const uint32_t raw0 = sm + C::kOffRaw + (w * kRpw + subr) * DP + chr * 16;
        const int copies = 2 * nu;
        if (!wait(sh.q_empty, (sidx & 1) ^ 1)) {
          alive = false;
          break;
        }
        queries();
        fence_async();
        arrive(sh.q_full);
#pragma unroll 1
        for (int n = 0; n < copies; ++n) {
          if (!wait(sh.raw_full[rawr.at], rawr.round) || !wait(sh.kv_empty[ring.at], ring.round ^ 1)) {
            alive = false;
            break;
          }
          const uint32_t raw = raw0 + rawr.at * C::kRaw;
          const uint32_t dst = sm + C::kOffSlots + ring.at * C::kSlot;
          bool any = false;
          if ((n & 1) && masked(n / 2)) {
#pragma unroll 1
            for (int x = 0; x < kCopies; ++x) {
              uint4 v = lds128(raw + x * 512);
              uint32_t *e = &v.x, bad = 0;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t m = __vcmpeq4(e[k] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                e[k] &= ~m;
                bad |= m;
              }
              if (bad) {
                sts128(raw + x * 512, v);
                any = true;
              }
            }
          }
          constexpr int kOnce = kCopies < 4 ? kCopies : 4;
#pragma unroll
          for (int x0 = 0; x0 < kCopies; x0 += kOnce) {
            uint4 v[kOnce];
#pragma unroll
            for (int x = 0; x < kOnce; ++x) v[x] = lds128(raw + (x0 + x) * 512);
#pragma unroll
            for (int x = 0; x < kOnce; ++x) {
              uint4 y0, y1;
              e4m3x4(v[x].x, y0.x, y0.y);
              e4m3x4(v[x].y, y0.z, y0.w);
              e4m3x4(v[x].z, y1.x, y1.y);
              e4m3x4(v[x].w, y1.z, y1.w);
              const int row = w * kRpw + (x0 + x) * kRpiRaw + subr;
              // (of 8 lanes that write at once, 4 write their second half first: the chunks of
              // channels 64 apart lie in the same banks)
              const bool turn = kCprRaw >= 8 && (chr & 4);
              sts128(dst + swz(kN, row, 2 * chr + turn), turn ? y1 : y0);
              sts128(dst + swz(kN, row, 2 * chr + !turn), turn ? y0 : y1);
            }
          }
          if (any) s.fix = 1;
          // (also before raw_empty: the next bulk copy to this place comes after what was written
          // to it above, and by the rows that kFetch copied)
          fence_async();
          arrive(sh.raw_empty[rawr.at]);
          arrive(sh.kv_full[ring.at]);
          ring = ring.after();
          rawr = rawr.after();
        }
      }
      tiles += 2 * nu;
      blocks += nu;
    }
    cp_wait<0>();
    // a block that gives up may have bulk copies under way: they land within microseconds
    if (!alive)
      for (const long long from = clock64(); clock64() - from < 2000000;) {
      }
  } else {
    regs_less<C::kRegsM>();
    if (warp == kMma || warp == kMma1) {
      // -------------------------------------------------------------- products
      const uint32_t half = 1u << 4 | (ES == 2 ? 1u << 7 | 1u << 10 : 0) | 8u << 24;
      const uint32_t dn = (c.D + 15) / 16 * 16;
      const uint32_t idesc_s = half | (uint32_t)(kN / 8) << 17;
      const uint32_t idesc_o = half | 1u << 16 | (dn / 8) << 17;
      const uint32_t tm = __shfl_sync(~0u, tmem, 0);
      // Each tile has a warp of its own: one looks after its barriers while the other's
      // instructions run.
      const int t = kTiles == 2 && warp == kMma1 ? 1 : 0;
      uint32_t done = 0, items = 0;          // blocks of this tile, items so far
      uint32_t turns = 0;                    // turns of this tile at the matrix unit so far
      Ring<C::kSlots> ring;                  // of the next copy, in the order K0, V0, K1, ...
      auto commit = [&](uint64_t &bar) {
        if (elect()) mma_commit(smem_addr(&bar));
      };
      const int steps = (c.D + 15) / 16;     // of 16 channels
      const uint32_t q_desc = desc_of(sm, 16);
      const uint32_t k_desc = desc_of(sm + C::kOffSlots, 16), v_desc = desc_of(sm + C::kOffSlots, kN * 128);
      // S of the keys in slot `at`; the other tile may go when the last half is on its way
      auto scores = [&](int buf, uint32_t at, bool pass, bool alone = false) {
        const uint32_t d = tm + buf * C::kS, q = q_desc + (alone ? 0 : t * (C::kQ / 16)), k = k_desc + at * (C::kSlot / 16);
        if (elect()) {
          if (!DIFF && steps == DP / 16) {
#pragma unroll
            for (int x = 0; x < DP / 16; ++x) {
              if (x == DP / 32 && pass) bar_arrive(smem_addr(&sh.turn[t ^ 1]));
              mma_ss(d, q + ((x >> 2) * (128 * 128) + (x & 3) * 32) / 16,
                     k + ((x >> 2) * (kN * 128) + (x & 3) * 32) / 16, idesc_s, x > 0);
            }
          } else {
            if (pass) bar_arrive(smem_addr(&sh.turn[t ^ 1]));
            // (the halves of a differential query have zeros in the other's channels)
            const int from = DIFF && kTiles == 2 && t ? c.D / 2 / 16 : 0;
            const int to = DIFF && kTiles == 2 && !t ? (c.D / 2 + 15) / 16 : steps;
#pragma unroll 1
            for (int x = from; x < to; ++x)
              mma_ss(d, q + ((x >> 2) * (128 * 128) + (x & 3) * 32) / 16,
                     k + ((x >> 2) * (kN * 128) + (x & 3) * 32) / 16, idesc_s, x > from);
          }
          mma_commit(smem_addr(&sh.s_full[buf]));
          mma_commit(smem_addr(&sh.kv_empty[at]));
          if (alone) mma_commit(smem_addr(&sh.kv_empty[at]));  // for both tiles
        }
        __syncwarp();
      };
      auto sums = [&](int buf, uint32_t at, bool add, bool alone = false) {  // O += P V, V in slot `at`
        const uint32_t d = tm + C::kO + t * DP, p = tm + buf * C::kS, v = v_desc + at * (C::kSlot / 16);
        if (elect()) {
#pragma unroll
          for (int x = 0; x < kN / 16; ++x) {
            if (C::kParts == 1) {
              mma_ts(d, p + x * 8, v + x * 2048 / 16, idesc_o, add || x > 0);
            } else {  // the parts of 32 tokens' weights lie next to each other
              mma_ts(d, p + (x >> 1) * 32 + (x & 1) * 8, v + x * 2048 / 16, idesc_o, add || x > 0);
              mma_ts(d, p + (x >> 1) * 32 + (x & 1) * 8 + 16, v + x * 2048 / 16, idesc_o, true);
            }
          }
          mma_commit(smem_addr(&sh.kv_empty[at]));
          if (alone) mma_commit(smem_addr(&sh.kv_empty[at]));
        }
        __syncwarp();
      };
#pragma unroll 1
      for (uint32_t sidx = 0;; ++sidx) {
        Seg &s = sh.seg[sidx & 1];
        if (!wait_work(sidx)) break;
        const int nu = __shfl_sync(~0u, s.nu, 0);
        const bool twin = kTiles == 2 && !DIFF && __shfl_sync(~0u, s.twin, 0);
        const bool two = kTiles == 2 && (DIFF || __shfl_sync(~0u, (int)(s.p0 + 128 < s.p1), 0));
        arrive(sh.seg_empty[sidx & 1]);
        if (nu < 0) break;
        if (nu == 0) {
          commit(sh.q_empty);  // its phases count segments
          continue;
        }
        if (!wait(sh.q_full, items++ & 1)) break;
        fence_after();
        bool ok = true;
        if (twin) {
          // every second block, with the first tile's queries; the other warp leaves its slots alone
          Ring<C::kSlots> r = ring.plus(2 * t);
          int u = t;
#pragma unroll 1
          for (; ok; u += 2) {
            if (!(ok = wait(sh.kv_full[r.at], r.round))) break;
            fence_after();
            scores(t, r.at, false, true);
            const bool more = u + 2 < nu;
            if (!more) commit(sh.q_empty);
            r = r.after();
            if (!(ok = wait(sh.kv_full[r.at], r.round) && wait(sh.p_full[t], done++ & 1))) break;
            fence_after();
            sums(t, r.at, u > t, true);
            if (!more) break;
            r = r.plus(3);
          }
          if (!ok) break;
          commit(sh.o_full[t]);
          ring = ring.plus(2 * nu);
          continue;
        }
        const bool mine = t == 0 || two;
#pragma unroll 1
        for (int u = -1; u < nu; ++u) {
          const Ring<C::kSlots> rv = ring, rk = u < 0 ? ring : ring.after();
          const bool more = u + 1 < nu;
          const uint32_t n = done + u;
          if (kTiles == 1) {
            // two buffers: the scores of block u + 1, whose buffer is free, then the sums of block u
            if (more) {
              if (!(ok = wait(sh.kv_full[rk.at], rk.round))) break;
              scores((n + 1) & 1, rk.at, false);
              if (u + 2 == nu) commit(sh.q_empty);
            }
            if (u >= 0) {
              if (!(ok = wait(sh.kv_full[rv.at], rv.round) && wait(sh.p_full[n & 1], (n >> 1) & 1))) break;
              fence_after();
              sums(n & 1, rv.at, u > 0);
              commit(sh.o_full[0]);
              if (!more) commit(sh.o_full[1]);
            }
          } else {
            // The sums of block u, the scores of block u + 1.  The tiles take turns at the matrix
            // unit: mixed, the instructions of both would take as long as both.
            if (u >= 0 && !(ok = wait(sh.kv_full[rv.at], rv.round))) break;
            if (two && more && !(ok = wait(sh.kv_full[rk.at], rk.round))) break;
            if (mine) {
              if (u >= 0 && !(ok = wait(sh.p_full[t], n & 1))) break;
              if (two && !(ok = wait(sh.turn[t], (turns++ & 1) ^ (t == 0)))) break;
              fence_after();
              if (u >= 0) sums(t, rv.at, u > 0);
            } else if (u >= 0) {
              commit(sh.kv_empty[rv.at]);
            }
            if (more) {
              if (!two && !(ok = wait(sh.kv_full[rk.at], rk.round))) break;
              if (mine) scores(t, rk.at, two);
              else commit(sh.kv_empty[rk.at]);
              if (u + 2 == nu) commit(sh.q_empty);
            } else {
              if (two) arrive(sh.turn[t ^ 1]);
              if (mine) commit(sh.o_full[t]);
            }
          }
          ring = more ? rk.after() : rv.after();
        }
        if (mine) done += nu;
        if (!ok) break;
      }
      // nothing of the matrix unit is in flight when the tensor memory is given back
      commit(sh.last);
      for (const long long from = clock64(); !bar_try(smem_addr(&sh.last), 0) && clock64() - from < kPatience;) {
      }
      __syncwarp();
    } else if (warp == kDeal) {
      // -------------------------------------------------------------- the work
      // Costs of all sequences; every lane owns `per` neighbouring ones.
      const int per = (a.batch + 31) / 32, b0 = lane * per;
      auto cost_of = [&](const Span &sp) -> uint32_t { return cut ? sp.units + C::kItemCost : 1; };
      auto one_cost = [&](const Entry &e) -> uint64_t {  // of one kv head, this lane alone
        uint64_t x = 0;
#pragma unroll 1
        for (int i = 0; i < e.items; ++i) x += cost_of(span_of<C>(a, group, e, i));
        return x;
      };
      auto warp_cost = [&](const Entry &e) -> uint64_t {  // the same, all lanes
        uint64_t x = 0;
#pragma unroll 1
        for (int i = lane; i < e.items; i += 32) x += cost_of(span_of<C>(a, group, e, i));
#pragma unroll
        for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
        return x;
      };
      constexpr int kFew = 4;
      uint64_t own = 0;
      Entry e;             // of the lane's last sequence, its only one in batches of up to 32
      uint32_t x = 0;      // and its cost, of one kv head
#pragma unroll 1
      for (int k = 0; k < per; ++k) {
        const int b = b0 + k;
        e.items = 0;
        if (b < a.batch) e = entry_of<C>(a, group, b, blockIdx.x == 0);
        x = 0;
        const bool big = e.items > kFew;
        if (!big) x = (uint32_t)one_cost(e);
#pragma unroll 1
        for (uint32_t todo = __ballot_sync(~0u, big); todo; todo &= todo - 1) {
          const int who = __ffs(todo) - 1;
          const uint32_t y = (uint32_t)warp_cost(from_lane(e, who));
          if (lane == who) x = y;
        }
        own += (uint64_t)x * c.heads;
      }
      uint64_t before = own;
#pragma unroll 1
      for (int o = 1; o < 32 && o < a.batch; o <<= 1) {
        const uint64_t y = __shfl_up_sync(~0u, before, o);
        if (lane >= o) before += y;
      }
      const uint64_t all = __shfl_sync(~0u, before, min(a.batch, 32) - 1);
      before -= own;
      uint32_t sidx = 0;
      Seg s;
      s.fix = 0;
      // hands a segment to the other warps (lane 0)
      auto hand = [&]() -> bool {
        if (!wait1(sh.seg_empty[sidx & 1], ((sidx >> 1) & 1) ^ 1, a.patience)) return false;
        sh.seg[sidx & 1] = s;
        bar_arrive(smem_addr(&sh.seg_full[sidx & 1]));
        ++sidx;
        return true;
      };
      Cut *cuts = reinterpret_cast<Cut *>(a.ws);
      const uint32_t W = (uint32_t)all;
      const bool good = all > 0 && all <= 0x7fffffffull;  // (starts that decrease may add up to more)
      if (all > 0x7fffffffull && lane == 0) atomicOr(c.status, kCacheArg);
      const uint32_t nblk = good ? max(1u, min(cut ? W / 2 : W, gridDim.x)) : 1;
      uint32_t pos = 0, stop = 0;
      if (good && blockIdx.x < nblk) {
        pos = deal(W, nblk, blockIdx.x);
        stop = deal(W, nblk, blockIdx.x + 1);
      }
      if (lane == 0 && cut) cuts[blockIdx.x].parts = 0;
      if (pos < stop) {
        // the sequence b, the kv head h and the item i that unit `pos` lies in
        const int owner = __ffs(__ballot_sync(~0u, pos < before + own)) - 1;
        uint32_t at = (uint32_t)__shfl_sync(~0u, before, owner);
        int b = owner * per;
        e = from_lane(e, owner);
        x = __shfl_sync(~0u, x, owner);
        if (per > 1) {
          e = entry_of<C>(a, group, b, false);
          x = (uint32_t)warp_cost(e);
#pragma unroll 1
          while (b + 1 < a.batch && pos >= at + x * c.heads) {
            at += x * c.heads;
            e = entry_of<C>(a, group, ++b, false);
            x = (uint32_t)warp_cost(e);
          }
        }
        const int h0 = x ? min((int)((pos - at) / x), c.heads - 1) : 0;
        at += x * h0;
        int i = 0;
#pragma unroll 1
        for (;;) {  // 32 items at a time
          const uint32_t mine = i + lane < e.items ? cost_of(span_of<C>(a, group, e, i + lane)) : 0;
          uint32_t y = mine;
#pragma unroll 1
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
#pragma unroll 1
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
            const int c0 = (int)(pos - at);
            const int c1 = (int)min(cost, (uint32_t)c0 + (stop - pos));
            const int u0 = cut ? max(c0 - C::kItemCost, 0) : 0;
            const int nu = cut ? c1 - C::kItemCost - u0 : sp.units;
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
              s.twin = kTiles == 2 && !DIFF && s.p1 - s.p0 <= 128 && nu > 1;
              if (s.part == 2) {
                Cut k;
                k.q0 = s.q0;
                k.p0 = s.p0;
                k.p1 = s.p1;
                k.h = h;
                // the blocks that begin in the rest of the item: shares differ by one at most
                const uint32_t rest = at + cost - stop;
                k.parts = 1 + rest / (W / nblk + 1);
                while (blockIdx.x + k.parts < nblk && deal(W, nblk, blockIdx.x + k.parts) < at + cost) ++k.parts;
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
    } else if (ES == 1 && warp == kFetch) {
      // -------------------------------------------------------------- codes
      // Blocks of codes to the ring of raw ones: in whole boxes of existing pages by the TMA, lane i
      // has box i, else row by row with zeros where there is nothing.
      constexpr int kCprRaw = DP / 16;
      Ring<(C::kRaws > 0 ? C::kRaws : 1)> ring;
      uint32_t blocks = 0;
      bool alive = true;
#pragma unroll 1
      for (uint32_t sidx = 0; alive; ++sidx) {
        Seg &s = sh.seg[sidx & 1];
        if (!wait_work(sidx)) break;
        const int nu = s.nu, lo = s.lo, hi = s.hi, first = s.t0;
        const uint32_t *tab_k =
            c.table + ((int64_t)s.slot * c.rows + ((int64_t)a.layer * 2) * c.heads + s.h) * c.blocks;
        const uint32_t *tab_v = tab_k + (int64_t)c.heads * c.blocks;
        arrive(sh.seg_empty[sidx & 1]);
        if (nu < 0) break;
        int blk = 0, off = 0;  // of this lane's box
        const bool has_box = box && lane * box < kN;
        if (has_box) {
          blk = a.by_page.of(first + lane * box);
          off = first + lane * box - blk * c.Tb;
        }
#pragma unroll 1
        for (int u = 0; u < nu && alive; ++u) {
          const int t0 = first + u * kN;
          uint32_t pk = 0, pv = 0;
          bool bulk = box && t0 >= lo && t0 + kN <= hi;
          if (bulk && has_box) {
            pk = tab_k[blk];
            pv = tab_v[blk];
          }
          bulk = __all_sync(~0u, bulk && (!has_box || (pk < c.pages && pv < c.pages)));
#pragma unroll 1
          for (int side = 0; side < 2; ++side) {
            if (!(alive = wait(sh.raw_empty[ring.at], ring.round ^ 1))) break;
            const uint32_t bar = smem_addr(&sh.raw_full[ring.at]);
            const uint32_t dst = sm + C::kOffRaw + ring.at * C::kRaw;
            if (bulk) {
              if (side == 0 && lane < 4) reinterpret_cast<uint32_t *>(&sh.holes[(blocks + u) % kHoles])[lane] = 0;
              if (lane == 0) bar_expect(bar, C::kRaw);
              else bar_arrive(bar);
              __syncwarp();
              if (has_box) copy_box(dst + lane * box * DP, &map, bar, 0, off, 0, side ? pv : pk);
            } else {
#pragma unroll 1
              for (int i = 0; i < kN / 32; ++i) {
                const int t = t0 + i * 32 + lane;
                const bool in = t >= lo && t < hi;
                uint64_t from = ~0ull;
                if (in) {
                  const int b = a.by_page.of(t);
                  const uint32_t qk = tab_k[b], qv = tab_v[b];
                  if (qk < c.pages && qv < c.pages)
                    from = (uint64_t)(side ? qv : qk) * c.page_bytes + (uint32_t)(t - b * c.Tb) * c.row_bytes;
                }
                const uint32_t gone = __ballot_sync(~0u, in && from == ~0ull);
                if (side == 0 && lane == 0) {
                  uint32_t *words = reinterpret_cast<uint32_t *>(&sh.holes[(blocks + u) % kHoles]);
                  if (kN == 128) {
                    words[i] = gone;
                  } else {
                    words[2 * i] = gone & 0xffffu;
                    words[2 * i + 1] = gone >> 16;
                  }
                  if (gone) atomicOr(c.status, kCacheArg);
                  __threadfence_block();
                }
#pragma unroll 4
                for (int y = 0; y < kCprRaw; ++y) {
                  const int row = (y * 32 + lane) / kCprRaw, ch = lane % kCprRaw;
                  const uint64_t b = __shfl_sync(~0u, from, row);
                  const bool on = b != ~0ull && ch * 16 < c.D;
                  cp_async16(dst + (i * 32 + row) * DP + ch * 16, c.pool + (on ? b + ch * 16 : 0), on);
                }
              }
              // this lane's arrival comes when its copies have
              asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
            }
            ring = ring.after();
          }
          if (has_box)
            for (off += kN; off >= c.Tb; off -= c.Tb) ++blk;
        }
        blocks += nu;
      }
      cp_wait<0>();
      if (!alive)
        for (const long long from = clock64(); clock64() - from < 2000000;) {
        }
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == kMma)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// Adds up the parts of the items that lie in several thread blocks, in their order: a warp per
// packed row and map, a lane has neighbouring channels.  blockIdx.x: the thread block that an
// item begins in.  Short code: it runs once, and is fetched while it runs.
constexpr int kJoin = 8;
template <int ES, int DP, bool DIFF>
__global__ void __launch_bounds__(kJoin * 32) k_chunk_join(ChunkArgs a) {
  using C = Cfg<ES, DP, DIFF>;
  constexpr int kVec = DP / 32;
  __shared__ float s_o[DIFF ? kJoin / 2 : 1][DIFF ? DP : 1];
  const CacheView &c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int map = DIFF ? warp & 1 : 0, slot = DIFF ? warp >> 1 : warp;
  constexpr int kRows = DIFF ? kJoin / 2 : kJoin;
  float unit = 1.f;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Cut k = reinterpret_cast<const Cut *>(a.ws)[blockIdx.x];
  const int parts = min(k.parts, (int)gridDim.x - (int)blockIdx.x);
  if (parts <= 0) return;
  const Part<C, DP> *part = reinterpret_cast<const Part<C, DP> *>(a.ws + kCutBytes) + blockIdx.x * 2;
  if (ES == 1 && c.scale) unit = c.scale[a.layer * c.heads + k.h];
#pragma unroll 1
  for (int rr = blockIdx.y * kRows + slot; rr < C::kItem; rr += gridDim.y * kRows) {
    const int p = k.p0 + rr;
    const bool on = p < k.p1;
    if (!DIFF && !on) break;
    const int j = a.by_group.of(p), head = k.h * (a.q_heads / c.heads) + p - j * (a.q_heads / c.heads);
    const int64_t oh = ((int64_t)k.q0 + j) * a.q_heads + head;
    const int row = !DIFF ? rr : C::kTiles == 2 ? map * 128 + rr : (rr >> 4) * 32 + map * 16 + (rr & 15);
    float M = -INFINITY, L = 0.f, o[kVec];
#pragma unroll
    for (int v = 0; v < kVec; ++v) o[v] = 0.f;
    if (on) {
      // the parts' maxima: the first 32 a lane each
      float m1 = -INFINITY, l1 = 0.f;
      if (lane < parts) {
        m1 = part[2 * lane + (lane == 0)].m[row];
        l1 = part[2 * lane + (lane == 0)].l[row];
      }
      M = m1;
#pragma unroll 1
      for (int i = lane + 32; i < parts; i += 32) M = fmaxf(M, part[2 * i].m[row]);
#pragma unroll 1
      for (int s = 16; s; s >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, s));
      const float m0 = M == -INFINITY ? 0.f : M;
#pragma unroll 4
      for (int i = 0; i < parts; ++i) {
        const Part<C, DP> &x = part[2 * i + (i == 0)];
        const float w = ex2((i < 32 ? __shfl_sync(~0u, m1, i & 31) : x.m[row]) - m0);
        L += w * (i < 32 ? __shfl_sync(~0u, l1, i & 31) : x.l[row]);
#pragma unroll
        for (int v = 0; v < kVec; v += 2) {
          const float2 y = *reinterpret_cast<const float2 *>(&x.o[row][lane * kVec + v]);
          o[v] += w * y.x;
          o[v + 1] += w * y.y;
        }
      }
      if (lane == 0 && a.lse) a.lse[oh * (DIFF ? 2 : 1) + map] = (m0 + log2f(L)) * kLn2;
    }
    float by = L == 0.f ? 0.f : unit / L;
    if (DIFF) {
      // the second map's warp hands its result to the first's
      if (on && map && L != 0.f) by *= a.lambda[head];
      if (map)
#pragma unroll
        for (int v = 0; v < kVec; ++v) s_o[slot][lane * kVec + v] = o[v] * by;
      __syncthreads();
      if (!map) {
        float q = 0.f;
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
          o[v] = o[v] * by - s_o[slot][lane * kVec + v];
          if (lane * kVec + v < c.D) q = fmaf(o[v], o[v], q);
        }
        by = 1.f;
        if (a.norm) {
#pragma unroll 1
          for (int s = 16; s; s >>= 1) q += __shfl_xor_sync(~0u, q, s);
          by = rsqrtf(q / c.D + a.eps);
          if (!Squares::enough(q, a.eps)) {  // the whole warp
            Squares all;
#pragma unroll
            for (int v = 0; v < kVec; ++v)
              if (lane * kVec + v < c.D) all.add(o[v]);
            all.add_lanes();
            by = all.inverse(c.D, a.eps);
          }
        }
      }
      __syncthreads();
    }
    if (on && !map)
#pragma unroll
      for (int v = 0; v < kVec; v += 2) {
        const int d = lane * kVec + v;
        if (d < c.D) {
          float f0 = by, f1 = by;
          if (DIFF && a.norm) {
            f0 *= a.norm[d];
            f1 *= a.norm[d + 1];
          }
          *reinterpret_cast<uint32_t *>(a.out + oh * c.D + d) = pack2<2>(o[v] * f0, o[v + 1] * f1);
        }
      }
  }
}

// Boxes of `rows` tokens of the pool's pages; false where the driver refuses them.  bf16: the
// channels in blocks of 64, one or all of them in a box; where they do not end with a block, and
// for codes, one block, filled up with zeros.
using Encode = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                            const cuuint64_t *, const cuuint32_t *, const cuuint32_t *,
                            CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                            CUtensorMapFloatOOBfill);
bool map_pages(CUtensorMap *map, const CacheView &c, int channels, int rows, int most) {
  static std::atomic<void *> known{nullptr};
  void *fn = known.load(std::memory_order_relaxed);
  if (!fn) {
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) !=
            cudaSuccess ||
        found != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      return false;
    }
    known.store(fn, std::memory_order_relaxed);
  }
  const bool codes = c.dtype == 1;
  const bool blocked = !codes && c.D % 64 == 0;
  const cuuint32_t blocks = blocked ? c.D / 64 : 1;
  const cuuint64_t dims[4] = {(cuuint64_t)(blocked ? 64 : c.D), (cuuint64_t)c.Tb, blocks, c.pages};
  const cuuint64_t strides[3] = {c.row_bytes, blocked ? 128u : c.row_bytes, c.page_bytes};
  const cuuint32_t sizes[4] = {(cuuint32_t)channels, (cuuint32_t)rows, rows == most ? blocks : 1, 1},
                   steps[4] = {1, 1, 1, 1};
  return reinterpret_cast<Encode>(fn)(
             map, codes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, c.pool, dims,
             strides, sizes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
             codes ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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
cudaError_t run(ChunkArgs a, cudaStream_t st) {
  using C = Cfg<ES, DP, DIFF>;
  a.by_group = Div(a.q_heads / a.c.heads);
  a.by_page = Div(a.c.Tb);
  a.patience = kPatience + a.batch * kPerSequence + a.max_len / C::kN * kPerBlock;
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
  // boxes of the largest power of two of tokens that pages are made of, 8 (a swizzle's) at least
  CUtensorMap map = {};
  int box = a.c.Tb & -a.c.Tb;
  if (box > C::kN) box = C::kN;
  if (box < 8 || a.c.pages > 0x7fffffff || !map_pages(&map, a.c, ES == 2 ? 64 : DP, box, C::kN)) box = 0;
  e = launch(kern, dim3((unsigned)grid), C::kThreads, smem, st, a, cut, box, map);
  if (e != cudaSuccess || !cut) return e;
  constexpr int kRows = DIFF ? kJoin / 2 : kJoin;
  return launch(k_chunk_join<ES, DP, DIFF>, dim3((unsigned)grid, (unsigned)(C::kItem / kRows)), kJoin * 32,
                0, st, a);
}

template <int ES, bool DIFF>
cudaError_t run_d(const ChunkArgs &a, cudaStream_t st) {
  if (a.c.D <= 64) return run<ES, 64, DIFF>(a, st);
  if (a.c.D <= 128) return run<ES, 128, DIFF>(a, st);
  return run<ES, 256, DIFF>(a, st);
}

}  // namespace

size_t chunk_ws_bytes(const CacheView &c, int32_t q_heads) {
  const int sms = sm_count();
  if (!sms) return 0;
  const size_t rows = c.D <= 128 ? 256 : 128, DP = c.D <= 64 ? 64 : c.D <= 128 ? 128 : 256;
  const size_t chunk = kCutBytes + (size_t)sms * 2 * rows * (DP + 2) * sizeof(float);
  const size_t one = attend_diff_ws_bytes(c, q_heads);
  return chunk > one ? chunk : one;
}

cudaError_t launch_chunk(const ChunkArgs &a, cudaStream_t st) {
  if (!a.lambda) return a.c.dtype == 1 ? run_d<1, false>(a, st) : run_d<2, false>(a, st);
  if (a.starts) return a.c.dtype == 1 ? run_d<1, true>(a, st) : run_d<2, true>(a, st);
  // one new token per sequence: nearly all of a tile's rows would be empty
  AttendArgs b;
  b.c = a.c;
  b.slots = a.slots;
  b.lens = a.lens;
  b.begins = a.begins;
  b.q = a.q;
  b.qs = a.qs;
  b.qhs = a.qhs;
  b.out = a.out;
  b.lse = a.lse;
  b.ws = a.ws;
  b.scale = a.scale;
  b.batch = a.batch;
  b.q_heads = a.q_heads;
  b.layer = a.layer;
  b.max_len = a.max_len;
  b.window = a.window;
  b.lambda = a.lambda;
  b.norm = a.norm;
  b.eps = a.eps;
  return launch_attend_diff(b, st);
}

}  // namespace skv
