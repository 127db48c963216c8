// skv_cache_attend.cuh -- attention of one new token per sequence over a paged KV cache, plain
// (instantiated in skv_cache_attend.cu) and differential (skv_cache_attend_diff.cu).
//
// o_h = sum_t p_t v_t / sum_t p_t with p_t = 2^(x_t - m), x_t = log2(e) * scale *
// q_h.k_t, m at a distance from the running maximum (softmax in one pass: when m grows
// to m', the sums so far are multiplied by 2^(m - m')).  Every key and value byte is used
// for 2 * group (bf16) or 4 * group (e4m3) operations, far below what the matrix
// units need per byte of HBM, so HBM bounds the call and the design is about
// keeping loads in flight:
//   - the work is cut into units of 4 warp tiles of one (sequence, kv head) row
//     and dealt evenly to one wave of persistent blocks, whatever the lengths;
//     a block may take parts of several rows, a row may lie in several blocks;
//   - a warp loads its own tiles (cp.async into its own ring of stages, rows
//     outside the range filled with zeros) and computes on them without any
//     block-wide barrier; the block's 4 warps are joined once per row;
//   - a row that lies in several blocks leaves a partial result in each (at most
//     two per block) and is joined by k_attend_join or, where few rows lie in many
//     blocks, k_attend_join_wide, in a fixed order;
//   - a batch of short rows is not cut: one block per row and no join.
// The products run on the matrix units transposed, tokens as rows and the group's
// query heads as the 8 columns of m16n8k16: S^T = K Q^T, O^T = V^T P^T, so a
// group of up to 8 heads wastes no row and the running maximum, the sum and O^T
// share one column layout (no exchange to rescale).  P goes from the accumulator
// to the operand layout by movmatrix.  e4m3 codes become fp16 (exact); q becomes
// fp16 after a power-of-two scale per head: the largest channel lies in [1, 2), so
// channels down to 2^-17 of it are exact and smaller ones are off by 2^-25 of it at most.
// Differential attention (DIFF) is the same with two columns per query head, one per map: a
// map's query has zeros in the other map's half of the channels, which costs the matrix units,
// far from busy, and no byte of the cache.  The first half of the columns is the first map.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "skv_cache.cuh"

namespace skv {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
// A row costs a block this many units more than it has: the stages run empty and the warps
// are joined between two rows.
constexpr int kRowCost = 2;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int ES, int DP, int NT>
struct Cfg {
  static constexpr int kRowB = DP * ES;              // bytes of a token's row in shared memory
  static constexpr int kCpr = kRowB / 16;            // 16-byte chunks of it
  static constexpr int kTok = kRowB <= 128 ? 32 : 16;  // tokens of a warp tile
  static constexpr int kTile = kTok * kRowB;         // bytes of a tile of K or V
  // 2 stages leave room for 3 blocks (12 warps) per SM, which hide one another's latency:
  // 107 us against 111 with 3 stages and 2 blocks for 32 rows of up to 16384 e4m3 tokens
  // (64 channels of e4m3, half as many bytes: 59.7 with 2, 61.8 with 3, 62.7 with 4; 25.9, 26.8
  // and 31.1 for 256 rows of up to 512).  256 channels: bf16 leaves one block of 4 warps per
  // SM either way, and 3 stages are better (197 us against 204 for 32 rows of up to 8192);
  // e4m3 has the room that the join of 16 heads takes (67 KB), though 2 would do for 8
  // heads (107 us against 110).
  static constexpr int kStages = DP == 256 ? 3 : 2;
  static constexpr int kUnit = kWarps * kTok;        // tokens of a unit
  static constexpr int kSmem = kWarps * kStages * 2 * kTile;
  static constexpr int kPerSm = 220 * 1024 / (kSmem + 1024) < 4 ? 220 * 1024 / (kSmem + 1024) : 4;
  static constexpr int kHeads = 8 * NT;
  // m is set kLift below the running maximum when x - m passes kMost, so p <= 2^kMost.  For
  // e4m3 p meets the values as fp16, which ends at 2^16 above, holds 11 bits down to 2^-14
  // and nothing below 2^-25: with the largest weight at 2^11 to 2^15, weights keep 11 bits
  // down to 2^-25 of it and the others are off by 2^-36 of it at most (105 us for 32 rows of
  // up to 16384 tokens and 39.2 for 256 of up to 512, as without).  bf16 has a float's
  // exponent.
  static constexpr float kLift = ES == 1 ? 11.f : 0.f, kMost = ES == 1 ? 15.f : 8.f;
  // floats of a head's row where the warps are joined: the 4 padding floats put what a
  // warp stores at once (8 channels of 4 heads) in different banks
  static constexpr int kPad = DP + 4;
  static_assert(kWarps * kHeads * (kPad + 2) * 4 <= kSmem, "the join of the warps reuses the stages");
};

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
template <bool TRANS>
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  if (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
template <int ES>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  if (ES == 2)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
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

// the upper halves of two floats, and what cutting p to its upper half leaves
__device__ __forceinline__ uint32_t high2(float a, float b) {
  return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
__device__ __forceinline__ float rest(float p) {
  return fmaf(p, 1.f + 0x1p-18f, -__uint_as_float(__float_as_uint(p) & 0xffff0000u));
}

// byte offset of 16-byte chunk c of row r in a tile: chunks are permuted so that
// the 8 rows one ldmatrix reads lie in 8 different bank groups
template <int CPR>
__device__ __forceinline__ uint32_t swz(int r, int c) {
  if (CPR >= 8) return (uint32_t)(r * CPR + ((c & ~7) | ((c ^ r) & 7))) * 16;
  return (uint32_t)(r * CPR + (c ^ ((r >> 1) & 3))) * 16;
}

// The tokens [begin, end) of batch entry b, its first tile's start and its units.
struct Span {
  int32_t slot, begin, end, start;
  int32_t units, cost;  // cost: units as they are dealt (see kRowCost)
};
__device__ __forceinline__ Span span_of(const AttendArgs &a, int b, int tok, int unit, bool tell) {
  Span s;
  s.slot = a.slots[b];
  const int32_t len = a.lens[b];
  s.begin = a.begins ? max(a.begins[b], 0) : 0;
  if (a.window) s.begin = max(s.begin, len - a.window);
  s.end = len;
  bool bad = len < 0 || len > a.max_len || (int64_t)len > (int64_t)a.c.blocks * a.c.Tb ||
             s.slot >= a.c.seqs;
  if (s.slot < 0) bad = false;  // padding
  if (bad && tell) atomicOr(a.c.status, kCacheArg);
  if (bad || s.slot < 0 || s.begin >= s.end) s.begin = s.end = 0;
  s.start = s.begin / tok * tok;
  s.units = (s.end - s.start + unit - 1) / unit;
  s.cost = s.units ? s.units + kRowCost : 0;
  return s;
}

// All units W of the batch (below 2^31, checked by the host); each lane owns `per`
// neighbouring entries with `mine` units, `before` of all lie before them; `below` lie
// before entry `upto`.  One warp, no block barrier: every warp of a block does the same.
struct Sums {
  uint32_t W, before, mine, below;
  int per;
};
template <typename C>
__device__ __forceinline__ Sums sums_of(const AttendArgs &a, int HV, int upto, bool tell) {
  const int lane = threadIdx.x & 31;
  Sums r;
  r.per = (a.batch + 31) / 32;
  uint32_t mine = 0, below = 0;
  const int lo = lane * r.per, hi = min(lo + r.per, a.batch);
#pragma unroll 4
  for (int b = lo; b < hi; ++b) {
    const uint32_t u = (uint32_t)span_of(a, b, C::kTok, C::kUnit, tell).cost * HV;
    mine += u;
    if (b < upto) below += u;
  }
  uint32_t x = mine;
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(~0u, x, o);
    if (lane >= o) x += y;
  }
  r.W = __shfl_sync(~0u, x, 31);
  r.mine = mine;
  r.before = x - mine;
  r.below = __reduce_add_sync(~0u, below);
  return r;
}

// How the units are dealt: block i of n takes [deal(i), deal(i + 1)), deal(i) =
// floor(i * W / n) = i * (W / n) + floor(i * (W % n) / n); n is at most a wave of blocks.
__device__ __forceinline__ uint32_t blocks_used(uint32_t W, uint32_t grid) {
  return max(1u, min(W / 2, grid));  // at least two units each
}
__device__ __forceinline__ uint32_t deal(uint32_t W, uint32_t n, uint32_t i) {
  const uint32_t q = W / n;
  return i * q + i * (W - q * n) / n;
}
// the block that unit u lies in: the largest i with i * W / n <= u
__device__ __forceinline__ int block_of(uint32_t W, uint32_t n, uint32_t u) {
  return (int)((((uint64_t)u + 1) * n - 1) / W);
}

// Partial results: per block two slots of kHeads x (DP sums, maximum, sum of weights).
template <int DP, int NT>
struct Part {
  float o[8 * NT][DP];
  float m[8 * NT], l[8 * NT];
};

// Zeros and -infinity for heads h0 .. h0 + nh - 1 of an entry without tokens.
template <bool DIFF>
__device__ __forceinline__ void write_empty(const AttendArgs &a, int b, int h0, int nh,
                                            int threads) {
  constexpr int kMaps = DIFF ? 2 : 1;
  const int64_t oh = (int64_t)b * a.q_heads + h0;
  for (int x = threadIdx.x; x < nh * a.c.D; x += threads) a.out[oh * a.c.D + x] = 0;
  for (int x = threadIdx.x; a.lse && x < nh * kMaps; x += threads) a.lse[oh * kMaps + x] = -INFINITY;
}

// ROWS: block i takes row i whole (entry i / HV); otherwise the units are dealt.
template <int ES, int DP, int NT, bool ROWS, bool DIFF>
__global__ void __launch_bounds__(kThreads, (Cfg<ES, DP, NT>::kPerSm)) k_attend(AttendArgs a,
                                                                              int head_tiles) {
  using C = Cfg<ES, DP, NT>;
  constexpr int kTileHeads = DIFF ? C::kHeads / 2 : C::kHeads;  // query heads of a row
  extern __shared__ __align__(128) uint8_t smem[];
  // In this order: k_attend_join reads the lengths before it waits, and it is launched once
  // every block here has seen the end of the work that wrote them.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const CacheView &c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int j = lane & 3, g8 = lane >> 2;
  const int HV = c.heads * head_tiles;  // rows per batch entry
  const int group = a.q_heads / c.heads;

  uint32_t pos, stop, before = 0;
  int b;
  if (ROWS) {
    b = blockIdx.x / HV;
    const int row = blockIdx.x - b * HV;
    const Span sp = span_of(a, b, C::kTok, C::kUnit, warp == 0 && row == 0);
    pos = row * sp.cost;
    stop = pos + sp.cost;
    if (!sp.units) {
      const int h = row / head_tiles, h0 = h * group + (row - h * head_tiles) * kTileHeads;
      write_empty<DIFF>(a, b, h0, min(kTileHeads, h * group + group - h0), kThreads);
      return;
    }
  } else {
    // this block's share of the units
    const Sums all = sums_of<C>(a, HV, 0, blockIdx.x == 0 && warp == 0);
    const uint32_t nblk = blocks_used(all.W, gridDim.x);
    if (blockIdx.x >= nblk) return;
    pos = deal(all.W, nblk, blockIdx.x);
    stop = deal(all.W, nblk, blockIdx.x + 1);
    if (pos >= stop) return;
    // the batch entry b that unit `pos` lies in, and the units before that entry
    const int owner = __ffs(__ballot_sync(~0u, pos < all.before + all.mine)) - 1;
    before = __shfl_sync(~0u, all.before, owner);
    b = owner * all.per;
    for (int b0 = b; all.per > 1 && b0 < a.batch; b0 += 32) {
      const int bb = b0 + lane;
      const uint32_t u =
          bb < a.batch ? (uint32_t)span_of(a, bb, C::kTok, C::kUnit, false).cost * HV : 0;
      uint32_t x = u;
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(~0u, x, o);
        if (lane >= o) x += y;
      }
      const uint32_t hit = __ballot_sync(~0u, pos < before + x);
      if (hit) {
        const int i = __ffs(hit) - 1;
        b = b0 + i;
        before += __shfl_sync(~0u, x - u, i);
        break;
      }
      before += __shfl_sync(~0u, x, 31);
    }
  }

  const uint32_t tile0 = smem_addr(smem) + warp * (C::kStages * 2 * C::kTile);
  const bool whole = c.Tb % C::kTok == 0;  // a tile lies in one page
  const bool plain = whole && c.row_bytes == C::kRowB;  // and is one run of bytes

  // (the bound on b: lengths that are overwritten meanwhile must not lead out of the arrays)
  while (pos < stop && b < a.batch) {
    Span sp = span_of(a, b, C::kTok, C::kUnit, false);
    if (pos >= before + (uint32_t)sp.cost * HV) {
      before += (uint32_t)sp.cost * HV;
      ++b;
      continue;
    }
    const int row = (pos - before) / (uint32_t)sp.cost;
    const int c0 = pos - before - (uint32_t)row * sp.cost;
    const int c1 = min((uint32_t)sp.cost, c0 + (stop - pos));
    pos += c1 - c0;
    const int u0 = max(c0 - kRowCost, 0), nu = c1 - kRowCost - u0;
    if (nu <= 0) continue;  // only the row's beginning
    const int h = row / head_tiles, h0 = h * group + (row - h * head_tiles) * kTileHeads;
    const int nh = min(kTileHeads, h * group + group - h0);  // query heads of this row
    const uint32_t *tab_k =
        c.table + ((int64_t)sp.slot * c.rows + ((int64_t)a.layer * 2) * c.heads + h) * c.blocks;
    const uint32_t *tab_v = tab_k + (int64_t)c.heads * c.blocks;

    // set when a token in the range has no page: its rows are zeros and it is masked
    bool holes = false;

    // block and token in it of this warp's next tile to load (tiles that lie in one page)
    int ld_t = sp.start + (u0 * kWarps + warp) * C::kTok;
    int ld_blk = ld_t / c.Tb, ld_off = ld_t - ld_blk * c.Tb;

    auto advance = [&]() {
      ld_t += C::kUnit;
      ld_off += C::kUnit;
      while (ld_off >= c.Tb) {
        ld_off -= c.Tb;
        ++ld_blk;
      }
    };
    auto load = [&](int u, int stage) {
      const int t0 = ld_t;
      if (u < nu && t0 < sp.end) {
        const uint32_t sk = tile0 + stage * 2 * C::kTile, sv = sk + C::kTile;
        // byte offsets in the pool of row 0 (the tile lies in one page) or of row lane % kTok
        int blk = ld_blk, tin = ld_off;
        if (!whole) {
          // (only pages of the range are looked up: there may be none outside)
          const int t = min(max(t0 + lane % C::kTok, sp.begin), sp.end - 1);
          blk = t / c.Tb;
          tin = t - blk * c.Tb;
        }
        const uint32_t pk = tab_k[blk], pv = tab_v[blk];
        const uint32_t off = (uint32_t)tin * c.row_bytes;
        const bool has = pk < c.pages && pv < c.pages;
        if (__any_sync(~0u, !has)) {
          holes = true;
          if (lane == 0) atomicOr(c.status, kCacheArg);
        }
        const uint64_t bk = has ? (uint64_t)pk * c.page_bytes + off : 0;
        const uint64_t bv = has ? (uint64_t)pv * c.page_bytes + off : 0;
        if (plain && has && t0 >= sp.begin && t0 + C::kTok <= sp.end) {
          // the tile is one run of bytes and all of it counts: only constants are added
          const uint8_t *gk = c.pool + bk + lane * 16, *gv = c.pool + bv + lane * 16;
#pragma unroll
          for (int i = 0; i < C::kTok * C::kCpr / 32; ++i) {
            constexpr int kRows = 32 / C::kCpr > 0 ? 32 / C::kCpr : 1;  // rows an instruction covers
            const uint32_t d = swz<C::kCpr>((i * kRows) % 8 + lane / C::kCpr, lane % C::kCpr) +
                               (i * kRows) / 8 * 8 * C::kRowB;
            cp_async16(sk + d, gk + i * 512);
            cp_async16(sv + d, gv + i * 512);
          }
          cp_commit();
          advance();
          return;
        }
#pragma unroll
        for (int i = 0; i < C::kTok * C::kCpr / 32; ++i) {
          const int id = i * 32 + lane, r = id / C::kCpr, ch = id % C::kCpr;
          const bool in = t0 + r >= sp.begin && t0 + r < sp.end && ch * 16 < (int)c.row_bytes;
          uint64_t rk, rv;
          bool ok;
          if (whole) {
            rk = bk + (uint32_t)r * c.row_bytes;
            rv = bv + (uint32_t)r * c.row_bytes;
            ok = has;
          } else {
            rk = __shfl_sync(~0u, bk, r);
            rv = __shfl_sync(~0u, bv, r);
            ok = __shfl_sync(~0u, (int)has, r);
          }
          const bool on = in && ok;
          cp_async16(sk + swz<C::kCpr>(r, ch), c.pool + (on ? rk + ch * 16 : 0), on);
          cp_async16(sv + swz<C::kCpr>(r, ch), c.pool + (on ? rv + ch * 16 : 0), on);
        }
      }
      cp_commit();
      if (whole) advance();
      else ld_t += C::kUnit;
    };

#pragma unroll
    for (int s = 0; s < C::kStages - 1; ++s) load(s, s);

    // q as the B operand: column n = head g8 (+ 8), rows k = channels.  e4m3 tiles
    // give lane j channels 4j..4j+3 of each 16, so q takes the same order.
    uint32_t qf[NT][DP / 16][2];
    float f[NT][2];  // x = f * (product), of heads 2j and 2j + 1
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int hq = DIFF ? (n * 8 + g8) % kTileHeads : n * 8 + g8;
      const uint16_t *qp = a.q + (int64_t)b * a.qs + (int64_t)(h0 + hq) * a.qhs;
      const bool on = hq < nh;
      // the channels of this column's query (DIFF: the halves end at a multiple of 8)
      const int d0 = DIFF && n * 8 + g8 >= kTileHeads ? c.D / 2 : 0;
      const int d1 = DIFF && n * 8 + g8 < kTileHeads ? c.D / 2 : c.D;
      float e = 1.f;
      if (ES == 2) {
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
          const int d = k * 16 + 2 * j;
          qf[n][k][0] = on && d >= d0 && d < d1 ? *reinterpret_cast<const uint32_t *>(qp + d) : 0;
          qf[n][k][1] = on && d + 8 >= d0 && d + 8 < d1 ? *reinterpret_cast<const uint32_t *>(qp + d + 8) : 0;
        }
      } else {
        float mx = 0.f;
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
          const int d = k * 16 + 4 * j;
          uint2 v = make_uint2(0, 0);
          if (on && d >= d0 && d < d1) v = *reinterpret_cast<const uint2 *>(qp + d);
          qf[n][k][0] = v.x;
          qf[n][k][1] = v.y;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t w = qf[n][k][i];
            mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(w << 16)),
                                 fabsf(__uint_as_float(w & 0xffff0000u))));
          }
        }
        mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 2));
        // the largest channel to [1, 2): e = 2^exponent, kept where 1/e is normal
        const uint32_t ex = __float_as_uint(mx) >> 23;
        if (ex >= 1 && ex < 253) e = __uint_as_float(ex << 23);
        const float r = 1.f / e;
#pragma unroll
        for (int k = 0; k < DP / 16; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t w = qf[n][k][i];
            qf[n][k][i] = pack2<1>(__uint_as_float(w << 16) * r,
                                   __uint_as_float(w & 0xffff0000u) * r);
          }
      }
      float s = a.scale * kLog2e;
      if (ES == 1 && c.scale) s *= c.scale[a.layer * c.heads + h];
      f[n][0] = s * __shfl_sync(~0u, e, 8 * j);      // head 2j: any lane of group 2j
      f[n][1] = s * __shfl_sync(~0u, e, 8 * j + 4);
    }

    float o[DP / 16][NT][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int d = 0; d < DP / 16; ++d)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[d][n][i] = 0.f;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
    }

    int stage = 0;
    for (int u = 0; u < nu; ++u) {
      cp_wait<C::kStages - 2>();
      __syncwarp();
      {
        int s = stage + C::kStages - 1;
        if (s >= C::kStages) s -= C::kStages;
        load(u + C::kStages - 1, s);
      }
      const int t0 = sp.start + ((u0 + u) * kWarps + warp) * C::kTok;
      const uint32_t sk = tile0 + stage * 2 * C::kTile, sv = sk + C::kTile;
      if (++stage == C::kStages) stage = 0;
      if (t0 >= sp.end) continue;  // the whole warp

      // S^T = K Q^T
      float x[C::kTok / 16][NT][4];
#pragma unroll
      for (int mt = 0; mt < C::kTok / 16; ++mt) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) x[mt][n][i] = 0.f;
        const int r = mt * 16 + (lane & 15);
        if (ES == 2) {
#pragma unroll
          for (int k = 0; k < DP / 16; ++k) {
            uint32_t t[4];
            ldsm4<false>(t, sk + swz<C::kCpr>(r, 2 * k + (lane >> 4)));
#pragma unroll
            for (int n = 0; n < NT; ++n)
              mma<ES>(x[mt][n], t[0], t[1], t[2], t[3], qf[n][k][0], qf[n][k][1]);
          }
        } else {
#pragma unroll
          for (int k = 0; k < DP / 16; k += 2) {
            uint32_t t[4];
            ldsm4<false>(t, sk + swz<C::kCpr>(r, k + (lane >> 4)));
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
              uint32_t a0, a1, a2, a3;
              e4m3x4(t[2 * kk], a0, a2);
              e4m3x4(t[2 * kk + 1], a1, a3);
#pragma unroll
              for (int n = 0; n < NT; ++n)
                mma<ES>(x[mt][n], a0, a1, a2, a3, qf[n][k + kk][0], qf[n][k + kk][1]);
            }
          }
        }
      }
      if (DIFF) {
        // The zeros of a column's query meet the other half's keys, and 0 * infinity is NaN: scores that
        // are NaN are made again of the column's own half.  (Their sum tells, one addition each.)
        float all = 0.f;
#pragma unroll
        for (int mt = 0; mt < C::kTok / 16; ++mt)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) all += x[mt][n][i];
        if (__any_sync(~0u, all != all)) {
          uint32_t todo = 0;
#pragma unroll
          for (int mt = 0; mt < C::kTok / 16; ++mt)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                todo |= (uint32_t)(x[mt][n][i] != x[mt][n][i]) << ((mt * NT + n) * 4 + i);
#pragma unroll 1
          for (; todo; todo &= todo - 1) {
            const int at = __ffs(todo) - 1, n = at / 4 % NT;
            const int t = t0 + at / (4 * NT) * 16 + g8 + (at & 2) * 4, col = n * 8 + 2 * j + (at & 1);
            const int map = col >= kTileHeads, hq = col - map * kTileHeads;
            if (hq >= nh || t < sp.begin || t >= sp.end) continue;
            const uint32_t pk = tab_k[t / c.Tb];
            if (pk >= c.pages) continue;
            // (x is of q over a power of two: f has it)
            float s = a.scale * kLog2e;
            if (ES == 1 && c.scale) s *= c.scale[a.layer * c.heads + h];
            const float fc = at & 1 ? (NT == 2 && n ? f[NT - 1][1] : f[0][1])
                                    : (NT == 2 && n ? f[NT - 1][0] : f[0][0]);
            const float y = half_score<ES>(
                a.q + (int64_t)b * a.qs + (int64_t)(h0 + hq) * a.qhs + map * (c.D / 2),
                c.pool + (uint64_t)pk * c.page_bytes + (uint32_t)(t % c.Tb) * c.row_bytes + map * (c.row_bytes / 2),
                c.D / 2) * (ES == 1 && fc != 0.f ? s / fc : 1.f);
#pragma unroll
            for (int mt = 0; mt < C::kTok / 16; ++mt)
#pragma unroll
              for (int m = 0; m < NT; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if ((mt * NT + m) * 4 + i == at) x[mt][m][i] = y;
          }
          __syncwarp();
        }
      }
      // scale, mask, running maximum
      const bool edge = holes || t0 < sp.begin || t0 + C::kTok > sp.end;
      bool grow = false;
      float top[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        top[n][0] = top[n][1] = -INFINITY;
#pragma unroll
        for (int mt = 0; mt < C::kTok / 16; ++mt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float v = x[mt][n][i] * f[n][i & 1];
            if (edge) {
              const int t = t0 + mt * 16 + g8 + (i >> 1) * 8;
              if (t < sp.begin || t >= sp.end) v = -INFINITY;
              else if (holes && (tab_k[t / c.Tb] >= c.pages || tab_v[t / c.Tb] >= c.pages))
                v = -INFINITY;
            }
            x[mt][n][i] = v;
            top[n][i & 1] = fmaxf(top[n][i & 1], v);
          }
        // (the difference that the weights are made of: no rounding can pass kMost)
        grow = grow || top[n][0] - m[n][0] > C::kMost || top[n][1] - m[n][1] > C::kMost;
      }
      if (__any_sync(~0u, grow)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float t = top[n][i];
            t = fmaxf(t, __shfl_xor_sync(~0u, t, 4));
            t = fmaxf(t, __shfl_xor_sync(~0u, t, 8));
            t = fmaxf(t, __shfl_xor_sync(~0u, t, 16));
            // (beyond 2^23 a float has no room for kLift)
            const float mn = fmaxf(m[n][i], fabsf(t) < 0x1p23f ? t - C::kLift : t);
            const float s = mn == -INFINITY ? 1.f : ex2(m[n][i] - mn);
            m[n][i] = mn;
            l[n][i] *= s;
#pragma unroll
            for (int d = 0; d < DP / 16; ++d) {
              o[d][n][i] *= s;
              o[d][n][i + 2] *= s;
            }
          }
      }
      // P, its sum, and P as the B operand.  bf16 holds 8 bits of a weight, so a weight is
      // cut to bf16 and what that leaves goes in a second bf16 operand (2^-16 in all; 57.3
      // us with it and 57.2 without for 16 x 8192 tokens); fp16 holds 11 bits.  The rest
      // is kept above 0 (p * 2^-18 more), so that no weight above 0 meets an infinite
      // value as 0 times it.
      uint32_t pf[C::kTok / 16][NT][2], pl[C::kTok / 16][NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float m0 = m[n][0] == -INFINITY ? 0.f : m[n][0];
        const float m1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
#pragma unroll
        for (int mt = 0; mt < C::kTok / 16; ++mt) {
          const float p0 = ex2(x[mt][n][0] - m0), p1 = ex2(x[mt][n][1] - m1);
          const float p2 = ex2(x[mt][n][2] - m0), p3 = ex2(x[mt][n][3] - m1);
          l[n][0] += p0 + p2;
          l[n][1] += p1 + p3;
          if (ES == 2) {
            pf[mt][n][0] = transpose8x8(high2(p0, p1));
            pf[mt][n][1] = transpose8x8(high2(p2, p3));
            pl[mt][n][0] = transpose8x8(pack2<ES>(rest(p0), rest(p1)));
            pl[mt][n][1] = transpose8x8(pack2<ES>(rest(p2), rest(p3)));
          } else {
            pf[mt][n][0] = transpose8x8(pack2<ES>(p0, p1));
            pf[mt][n][1] = transpose8x8(pack2<ES>(p2, p3));
          }
        }
      }
      // O^T += V^T P^T
#pragma unroll
      for (int mt = 0; mt < C::kTok / 16; ++mt) {
        if (ES == 2) {
          const int r = mt * 16 + (lane & 7) + (lane >> 4) * 8;
#pragma unroll
          for (int d = 0; d < DP / 16; ++d) {
            uint32_t t[4];
            ldsm4<true>(t, sv + swz<C::kCpr>(r, 2 * d + ((lane >> 3) & 1)));
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma<ES>(o[d][n], t[0], t[1], t[2], t[3], pf[mt][n][0], pf[mt][n][1]);
              mma<ES>(o[d][n], t[0], t[1], t[2], t[3], pl[mt][n][0], pl[mt][n][1]);
            }
          }
        } else {
          const int r = mt * 16 + (lane & 15);
#pragma unroll
          for (int d = 0; d < DP / 16; d += 2) {
            uint32_t t[4];
            ldsm4<true>(t, sv + swz<C::kCpr>(r, d + (lane >> 4)));
#pragma unroll
            for (int dd = 0; dd < 2; ++dd) {
              // bytes: token 2j channels (2r, 2r+1), token 2j+1 the same
              uint32_t a0, a1, a2, a3;
              e4m3x4(__byte_perm(t[2 * dd], 0, 0x3120), a0, a1);
              e4m3x4(__byte_perm(t[2 * dd + 1], 0, 0x3120), a2, a3);
#pragma unroll
              for (int n = 0; n < NT; ++n)
                mma<ES>(o[d + dd][n], a0, a1, a2, a3, pf[mt][n][0], pf[mt][n][1]);
            }
          }
        }
      }
    }
    cp_wait<0>();

    // join the warps in the stages' memory, then write the row or a partial result
    float *so = reinterpret_cast<float *>(smem);
    float *sm = so + kWarps * C::kHeads * C::kPad, *sl = sm + kWarps * C::kHeads;
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float s = l[n][i];
        s += __shfl_xor_sync(~0u, s, 4);
        s += __shfl_xor_sync(~0u, s, 8);
        s += __shfl_xor_sync(~0u, s, 16);
        const int hh = n * 8 + 2 * j + i;
        if (g8 == 0) {
          sm[warp * C::kHeads + hh] = m[n][i];
          sl[warp * C::kHeads + hh] = s;
        }
#pragma unroll
        for (int d = 0; d < DP / 16; ++d) {
          const int d0 = ES == 2 ? d * 16 + g8 : d * 16 + 2 * g8;
          const int d1 = ES == 2 ? d0 + 8 : d0 + 1;
          so[(warp * C::kHeads + hh) * C::kPad + d0] = o[d][n][i];
          so[(warp * C::kHeads + hh) * C::kPad + d1] = o[d][n][i + 2];
        }
      }
    __syncthreads();
    constexpr int kMaps = DIFF ? 2 : 1;
    const bool done = ROWS || (u0 == 0 && nu == sp.units);
    Part<DP, NT> *part = reinterpret_cast<Part<DP, NT> *>(a.ws) + ((int64_t)blockIdx.x * 2 + (u0 == 0));
    float osc = 1.f;
    if (ES == 1 && c.scale) osc = c.scale[a.layer * c.heads + h];
    for (int x = threadIdx.x; x < nh * kMaps * (DP / 4); x += kThreads) {
      // (DIFF: column hq % kTileHeads of either half)
      const int hc = x / (DP / 4), d = (x - hc * (DP / 4)) * 4;
      const int map = DIFF && hc >= nh, hh = map ? hc - nh + kTileHeads : hc;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm[w * C::kHeads + hh]);
      const float m0 = M == -INFINITY ? 0.f : M;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      float L = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float s = ex2(sm[w * C::kHeads + hh] - m0);
        const float4 t = *reinterpret_cast<const float4 *>(so + (w * C::kHeads + hh) * C::kPad + d);
        v.x += s * t.x;
        v.y += s * t.y;
        v.z += s * t.z;
        v.w += s * t.w;
        L += s * sl[w * C::kHeads + hh];
      }
      if (DIFF && done) {
        // kept in the first warp's place, which no other thread reads, until both maps are there
        const float r = (L == 0.f ? 0.f : osc / L) * (map ? a.lambda[h0 + hc - nh] : 1.f);
        *reinterpret_cast<float4 *>(so + hh * C::kPad + d) =
            make_float4(v.x * r, v.y * r, v.z * r, v.w * r);
        if (d == 0 && a.lse)
          a.lse[((int64_t)b * a.q_heads + h0 + hc - map * nh) * 2 + map] = (m0 + log2f(L)) * kLn2;
      } else if (done) {
        const int64_t oh = (int64_t)b * a.q_heads + h0 + hh;
        if (d < c.D) {
          const float r = L == 0.f ? 0.f : osc / L;
          *reinterpret_cast<uint2 *>(a.out + oh * c.D + d) =
              make_uint2(pack2<2>(v.x * r, v.y * r), pack2<2>(v.z * r, v.w * r));
        }
        if (d == 0 && a.lse) a.lse[oh] = (m0 + log2f(L)) * kLn2;
      } else {
        *reinterpret_cast<float4 *>(&part->o[hh][d]) = v;
        if (d == 0) {
          part->m[hh] = M;
          part->l[hh] = L;
        }
      }
    }
    if (DIFF && done) {
      __syncthreads();
      for (int hh = warp; hh < nh; hh += kWarps) {
        const int64_t oh = (int64_t)b * a.q_heads + h0 + hh;
        Squares q;
        for (int d = lane; a.norm && d < c.D; d += 32)
          q.add(so[hh * C::kPad + d] - so[(hh + kTileHeads) * C::kPad + d]);
        q.add_lanes();
        const float r = !a.norm ? 1.f : q.inverse(c.D, a.eps);
        for (int d = lane * 2; d < c.D; d += 64) {
          float y[2];
#pragma unroll
          for (int i = 0; i < 2; ++i)
            y[i] = (so[hh * C::kPad + d + i] - so[(hh + kTileHeads) * C::kPad + d + i]) * r *
                   (a.norm ? a.norm[d + i] : 1.f);
          *reinterpret_cast<uint32_t *>(a.out + oh * c.D + d) = pack2<2>(y[0], y[1]);
        }
      }
    }
    __syncthreads();
  }
}

// A row as the joins see it: the blocks that share it and where its parts lie.
struct Row {
  int b, hq, hh;  // batch entry, query head, the head's place in the parts
  int c0, n;      // the first block, how many; n = 0: no tokens
};
template <typename C, bool DIFF>
__device__ __forceinline__ Row row_of(const AttendArgs &a, int head_tiles, int grid, int x) {
  Row r;
  r.b = x / a.q_heads;
  r.hq = x - r.b * a.q_heads;
  const int HV = a.c.heads * head_tiles, group = a.q_heads / a.c.heads;
  const Sums all = sums_of<C>(a, HV, r.b, false);
  const int cost = span_of(a, r.b, C::kTok, C::kUnit, false).cost;
  const int h = r.hq / group, in = r.hq - h * group;
  constexpr int kTileHeads = DIFF ? C::kHeads / 2 : C::kHeads;
  r.hh = in % kTileHeads;
  const uint32_t lo = all.below + (uint32_t)(h * head_tiles + in / kTileHeads) * cost;
  const uint32_t nblk = blocks_used(all.W, grid);
  r.c0 = r.n = 0;
  if (cost) {  // the blocks of the row's first and last unit
    r.c0 = block_of(all.W, nblk, lo + kRowCost);
    r.n = min(block_of(all.W, nblk, lo + cost - 1), (int)nblk - 1) - r.c0 + 1;
  }
  return r;
}

// The joins add up the parts of a row that lies in several blocks (the first block's part is
// the one that begins the row, slot 1) and write rows without tokens.  They are launched
// while k_attend still runs and find their parts before they wait, so that only the reading
// of the parts comes after k_attend's end.  Every block waits, also one whose row is
// complete: what follows in the stream waits for the join alone, so it must not end before
// k_attend.  (It does not let its successor start early: the next call's blocks would take
// the places of its own.)

// Many rows: one block of two warps per (batch entry, query head); each warp takes every
// second part, the first kPre of them in one round of loads.
template <int ES, int DP, int NT>
__global__ void __launch_bounds__(64) k_attend_join(AttendArgs a, int head_tiles, int grid) {
  using C = Cfg<ES, DP, NT>;
  constexpr int kVec = DP / 32;  // channels per lane
  constexpr int kPre = 4;
  __shared__ float s_o[2][DP];
  const CacheView &c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Row r = row_of<C, false>(a, head_tiles, grid, blockIdx.x);
  const int64_t oh = (int64_t)r.b * a.q_heads + r.hq;
  const int n = r.n, hh = r.hh;
  const Part<DP, NT> *parts = reinterpret_cast<const Part<DP, NT> *>(a.ws) + r.c0 * 2;
  float osc = 1.f;
  if (ES == 1 && c.scale) osc = c.scale[a.layer * c.heads + r.hq / (a.q_heads / c.heads)];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (n == 0) write_empty<false>(a, r.b, r.hq, 1, 64);
  if (n <= 1) return;
  float pm[kPre], po[kPre][kVec];
#pragma unroll
  for (int i = 0; i < kPre; ++i) {
    const int k = warp + i * 2;
    pm[i] = -INFINITY;
    if (k < n) {
      const Part<DP, NT> &p = parts[2 * k + (k == 0)];
      pm[i] = p.m[hh];
#pragma unroll
      for (int v = 0; v < kVec; ++v) po[i][v] = p.o[hh][v * 32 + lane];
    }
  }
  float m1 = -INFINITY, l1 = 0.f;  // of part `lane`
  if (lane < n) {
    const Part<DP, NT> &p = parts[2 * lane + (lane == 0)];
    m1 = p.m[hh];
    l1 = p.l[hh];
  }
  float M = m1;
  for (int i = lane + 32; i < n; i += 32) M = fmaxf(M, parts[2 * i].m[hh]);
#pragma unroll
  for (int s = 16; s; s >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, s));
  const float m0 = M == -INFINITY ? 0.f : M;
  float L = ex2(m1 - m0) * l1;
  for (int i = lane + 32; i < n; i += 32) L += ex2(parts[2 * i].m[hh] - m0) * parts[2 * i].l[hh];
  float acc[kVec];
#pragma unroll
  for (int v = 0; v < kVec; ++v) acc[v] = 0.f;
#pragma unroll
  for (int i = 0; i < kPre; ++i)
    if (warp + i * 2 < n) {
      const float w = ex2(pm[i] - m0);
#pragma unroll
      for (int v = 0; v < kVec; ++v) acc[v] += w * po[i][v];
    }
#pragma unroll 4
  for (int i = warp + kPre * 2; i < n; i += 2) {
    const Part<DP, NT> &p = parts[2 * i];
    const float w = ex2(p.m[hh] - m0);
#pragma unroll
    for (int v = 0; v < kVec; ++v) acc[v] += w * p.o[hh][v * 32 + lane];
  }
#pragma unroll
  for (int s = 16; s; s >>= 1) L += __shfl_xor_sync(~0u, L, s);
#pragma unroll
  for (int v = 0; v < kVec; ++v) s_o[warp][v * 32 + lane] = acc[v];
  __syncthreads();
  for (int d = threadIdx.x; d < c.D; d += 64) {
    const __nv_bfloat16 v =
        __float2bfloat16_rn(L == 0.f ? 0.f : (s_o[0][d] + s_o[1][d]) / L * osc);
    a.out[oh * c.D + d] = *reinterpret_cast<const uint16_t *>(&v);
  }
  if (threadIdx.x == 0 && a.lse) a.lse[oh] = (m0 + log2f(L)) * kLn2;
}

// Few rows with many parts each: one block of 8 warps per (batch entry, query head) and 32
// channels; each warp takes every 8th part, 32 of them in one round of loads.
constexpr int kWide = 8;
constexpr int kMostParts = 4 * 160;  // blocks that can share a row
template <int ES, int DP, int NT>
__global__ void __launch_bounds__(kWide * 32) k_attend_join_wide(AttendArgs a, int head_tiles,
                                                                 int grid) {
  using C = Cfg<ES, DP, NT>;
  constexpr int kPre = 32, kCols = DP / 32;
  __shared__ float s_w[kMostParts], s_o[kWide][32], s_m[kWide], s_l[kWide];
  const CacheView &c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int x = blockIdx.x / kCols, col = blockIdx.x - x * kCols;
  const Row r = row_of<C, false>(a, head_tiles, grid, x);
  const int64_t oh = (int64_t)r.b * a.q_heads + r.hq;
  const int n = min(r.n, kMostParts), hh = r.hh, d = col * 32 + lane;
  const Part<DP, NT> *parts = reinterpret_cast<const Part<DP, NT> *>(a.ws) + r.c0 * 2;
  float osc = 1.f;
  if (ES == 1 && c.scale) osc = c.scale[a.layer * c.heads + r.hq / (a.q_heads / c.heads)];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (n == 0 && col == 0) write_empty<false>(a, r.b, r.hq, 1, kWide * 32);
  if (n <= 1) return;
  float po[kPre];
#pragma unroll
  for (int i = 0; i < kPre; ++i) {
    const int k = warp + i * kWide;
    po[i] = k < n ? parts[2 * k + (k == 0)].o[hh][d] : 0.f;
  }
  float M = -INFINITY;
  for (int k = threadIdx.x; k < n; k += kWide * 32) {
    const float m = parts[2 * k + (k == 0)].m[hh];
    s_w[k] = m;
    M = fmaxf(M, m);
  }
#pragma unroll
  for (int s = 16; s; s >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, s));
  if (lane == 0) s_m[warp] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWide; ++w) M = fmaxf(M, s_m[w]);
  const float m0 = M == -INFINITY ? 0.f : M;
  float L = 0.f;
  for (int k = threadIdx.x; k < n; k += kWide * 32) {
    const float w = ex2(s_w[k] - m0);
    s_w[k] = w;
    L += w * parts[2 * k + (k == 0)].l[hh];
  }
#pragma unroll
  for (int s = 16; s; s >>= 1) L += __shfl_xor_sync(~0u, L, s);
  if (lane == 0) s_l[warp] = L;
  __syncthreads();
  float acc = 0.f;
#pragma unroll
  for (int i = 0; i < kPre; ++i)
    if (warp + i * kWide < n) acc += s_w[warp + i * kWide] * po[i];
#pragma unroll 8
  for (int k = warp + kPre * kWide; k < n; k += kWide) acc += s_w[k] * parts[2 * k].o[hh][d];
  s_o[warp][lane] = acc;
  __syncthreads();
  if (warp) return;
  acc = L = 0.f;
#pragma unroll
  for (int w = 0; w < kWide; ++w) {
    acc += s_o[w][lane];
    L += s_l[w];
  }
  if (d < c.D) {
    const __nv_bfloat16 v = __float2bfloat16_rn(L == 0.f ? 0.f : acc / L * osc);
    a.out[oh * c.D + d] = *reinterpret_cast<const uint16_t *>(&v);
  }
  if (col == 0 && lane == 0 && a.lse) a.lse[oh] = (m0 + log2f(L)) * kLn2;
}

// Differential attention: one block of 8 warps per (batch entry, query head) for any number of
// parts; each warp takes every 8th part of both maps, the norm needs all channels.
template <int ES, int DP, int NT>
__global__ void __launch_bounds__(kWide * 32) k_attend_join_diff(AttendArgs a, int head_tiles, int grid) {
  using C = Cfg<ES, DP, NT>;
  constexpr int kVec = DP / 32;
  __shared__ float s_w[2][kMostParts], s_o[kWide][2][DP], s_m[2][kWide], s_l[2][kWide];
  __shared__ Squares s_q[kWide];
  const CacheView &c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Row r = row_of<C, true>(a, head_tiles, grid, blockIdx.x);
  const int64_t oh = (int64_t)r.b * a.q_heads + r.hq;
  const int n = min(r.n, kMostParts);
  const Part<DP, NT> *parts = reinterpret_cast<const Part<DP, NT> *>(a.ws) + r.c0 * 2;
  float osc = 1.f;
  if (ES == 1 && c.scale) osc = c.scale[a.layer * c.heads + r.hq / (a.q_heads / c.heads)];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (n == 0) write_empty<true>(a, r.b, r.hq, 1, kWide * 32);
  if (n <= 1) return;
  float M[2] = {-INFINITY, -INFINITY}, L[2] = {0.f, 0.f};
#pragma unroll
  for (int map = 0; map < 2; ++map) {
    for (int k = threadIdx.x; k < n; k += kWide * 32) {
      const float m = parts[2 * k + (k == 0)].m[r.hh + map * (C::kHeads / 2)];
      s_w[map][k] = m;
      M[map] = fmaxf(M[map], m);
    }
#pragma unroll
    for (int s = 16; s; s >>= 1) M[map] = fmaxf(M[map], __shfl_xor_sync(~0u, M[map], s));
    if (lane == 0) s_m[map][warp] = M[map];
  }
  __syncthreads();
#pragma unroll
  for (int map = 0; map < 2; ++map) {
#pragma unroll
    for (int w = 0; w < kWide; ++w) M[map] = fmaxf(M[map], s_m[map][w]);
    M[map] = M[map] == -INFINITY ? 0.f : M[map];
    for (int k = threadIdx.x; k < n; k += kWide * 32) {
      const float w = ex2(s_w[map][k] - M[map]);
      s_w[map][k] = w;
      L[map] += w * parts[2 * k + (k == 0)].l[r.hh + map * (C::kHeads / 2)];
    }
#pragma unroll
    for (int s = 16; s; s >>= 1) L[map] += __shfl_xor_sync(~0u, L[map], s);
    if (lane == 0) s_l[map][warp] = L[map];
  }
  __syncthreads();
  float acc[2][kVec];
#pragma unroll
  for (int map = 0; map < 2; ++map)
#pragma unroll
    for (int v = 0; v < kVec; ++v) acc[map][v] = 0.f;
#pragma unroll 4
  for (int k = warp; k < n; k += kWide) {
    const Part<DP, NT> &p = parts[2 * k + (k == 0)];
#pragma unroll
    for (int map = 0; map < 2; ++map)
#pragma unroll
      for (int v = 0; v < kVec; ++v)
        acc[map][v] += s_w[map][k] * p.o[r.hh + map * (C::kHeads / 2)][v * 32 + lane];
  }
#pragma unroll
  for (int map = 0; map < 2; ++map) {
#pragma unroll
    for (int v = 0; v < kVec; ++v) s_o[warp][map][v * 32 + lane] = acc[map][v];
    L[map] = 0.f;
#pragma unroll
    for (int w = 0; w < kWide; ++w) L[map] += s_l[map][w];
  }
  __syncthreads();
  const int d = threadIdx.x;  // DP is at most the block's threads
  float y = 0.f;
  if (d < c.D) {
    float o[2] = {0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kWide; ++w)
#pragma unroll
      for (int map = 0; map < 2; ++map) o[map] += s_o[w][map][d];
    const float f0 = L[0] == 0.f ? 0.f : osc / L[0];
    const float f1 = (L[1] == 0.f ? 0.f : osc / L[1]) * a.lambda[r.hq];
    y = o[0] * f0 - o[1] * f1;
  }
  if (a.norm) {
    Squares q;
    q.add(y);
    q.add_lanes();
    if (lane == 0) s_q[warp] = q;
    __syncthreads();
    q = s_q[0];
#pragma unroll
    for (int w = 1; w < kWide; ++w) q.add(s_q[w]);
    if (d < c.D) y = y * q.inverse(c.D, a.eps) * a.norm[d];
  }
  if (d < c.D) {
    const __nv_bfloat16 v = __float2bfloat16_rn(y);
    a.out[oh * c.D + d] = *reinterpret_cast<const uint16_t *>(&v);
  }
  if (threadIdx.x < 2 && a.lse) {
    const int map = threadIdx.x;
    a.lse[oh * 2 + map] = map ? (M[1] + log2f(L[1])) * kLn2 : (M[0] + log2f(L[0])) * kLn2;
  }
}

int sm_count() {
  static std::atomic<int> known[64];  // by device; a device's SMs do not change
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed))) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (n > kMostParts / 4) n = kMostParts / 4;
  if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

template <int ES, int DP, int NT, bool DIFF>
cudaError_t run(const AttendArgs &a, int head_tiles, cudaStream_t st) {
  using C = Cfg<ES, DP, NT>;
  const int sms = sm_count();
  if (!sms) return cudaErrorInvalidDevice;
  const int64_t rows = (int64_t)a.batch * a.c.heads * head_tiles;
  // a tile may start up to kTok - 1 tokens before the range
  const int64_t row_units = ((int64_t)a.max_len + C::kTok - 1 + C::kUnit - 1) / C::kUnit;
  const int64_t wave = (int64_t)sms * C::kPerSm;
  // One block per row, and no join, where a block takes little longer for a row than the
  // cut and the join do; with many rows the blocks that start as others end also even out
  // what is left.  A unit takes a block that has its SM to itself 0.3 us (bf16: what the
  // SM's shared memory takes in and out) or 0.8 us (e4m3: the conversions).  Cut / not cut,
  // 128 channels, us: bf16, 8 rows of 9 units 7.1 / 7.8; 64 rows of 9 8.1 / 8.4, of 17 9.3 /
  // 12.9; 256 rows of 17 22.0 / 21.1, of 33 33.6 / 36.7; 512 rows of 33 61.2 / 59.2, of 65
  // 108 / 117; 2048 rows of 9 78.8 / 56.8.  e4m3, 64 rows of 5 units 8.6 / 7.2, of 9 8.9 /
  // 10.2; 256 rows of 9 16.2 / 14.7, of 17 22.3 / 23.5; 1024 rows of 17 61.2 / 58.3; 2048
  // rows of 5 49.3 / 38.6.
  // A unit is 64 or 128 tokens: 32 KB of keys and values as at 128 channels for bf16 of 64
  // and e4m3 of 256 channels, half of that for e4m3 of 64, twice that for bf16 of 256.  The
  // same rule, rows of one length, cut / not cut, us: bf16 of 64, 8 rows of 9 units 7.7 /
  // 10.2, 256 of 17 29.8 / 26.9, of 33 47.8 / 46.6, 512 of 33 87 / 100 (the last blocks
  // run alone), 2048 of 33 325 / 313; e4m3 of 64, 64 of 9 9.3 / 9.9, 256 of 17 19.6 / 18.0,
  // 512 of 33 51.4 / 48.7, 2048 of 9 64 / 55, of 33 187 / 172; bf16 of 256, 8 of 9 9.0 /
  // 11.8, 64 of 9 15.4 / 13.1, of 17 19.5 / 20.4, 256 of 17 50.2 / 49.1, 512 of 33 163 /
  // 171; e4m3 of 256, 64 of 9 12.8 / 11.8, 256 of 17 31.9 / 28.1, of 33 51.7 / 47.4, 2048 of
  // 33 339 / 319.  The rule's side is the slower one, by up to 15%, for rows in two waves
  // (512 of 17 to 33 units, bf16) and by up to 14% for 256 and more rows of 17 to 33 units of
  // e4m3, by 10% for 64 rows of 9 (bf16), elsewhere by less than 9% or not at all.
  const int64_t whole = ES == 2 ? (rows < 448 ? 5 + rows / 16 : 33)
                                : (rows < 768 ? 5 + rows / 64 : 17);
  if (row_units <= whole) {
    auto kern = k_attend<ES, DP, NT, true, DIFF>;
    cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    return launch(kern, dim3((unsigned)rows), kThreads, C::kSmem, st, a, head_tiles);
  }
  auto kern = k_attend<ES, DP, NT, false, DIFF>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  int64_t grid = rows * row_units / 2;
  if (grid > wave) grid = wave;
  if (grid < 1) grid = 1;
  e = launch(kern, dim3((unsigned)grid), kThreads, C::kSmem, st, a, head_tiles);
  if (e != cudaSuccess) return e;
  const int64_t joins = (int64_t)a.batch * a.q_heads;
  if constexpr (DIFF) {
    return launch(k_attend_join_diff<ES, DP, NT>, dim3((unsigned)joins), kWide * 32, 0, st, a, head_tiles,
                  (int)grid);
  } else {
  // Few rows with many parts each: one row of 31394 tokens 8.7 us against 21.1, 8 of 131071
  // 47.1 against 50.9; but 8 of 2048 (17 parts) 8.5 against 8.0, and 16 of 8192 with 8 query
  // heads (512 blocks) 19.9 against 19.0.
  if (grid / rows >= 24 && joins * (DP / 32) <= 2 * sms)
    return launch(k_attend_join_wide<ES, DP, NT>, dim3((unsigned)(joins * (DP / 32))), kWide * 32,
                  0, st, a, head_tiles, (int)grid);
  return launch(k_attend_join<ES, DP, NT>, dim3((unsigned)joins), 64, 0, st, a, head_tiles,
                (int)grid);
  }
}

template <int ES, int DP, bool DIFF>
cudaError_t run_nt(const AttendArgs &a, cudaStream_t st) {
  const int columns = a.q_heads / a.c.heads * (DIFF ? 2 : 1);
  if (columns <= 8) return run<ES, DP, 1, DIFF>(a, 1, st);
  return run<ES, DP, 2, DIFF>(a, (columns + 15) / 16, st);
}

template <int ES, bool DIFF>
cudaError_t run_d(const AttendArgs &a, cudaStream_t st) {
  if (a.c.D <= 64) return run_nt<ES, 64, DIFF>(a, st);
  if (a.c.D <= 128) return run_nt<ES, 128, DIFF>(a, st);
  return run_nt<ES, 256, DIFF>(a, st);
}

size_t ws_bytes(const CacheView &c, int columns) {
  const int sms = sm_count();
  if (!sms) return 0;
  const int heads = columns <= 8 ? 8 : 16;
  const int DP = c.D <= 64 ? 64 : c.D <= 128 ? 128 : 256;
  // two partial results for each of at most two blocks per SM
  return (size_t)sms * 4 * 2 * heads * (DP + 2) * sizeof(float);
}

}  // namespace
}  // namespace skv
