// skv_cache_append.cu -- new tokens into a paged KV cache: rotary positions on
// one or more axes applied to q and k, keys and values rounded to the cache's
// type and written to their pages.
//
// Pair p of a token turns by a = position[axis_p] * freq_p.  The angle is formed
// in fp64 in turns, t = position * (freq / 2 pi), and only its fraction in
// [-1/2, 1/2] goes to fp32: position 2^20 at freq 1 leaves 2^-33 turns of error
// where an fp32 product would leave 2^-6 radians.  That is two fp64 products per
// (token, pair), shared by all heads through shared memory, so the fp64 rate
// does not bound the call.  Everything else is one read of q, k, v and one write
// of q and the cache rows: the call is bound by HBM.
//
// A block takes a few tokens.  Their units of 16 channels (two 16-byte vectors: the two
// halves of 8 pairs, or 16 neighbouring channels) are cut into tasks of 32 units of one
// kind for a warp -- q or k channels that turn, q, k or v channels that pass -- so no
// warp diverges; where each (token, head) is read from and goes to lies in shared
// memory, so a unit costs one division by multiplication and few address operations
// (53% of the issue slots are busy for e4m3, 63% for bf16).  A task's vectors
// are loaded before the one before it is turned, the first ones before the block forms
// its angles and looks up its pages.
//
// 8190 tokens of 64 + 8 + 8 heads of 128 (336 MB): 53.3 us, 6.3 TB/s; 16001 tokens of
// 32 + 8 + 8 heads into e4m3 (361 MB): 62.8 us, 5.7 TB/s.  Loading two or three tasks
// ahead, or passing the tokens through shared memory by bulk copies, is slower (63 to 75
// us and 75 to 115 us): more of the registers or of the SM's memory per warp, fewer warps.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "skv_cache.cuh"

namespace skv {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
// Blocks per SM (bounds the registers) and units of a block, for bf16 and e4m3 caches:
// 54.6 and 68.5 us with 9 and 8 blocks, 75.8 and 73.8 with 11 and 10 (the two calls above);
// 55.6 and 63.6 with 1024 units, 66.2 with 2048 (e4m3).
constexpr int kBlocks[2] = {10, 9};
constexpr int kUnits[2] = {640, 1536};
constexpr int kMostToks = 16;

__device__ __forceinline__ void unpack(const uint4 &v, float *x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack_bf16(const float *x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// x * inv as e4m3, rounded to nearest even, saturating; NaN stays NaN.
__device__ __forceinline__ uint2 pack_e4m3(const float *x, float inv) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t h[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
      h[j] = __nv_cvt_float2_to_fp8x2(
          make_float2(x[4 * i + 2 * j] * inv, x[4 * i + 2 * j + 1] * inv), __NV_SATFINITE,
          __NV_E4M3);
    w[i] = h[0] | h[1] << 16;
  }
  return make_uint2(w[0], w[1]);
}

// The kinds of units.  A block's rows are its tokens' q heads, then their k heads, then
// their v heads (token-major in each).
enum { kQTurn, kKTurn, kQPass, kKPass, kV, kKinds };
struct Kind {
  int task0, n;      // its first task, its units
  int per, from;     // units of a row, the first of them
  uint32_t magic;    // x / per = (x * magic) >> 32, or x where it is 0 (see magic_of)
  int row0;          // its first row
  int turns, q;
};

// How the work is cut (built by the host).
struct Plan {
  int toks;           // tokens of a block, at most 16
  int units, turned;  // 16-channel units of a head, those that turn
  uint32_t by_units, by_turned, by_pass;  // magics
};

// (a, b) turned by (cos, sin).
__device__ __forceinline__ void turn(float &a, float &b, float co, float s) {
  const float x = a, y = b;
  a = x * co - y * s;
  b = x * s + y * co;
}

// One lane's unit of a task: its vectors, row and place in the row; row < 0: none.
struct Unit {
  uint4 v0, v1;
  int row, u, kind, tk;
};

template <bool E4M3>
__global__ void __launch_bounds__(kThreads, kBlocks[E4M3]) k_append(AppendArgs a, Plan pl) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Kind kinds[kKinds];
  begin();
  const CacheView &c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pairs = a.rotary / 2, kv = 2 * c.heads, heads = a.q_heads + kv;
  float2 *cs = reinterpret_cast<float2 *>(smem);                        // [toks][pairs], see below
  uint64_t *srcs = reinterpret_cast<uint64_t *>(cs + pl.toks * pairs);  // [rows]: address | token
  uint64_t *dsts = srcs + pl.toks * heads;                              // [rows], 0: nowhere
  float *invs = reinterpret_cast<float *>(dsts + pl.toks * heads);      // [heads], e4m3
  const int64_t i0 = (int64_t)blockIdx.x * pl.toks;
  const int nt = (int)min((int64_t)pl.toks, (int64_t)a.n - i0);
  const int nq = nt * a.q_heads, nk = nt * c.heads;
  const int passing = pl.units - pl.turned;
  // tasks of each kind in turn, 32 units each
  const int e0 = (nq * pl.turned + 31) / 32, e1 = e0 + (nk * pl.turned + 31) / 32;
  const int e2 = e1 + (nq * passing + 31) / 32, e3 = e2 + (nk * passing + 31) / 32;
  const int e4 = e3 + (nk * pl.units + 31) / 32;
  if (threadIdx.x < kKinds) {
    const int k = threadIdx.x;
    Kind x;
    x.turns = k == kQTurn || k == kKTurn;
    x.q = k == kQTurn || k == kQPass;
    x.per = x.turns ? pl.turned : k == kV ? pl.units : passing;
    x.from = k == kQPass || k == kKPass ? pl.turned : 0;
    x.magic = x.turns ? pl.by_turned : k == kV ? pl.by_units : pl.by_pass;
    x.n = (x.q ? nq : nk) * x.per;
    x.task0 = k == kQTurn ? 0 : k == kKTurn ? e0 : k == kQPass ? e1 : k == kKPass ? e2 : e3;
    x.row0 = x.q ? 0 : k == kV ? nq + nk : nq;
    kinds[k] = x;
  }
  for (int x = threadIdx.x; x < nt * heads; x += kThreads) {
    const uint16_t *p;
    int tk;
    if (x < nq) {
      tk = x / a.q_heads;
      p = a.q + (i0 + tk) * a.qs + (x - tk * a.q_heads) * a.qhs;
      dsts[x] = reinterpret_cast<uint64_t>(a.q_out + (i0 * a.q_heads + x) * c.D);
    } else {
      const int y = x - nq < nk ? x - nq : x - nq - nk;
      tk = y / c.heads;
      const int h = y - tk * c.heads;
      p = x - nq < nk ? a.k + (i0 + tk) * a.ks + h * a.khs : a.v + (i0 + tk) * a.vs + h * a.vhs;
    }
    srcs[x] = reinterpret_cast<uint64_t>(p) | (uint64_t)tk;  // 16-byte aligned
  }
  __syncthreads();

  auto fetch = [&](int task) {
    Unit t;
    t.row = -1;
    if (task >= e4) return t;
    t.kind = (task >= e0) + (task >= e1) + (task >= e2) + (task >= e3);
    const Kind k = kinds[t.kind];
    const uint32_t x = (task - k.task0) * 32 + lane;
    if (x >= (uint32_t)k.n) return t;
    const uint32_t r = k.magic ? __umulhi(x, k.magic) : x;
    t.u = x - r * k.per + k.from;
    t.row = k.row0 + r;
    const uint64_t s = srcs[t.row];
    t.tk = (int)(s & 15);
    const uint16_t *src = reinterpret_cast<const uint16_t *>(s & ~15ull);
    const bool halves = k.turns && !a.interleaved;
    const int d0 = halves ? 8 * t.u : 16 * t.u, d1 = halves ? d0 + pairs : d0 + 8;
    t.v0 = __ldcs(reinterpret_cast<const uint4 *>(src + d0));
    t.v1 = d1 < c.D ? __ldcs(reinterpret_cast<const uint4 *>(src + d1)) : make_uint4(0, 0, 0, 0);
    return t;
  };

  Unit next = fetch(warp);

  // where the tokens' keys and values go (0: nowhere), and the tokens' angles
  for (int x = threadIdx.x; x < 2 * nk; x += kThreads) {
    const int side = x >= nk, y = x - side * nk, tk = y / c.heads, h = y - tk * c.heads;
    const int32_t slot = a.slots[i0 + tk], at = a.at[i0 + tk], blk = at / c.Tb;
    uint64_t dst = 0;
    bool bad = slot >= 0;
    if (slot >= 0 && slot < c.seqs && at >= 0 && blk < c.blocks) {
      const uint32_t page =
          c.table[((int64_t)slot * c.rows + ((int64_t)a.layer * 2 + side) * c.heads + h) *
                      c.blocks + blk];
      if (page < c.pages && c.refs[page] == 1) {
        bad = false;
        dst = reinterpret_cast<uint64_t>(c.pool + (uint64_t)page * c.page_bytes +
                                         (uint32_t)(at - blk * c.Tb) * c.row_bytes);
      }
    }
    if (bad) atomicOr(c.status, kCacheArg);
    dsts[nq + x] = dst;
  }
  if (E4M3)
    for (int h = threadIdx.x; h < c.heads; h += kThreads)
      invs[h] = c.scale ? 1.f / c.scale[a.layer * c.heads + h] : 1.f;
  // from the other end of the block: the first threads are at the pages
  for (int x = kThreads - 1 - threadIdx.x; x < nt * pairs; x += kThreads) {
    const int tk = x / pairs, p = x - tk * pairs;
    const int ax = a.axis ? a.axis[p] : 0;
    float s = 0.f, co = 1.f;
    if (ax < a.axes) {
      const double turns = (double)a.positions[(int64_t)ax * a.n + i0 + tk] *
                           (a.freqs[p] * 0.15915494309189533577);  // 1 / (2 pi)
      sincospif(2.f * (float)(turns - rint(turns)), &s, &co);
    } else {
      atomicOr(c.status, kCacheArg);
    }
    // pairs 8u + 2j and 8u + 2j + 1 at [token][j][u]: the units a warp reads at once lie
    // next to each other
    const int u = p >> 3, j = (p >> 1) & 3;
    cs[tk * pairs + (j * pl.turned + u) * 2 + (p & 1)] = make_float2(co, s);
  }
  __syncthreads();

  for (int task = warp; task < e4; task += kWarps) {
    const Unit t = next;
    next = fetch(task + kWarps);
    if (t.row < 0) continue;
    uint8_t *o = reinterpret_cast<uint8_t *>(dsts[t.row]);
    if (!o) continue;
    const bool turns = t.kind <= kKTurn, q = t.kind == kQTurn || t.kind == kQPass;
    const bool halves = turns && !a.interleaved;
    const int d0 = halves ? 8 * t.u : 16 * t.u, d1 = halves ? d0 + pairs : d0 + 8;
    if (!turns && (q || !E4M3)) {
      __stcs(reinterpret_cast<uint4 *>(o + 2 * d0), t.v0);
      if (d1 < c.D) __stcs(reinterpret_cast<uint4 *>(o + 2 * d1), t.v1);
      continue;
    }
    float x0[8], x1[8];
    unpack(t.v0, x0);
    unpack(t.v1, x1);
    if (turns) {
      const float4 *w = reinterpret_cast<const float4 *>(cs + t.tk * pairs) + t.u;
      if (halves) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 f = w[j * pl.turned];
          turn(x0[2 * j], x1[2 * j], f.x, f.y);
          turn(x0[2 * j + 1], x1[2 * j + 1], f.z, f.w);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float4 f = w[j * pl.turned], g = w[(2 + j) * pl.turned];
          turn(x0[4 * j], x0[4 * j + 1], f.x, f.y);
          turn(x0[4 * j + 2], x0[4 * j + 3], f.z, f.w);
          turn(x1[4 * j], x1[4 * j + 1], g.x, g.y);
          turn(x1[4 * j + 2], x1[4 * j + 3], g.z, g.w);
        }
      }
    }
    if (E4M3 && !q) {
      const int y = t.row - nq < nk ? t.row - nq : t.row - nq - nk;
      const float inv = invs[y - t.tk * c.heads];
      const uint2 c0 = pack_e4m3(x0, inv), c1 = pack_e4m3(x1, inv);
      if (halves) {
        __stcs(reinterpret_cast<uint2 *>(o + d0), c0);
        __stcs(reinterpret_cast<uint2 *>(o + d1), c1);
      } else {  // 16 neighbouring channels (D % 16 == 0)
        __stcs(reinterpret_cast<uint4 *>(o + d0), make_uint4(c0.x, c0.y, c1.x, c1.y));
      }
    } else {
      __stcs(reinterpret_cast<uint4 *>(o + 2 * d0), pack_bf16(x0));
      __stcs(reinterpret_cast<uint4 *>(o + 2 * d1), pack_bf16(x1));
    }
  }
}

// ceil(2^32 / d), with which x / d is exact where x * d is below 2^32; 0 for d = 1.
uint32_t magic_of(int d) { return d > 1 ? (uint32_t)(((1ull << 32) + d - 1) / d) : 0u; }

}  // namespace

cudaError_t launch_append(const AppendArgs &a, cudaStream_t st) {
  const CacheView &c = a.c;
  const int pairs = a.rotary / 2;
  Plan p;
  p.units = (c.D + 15) / 16;
  p.turned = a.rotary / 16;
  // tokens of a block: one while these fill no more than a wave of blocks, else as many as
  // make kUnits units
  const int64_t units = ((int64_t)a.q_heads + 2 * c.heads) * p.units;
  const int64_t toks = a.n <= 152 * 8 ? 1 : (kUnits[c.dtype == 1] + units / 2) / units;
  p.toks = (int)(toks < 1 ? 1 : toks > kMostToks ? kMostToks : toks);
  p.by_units = magic_of(p.units);
  p.by_turned = magic_of(p.turned);
  p.by_pass = magic_of(p.units - p.turned);
  const size_t heads = (size_t)a.q_heads + 2 * (size_t)c.heads;
  const size_t smem = (size_t)p.toks * (sizeof(float2) * pairs + 2 * sizeof(uint64_t) * heads) +
                      (c.dtype == 1 ? sizeof(float) * (size_t)c.heads : 0);
  auto kern = c.dtype == 1 ? k_append<true> : k_append<false>;
  // A launch has 48 KB, the kernel's own variables among them.  What is asked for is the most
  // that any call takes (one token of 8192 heads, 512 pairs, 4096 scales), so that threads
  // that launch at the same time do not lower it for one another.
  constexpr int kFree = 47 * 1024, kMost = 148 * 1024;
  if (smem > (size_t)kFree) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (e != cudaSuccess) return e;
  }
  return launch(kern, dim3((unsigned)((a.n + p.toks - 1) / p.toks)), kThreads, smem, st, a, p);
}

}  // namespace skv
