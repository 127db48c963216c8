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
// warp diverges; a task's vectors are loaded before the one before it is turned, the
// first ones before the block forms its angles and looks up its pages.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "skv_cache.cuh"

namespace skv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kToks = 4;  // tokens of a block

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

// x / d where x * d is below 2^32: magic = ceil(2^32 / d), 0 for d = 1.
struct Div {
  uint32_t magic;
};
__device__ __forceinline__ uint32_t div_of(uint32_t x, const Div &v) {
  return v.magic ? __umulhi(x, v.magic) : x;
}

// How the work is cut (built by the host).
struct Plan {
  int toks;           // tokens of a block
  int units, turned;  // 16-channel units of a head, those that turn
  Div by_units, by_turned, by_pass, by_q, by_kv;
};

enum Kind { kQTurn, kKTurn, kQPass, kKPass, kV, kKinds };

// (a, b) turned by (cos, sin).
__device__ __forceinline__ void turn(float &a, float &b, float co, float s) {
  const float x = a, y = b;
  a = x * co - y * s;
  b = x * s + y * co;
}

// One lane's unit of a task.
struct Unit {
  uint4 v0, v1;
  int kind, tk, h, u;  // kind < 0: none
};

template <bool E4M3>
__global__ void __launch_bounds__(kThreads, 5) k_append(AppendArgs a, Plan pl) {
  extern __shared__ __align__(16) uint8_t smem[];
  begin();
  const CacheView &c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pairs = a.rotary / 2, kv = 2 * c.heads;
  float2 *cs = reinterpret_cast<float2 *>(smem);                            // [toks][pairs], see below
  uint64_t *dsts = reinterpret_cast<uint64_t *>(cs + pl.toks * pairs);      // [toks][2][heads]
  float *invs = reinterpret_cast<float *>(dsts + pl.toks * kv);             // [heads], e4m3
  const int64_t i0 = (int64_t)blockIdx.x * pl.toks;
  const int nt = (int)min((int64_t)pl.toks, (int64_t)a.n - i0);
  const int passing = pl.units - pl.turned;

  // tasks [0, e0) are of kind 0, [e0, e1) of kind 1, ...
  const int n0 = nt * a.q_heads * pl.turned, n1 = nt * c.heads * pl.turned;
  const int n2 = nt * a.q_heads * passing, n3 = nt * c.heads * passing;
  const int n4 = nt * c.heads * pl.units;
  const int e0 = (n0 + 31) / 32, e1 = e0 + (n1 + 31) / 32, e2 = e1 + (n2 + 31) / 32;
  const int e3 = e2 + (n3 + 31) / 32, e4 = e3 + (n4 + 31) / 32;

  auto fetch = [&](int task) {
    Unit t;
    t.kind = -1;
    if (task >= e4) return t;
    int kind, x, n;
    if (task < e0) kind = kQTurn, x = task, n = n0;
    else if (task < e1) kind = kKTurn, x = task - e0, n = n1;
    else if (task < e2) kind = kQPass, x = task - e1, n = n2;
    else if (task < e3) kind = kKPass, x = task - e2, n = n3;
    else kind = kV, x = task - e3, n = n4;
    x = x * 32 + lane;
    if (x >= n) return t;
    const bool turns = kind <= kKTurn, q = kind == kQTurn || kind == kQPass;
    const int th = div_of(x, turns ? pl.by_turned : kind == kV ? pl.by_units : pl.by_pass);
    t.u = x - th * (turns ? pl.turned : kind == kV ? pl.units : passing);
    if (kind == kQPass || kind == kKPass) t.u += pl.turned;
    t.tk = div_of(th, q ? pl.by_q : pl.by_kv);
    t.h = th - t.tk * (q ? a.q_heads : c.heads);
    t.kind = kind;
    const int64_t i = i0 + t.tk;
    const uint16_t *src = q             ? a.q + i * a.qs + t.h * a.qhs
                          : kind == kV  ? a.v + i * a.vs + t.h * a.vhs
                                        : a.k + i * a.ks + t.h * a.khs;
    const bool halves = turns && !a.interleaved;
    const int d0 = halves ? 8 * t.u : 16 * t.u, d1 = halves ? d0 + pairs : d0 + 8;
    t.v0 = __ldcs(reinterpret_cast<const uint4 *>(src + d0));
    t.v1 = d1 < c.D ? __ldcs(reinterpret_cast<const uint4 *>(src + d1)) : make_uint4(0, 0, 0, 0);
    return t;
  };

  Unit next = fetch(warp);

  // the tokens' angles, and where their keys and values go (0: nowhere)
  for (int x = threadIdx.x; x < nt * kv; x += kThreads) {
    const int tk = x / kv, r = x - tk * kv;
    const int32_t slot = a.slots[i0 + tk], at = a.at[i0 + tk], blk = at / c.Tb;
    uint64_t dst = 0;
    bool bad = slot >= 0;
    if (slot >= 0 && slot < c.seqs && at >= 0 && blk < c.blocks) {
      const uint32_t page =
          c.table[((int64_t)slot * c.rows + (int64_t)a.layer * kv + r) * c.blocks + blk];
      if (page < c.pages && c.refs[page] == 1) {
        bad = false;
        dst = reinterpret_cast<uint64_t>(c.pool + (uint64_t)page * c.page_bytes +
                                         (uint32_t)(at - blk * c.Tb) * c.row_bytes);
      }
    }
    if (bad) atomicOr(c.status, kCacheArg);
    dsts[x] = dst;
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
    if (t.kind < 0) continue;
    const bool turns = t.kind <= kKTurn, q = t.kind == kQTurn || t.kind == kQPass;
    uint8_t *o = q ? reinterpret_cast<uint8_t *>(a.q_out + ((i0 + t.tk) * a.q_heads + t.h) * c.D)
                   : reinterpret_cast<uint8_t *>(
                         dsts[t.tk * kv + (t.kind == kV ? c.heads : 0) + t.h]);
    if (!o) continue;
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
      const float inv = invs[t.h];
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

Div make_div(int d) {
  return Div{d > 1 ? (uint32_t)(((1ull << 32) + d - 1) / d) : 0u};
}

}  // namespace

cudaError_t launch_append(const AppendArgs &a, cudaStream_t st) {
  const CacheView &c = a.c;
  const int pairs = a.rotary / 2;
  Plan p;
  p.units = (c.D + 15) / 16;
  p.turned = a.rotary / 16;
  // one token per block while that fills no more than a wave of blocks, and where its units
  // are many (div_of)
  const int64_t units = ((int64_t)a.q_heads + 2 * c.heads) * p.units;
  p.toks = a.n <= 152 * 4 || units > 4096 ? 1 : kToks;
  p.by_units = make_div(p.units);
  p.by_turned = make_div(p.turned);
  p.by_pass = make_div(p.units - p.turned);
  p.by_q = make_div(a.q_heads);
  p.by_kv = make_div(c.heads);
  const size_t smem = (size_t)p.toks * (sizeof(float2) * pairs + sizeof(uint64_t) * 2 * c.heads) +
                      (c.dtype == 1 ? sizeof(float) * (size_t)c.heads : 0);
  auto kern = c.dtype == 1 ? k_append<true> : k_append<false>;
  if (smem > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem);
    if (e != cudaSuccess) return e;
  }
  return launch(kern, dim3((unsigned)((a.n + p.toks - 1) / p.toks)), kThreads, smem, st, a, p);
}

}  // namespace skv
