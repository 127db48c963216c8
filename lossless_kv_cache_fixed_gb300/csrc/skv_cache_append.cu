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
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "skv_cache.cuh"

namespace skv {
namespace {

constexpr int kThreads = 256;

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

// x / scale as e4m3, one rounding to nearest even, saturating; NaN stays NaN.
__device__ __forceinline__ uint2 pack_e4m3(const float *x, float scale) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t h[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
      h[j] = __nv_cvt_float2_to_fp8x2(
          make_float2(__fdiv_rn(x[4 * i + 2 * j], scale), __fdiv_rn(x[4 * i + 2 * j + 1], scale)),
          __NV_SATFINITE, __NV_E4M3);
    w[i] = h[0] | h[1] << 16;
  }
  return make_uint2(w[0], w[1]);
}

// A block takes `tt` tokens.  Its threads first fill the tokens' cos/sin table,
// then take units of two 8-channel vectors of one (token, head): the two halves
// of 8 pairs, 16 neighbouring channels with 8 pairs, or 16 channels that pass.
template <bool E4M3>
__global__ void __launch_bounds__(kThreads) k_append(AppendArgs a, int tt) {
  extern __shared__ float2 cs[];  // [tt][rotary / 2]
  const CacheView &c = a.c;
  const int64_t i0 = (int64_t)blockIdx.x * tt;
  const int nt = (int)min((int64_t)tt, (int64_t)a.n - i0);
  const int pairs = a.rotary / 2;
  for (int x = threadIdx.x; x < nt * pairs; x += kThreads) {
    const int t = x / pairs, p = x - t * pairs;
    const int ax = a.axis ? a.axis[p] : 0;
    float s = 0.f, co = 1.f;
    if (ax < a.axes) {
      const double turns = (double)a.positions[(int64_t)ax * a.n + i0 + t] *
                           (a.freqs[p] * 0.15915494309189533577);  // 1 / (2 pi)
      sincospif(2.f * (float)(turns - rint(turns)), &s, &co);
    } else {
      atomicOr(c.status, kCacheArg);
    }
    cs[x] = make_float2(co, s);
  }
  __syncthreads();
  const uint32_t U = (uint32_t)(c.D + 15) / 16;
  const uint32_t heads = (uint32_t)(a.q_heads + 2 * c.heads);
  const uint32_t total = (uint32_t)nt * heads * U;
  const uint32_t turned = (uint32_t)a.rotary / 16;
  for (uint32_t x = threadIdx.x; x < total; x += kThreads) {
    const uint32_t th = x / U, u = x - th * U;
    const uint32_t t = th / heads;
    int h = (int)(th - t * heads);
    const int64_t i = i0 + t;
    const int kind = h < a.q_heads ? 0 : h < a.q_heads + c.heads ? 1 : 2;
    h -= kind == 0 ? 0 : kind == 1 ? a.q_heads : a.q_heads + c.heads;
    const bool turn = kind < 2 && u < turned;
    const bool inter = turn && !a.interleaved;
    const int d0 = inter ? 8 * u : 16 * u, d1 = inter ? 8 * u + pairs : 16 * u + 8;
    const bool two = d1 < c.D;
    const uint16_t *src = kind == 0   ? a.q + i * a.qs + h * a.qhs
                          : kind == 1 ? a.k + i * a.ks + h * a.khs
                                      : a.v + i * a.vs + h * a.vhs;
    // where it goes
    uint8_t *dst;
    if (kind == 0) {
      dst = reinterpret_cast<uint8_t *>(a.q_out + (i * a.q_heads + h) * c.D);
    } else {
      const int32_t slot = a.slots[i], at = a.at[i];
      if (slot < 0) continue;
      const int32_t blk = at / c.Tb;
      if (slot >= c.seqs || at < 0 || blk >= c.blocks) {
        atomicOr(c.status, kCacheArg);
        continue;
      }
      const uint32_t page =
          c.table[((int64_t)slot * c.rows + ((int64_t)a.layer * 2 + kind - 1) * c.heads + h) *
                      c.blocks + blk];
      if (page >= c.pages || c.refs[page] != 1) {
        atomicOr(c.status, kCacheArg);
        continue;
      }
      dst = c.pool + (uint64_t)page * c.page_bytes + (uint32_t)(at - blk * c.Tb) * c.row_bytes;
    }
    uint4 v0 = ld_stream(src + d0), v1 = make_uint4(0, 0, 0, 0);
    if (two) v1 = ld_stream(src + d1);
    if (turn || (E4M3 && kind)) {
      float x0[8], x1[8];
      unpack(v0, x0);
      unpack(v1, x1);
      if (turn) {
        const float4 *w = reinterpret_cast<const float4 *>(cs + t * pairs + 8 * u);
        float f[16];
#pragma unroll
        for (int j = 0; j < 4; ++j) *reinterpret_cast<float4 *>(f + 4 * j) = w[j];
        if (inter) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float p = x0[j], q = x1[j];
            x0[j] = p * f[2 * j] - q * f[2 * j + 1];
            x1[j] = p * f[2 * j + 1] + q * f[2 * j];
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float p = x0[2 * j], q = x0[2 * j + 1];
            x0[2 * j] = p * f[2 * j] - q * f[2 * j + 1];
            x0[2 * j + 1] = p * f[2 * j + 1] + q * f[2 * j];
            p = x1[2 * j], q = x1[2 * j + 1];
            x1[2 * j] = p * f[8 + 2 * j] - q * f[9 + 2 * j];
            x1[2 * j + 1] = p * f[9 + 2 * j] + q * f[8 + 2 * j];
          }
        }
      }
      if (E4M3 && kind) {
        const float scale = c.scale ? c.scale[a.layer * c.heads + h] : 1.f;
        *reinterpret_cast<uint2 *>(dst + d0) = pack_e4m3(x0, scale);
        if (two) *reinterpret_cast<uint2 *>(dst + d1) = pack_e4m3(x1, scale);
        continue;
      }
      v0 = pack_bf16(x0);
      v1 = pack_bf16(x1);
    }
    st_stream(dst + 2 * d0, v0);
    if (two) st_stream(dst + 2 * d1, v1);
  }
}

}  // namespace

cudaError_t launch_append(const AppendArgs &a, cudaStream_t st) {
  // one token per block while that fills no more than a wave of blocks
  const int tt = a.n <= 152 * 8 ? 1 : 4;
  const unsigned grid = (unsigned)((a.n + tt - 1) / tt);
  const size_t smem = sizeof(float2) * (size_t)tt * (a.rotary / 2);
  if (a.c.dtype == 1) k_append<true><<<grid, kThreads, smem, st>>>(a, tt);
  else k_append<false><<<grid, kThreads, smem, st>>>(a, tt);
  return cudaGetLastError();
}

}  // namespace skv
