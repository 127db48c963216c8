// skv_cache_chunk.cu -- attention of the new tokens of each sequence over a paged KV
// cache, plain and differential.
//
// o_h = sum_t p_t v_t / sum_t p_t with p_t = 2^(x_t - m), x_t = log2(e) * scale * q_h.k_t, m
// the running maximum (softmax in one pass: when m grows to m', the sums so far are multiplied
// by 2^(m - m')).  Differential attention runs the halves of q and k as two such maps over the
// same values and subtracts lambda times the second result.
//
// The simplest form: one warp per (row, query head), 32 tokens at a time, a lane per token for
// the scores and 32 channels per step for the sums, all in fp32 without matrix instructions.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "skv_cache.cuh"

namespace skv {
namespace {

constexpr int kWarps = 8;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float scalar(const uint8_t *p, int dtype, int d) {
  if (dtype == 0) return __uint_as_float((uint32_t) reinterpret_cast<const uint16_t *>(p)[d] << 16);
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)p[d]));
  return __half2float(__ushort_as_half((unsigned short)(h & 0xffff)));
}

// The sequence that row i belongs to, -1 if none.
__device__ __forceinline__ int sequence_of(const ChunkArgs &a, int i) {
  if (!a.starts) return i;
  for (int b = 0; b < a.batch; ++b)
    if (a.starts[b] <= i && i < a.starts[b + 1] && a.starts[b] >= 0 && a.starts[b + 1] <= a.tokens)
      return b;
  return -1;
}

__global__ void __launch_bounds__(kWarps * 32) k_chunk(ChunkArgs a) {
  begin();
  const CacheView &c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // what is wrong with the sequences themselves
  for (int b = blockIdx.x * blockDim.x + threadIdx.x; b < a.batch; b += gridDim.x * blockDim.x) {
    const int32_t len = a.lens[b], slot = a.slots[b];
    bool bad = slot >= 0 && (len < 0 || len > a.max_len || (int64_t)len > (int64_t)c.blocks * c.Tb ||
                             slot >= c.seqs);
    if (a.starts)
      bad = bad || a.starts[b] < 0 || a.starts[b + 1] > a.tokens || a.starts[b] > a.starts[b + 1];
    if (bad) atomicOr(c.status, kCacheArg);
  }
  const int64_t id = (int64_t)blockIdx.x * kWarps + warp;
  if (id >= (int64_t)a.tokens * a.q_heads) return;
  const int i = id / a.q_heads, h = id - (int64_t)i * a.q_heads, kvh = h / (a.q_heads / c.heads);
  const int b = sequence_of(a, i);
  if (b < 0) return;
  const int32_t len = a.lens[b], slot = a.slots[b];
  int lo = a.begins ? max(a.begins[b], 0) : 0, hi = len;
  {
    const int last = a.starts ? a.starts[b + 1] : i + 1;
    const int64_t at = (int64_t)len - (last - i);
    if (!a.full) hi = (int)min((int64_t)hi, at + 1);
    if (a.window) lo = (int)max((int64_t)lo, at - a.window + 1);
    if (at < 0 || slot < 0 || slot >= c.seqs || len > a.max_len ||
        (int64_t)len > (int64_t)c.blocks * c.Tb)
      hi = lo = 0;
  }
  const uint32_t *tab_k =
      c.table + ((int64_t)max(slot, 0) * c.rows + ((int64_t)a.layer * 2) * c.heads + kvh) * c.blocks;
  const uint32_t *tab_v = tab_k + (int64_t)c.heads * c.blocks;
  const uint16_t *q = a.q + i * a.qs + h * a.qhs;
  const float unit = c.scale ? c.scale[a.layer * c.heads + kvh] : 1.f;
  const float f = a.scale * kLog2e * unit;
  const int maps = a.lambda ? 2 : 1, width = c.D / maps;
  float res[8];
  for (int m = 0; m < maps; ++m) {
    float o[8], top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) o[k] = 0.f;
    for (int t0 = lo; t0 < hi; t0 += 32) {
      const int t = t0 + lane;
      float x = -INFINITY;
      const uint8_t *row_v = nullptr;
      if (t < hi) {
        const uint32_t pk = tab_k[t / c.Tb], pv = tab_v[t / c.Tb];
        if (pk < c.pages && pv < c.pages) {
          const uint32_t off = (uint32_t)(t % c.Tb) * c.row_bytes;
          const uint8_t *row_k = c.pool + (uint64_t)pk * c.page_bytes + off;
          row_v = c.pool + (uint64_t)pv * c.page_bytes + off;
          float s = 0.f;
          for (int d = m * width; d < (m + 1) * width; ++d)
            s += scalar(row_k, c.dtype, d) * __uint_as_float((uint32_t)q[d] << 16);
          x = s * f;
        } else {
          atomicOr(c.status, kCacheArg);
        }
      }
      float best = x;
      for (int s = 16; s; s >>= 1) best = fmaxf(best, __shfl_xor_sync(~0u, best, s));
      best = fmaxf(best, top);
      const float by = best == -INFINITY ? 1.f : exp2f(top - best);
      const float p = row_v ? (best == -INFINITY && x == best ? 0.f : exp2f(x - best)) : 0.f;
      top = best;
      sum = sum * by + p;
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] *= by;
      for (int l = 0; l < 32; ++l) {
        const uint8_t *r = reinterpret_cast<const uint8_t *>(
            __shfl_sync(~0u, reinterpret_cast<unsigned long long>(row_v), l));
        const float w = __shfl_sync(~0u, p, l);
        if (!r) continue;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k * 32 + lane < c.D) o[k] += w * scalar(r, c.dtype, k * 32 + lane);
      }
    }
    for (int s = 16; s; s >>= 1) sum += __shfl_xor_sync(~0u, sum, s);
    const float by = (sum == 0.f ? 0.f : unit / sum) * (m ? a.lambda[h] : 1.f);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (sum == 0.f) o[k] = 0.f;
      res[k] = m ? res[k] - o[k] * by : o[k] * by;
    }
    if (lane == 0 && a.lse)
      a.lse[id * maps + m] = top == -INFINITY ? top : (top + log2f(sum)) * kLn2;
  }
  float by = 1.f;
  if (a.norm) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k * 32 + lane < c.D) s += res[k] * res[k];
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(~0u, s, x);
    by = rsqrtf(s / c.D + a.eps);
    if (s == 0.f) by = 0.f;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int d = k * 32 + lane;
    if (d < c.D) {
      const __nv_bfloat16 v = __float2bfloat16_rn(res[k] * by * (a.norm ? a.norm[d] : 1.f));
      a.out[id * c.D + d] = *reinterpret_cast<const uint16_t *>(&v);
    }
  }
}

}  // namespace

size_t chunk_ws_bytes(const CacheView &, int32_t) { return 256; }

cudaError_t launch_chunk(const ChunkArgs &a, cudaStream_t st) {
  const int64_t blocks = ((int64_t)a.tokens * a.q_heads + kWarps - 1) / kWarps;
  return launch(k_chunk, dim3((unsigned)blocks), kWarps * 32, 0, st, a);
}

}  // namespace skv
