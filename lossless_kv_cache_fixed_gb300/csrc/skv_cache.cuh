// skv_cache.cuh -- what the paged-cache kernels (skv_cache_pages.cu,
// skv_cache_append.cu, skv_cache_attend*, skv_cache_chunk.cu) and their C ABI
// (skv_cache_api.cu) share.  Not installed; not part of the ABI.
#pragma once
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace skv {

constexpr uint32_t kNoPage = 0xffffffffu;

// bits of the cache's status word
constexpr uint32_t kCacheArg = 1u;       // a slot, length or page out of range
constexpr uint32_t kCacheCapacity = 2u;  // not enough free pages
constexpr uint32_t kCacheStuck = 4u;     // a kernel gave up waiting for a part of itself

// The cache as the kernels see it.  Row r of a sequence is (layer*2 + kv)*heads
// + head; its table entries are at (slot*rows + r)*blocks.
struct CacheView {
  int32_t dtype, layers, heads, D, Tb, seqs, blocks;
  int64_t rows;        // layers * 2 * heads
  uint64_t pages;
  uint32_t page_bytes;  // Tb * D * scalar size, a multiple of 16
  uint32_t row_bytes;   // D * scalar size, a multiple of 16
  uint8_t *pool;
  uint32_t *table;
  uint32_t *refs;
  uint32_t *status;
  const float *scale;
};

// 16 bytes of a streaming copy: read once, written once.
__device__ __forceinline__ uint4 ld_stream(const void *p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
__device__ __forceinline__ void st_stream(void *p, const uint4 &v) {
  asm volatile("st.global.L1::no_allocate.v4.u32 [%0], {%1,%2,%3,%4};" ::"l"(p), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
}

// Every kernel of the paged cache is launched while the one before it in the stream may
// still run (programmatic dependent launch), which hides its launch, and calls begin()
// (k_attend and k_attend_join: their own order of the two) before its first read: it
// returns when all of the earlier work is complete.
__device__ __forceinline__ void begin() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
template <typename... P, typename... A>
cudaError_t launch(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st,
                   A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

// ---- launchers (each enqueues on the stream and returns the launch status) ----

// Workspace of the page operations, byte offsets (see skv_cache_pages.cu).
struct PagesWs {
  size_t go, base, need, bad, counts, list, rank, top_refs, total;
};
PagesWs pages_ws(uint64_t pages, int64_t n);

cudaError_t launch_reserve(const CacheView &c, const int32_t *slots, const int32_t *old_len,
                           const int32_t *new_len, int32_t n, uint8_t *ws, cudaStream_t st);
cudaError_t launch_fork(const CacheView &c, const int32_t *parents, const int32_t *children,
                        const int32_t *lens, int32_t n, uint8_t *ws, cudaStream_t st);
cudaError_t launch_free(const CacheView &c, const int32_t *slots, int32_t n, cudaStream_t st);
cudaError_t launch_compact(const CacheView &c, uint32_t *table_out, uint32_t *refs_out,
                           uint8_t *ws, cudaStream_t st);
cudaError_t launch_copy_pages(const CacheView &c, const uint8_t *src_pool, uint64_t src_pages,
                              const uint32_t *src, uint8_t *dst_pool, uint64_t dst_pages,
                              const uint32_t *dst, int64_t n, cudaStream_t st);

struct AppendArgs {
  CacheView c;
  const uint16_t *q, *k, *v;
  int64_t qs, qhs, ks, khs, vs, vhs;  // strides in elements
  const int32_t *slots, *at, *positions;
  uint16_t *q_out;
  const double *freqs;
  const uint8_t *axis;
  int32_t n, q_heads, layer, rotary, axes, interleaved;
};
cudaError_t launch_append(const AppendArgs &a, cudaStream_t st);

struct AttendArgs {
  CacheView c;
  const int32_t *slots, *lens, *begins;
  const uint16_t *q;
  int64_t qs, qhs;
  uint16_t *out;
  float *lse;
  uint8_t *ws;
  float scale;
  int32_t batch, q_heads, layer, max_len;
  int32_t window = 0;                               // tokens that are seen; 0: all
  const float *lambda = nullptr, *norm = nullptr;   // differential attention
  float eps = 0.f;
};
size_t attend_ws_bytes(const CacheView &c, int32_t q_heads);
cudaError_t launch_attend(const AttendArgs &a, cudaStream_t st);
size_t attend_diff_ws_bytes(const CacheView &c, int32_t q_heads);
cudaError_t launch_attend_diff(const AttendArgs &a, cudaStream_t st);

// Division by a number that the host knows, of numbers below 2^31 (Granlund and Montgomery:
// n / d = (n + floor(n m / 2^32)) >> s with s = ceil(log2 d), m = floor(2^32 (2^s - d) / d) + 1).
struct Div {
  uint32_t mul = 1, shift = 0;
  Div() = default;
  explicit Div(uint32_t d) {
    while ((1ull << shift) < d) ++shift;
    mul = (uint32_t)(((1ull << 32) * ((1ull << shift) - d)) / d + 1);
  }
  __device__ __forceinline__ int of(int n) const {
    return (int)(((uint32_t)n + __umulhi((uint32_t)n, mul)) >> shift);
  }
};

// four e4m3 codes to halves: the two in the low 16 bits, the two in the high
__device__ __forceinline__ void e4m3x4(uint32_t v, uint32_t &lo, uint32_t &hi) {
  asm("{.reg .b16 a, b; mov.b32 {a, b}, %2; cvt.rn.f16x2.e4m3x2 %0, a; cvt.rn.f16x2.e4m3x2 %1, b;}"
      : "=r"(lo), "=r"(hi)
      : "r"(v));
}
// q . k over n channels, a multiple of 8 (e4m3 codes or bf16): scores that a matrix product did not give
template <int ES>
static __device__ __noinline__ float half_score(const uint16_t *q, const uint8_t *k, int n) {
  float y = 0.f;
#pragma unroll 1
  for (int d = 0; d < n; d += 2) {
    const uint32_t w = *reinterpret_cast<const uint32_t *>(q + d);
    uint32_t u;
    if (ES == 2) {
      u = *reinterpret_cast<const uint32_t *>(k + d * 2);
      y = fmaf(__uint_as_float(w << 16), __uint_as_float(u << 16), y);
      y = fmaf(__uint_as_float(w & 0xffff0000u), __uint_as_float(u & 0xffff0000u), y);
    } else {
      uint32_t none;
      e4m3x4(*reinterpret_cast<const uint16_t *>(k + d), u, none);
      const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&u));
      y = fmaf(__uint_as_float(w << 16), v.x, y);
      y = fmaf(__uint_as_float(w & 0xffff0000u), v.y, y);
    }
  }
  return y;
}

// The mean square of a result's channels, whatever power of two they lie at: the squares of
// numbers beyond 2^64 or below 2^-63 leave the range of a float, so two more sums are taken of the
// channels times 2^-70 and 2^70.
struct Squares {
  float q = 0.f, big = 0.f, tiny = 0.f;
  // whether a sum of squares does without the other two (where eps is 2^-60 or more, squares
  // below 2^-80 do not count next to it)
  static __device__ __forceinline__ bool enough(float q, float eps) {
    return q <= 0x1p100f && (q >= 0x1p-80f || eps >= 0x1p-60f);
  }
  __device__ __forceinline__ void add(float x) {
    const float b = x * 0x1p-70f, t = x * 0x1p70f;
    q = fmaf(x, x, q);
    big = fmaf(b, b, big);
    tiny = fmaf(t, t, tiny);
  }
  __device__ __forceinline__ void add(const Squares &o) {
    q += o.q;
    big += o.big;
    tiny += o.tiny;
  }
  __device__ __forceinline__ void add_lanes() {
    for (int s = 16; s; s >>= 1) {
      q += __shfl_xor_sync(~0u, q, s);
      big += __shfl_xor_sync(~0u, big, s);
      tiny += __shfl_xor_sync(~0u, tiny, s);
    }
  }
  // 1 / sqrt(mean + eps), 0 for a result of zeros
  __device__ __forceinline__ float inverse(int n, float eps) const {
    if (enough(q, eps)) return rsqrtf(q / n + eps);
    if (big >= 0x1p-60f) return rsqrtf(big / n + eps * 0x1p-70f * 0x1p-70f) * 0x1p-70f;
    if (tiny == 0.f) return 0.f;
    // (eps is below 2^-60, or the sum is NaN)
    return rsqrtf(tiny / n + eps * 0x1p70f * 0x1p70f) * 0x1p70f;
  }
};

struct ChunkArgs {
  CacheView c;
  Div by_group, by_page;  // query heads of a kv head; tokens of a page
  const int32_t *slots, *lens, *begins, *starts;
  const uint16_t *q;
  int64_t qs, qhs;
  uint16_t *out;
  float *lse;
  const float *lambda, *norm;  // differential attention: lambda is not null
  uint8_t *ws;
  float scale, eps;
  int32_t batch, tokens, q_heads, layer, max_len, window, full;
  long long patience;  // clocks that a wait may take
};
size_t chunk_ws_bytes(const CacheView &c, int32_t q_heads);
cudaError_t launch_chunk(const ChunkArgs &a, cudaStream_t st);

}  // namespace skv
