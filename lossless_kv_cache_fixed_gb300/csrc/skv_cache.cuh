// skv_cache.cuh -- what the paged-cache kernels (skv_cache_pages.cu,
// skv_cache_append.cu, skv_cache_attend.cu) and their C ABI (skv_cache_api.cu)
// share.  Not installed; not part of the ABI.
#pragma once
#include <cuda_runtime.h>
#include <cstdint>

namespace skv {

constexpr uint32_t kNoPage = 0xffffffffu;

// bits of the cache's status word
constexpr uint32_t kCacheArg = 1u;       // a slot, length or page out of range
constexpr uint32_t kCacheCapacity = 2u;  // not enough free pages

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
};
size_t attend_ws_bytes(const CacheView &c, int32_t q_heads);
cudaError_t launch_attend(const AttendArgs &a, cudaStream_t st);

}  // namespace skv
