// skv_cache_api.cu -- the C ABI of the paged cache declared in include/skv.h:
// argument checks, launches and the status word.
#include <cuda_runtime.h>

#include <climits>

#include "../../include/skv.h"
#include "skv_cache.cuh"

using namespace skv;

namespace {

constexpr size_t kAlign = 256;
constexpr int32_t kMaxList = 4096;  // sequences of one page operation
bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }
cudaStream_t stream_of(skv_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }
// An error is reported here, once: left with the runtime, the coder's next launch would
// report it as its own.
int status_of(cudaError_t e) {
  if (e == cudaSuccess) return SKV_OK;
  cudaGetLastError();
  return SKV_ERR_CUDA;
}

int make_view(const skv_cache *k, CacheView *out) {
  if (!k || k->flags) return SKV_ERR_ARG;
  if (k->dtype != SKV_BF16 && k->dtype != SKV_E4M3) return SKV_ERR_ARG;
  const int size = k->dtype == SKV_BF16 ? 2 : 1;
  if (k->layers <= 0 || k->heads <= 0 || k->head_dim <= 0 || k->page_tokens <= 0 ||
      k->max_seqs <= 0 || k->max_blocks <= 0)
    return SKV_ERR_ARG;
  if (k->head_dim * (int64_t)size % 16) return SKV_ERR_ARG;
  if (k->num_pages == 0 || k->num_pages >= SKV_NO_PAGE) return SKV_ERR_ARG;
  if (!k->pool || !k->table || !k->refs || !k->status) return SKV_ERR_ARG;
  if (!aligned(k->pool, 16) || !aligned(k->table, 16) || !aligned(k->refs, 16) ||
      !aligned(k->status, 4) || !aligned(k->scale, 4))
    return SKV_ERR_ARG;
  if (k->scale && k->dtype != SKV_E4M3) return SKV_ERR_ARG;
  const int64_t page = (int64_t)k->page_tokens * k->head_dim * size;
  const int64_t heads2 = 2ll * k->layers * k->heads;
  // a page's bytes, a sequence's table entries and its tokens are 32-bit in the kernels
  if (page > INT_MAX || heads2 > INT_MAX || heads2 * k->max_blocks > INT_MAX ||
      (int64_t)k->max_blocks * k->page_tokens > INT_MAX)
    return SKV_ERR_ARG;
  CacheView &c = *out;
  c.dtype = k->dtype;
  c.layers = k->layers;
  c.heads = k->heads;
  c.D = k->head_dim;
  c.Tb = k->page_tokens;
  c.seqs = k->max_seqs;
  c.blocks = k->max_blocks;
  c.rows = heads2;
  c.pages = k->num_pages;
  c.page_bytes = (uint32_t)page;
  c.row_bytes = (uint32_t)(k->head_dim * size);
  c.pool = static_cast<uint8_t *>(k->pool);
  c.table = k->table;
  c.refs = k->refs;
  c.status = k->status;
  c.scale = k->scale;
  return SKV_OK;
}

// A list of n sequences for the page operations.
int check_list(const int32_t *p, int32_t n) {
  if (n < 0 || n > kMaxList || (n && !p) || !aligned(p, 4)) return SKV_ERR_ARG;
  return SKV_OK;
}

int check_pages_ws(const CacheView &c, int32_t n, const void *ws, size_t bytes) {
  if (!ws || !aligned(ws, kAlign)) return SKV_ERR_ARG;
  return bytes < pages_ws(c.pages, n).total ? SKV_ERR_CAPACITY : SKV_OK;
}

// What skv_cache_attend_chunk and skv_cache_attend_diff share; diff is null for the former.
int attend_chunk(const skv_cache *cache, int32_t layer, const skv_chunk *k, const skv_diff *diff,
                 const void *q, int64_t q_stride, int64_t q_head_stride, int32_t q_heads,
                 float softmax_scale, void *out, float *lse, void *workspace,
                 size_t workspace_bytes, skv_stream_t stream) {
  ChunkArgs a;
  if (int rc = make_view(cache, &a.c)) return rc;
  const CacheView &c = a.c;
  if (!k || layer < 0 || layer >= c.layers || q_heads <= 0 || q_heads % c.heads || c.D > 256 ||
      (k->flags & ~SKV_CHUNK_FULL) || k->reserved || k->batch < 0 || k->tokens < 0 ||
      k->window < 0 || k->max_len < 0 || k->max_len > INT_MAX - 1024)
    return SKV_ERR_ARG;
  if (!k->starts && k->tokens != k->batch) return SKV_ERR_ARG;
  // The units of all rows are 32-bit: an item has max_len / 64 + 2 blocks at most and counts for up
  // to 8 more (kItemCost).  So are the rows of all heads, up to the end of the last item (256 rows).
  const int64_t group = q_heads / c.heads;
  const int64_t items = (k->tokens * group / 64 + k->batch) * c.heads;
  if (k->tokens * (int64_t)q_heads > INT_MAX - 512 || items > INT_MAX ||
      items * (k->max_len / 64 + 12) > INT_MAX ||
      (!k->starts && (int64_t)k->batch * q_heads * (k->max_len / 64 + 4) > INT_MAX))
    return SKV_ERR_ARG;
  a.lambda = a.norm = nullptr;
  a.eps = 0.f;
  if (diff) {
    if (!diff->lambda || !aligned(diff->lambda, 4) || !aligned(diff->norm, 4) || diff->reserved ||
        !(diff->eps >= 0.f) || c.D % 16)
      return SKV_ERR_ARG;
    a.lambda = diff->lambda;
    a.norm = diff->norm;
    a.eps = diff->eps;
  }
  if (!k->batch || !k->tokens) return SKV_OK;
  if (!k->slots || !k->lens || !q || !out || !aligned(k->slots, 4) || !aligned(k->lens, 4) ||
      !aligned(k->begins, 4) || !aligned(k->starts, 4) || !aligned(q, 16) || !aligned(out, 16) ||
      !aligned(lse, 4))
    return SKV_ERR_ARG;
  if (q_stride % 8 || q_head_stride % 8) return SKV_ERR_ARG;
  if (!workspace || !aligned(workspace, kAlign)) return SKV_ERR_ARG;
  const size_t need = chunk_ws_bytes(c, q_heads);
  if (!need) return status_of(cudaErrorInvalidDevice);
  if (workspace_bytes < need) return SKV_ERR_CAPACITY;
  a.slots = k->slots;
  a.lens = k->lens;
  a.begins = k->begins;
  a.starts = k->starts;
  a.q = static_cast<const uint16_t *>(q);
  a.qs = q_stride;
  a.qhs = q_head_stride;
  a.out = static_cast<uint16_t *>(out);
  a.lse = lse;
  a.ws = static_cast<uint8_t *>(workspace);
  a.scale = softmax_scale;
  a.batch = k->batch;
  a.tokens = k->tokens;
  a.q_heads = q_heads;
  a.layer = layer;
  a.max_len = k->max_len;
  a.window = k->window;
  a.full = (k->flags & SKV_CHUNK_FULL) ? 1 : 0;
  return status_of(launch_chunk(a, stream_of(stream)));
}

}  // namespace

extern "C" {

int skv_cache_init(const skv_cache *cache, skv_stream_t stream) {
  CacheView c;
  if (int rc = make_view(cache, &c)) return rc;
  cudaStream_t st = stream_of(stream);
  const size_t entries = (size_t)c.seqs * (size_t)c.rows * (size_t)c.blocks;
  cudaError_t e = cudaMemsetAsync(c.table, 0xff, sizeof(uint32_t) * entries, st);
  if (e == cudaSuccess) e = cudaMemsetAsync(c.refs, 0, sizeof(uint32_t) * (size_t)c.pages, st);
  if (e == cudaSuccess) e = cudaMemsetAsync(c.status, 0, sizeof(uint32_t), st);
  return status_of(e);
}

int skv_cache_status(const skv_cache *cache, skv_stream_t stream) {
  CacheView c;
  if (int rc = make_view(cache, &c)) return rc;
  cudaStream_t st = stream_of(stream);
  uint32_t v = 0;
  cudaError_t e = cudaMemcpyAsync(&v, c.status, sizeof(v), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaMemsetAsync(c.status, 0, sizeof(v), st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (int rc = status_of(e)) return rc;
  if (v & kCacheStuck) return SKV_ERR_CUDA;
  if (v & kCacheArg) return SKV_ERR_ARG;
  return v & kCacheCapacity ? SKV_ERR_CAPACITY : SKV_OK;
}

size_t skv_cache_workspace_bytes(const skv_cache *cache, int32_t n) {
  CacheView c;
  if (make_view(cache, &c) || n < 0 || n > kMaxList) return 0;
  return pages_ws(c.pages, n).total;
}

int skv_cache_reserve(const skv_cache *cache, const int32_t *slots, const int32_t *old_len,
                      const int32_t *new_len, int32_t n, void *workspace,
                      size_t workspace_bytes, skv_stream_t stream) {
  CacheView c;
  int rc = make_view(cache, &c);
  if (rc || (rc = check_list(slots, n)) || (rc = check_list(old_len, n)) ||
      (rc = check_list(new_len, n)) || (rc = check_pages_ws(c, n, workspace, workspace_bytes)))
    return rc;
  if (!n) return SKV_OK;
  return status_of(launch_reserve(c, slots, old_len, new_len, n, static_cast<uint8_t *>(workspace),
                                  stream_of(stream)));
}

int skv_cache_fork(const skv_cache *cache, const int32_t *parents, const int32_t *children,
                   const int32_t *lens, int32_t n, void *workspace, size_t workspace_bytes,
                   skv_stream_t stream) {
  CacheView c;
  int rc = make_view(cache, &c);
  if (rc || (rc = check_list(parents, n)) || (rc = check_list(children, n)) ||
      (rc = check_list(lens, n)) || (rc = check_pages_ws(c, n, workspace, workspace_bytes)))
    return rc;
  if (!n) return SKV_OK;
  if (c.rows * n > INT_MAX) return SKV_ERR_ARG;  // one block per (row, child)
  return status_of(launch_fork(c, parents, children, lens, n, static_cast<uint8_t *>(workspace),
                               stream_of(stream)));
}

int skv_cache_free(const skv_cache *cache, const int32_t *slots, int32_t n, skv_stream_t stream) {
  CacheView c;
  int rc = make_view(cache, &c);
  if (rc || (rc = check_list(slots, n))) return rc;
  if (!n) return SKV_OK;
  return status_of(launch_free(c, slots, n, stream_of(stream)));
}

int skv_cache_compact(const skv_cache *cache, uint32_t *table_out, uint32_t *refs_out,
                      void *workspace, size_t workspace_bytes, skv_stream_t stream) {
  CacheView c;
  int rc = make_view(cache, &c);
  if (rc) return rc;
  if (!table_out != !refs_out || !aligned(table_out, 16) || !aligned(refs_out, 16))
    return SKV_ERR_ARG;
  if (!table_out) {
    table_out = c.table;
    refs_out = c.refs;
  } else if ((table_out == c.table) != (refs_out == c.refs)) {
    return SKV_ERR_ARG;
  }
  if ((rc = check_pages_ws(c, 0, workspace, workspace_bytes))) return rc;
  return status_of(launch_compact(c, table_out, refs_out, static_cast<uint8_t *>(workspace),
                                  stream_of(stream)));
}

int skv_cache_copy_pages(const skv_cache *cache, const void *src_pool, uint64_t src_pages,
                         const uint32_t *src, void *dst_pool, uint64_t dst_pages,
                         const uint32_t *dst, int64_t n, skv_stream_t stream) {
  CacheView c;
  if (int rc = make_view(cache, &c)) return rc;
  if (n < 0 || n >= (int64_t)SKV_NO_PAGE || !aligned(src_pool, 16) || !aligned(dst_pool, 16))
    return SKV_ERR_ARG;
  if (!n) return SKV_OK;
  if (!src || !dst || !aligned(src, 4) || !aligned(dst, 4)) return SKV_ERR_ARG;
  if (!src_pool) {
    src_pool = c.pool;
    src_pages = c.pages;
  }
  if (!dst_pool) {
    dst_pool = c.pool;
    dst_pages = c.pages;
  }
  return status_of(launch_copy_pages(c, static_cast<const uint8_t *>(src_pool), src_pages, src,
                                     static_cast<uint8_t *>(dst_pool), dst_pages, dst, n,
                                     stream_of(stream)));
}

int skv_cache_append(const skv_cache *cache, int32_t layer, const skv_rope *rope,
                     const skv_tokens *tokens, const int32_t *slots, const int32_t *at,
                     const int32_t *positions, int32_t n, int32_t q_heads, void *q_out,
                     skv_stream_t stream) {
  AppendArgs a;
  if (int rc = make_view(cache, &a.c)) return rc;
  const CacheView &c = a.c;
  if (!tokens || layer < 0 || layer >= c.layers || n < 0 || q_heads < 0) return SKV_ERR_ARG;
  a.rotary = a.interleaved = 0;
  a.axes = 1;
  a.freqs = nullptr;
  a.axis = nullptr;
  if (rope) {
    if (rope->rotary_dim < 0 || rope->rotary_dim % 16 || rope->rotary_dim > c.D ||
        rope->rotary_dim > 1024 || rope->axes < 1 || rope->axes > 4 || rope->reserved ||
        (rope->flags & ~SKV_ROPE_INTERLEAVED))
      return SKV_ERR_ARG;
    if (rope->rotary_dim && (!rope->freqs || !aligned(rope->freqs, 8))) return SKV_ERR_ARG;
    a.rotary = rope->rotary_dim;
    a.axes = rope->axes;
    a.interleaved = (rope->flags & SKV_ROPE_INTERLEAVED) ? 1 : 0;
    a.freqs = rope->freqs;
    a.axis = rope->axis_of_pair;
  }
  if (!n) return SKV_OK;
  if (a.rotary && (!positions || !aligned(positions, 4))) return SKV_ERR_ARG;
  if (!slots || !at || !aligned(slots, 4) || !aligned(at, 4)) return SKV_ERR_ARG;
  if (!tokens->k || !tokens->v || !aligned(tokens->k, 16) || !aligned(tokens->v, 16))
    return SKV_ERR_ARG;
  if (q_heads && (!tokens->q || !q_out || !aligned(tokens->q, 16) || !aligned(q_out, 16)))
    return SKV_ERR_ARG;
  if ((q_heads && (tokens->q_stride % 8 || tokens->q_head_stride % 8)) || tokens->k_stride % 8 ||
      tokens->k_head_stride % 8 || tokens->v_stride % 8 || tokens->v_head_stride % 8)
    return SKV_ERR_ARG;
  // the kernel's index arithmetic; a token's rows and scales fit shared memory
  if (c.D > 4096 || (int64_t)q_heads + 2ll * c.heads > 8192) return SKV_ERR_ARG;
  a.q = static_cast<const uint16_t *>(tokens->q);
  a.k = static_cast<const uint16_t *>(tokens->k);
  a.v = static_cast<const uint16_t *>(tokens->v);
  a.qs = tokens->q_stride;
  a.qhs = tokens->q_head_stride;
  a.ks = tokens->k_stride;
  a.khs = tokens->k_head_stride;
  a.vs = tokens->v_stride;
  a.vhs = tokens->v_head_stride;
  a.slots = slots;
  a.at = at;
  a.positions = positions;
  a.q_out = static_cast<uint16_t *>(q_out);
  a.n = n;
  a.q_heads = q_heads;
  a.layer = layer;
  return status_of(launch_append(a, stream_of(stream)));
}

size_t skv_cache_attend_workspace_bytes(const skv_cache *cache, int32_t batch, int32_t q_heads) {
  CacheView c;
  if (make_view(cache, &c) || batch < 0 || q_heads <= 0 || q_heads % c.heads || c.D > 256) return 0;
  const size_t need = attend_ws_bytes(c, q_heads);
  if (!need) cudaGetLastError();  // no device
  return need;
}

int skv_cache_attend(const skv_cache *cache, int32_t layer, const int32_t *slots,
                     const int32_t *lens, const int32_t *begins, int32_t batch, const void *q,
                     int64_t q_stride, int64_t q_head_stride, int32_t q_heads,
                     float softmax_scale, int32_t max_len, void *out, float *lse,
                     void *workspace, size_t workspace_bytes, skv_stream_t stream) {
  AttendArgs a;
  if (int rc = make_view(cache, &a.c)) return rc;
  const CacheView &c = a.c;
  if (layer < 0 || layer >= c.layers || batch < 0 || q_heads <= 0 || q_heads % c.heads ||
      c.D > 256 || max_len < 0 || max_len > INT_MAX - 1024)
    return SKV_ERR_ARG;
  // one block of the join per (entry, query head); the units of all rows are 32-bit
  if ((int64_t)batch * q_heads > INT_MAX ||
      (int64_t)batch * q_heads * (max_len / 64 + 4) > INT_MAX)
    return SKV_ERR_ARG;
  if (!batch) return SKV_OK;
  if (!slots || !lens || !q || !out || !aligned(slots, 4) || !aligned(lens, 4) ||
      !aligned(begins, 4) || !aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4))
    return SKV_ERR_ARG;
  if (q_stride % 8 || q_head_stride % 8) return SKV_ERR_ARG;
  if (!workspace || !aligned(workspace, kAlign)) return SKV_ERR_ARG;
  const size_t need = attend_ws_bytes(c, q_heads);
  if (!need) return status_of(cudaErrorInvalidDevice);
  if (workspace_bytes < need) return SKV_ERR_CAPACITY;
  a.slots = slots;
  a.lens = lens;
  a.begins = begins;
  a.q = static_cast<const uint16_t *>(q);
  a.qs = q_stride;
  a.qhs = q_head_stride;
  a.out = static_cast<uint16_t *>(out);
  a.lse = lse;
  a.ws = static_cast<uint8_t *>(workspace);
  a.scale = softmax_scale;
  a.batch = batch;
  a.q_heads = q_heads;
  a.layer = layer;
  a.max_len = max_len;
  return status_of(launch_attend(a, stream_of(stream)));
}

size_t skv_cache_attend_chunk_workspace_bytes(const skv_cache *cache, int32_t q_heads) {
  CacheView c;
  if (make_view(cache, &c) || q_heads <= 0 || q_heads % c.heads || c.D > 256) return 0;
  const size_t need = chunk_ws_bytes(c, q_heads);
  if (!need) cudaGetLastError();  // no device
  return need;
}

int skv_cache_attend_chunk(const skv_cache *cache, int32_t layer, const skv_chunk *chunk,
                           const void *q, int64_t q_stride, int64_t q_head_stride,
                           int32_t q_heads, float softmax_scale, void *out, float *lse,
                           void *workspace, size_t workspace_bytes, skv_stream_t stream) {
  return attend_chunk(cache, layer, chunk, nullptr, q, q_stride, q_head_stride, q_heads,
                      softmax_scale, out, lse, workspace, workspace_bytes, stream);
}

int skv_cache_attend_diff(const skv_cache *cache, int32_t layer, const skv_chunk *chunk,
                          const skv_diff *diff, const void *q, int64_t q_stride,
                          int64_t q_head_stride, int32_t q_heads, float softmax_scale,
                          void *out, float *lse, void *workspace, size_t workspace_bytes,
                          skv_stream_t stream) {
  if (!diff) return SKV_ERR_ARG;
  return attend_chunk(cache, layer, chunk, diff, q, q_stride, q_head_stride, q_heads,
                      softmax_scale, out, lse, workspace, workspace_bytes, stream);
}

}  // extern "C"
