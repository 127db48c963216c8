// skv_cache_attend.cu -- attention of one new token per sequence: see skv_cache_attend.cuh.
#include "skv_cache_attend.cuh"

namespace skv {

size_t attend_ws_bytes(const CacheView &c, int32_t q_heads) { return ws_bytes(c, q_heads / c.heads); }

cudaError_t launch_attend(const AttendArgs &a, cudaStream_t st) {
  return a.c.dtype == 1 ? run_d<1, false>(a, st) : run_d<2, false>(a, st);
}

}  // namespace skv
