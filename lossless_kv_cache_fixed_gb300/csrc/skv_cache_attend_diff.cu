// skv_cache_attend_diff.cu -- differential attention of one new token per sequence: see
// skv_cache_attend.cuh.
#include "skv_cache_attend.cuh"

namespace skv {

size_t attend_diff_ws_bytes(const CacheView &c, int32_t q_heads) {
  return ws_bytes(c, q_heads / c.heads * 2);
}

cudaError_t launch_attend_diff(const AttendArgs &a, cudaStream_t st) {
  return a.c.dtype == 1 ? run_d<1, true>(a, st) : run_d<2, true>(a, st);
}

}  // namespace skv
