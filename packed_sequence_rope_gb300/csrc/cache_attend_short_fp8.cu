// Attention of few new tokens over the paged cache, 8-bit pages: cache_attend_short.cuh.
#include "cache_attend_short.cuh"

namespace aa {

cudaError_t launch_attend_short_fp8(const aa_cache_s* c, const AttendParams& P, int max_q, void* workspace, cudaStream_t s) {
  return launch_short<true>(c, P, max_q, workspace, s);
}

}  // namespace aa
