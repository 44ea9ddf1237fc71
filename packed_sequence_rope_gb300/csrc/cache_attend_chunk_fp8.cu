// Attention of chunks of new tokens over the paged cache, 8-bit pages: cache_attend_chunk.cuh.
#include "cache_attend_chunk.cuh"

namespace aa {

aa_status launch_attend_chunk_fp8(const aa_cache_s* c, const AttendParams& P, void* workspace, cudaStream_t s) {
  return launch_chunk<kFromCodes>(c, P, c->k_map64, c->v_map64, 0, workspace, s);
}

}  // namespace aa
