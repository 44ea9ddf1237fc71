// Attention of few new tokens over the paged cache, 16-bit pages: cache_attend_short.cuh.
#include "cache_attend_short.cuh"

namespace aa {

size_t short_workspace_bytes(const aa_cache_s* c, int num_seqs, int total_tokens, int max_q, int table_width, int group) {
  const ShortShape f = shape_of(c, num_seqs, max_q, table_width, group);
  const size_t rows = (size_t)total_tokens * c->cfg.num_kv_heads * group;
  return f.splits == 1 ? 256 : align256(f.splits * rows * c->cfg.head_dim * 4) + align256(f.splits * rows * 8);
}

cudaError_t launch_attend_short(const aa_cache_s* c, const AttendParams& P, int max_q, void* workspace, cudaStream_t s) {
  return launch_short<false>(c, P, max_q, workspace, s);
}

}  // namespace aa
