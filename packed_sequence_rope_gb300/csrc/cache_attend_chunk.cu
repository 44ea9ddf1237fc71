// Attention of chunks of new tokens over the paged cache, 16-bit pages: cache_attend_chunk.cuh.
#include "cache_attend_chunk.cuh"

namespace aa {

size_t chunk_workspace_bytes(const aa_cache_s* c, int num_seqs, int total_tokens, int table_width, int group, bool from_codes) {
  if (whole_units(table_width, __builtin_ctz((unsigned)c->cfg.page_size))) return 256;  // nothing is kept
  const size_t slots = slots_for(total_tokens, num_seqs, tiles_of(from_codes) * (128 / group)), ctas = ctas_for(c);
  return align256(ctas * 4 * 128 * c->cfg.head_dim * 4) + align256(ctas * 4 * 128 * 8) + align256(ctas * sizeof(Cut)) +
         align256(slots * sizeof(Unit)) + align256((slots + 1) * 8);
}

aa_status launch_attend_chunk(const aa_cache_s* c, const AttendParams& P, void* workspace, cudaStream_t s) {
  return launch_chunk<kFromPages>(c, P, c->k_map64, c->v_map64, 0, workspace, s);
}

}  // namespace aa
