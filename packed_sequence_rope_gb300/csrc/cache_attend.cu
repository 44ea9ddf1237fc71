// Attention of new tokens over the paged cache (aa_cache_attend).
//
// For new token i of sequence b, at position p = kv_len - n_b + i, and query
// head h ("When Precision Meets Position", architecture page §3.4
// "AnchorAttention: The Shared Anchor Design", "Mask construction"):
//   visible keys: [max(key_lo, 0), p], and key 0 with the anchor (p >= 0)
//   O_i = sum_j softmax_j(scale * q_i . k_j) v_j, LSE_i = ln sum_j exp(...)
// in one pass with the running maximum and sum of the softmax. This file checks the
// arguments and chooses between cache_attend_short.cu (few rows per sequence: the
// keys are read once, HBM-bound) and cache_attend_chunk.cu (tcgen05 products).
#include <algorithm>
#include <cmath>

#include "cache_attend.cuh"

using namespace aa;

// Few rows: the kernel for them, whose row tile holds kShortRows. Its warps share a
// 16-row tile's keys at 16 rows, but at 33 to 64 take 16 rows each and all keys,
// which at D = 128 costs more than HBM does; there the other kernel takes the calls
// with work for every SM, and those of short contexts. Up to 32 rows stay here over
// short contexts too, where many sequences would be faster there (first line). 64
// units and kWholeKeys are where the two met on 152 SMs. Measured, microseconds
// of this one / the other, 8 kv heads of 128, group 4:
//   rows, sequences   300 keys     2048        16384
//   32, 1             10.1 / 10.5  9.6 / 16.7  20.6 / 27.1
//   32, 42            31.8 / 27.2  81.1 / 89.1 457 / 534
//   64, 1             15.1 / 10.7  14.2 / 17.3 29.2 / 28.8
//   64, 8             15.1 / 11.6  33.9 / 29.6 131 / 118
//   64, 42            49.1 / 27.7  117 / 92.0  621 / 537
// With D = 64: 64 rows of 42 sequences 24.4 / 25.0, 56.9 / 76.2 and 314 / 469.
static bool takes_short(const aa_cache_s* c, int num_seqs, int max_q, int table_width, int group) {
  const int64_t rows = (int64_t)std::max(max_q, 1) * group;
  if (rows <= 32 || c->cfg.head_dim == 64) return rows <= kShortRows;
  return rows <= kShortRows && (int64_t)table_width * c->cfg.page_size > kWholeKeys &&
         (int64_t)num_seqs * c->cfg.num_kv_heads < 64;
}

extern "C" size_t aa_cache_attend_workspace_bytes(aa_cache_t c, int32_t num_seqs, int32_t total_tokens, int32_t max_q,
                                                  int32_t table_width, int32_t q_heads) {
  if (!c || num_seqs < 1 || total_tokens < 0 || max_q < 0 || table_width < 1 || q_heads < 1) return 0;
  const int Hkv = c->cfg.num_kv_heads;
  if (c->host_only || q_heads % Hkv || q_heads / Hkv > 64) return 0;
  if (total_tokens >= (1 << 30) || num_seqs > (1 << 20) || (int64_t)table_width * c->cfg.page_size >= (1ll << 30)) return 0;
  if (takes_short(c, num_seqs, max_q, table_width, q_heads / Hkv))
    return short_workspace_bytes(c, num_seqs, total_tokens, max_q, table_width, q_heads / Hkv);
  return chunk_workspace_bytes(c, num_seqs, total_tokens, table_width, q_heads / Hkv);
}

extern "C" aa_status aa_cache_attend(aa_cache_t c, const aa_cache_batch* batch, const void* q, int64_t q_stride,
                                     int32_t q_heads, int32_t max_q, const int32_t* key_lo, int32_t anchor,
                                     float softmax_scale, void* o, float* lse, void* workspace, size_t workspace_bytes,
                                     aa_stream_t stream) {
  aa_status st = check_compute_cache(c);
  if (st != AA_OK) return st;
  if ((st = check_batch(c, batch)) != AA_OK) return st;
  const int D = c->cfg.head_dim, Hkv = c->cfg.num_kv_heads, T = batch->total_tokens;
  if (q_heads < 1 || q_heads % Hkv || q_heads / Hkv > 64)
    return fail(AA_ERR_INVALID_ARG, "q_heads must be a multiple of Hkv, at most 64 per kv head");
  if ((int64_t)batch->num_seqs * Hkv >= (1 << 27))
    return fail(AA_ERR_INVALID_ARG, "num_seqs * Hkv must stay below 2^27");
  if (max_q < 0) return fail(AA_ERR_INVALID_ARG, "max_q must be >= 0");
  if ((int64_t)q_heads * T >= (1ll << 31)) return fail(AA_ERR_INVALID_ARG, "q_heads * total_tokens must stay below 2^31");
  if (!std::isfinite(softmax_scale)) return fail(AA_ERR_INVALID_ARG, "softmax_scale is not finite");
  if (T == 0) return AA_OK;
  if ((st = check_rows("q", q, q_stride, q_heads, D)) != AA_OK) return st;
  if (!o || !aligned16(o)) return fail(AA_ERR_INVALID_ARG, "o must be a 16-byte aligned device pointer");
  if ((reinterpret_cast<uintptr_t>(lse) & 3u) || (reinterpret_cast<uintptr_t>(key_lo) & 3u))
    return fail(AA_ERR_INVALID_ARG, "lse and key_lo must be 4-byte aligned device pointers");
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return fail(AA_ERR_INVALID_ARG, "workspace must be a 256-byte aligned device pointer");
  const size_t used = aa_cache_attend_workspace_bytes(c, batch->num_seqs, T, max_q, batch->table_width, q_heads);
  if (workspace_bytes < used)
    return fail(AA_ERR_INVALID_ARG, "workspace is smaller than aa_cache_attend_workspace_bytes()");
  // what the call writes lies apart: the kernels' index ranges come from the workspace
  const struct {
    const char* name;
    const void* at;
    size_t bytes;
  } written[] = {{"o", o, (size_t)T * q_heads * D * 2},
                 {"lse", lse, (size_t)T * q_heads * 4},
                 {"the workspace", workspace, used > 256 ? used : 0}},  // 256: none is in use
    read[] = {{"q", q, rows_span(T, q_stride, q_heads, D)},
              {"key_lo", key_lo, (size_t)T * 4},
              {"page_table", batch->page_table, (size_t)batch->num_seqs * batch->table_width * 4},
              {"cu_q", batch->cu_q, ((size_t)batch->num_seqs + 1) * 4},
              {"kv_len", batch->kv_len, (size_t)batch->num_seqs * 4}};
  for (const auto& x : written) {
    if (!x.at || !x.bytes) continue;
    if ((st = check_outside_pool(c, x.name, x.at, x.bytes)) != AA_OK) return st;
    auto apart = [&](const auto& y) {
      return !y.at || !y.bytes || &y == &x || !overlap(x.at, x.bytes, y.at, y.bytes);
    };
    for (const auto& y : written)
      if (!apart(y)) return fail(AA_ERR_INVALID_ARG, std::string(x.name) + " overlaps " + y.name);
    for (const auto& y : read)
      if (!apart(y)) return fail(AA_ERR_INVALID_ARG, std::string(x.name) + " overlaps " + y.name);
  }
  AttendParams P;
  P.batch = batch_params(c, batch);
  P.q = static_cast<const __nv_bfloat16*>(q);
  P.o = static_cast<__nv_bfloat16*>(o);
  P.lse = lse;
  P.key_lo = key_lo;
  P.q_stride = q_stride;
  P.Hq = q_heads;
  P.group = q_heads / Hkv;
  P.anchor = anchor != 0;
  P.page_shift = __builtin_ctz((unsigned)c->cfg.page_size);
  P.scale_log2 = (float)((softmax_scale > 0.f ? (double)softmax_scale : 1.0 / std::sqrt((double)D)) * 1.4426950408889634);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (!takes_short(c, batch->num_seqs, max_q, batch->table_width, P.group)) return launch_attend_chunk(c, P, workspace, s);
  cudaError_t e = launch_attend_short(c, P, max_q, workspace, s);
  return e == cudaSuccess ? AA_OK : cuda_fail(e, "attend_short_kernel launch");
}
