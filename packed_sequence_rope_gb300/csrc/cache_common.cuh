// Device helpers shared by the paged cache's kernels: which sequence a row
// belongs to, and where its positions lie in the pool.
#pragma once

#include "cache_internal.h"
#include "kcommon.cuh"

namespace aa {

// The sequence of row t: the last b with cu_q[b] <= t, for cu_q[0] <= t (a
// whole warp asks for one row; sequences without new tokens are passed over).
// 33-ary search: one load latency for up to 32 sequences, two for 1056.
__device__ __forceinline__ int warp_find_seq(const int32_t* __restrict__ cu_q, int num_seqs, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = num_seqs;  // the answer lies in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 32) / 33;  // lanes look at the last entry of 32 of the 33 parts
    const int at = (lane + 1) * step;
    const bool le = at < n && __ldg(cu_q + lo + at) <= t;
    const int parts = __popc(__ballot_sync(0xffffffffu, le));  // cu_q does not decrease
    lo += parts * step;
    n = min(step, n - parts * step);
  }
  return lo;
}

// One batch as the kernels see it.
struct BatchParams {
  const int32_t *table, *cu_q, *kv_len;
  int B, W, T;
  int num_pages, Hkv;
  int64_t layer_page0;  // layer * num_pages
  int32_t* err;
};

inline BatchParams batch_params(const aa_cache_s* c, const aa_cache_batch* b) {
  BatchParams p;
  p.table = b->page_table;
  p.cu_q = b->cu_q;
  p.kv_len = b->kv_len;
  p.B = b->num_seqs;
  p.W = b->table_width;
  p.T = b->total_tokens;
  p.num_pages = c->cfg.num_pages;
  p.Hkv = c->cfg.num_kv_heads;
  p.layer_page0 = (int64_t)b->layer * c->cfg.num_pages;
  p.err = c->err;
  return p;
}

}  // namespace aa
