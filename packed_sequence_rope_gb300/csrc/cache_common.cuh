// Device helpers shared by the paged cache's kernels: which sequence a row
// belongs to, and where its positions lie in the pool.
#pragma once

#include "cache_internal.h"
#include "kcommon.cuh"

namespace aa {

// The last i in [0, n) for which `holds` does, where it holds for 0 and, from
// some i on, no longer. A whole warp asks; 33-ary search: one load latency for
// up to 33 entries, two for 1089.
template <class Holds>
__device__ __forceinline__ int warp_last(int n, Holds holds) {
  const int lane = threadIdx.x & 31;
  int lo = 0;  // the answer lies in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 32) / 33;  // lanes look at the first entry of all of the 33 parts but one
    const int at = (lane + 1) * step;
    const bool yes = at < n && holds(lo + at);
    const int parts = __popc(__ballot_sync(0xffffffffu, yes));
    lo += parts * step;
    n = min(step, n - parts * step);
  }
  return lo;
}

// The sequence of row t >= cu_q[0] (sequences without new tokens are passed over).
__device__ __forceinline__ int warp_find_seq(const int32_t* __restrict__ cu_q, int num_seqs, int t) {
  return warp_last(num_seqs, [&](int i) { return __ldg(cu_q + i) <= t; });
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
