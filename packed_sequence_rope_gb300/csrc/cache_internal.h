// Declarations shared by the paged cache's host bookkeeping and its kernels.
#pragma once

#include <cuda.h>

#include "aa_internal.h"

// One sequence of the host bookkeeping: its length and the pages of its
// positions in order.
struct aa_cache_seq {
  int32_t len = 0;
  std::vector<int32_t> pages;
};

struct aa_cache_s {
  aa_cache_config cfg;
  bool host_only = false;
  int device = 0, num_sms = 0;
  void *k_pages = nullptr, *v_pages = nullptr;
  // 8-bit pages: a byte per token and kv head, [num_layers, num_pages, Hkv, page_size]; else NULL
  uint8_t *k_scales = nullptr, *v_scales = nullptr;
  int32_t* err = nullptr;        // device error word (0 = ok)
  // the pool as [num_layers * num_pages * Hkv * page_size, D] rows, in boxes of
  // a page's rows (at most 64) by 64 channels (8-bit pages: by all channels)
  CUtensorMap k_map64, v_map64;
  std::vector<aa_cache_seq> seqs;
  std::vector<int32_t> refs;     // [num_pages] sequences holding the page
  std::vector<int32_t> free;     // pages with refs == 0, the lowest last
  bool fp8() const { return k_scales != nullptr; }
  int64_t page_bytes() const { return page_elems() * (fp8() ? 1 : 2); }
  int64_t page_elems() const { return (int64_t)cfg.num_kv_heads * cfg.page_size * cfg.head_dim; }
};

namespace aa {

// Error word of the cache's device calls.
constexpr int32_t kCacheBadPage = 1, kCacheBadPosition = 2, kCacheBadTree = 3, kCacheBadPath = 4;

// Words of 64 new tokens in a row of a drafted tree's masks, at most.
constexpr int kMaxTreeWords = 1 << 14;

// Refuses NULL, host-only handles and a current device that is not the handle's.
aa_status check_compute_cache(const aa_cache_s* c);
aa_status check_batch(const aa_cache_s* c, const aa_cache_batch* b);
// Refuses an output that lies in the pool.
aa_status check_outside_pool(const aa_cache_s* c, const char* what, const void* out, size_t bytes);

// One (source, target) pair of a page copy.
struct PagePair {
  int32_t src, dst;
};
aa_status launch_copy_pages(const aa_cache_s* c, const std::vector<PagePair>& pairs, cudaStream_t s);

// Tensor map over the pool's rows [rows, D], box {64, box_rows}, 128-byte
// swizzle; for 8-bit pages box {D, box_rows}, a swizzle of D bytes (rope.cu).
aa_status make_pool_map(CUtensorMap* m, const void* base, int64_t rows, int D, int box_rows);
aa_status make_pool_map_fp8(CUtensorMap* m, const void* base, int64_t rows, int D, int box_rows);

// Tensor map over q [T, Hkv, group, D] with `stride` elements from token to
// token, box {64, group, 1, tokens} (rope.cu).
aa_status make_query_map(CUtensorMap* m, const void* q, int T, int64_t stride, int Hkv, int group, int D, int tokens);

// Checks shared with aa_rope_axes_apply (rope_axes.cu).
size_t rows_span(int64_t T, int64_t stride, int H, int D);
bool overlap(const void* a, size_t na, const void* b, size_t nb);
aa_status check_rows(const char* what, const void* x, int64_t stride, int H, int D);
aa_status check_turned(const char* what, const void* x, int64_t stride, const void* out, int H, int D, int64_t T);

}  // namespace aa
