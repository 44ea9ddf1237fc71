// Host side of the paged key/value cache: the handle, and which page belongs to
// which sequence.
//
// A page is free (reference count 0) or held by one or more sequences. Only
// the last page of a sequence can be partly filled, and only growing writes to
// it, so sharing is safe until a sequence grows into a shared, partly filled
// page: aa_cache_resize then gives it a copy of its own first. Every call
// works out its whole result before it changes anything, launches the copies it
// needs, and only then takes the result over.
#include <algorithm>
#include <cstdio>
#include <new>

#include "cache_internal.h"

namespace aa {

aa_status check_compute_cache(const aa_cache_s* c) {
  if (!c) return fail(AA_ERR_INVALID_ARG, "cache is NULL");
  if (c->host_only) return fail(AA_ERR_INVALID_ARG, "cache was created with host_only = 1");
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "device query");
  if (dev != c->device)
    return fail(AA_ERR_INVALID_ARG, "the cache lives on device " + std::to_string(c->device) + ", the current one is " +
                                        std::to_string(dev));
  return AA_OK;
}

aa_status check_batch(const aa_cache_s* c, const aa_cache_batch* b) {
  if (!b) return fail(AA_ERR_INVALID_ARG, "batch is NULL");
  if (b->num_seqs < 1 || b->num_seqs > (1 << 20)) return fail(AA_ERR_INVALID_ARG, "num_seqs must be in [1, 2^20]");
  if (b->total_tokens < 0 || b->total_tokens >= (1 << 30))
    return fail(AA_ERR_INVALID_ARG, "total_tokens must be in [0, 2^30)");
  if (b->table_width < 1 || (int64_t)b->table_width * c->cfg.page_size >= (1ll << 30))
    return fail(AA_ERR_INVALID_ARG, "table_width must be >= 1 and hold fewer than 2^30 positions");
  if (b->layer < 0 || b->layer >= c->cfg.num_layers) return fail(AA_ERR_INVALID_ARG, "layer must be in [0, num_layers)");
  for (const int32_t* p : {b->page_table, b->cu_q, b->kv_len})
    if (!p || (reinterpret_cast<uintptr_t>(p) & 3u))
      return fail(AA_ERR_INVALID_ARG, "page_table, cu_q and kv_len must be device pointers to int32");
  return AA_OK;
}

aa_status check_outside_pool(const aa_cache_s* c, const char* what, const void* out, size_t bytes) {
  const size_t pool = (size_t)c->cfg.num_layers * c->cfg.num_pages * c->page_elems() * 2;
  if (overlap(out, bytes, c->k_pages, pool) || overlap(out, bytes, c->v_pages, pool))
    return fail(AA_ERR_INVALID_ARG, std::string(what) + " overlaps the cache's pages");
  return AA_OK;
}

namespace {

aa_status check_seq(const aa_cache_s* c, int32_t s) {
  if (s < 0 || s >= (int32_t)c->seqs.size())
    return fail(AA_ERR_INVALID_ARG, "sequence " + std::to_string(s) + " must be in [0, max_seqs)");
  return AA_OK;
}

aa_status refuse_capture(cudaStream_t s, const char* what) {
  cudaStreamCaptureStatus st = cudaStreamCaptureStatusNone;
  cudaError_t e = cudaStreamIsCapturing(s, &st);
  if (e != cudaSuccess) return cuda_fail(e, "stream query");
  if (st != cudaStreamCaptureStatusNone)
    return fail(AA_ERR_INVALID_ARG, std::string(what) +
                                        " would copy pages while the stream is captured: its bookkeeping changes at once, "
                                        "the copy only in a replay");
  return AA_OK;
}

// Copies before the bookkeeping is taken over; a host-only handle has none.
aa_status copy_now(const aa_cache_s* c, const std::vector<PagePair>& pairs, cudaStream_t s, const char* what) {
  if (pairs.empty() || c->host_only) return AA_OK;
  aa_status st = check_compute_cache(c);
  if (st == AA_OK) st = refuse_capture(s, what);
  return st == AA_OK ? launch_copy_pages(c, pairs, s) : st;
}

aa_status resize(aa_cache_s* c, const int32_t* ids, const int32_t* lens, int32_t n, cudaStream_t stream) {
  if (n < 0 || (n > 0 && (!ids || !lens))) return fail(AA_ERR_INVALID_ARG, "seqs and lens must be host arrays of n");
  const int64_t ps = c->cfg.page_size;
  std::vector<char> named(c->seqs.size(), 0);
  for (int32_t i = 0; i < n; ++i) {
    aa_status st = check_seq(c, ids[i]);
    if (st != AA_OK) return st;
    if (named[ids[i]]) return fail(AA_ERR_INVALID_ARG, "sequence " + std::to_string(ids[i]) + " is named twice");
    named[ids[i]] = 1;
    if (lens[i] < 0 || lens[i] >= (1 << 30)) return fail(AA_ERR_INVALID_ARG, "lengths must be in [0, 2^30)");
  }
  std::vector<int32_t> refs = c->refs, free = c->free;
  std::vector<aa_cache_seq> after(n);
  bool returned = false;
  for (int32_t i = 0; i < n; ++i) {  // what shrinking gives back may serve the growing
    after[i] = c->seqs[ids[i]];
    const size_t keep = (size_t)((lens[i] + ps - 1) / ps);
    while (after[i].pages.size() > keep) {
      const int32_t p = after[i].pages.back();
      after[i].pages.pop_back();
      if (--refs[p] == 0) {
        free.push_back(p);
        returned = true;
      }
    }
  }
  // the lowest page is handed out first: pages stay at the front of the pool
  if (returned) std::sort(free.begin(), free.end(), std::greater<int32_t>());
  std::vector<PagePair> copies;
  for (int32_t i = 0; i < n; ++i) {
    aa_cache_seq& q = after[i];
    const int32_t len = std::min(q.len, lens[i]);  // tokens that are kept
    if (lens[i] > len && len % ps) {
      int32_t& last = q.pages[len / ps];
      if (refs[last] > 1) {
        if (free.empty()) return fail(AA_ERR_NO_MEMORY, "the cache has no free page left");
        const int32_t own = free.back();
        free.pop_back();
        copies.push_back({last, own});
        --refs[last];
        refs[own] = 1;
        last = own;
      }
    }
    const size_t need = (size_t)((lens[i] + ps - 1) / ps);
    while (q.pages.size() < need) {
      if (free.empty()) return fail(AA_ERR_NO_MEMORY, "the cache has no free page left");
      q.pages.push_back(free.back());
      refs[free.back()] = 1;
      free.pop_back();
    }
    q.len = lens[i];
  }
  aa_status st = copy_now(c, copies, stream, "aa_cache_resize");
  if (st != AA_OK) return st;
  for (int32_t i = 0; i < n; ++i) c->seqs[ids[i]] = std::move(after[i]);
  c->refs.swap(refs);
  c->free.swap(free);
  return AA_OK;
}

aa_status compact(aa_cache_s* c, cudaStream_t stream, int32_t* moved) {
  if (moved) *moved = 0;
  const int32_t P = c->cfg.num_pages;
  const int32_t used = P - (int32_t)c->free.size();
  std::vector<int32_t> to(P, -1);
  std::vector<PagePair> copies;
  int32_t hole = 0;
  for (int32_t p = used; p < P; ++p) {
    if (c->refs[p] == 0) continue;
    while (c->refs[hole] != 0) ++hole;  // as many holes below `used` as pages in use above it
    to[p] = hole;
    copies.push_back({p, hole});
    ++hole;
  }
  if (copies.empty()) return AA_OK;
  std::vector<int32_t> refs(P, 0), free;
  free.reserve(P - used);
  for (int32_t p = 0; p < P; ++p)
    if (c->refs[p]) refs[to[p] >= 0 ? to[p] : p] = c->refs[p];
  for (int32_t p = P - 1; p >= used; --p) free.push_back(p);
  aa_status st = copy_now(c, copies, stream, "aa_cache_compact");
  if (st != AA_OK) return st;
  for (aa_cache_seq& q : c->seqs)
    for (int32_t& p : q.pages)
      if (to[p] >= 0) p = to[p];
  c->refs.swap(refs);
  c->free.swap(free);
  if (moved) *moved = (int32_t)copies.size();
  return AA_OK;
}

aa_status copy_pages(const aa_cache_s* c, const int32_t* src, const int32_t* dst, int32_t n, cudaStream_t stream) {
  if (n < 0 || (n > 0 && (!src || !dst))) return fail(AA_ERR_INVALID_ARG, "src and dst must be host arrays of n");
  const int32_t P = c->cfg.num_pages;
  std::vector<PagePair> pairs;
  pairs.reserve(n);
  for (int32_t i = 0; i < n; ++i) {
    if (src[i] < 0 || src[i] >= P || dst[i] < 0 || dst[i] >= P)
      return fail(AA_ERR_INVALID_ARG, "pair " + std::to_string(i) + ": page numbers must be in [0, num_pages)");
    if (src[i] != dst[i]) pairs.push_back({src[i], dst[i]});
  }
  // a target twice, or a target that is also read: the copies run at once
  std::vector<int32_t> targets(pairs.size());
  for (size_t i = 0; i < pairs.size(); ++i) targets[i] = pairs[i].dst;
  std::sort(targets.begin(), targets.end());
  if (std::adjacent_find(targets.begin(), targets.end()) != targets.end())
    return fail(AA_ERR_INVALID_ARG, "a page is the target of two pairs");
  for (int32_t i = 0; i < n; ++i)
    if (std::binary_search(targets.begin(), targets.end(), src[i]))
      return fail(AA_ERR_INVALID_ARG, "page " + std::to_string(src[i]) + " is both a source and a target");
  return pairs.empty() ? AA_OK : launch_copy_pages(c, pairs, stream);
}

// C++ exceptions (an allocation that fails) end at the C boundary.
template <class Fn>
aa_status guarded(Fn fn) {
  try {
    return fn();
  } catch (const std::bad_alloc&) {
    return fail(AA_ERR_NO_MEMORY, "host allocation");
  } catch (const std::exception& e) {
    return fail(AA_ERR_INVALID_ARG, e.what());
  }
}

}  // namespace
}  // namespace aa

using namespace aa;

extern "C" aa_status aa_cache_create(const aa_cache_config* cfg, void* k_pages, void* v_pages, aa_cache_t* out) {
  if (!out) return fail(AA_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  if (!cfg) return fail(AA_ERR_INVALID_ARG, "config is NULL");
  if (cfg->head_dim != 64 && cfg->head_dim != 128) return fail(AA_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
  if (cfg->page_size != 16 && cfg->page_size != 32 && cfg->page_size != 64 && cfg->page_size != 128)
    return fail(AA_ERR_UNSUPPORTED, "page_size must be 16, 32, 64 or 128");
  if (cfg->num_layers < 1 || cfg->num_pages < 1 || cfg->num_kv_heads < 1)
    return fail(AA_ERR_INVALID_ARG, "num_layers, num_pages and num_kv_heads must be >= 1");
  if (cfg->max_seqs < 0 || cfg->max_seqs > (1 << 24)) return fail(AA_ERR_INVALID_ARG, "max_seqs must be in [0, 2^24]");
  double rows = (double)cfg->num_layers * cfg->num_pages * cfg->num_kv_heads * cfg->page_size;
  if (rows >= 2147483648.0)
    return fail(AA_ERR_INVALID_ARG, "num_layers * num_pages * Hkv * page_size must stay below 2^31");
  const bool host_only = cfg->host_only != 0;
  if (!host_only) {
    if (!k_pages || !v_pages || !aligned16(k_pages) || !aligned16(v_pages))
      return fail(AA_ERR_INVALID_ARG, "k_pages and v_pages must be 16-byte aligned device pointers");
    const size_t bytes = (size_t)rows * cfg->head_dim * 2;
    const uintptr_t a = reinterpret_cast<uintptr_t>(k_pages), b = reinterpret_cast<uintptr_t>(v_pages);
    if (a < b + bytes && b < a + bytes) return fail(AA_ERR_INVALID_ARG, "k_pages and v_pages overlap");
  }
  aa_cache_s* c = nullptr;
  aa_status st = guarded([&] {
    c = new aa_cache_s();
    c->cfg = *cfg;
    c->host_only = host_only;
    c->k_pages = k_pages;
    c->v_pages = v_pages;
    c->seqs.resize(cfg->max_seqs);
    if (cfg->max_seqs) {
      c->refs.assign(cfg->num_pages, 0);
      c->free.resize(cfg->num_pages);
      for (int32_t p = 0; p < cfg->num_pages; ++p) c->free[p] = cfg->num_pages - 1 - p;
    }
    return AA_OK;
  });
  if (st == AA_OK && !host_only) {
    cudaError_t e = cudaGetDevice(&c->device);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&c->num_sms, cudaDevAttrMultiProcessorCount, c->device);
    if (e == cudaSuccess) e = cudaMalloc((void**)&c->err, sizeof(int32_t));
    if (e == cudaSuccess) e = cudaMemset(c->err, 0, sizeof(int32_t));
    // the clear runs on the legacy stream: done before any call on another one
    if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);
    if (e != cudaSuccess) st = cuda_fail(e, "cache set-up");
    const int box = std::min(cfg->page_size, 64);
    if (st == AA_OK) st = make_pool_map(&c->k_map64, k_pages, (int64_t)rows, cfg->head_dim, box);
    if (st == AA_OK) st = make_pool_map(&c->v_map64, v_pages, (int64_t)rows, cfg->head_dim, box);
  }
  if (st != AA_OK) {
    if (c && c->err) cudaFree(c->err);
    delete c;
    return st;
  }
  *out = c;
  return AA_OK;
}

extern "C" aa_status aa_cache_destroy(aa_cache_t c) {
  if (!c) return AA_OK;
  if (!c->host_only) {
    int dev = -1;
    const bool moved = cudaGetDevice(&dev) == cudaSuccess && dev != c->device && cudaSetDevice(c->device) == cudaSuccess;
    cudaDeviceSynchronize();
    cudaFree(c->err);
    if (moved) cudaSetDevice(dev);
  }
  delete c;
  return AA_OK;
}

extern "C" aa_status aa_cache_resize(aa_cache_t c, const int32_t* seqs, const int32_t* lens, int32_t n,
                                     aa_stream_t stream) {
  if (!c) return fail(AA_ERR_INVALID_ARG, "cache is NULL");
  return guarded([&] { return resize(c, seqs, lens, n, reinterpret_cast<cudaStream_t>(stream)); });
}

extern "C" aa_status aa_cache_fork(aa_cache_t c, int32_t src, int32_t dst) {
  if (!c) return fail(AA_ERR_INVALID_ARG, "cache is NULL");
  return guarded([&] {
    aa_status st = check_seq(c, src);
    if (st == AA_OK) st = check_seq(c, dst);
    if (st != AA_OK) return st;
    if (c->seqs[dst].len != 0) return fail(AA_ERR_INVALID_ARG, "dst must be an empty sequence");
    if (src == dst) return AA_OK;  // an empty one
    aa_cache_seq both = c->seqs[src];
    for (int32_t p : both.pages) ++c->refs[p];
    c->seqs[dst] = std::move(both);
    return AA_OK;
  });
}

extern "C" aa_status aa_cache_compact(aa_cache_t c, aa_stream_t stream, int32_t* moved) {
  if (!c) return fail(AA_ERR_INVALID_ARG, "cache is NULL");
  if (c->seqs.empty()) return fail(AA_ERR_INVALID_ARG, "the cache keeps no sequences (max_seqs = 0)");
  return guarded([&] { return compact(c, reinterpret_cast<cudaStream_t>(stream), moved); });
}

extern "C" aa_status aa_cache_tables(aa_cache_t c, const int32_t* seqs, int32_t n, int32_t* table, int32_t width,
                                     int32_t* lens) {
  if (!c) return fail(AA_ERR_INVALID_ARG, "cache is NULL");
  if (n < 0 || (n > 0 && !seqs)) return fail(AA_ERR_INVALID_ARG, "seqs must be a host array of n");
  if (table && width < 1) return fail(AA_ERR_INVALID_ARG, "table_width must be >= 1");
  return guarded([&] {
    for (int32_t i = 0; i < n; ++i) {
      aa_status st = check_seq(c, seqs[i]);
      if (st != AA_OK) return st;
      if (table && c->seqs[seqs[i]].pages.size() > (size_t)width)
        return fail(AA_ERR_INVALID_ARG, "sequence " + std::to_string(seqs[i]) + " has " +
                                            std::to_string(c->seqs[seqs[i]].pages.size()) + " pages, table_width is " +
                                            std::to_string(width));
    }
    for (int32_t i = 0; i < n; ++i) {
      const aa_cache_seq& q = c->seqs[seqs[i]];
      if (table) {
        std::fill(table + (size_t)i * width, table + (size_t)(i + 1) * width, -1);
        std::copy(q.pages.begin(), q.pages.end(), table + (size_t)i * width);
      }
      if (lens) lens[i] = q.len;
    }
    return AA_OK;
  });
}

extern "C" aa_status aa_cache_stats(aa_cache_t c, int32_t* free_pages, int32_t* shared_pages, int32_t* longest) {
  if (!c) return fail(AA_ERR_INVALID_ARG, "cache is NULL");
  if (free_pages) *free_pages = (int32_t)c->free.size();
  if (shared_pages) *shared_pages = (int32_t)std::count_if(c->refs.begin(), c->refs.end(), [](int32_t r) { return r > 1; });
  if (longest) {
    *longest = 0;
    for (const aa_cache_seq& q : c->seqs) *longest = std::max(*longest, (int32_t)q.pages.size());
  }
  return AA_OK;
}

extern "C" aa_status aa_cache_copy_pages(aa_cache_t c, const int32_t* src, const int32_t* dst, int32_t n,
                                         aa_stream_t stream) {
  aa_status st = check_compute_cache(c);
  if (st != AA_OK) return st;
  return guarded([&] { return copy_pages(c, src, dst, n, reinterpret_cast<cudaStream_t>(stream)); });
}

extern "C" aa_status aa_cache_check_error(aa_cache_t c, aa_stream_t stream) {
  aa_status st = check_compute_cache(c);
  if (st != AA_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int32_t word = 0;
  cudaError_t e = cudaMemcpyAsync(&word, c->err, sizeof(word), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return cuda_fail(e, "reading the device error word");
  if (word == 0) return AA_OK;
  e = cudaMemsetAsync(c->err, 0, sizeof(int32_t), s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return cuda_fail(e, "clearing the device error word");
  if (word == kCacheBadPage) return fail(AA_ERR_INVALID_ARG, "a page table holds a page number outside the pool");
  if (word == kCacheBadPosition)
    return fail(AA_ERR_INVALID_ARG, "a position lies outside its page table (kv_len below the new tokens, or the table too narrow)");
  char buf[96];
  std::snprintf(buf, sizeof buf, "device-side wait timed out or launch check failed (site code %d)", (int)word);
  return fail(AA_ERR_TIMEOUT, buf);
}
