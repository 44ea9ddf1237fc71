// Drafted trees: from each drafted token's parent the masks and positions that
// aa_cache_attend_tree and the rotation take (aa_cache_tree_masks), and moving the
// accepted tokens up behind the cached ones (aa_cache_accept).
#include "cache_common.cuh"

namespace aa {
namespace {

constexpr int kThreads = 256;

struct MaskParams {
  const int32_t *parents, *cu_q, *kv_len;
  uint64_t* mask;
  int32_t *pos, *err;
  int B, T, words;
};

// One thread per new token i walks up its ancestors, whose indices fall: each word of
// its row is complete when the walk leaves it.
__global__ void __launch_bounds__(kThreads) tree_masks_kernel(const MaskParams P) {
  const int t0 = (int)blockIdx.x * kThreads + (int)(threadIdx.x & ~31u), t = t0 + (int)(threadIdx.x & 31);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (t0 >= P.T) return;
  // the sequence of the warp's first token; later ones follow from it
  int seq = warp_find_seq(P.cu_q, P.B, t0);
  if (t >= P.T || t < __ldg(P.cu_q) || t >= __ldg(P.cu_q + P.B)) return;
  while (seq + 1 < P.B && t >= __ldg(P.cu_q + seq + 1)) ++seq;
  const int q0 = __ldg(P.cu_q + seq), n = __ldg(P.cu_q + seq + 1) - q0, i = t - q0;
  if (q0 < 0 || i < 0 || i >= n) return;  // a cu_q that is none
  uint64_t* row = P.mask + (int64_t)t * P.words;
  int w = P.words - 1, depth = 0;
  uint64_t bits = 0;
  for (int at = i;;) {
    const int in = at >> 6;
    for (; w > in; --w) {
      row[w] = bits;
      bits = 0;
    }
    if (in == w) bits |= 1ull << (at & 63);  // else past the masks' width
    int up = __ldg(P.parents + q0 + at);
    if (up < -1 || up >= at) {
      atomicCAS(P.err, 0, kCacheBadTree);
      up = -1;
    }
    if (up < 0) break;
    at = up;
    ++depth;
  }
  for (; w >= 0; --w) {
    row[w] = bits;
    bits = 0;
  }
  P.pos[t] = __ldg(P.kv_len + seq) - n + depth;
}

struct AcceptParams {
  BatchParams batch;
  const int32_t* path;
  uint8_t *k_pages, *v_pages, *k_scales, *v_scales;
  int width, page_shift, row_shift;  // row_shift: log2 of a row's 16-byte chunks
};

constexpr int kMoves = 2;  // 16-byte chunks of keys, and of values, that a thread moves at a time

// One block per layer and sequence. Row path[i] goes to row i of the new
// tokens. Since the path ascends, path[i] >= i: a row is overwritten only after it has
// been read if the rows are moved in order, a batch at a time, all loads of a batch
// before its stores.
// The warps read the path for themselves: nothing stands between it and the rows' loads
// but the page table.
__global__ void __launch_bounds__(kThreads) accept_kernel(const __grid_constant__ AcceptParams P) {
  const BatchParams& b = P.batch;
  const int seq = (int)blockIdx.y, layer = (int)blockIdx.x, lane = threadIdx.x & 31;
  const int32_t* path = P.path + (int64_t)seq * P.width;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int n = __ldg(b.cu_q + seq + 1) - __ldg(b.cu_q + seq), base = __ldg(b.kv_len + seq) - n;
  int count = 0, last = -1;
  bool bad_path = false;
  for (bool more = true; more && count < P.width;) {
    const int at = count + lane, x = at < P.width ? __ldg(path + at) : -1;
    const uint32_t none = __ballot_sync(0xffffffffu, x < 0);
    const int some = none ? __ffs((int)none) - 1 : 32;
    int before = __shfl_up_sync(0xffffffffu, x, 1);
    if (lane == 0) before = last;
    bad_path |= __any_sync(0xffffffffu, lane < some && (x >= n || x <= before));
    last = __shfl_sync(0xffffffffu, x, max(some - 1, 0));
    count += some;
    more = none == 0;
  }
  if (count == 0) return;
  if (bad_path || base < 0 || (int64_t)base + n > (int64_t)b.W << P.page_shift) {  // nothing of the sequence is moved
    if (threadIdx.x == 0) atomicCAS(b.err, 0, bad_path ? kCacheBadPath : kCacheBadPosition);
    return;
  }
  const int chunks = 1 << P.row_shift;
  // pool row of position p for kv head g; -1: no page
  auto row_of = [&](int p, int g) -> int64_t {
    const int page = __ldg(b.table + (int64_t)seq * b.W + (p >> P.page_shift));
    if (page < 0 || page >= b.num_pages) {
      atomicCAS(b.err, 0, kCacheBadPage);
      return -1;
    }
    return (((((int64_t)layer * b.num_pages + page) * b.Hkv) + g) << P.page_shift) + (p & ((1 << P.page_shift) - 1));
  };
  const int64_t all = (int64_t)count * b.Hkv << P.row_shift;
  for (int64_t x0 = 0; x0 < all; x0 += kThreads * kMoves) {
    uint4 k[kMoves], v[kMoves];
    uint8_t k_scale[kMoves], v_scale[kMoves];
    int64_t to[kMoves];
#pragma unroll
    for (int m = 0; m < kMoves; ++m) {
      const int64_t x = x0 + m * kThreads + threadIdx.x;
      to[m] = -1;
      if (x >= all) continue;
      const int r = (int)(x >> P.row_shift), i = r / b.Hkv, g = r - i * b.Hkv, from_i = __ldg(path + i);
      if (from_i == i) continue;
      const int64_t from = row_of(base + from_i, g), into = row_of(base + i, g);
      if (from < 0 || into < 0) continue;
      to[m] = into;
      const int64_t at = ((from << P.row_shift) + (x & (chunks - 1))) << 4;
      k[m] = *reinterpret_cast<const uint4*>(P.k_pages + at);
      v[m] = *reinterpret_cast<const uint4*>(P.v_pages + at);
      if (P.k_scales) {
        k_scale[m] = P.k_scales[from];
        v_scale[m] = P.v_scales[from];
      }
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < kMoves; ++m) {
      if (to[m] < 0) continue;
      const int64_t chunk = (x0 + m * kThreads + threadIdx.x) & (chunks - 1), at = ((to[m] << P.row_shift) + chunk) << 4;
      *reinterpret_cast<uint4*>(P.k_pages + at) = k[m];
      *reinterpret_cast<uint4*>(P.v_pages + at) = v[m];
      if (P.k_scales && chunk == 0) {
        P.k_scales[to[m]] = k_scale[m];
        P.v_scales[to[m]] = v_scale[m];
      }
    }
    __syncthreads();
  }
}

}  // namespace
}  // namespace aa

using namespace aa;

extern "C" aa_status aa_cache_tree_masks(aa_cache_t c, const int32_t* parents, const int32_t* cu_q, const int32_t* kv_len,
                                         int32_t num_seqs, int32_t total_tokens, int32_t tree_words, uint64_t* mask,
                                         int32_t* pos, aa_stream_t stream) {
  aa_status st = check_compute_cache(c);
  if (st != AA_OK) return st;
  if (num_seqs < 1 || num_seqs > (1 << 20)) return fail(AA_ERR_INVALID_ARG, "num_seqs must be in [1, 2^20]");
  if (total_tokens < 0 || total_tokens >= (1 << 30)) return fail(AA_ERR_INVALID_ARG, "total_tokens must be in [0, 2^30)");
  if (tree_words < 1 || tree_words > kMaxTreeWords)
    return fail(AA_ERR_INVALID_ARG, "tree_words must be in [1, " + std::to_string(kMaxTreeWords) + "]");
  if (total_tokens == 0) return AA_OK;
  const size_t T = (size_t)total_tokens;
  const struct {
    const char* name;
    const void* at;
    size_t bytes;
  } all[] = {{"mask", mask, T * tree_words * 8},     {"pos", pos, T * 4},
             {"parents", parents, T * 4},            {"cu_q", cu_q, ((size_t)num_seqs + 1) * 4},
             {"kv_len", kv_len, (size_t)num_seqs * 4}};
  for (const auto& x : all)
    if (!x.at || (reinterpret_cast<uintptr_t>(x.at) & (x.at == mask ? 7u : 3u)))
      return fail(AA_ERR_INVALID_ARG, std::string(x.name) + " must be an aligned device pointer");
  for (int w = 0; w < 2; ++w) {
    if ((st = check_outside_pool(c, all[w].name, all[w].at, all[w].bytes)) != AA_OK) return st;
    for (int r = w + 1; r < 5; ++r)
      if (overlap(all[w].at, all[w].bytes, all[r].at, all[r].bytes))
        return fail(AA_ERR_INVALID_ARG, std::string(all[w].name) + " overlaps " + all[r].name);
  }
  const MaskParams P{parents, cu_q, kv_len, mask, pos, c->err, num_seqs, total_tokens, tree_words};
  const cudaError_t e = launch_after(tree_masks_kernel, dim3((unsigned)((T + kThreads - 1) / kThreads)), kThreads, 0,
                                     reinterpret_cast<cudaStream_t>(stream), P);
  return e == cudaSuccess ? AA_OK : cuda_fail(e, "tree_masks_kernel launch");
}

extern "C" aa_status aa_cache_accept(aa_cache_t c, const aa_cache_batch* batch, const int32_t* path, int32_t path_width,
                                     aa_stream_t stream) {
  aa_status st = check_compute_cache(c);
  if (st != AA_OK) return st;
  if ((st = check_batch(c, batch)) != AA_OK) return st;
  if (path_width < 0 || path_width >= (1 << 30)) return fail(AA_ERR_INVALID_ARG, "path_width must be in [0, 2^30)");
  if ((int64_t)path_width * c->cfg.num_kv_heads >= (1ll << 31))
    return fail(AA_ERR_INVALID_ARG, "path_width * Hkv must stay below 2^31");
  if (path_width == 0) return AA_OK;
  if (!path || (reinterpret_cast<uintptr_t>(path) & 3u))
    return fail(AA_ERR_INVALID_ARG, "path must be a device pointer to int32");
  AcceptParams P;
  P.batch = batch_params(c, batch);
  P.path = path;
  P.k_pages = static_cast<uint8_t*>(c->k_pages);
  P.v_pages = static_cast<uint8_t*>(c->v_pages);
  P.k_scales = c->k_scales;
  P.v_scales = c->v_scales;
  P.width = path_width;
  P.page_shift = __builtin_ctz((unsigned)c->cfg.page_size);
  P.row_shift = __builtin_ctz((unsigned)(c->cfg.head_dim * (c->fp8() ? 1 : 2) / 16));
  // sequences in slices of what a grid's second dimension holds
  for (int first = 0; first < batch->num_seqs; first += 65535) {
    const int some = batch->num_seqs - first < 65535 ? batch->num_seqs - first : 65535;
    AcceptParams S = P;
    S.batch.table += (int64_t)first * S.batch.W;
    S.batch.cu_q += first;
    S.batch.kv_len += first;
    S.path += (int64_t)first * path_width;
    const cudaError_t e = launch_after(accept_kernel, dim3((unsigned)c->cfg.num_layers, (unsigned)some), kThreads, 0,
                                       reinterpret_cast<cudaStream_t>(stream), S);
    if (e != cudaSuccess) return cuda_fail(e, "accept_kernel launch");
  }
  return AA_OK;
}
