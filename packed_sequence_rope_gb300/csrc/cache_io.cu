// Writing to the paged cache: aa_cache_append (new keys rotated into their
// pages, values beside them, queries rotated on the way; quantised as they are
// written where the pages hold 8 bits), aa_cache_read, which brings tokens back, and
// the page copies of aa_cache_copy_pages, aa_cache_resize and aa_cache_compact.
//
// 8-bit pages: a row of D values is stored as e4m3 codes c with x = c * 2^e, e the
// smallest integer in [-100, 119] that keeps max |x| within 448 * 2^e, and a byte e + 127.
// A power of two costs a floating-point code no accuracy, and makes what a page
// holds exact in bf16 (4-bit significands). e >= -100 keeps a weight times 2^e of the
// attention in bf16's normal range, e <= 119 what a page holds within its range. A row with a value that is not finite has byte
// 255, which makes all of it NaN.
//
// They are bound by HBM (a decoding step's few rows by the launch): every byte
// is read and written once, in 16-byte accesses. A compaction of 256 pages of
// 128 KB in 32 layers takes 615 us, 7.0 TB/s (a copy of the same bytes: 6.77).
#include <algorithm>

#include "cache_common.cuh"
#include "rope_axes.cuh"

namespace aa {
namespace {

constexpr int kThreads = 256;
// Up to here a block takes one token, above two. 64 tokens of 32 + 8 + 8 heads:
// 3.0 us with one, 3.2 with two; 1024 tokens: 6.7 and 5.8 us; 13.7 thousand: 58 us
// with two (5.8 TB/s), 60 with four.
constexpr int kFewTokens = 128;

struct AppendParams {
  AxesTable tab;
  BatchParams batch;
  const int32_t* pos;
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16 *q_out, *k_pages, *v_pages;
  uint8_t *k_scales, *v_scales;  // 8-bit pages; k_pages and v_pages are then bytes
  int64_t q_stride, k_stride, v_stride;
  int Hq, page_shift;
};

// Sixteen values of a row in fp32, eight from each of the places where Pairs8 has them; with
// kHalved half of them, which fp32 also holds where a rotation makes bf16's largest longer by
// sqrt 2. (Of values, which are not rotated, too: keys alone cost a register more, 1.7 %; both 0.4.)
template <int HD, int L, bool kHalved>
struct Values16 {
  static constexpr float kBy = kHalved ? 0.5f : 1.f;
  float a[8], b[8];
  __device__ __forceinline__ explicit Values16(const Pairs8<HD, L>& x) {
    const uint32_t u[8] = {x.a.x, x.a.y, x.a.z, x.a.w, x.b.x, x.b.y, x.b.z, x.b.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 va = ptx::unpack_bf16x2(u[e]), vb = ptx::unpack_bf16x2(u[4 + e]);
      a[2 * e] = kBy * va.x;
      a[2 * e + 1] = kBy * va.y;
      b[2 * e] = kBy * vb.x;
      b[2 * e + 1] = kBy * vb.y;
    }
  }
  __device__ __forceinline__ void turn(const float2* cs) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if constexpr (L == 0) {
        float* x = e < 4 ? a + 2 * e : b + 2 * e - 8;
        rope_pair(x[0], x[1], cs[e].x, cs[e].y);
      } else {
        rope_pair(a[e], b[e], cs[e].x, cs[e].y);
      }
    }
  }
  // Quantises the row, which HD / 16 neighbouring lanes hold, into `row`; its scale's
  // byte goes to *scale.
  __device__ __forceinline__ void store(uint8_t* row, uint8_t* scale, int chunk) const {
    constexpr int kLanes = HD / 16;
    const uint32_t lanes = ((1u << kLanes) - 1u) << ((threadIdx.x & 31) & ~(kLanes - 1));
    uint32_t top = 0;  // the largest magnitude's bits; NaN and infinity are above all numbers
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, max(__float_as_uint(a[e]) & 0x7fffffffu, __float_as_uint(b[e]) & 0x7fffffffu));
#pragma unroll
    for (int d = 1; d < kLanes; d *= 2) top = max(top, __shfl_xor_sync(lanes, top, d));
    // 448 = 1.75 * 2^8
    const int e = min(max((int)(top >> 23) - 135 + kHalved + ((top & 0x7fffffu) > 0x600000u ? 1 : 0), -100), 119);
    const float down = __uint_as_float((uint32_t)(127 - e + kHalved) << 23);
    uint32_t w[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const float* v = x < 2 ? a + 4 * x : b + 4 * x - 8;
      w[x] = ptx::pack_e4m3x2(v[0] * down, v[1] * down) | ptx::pack_e4m3x2(v[2] * down, v[3] * down) << 16;
    }
    if constexpr (L == 0) {
      *reinterpret_cast<uint4*>(row + 16 * chunk) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      *reinterpret_cast<uint2*>(row + 8 * chunk) = make_uint2(w[0], w[1]);
      *reinterpret_cast<uint2*>(row + HD / 2 + 8 * chunk) = make_uint2(w[2], w[3]);
    }
    if (chunk == 0) *scale = top >= 0x7f800000u ? 255 : (uint8_t)(e + 127);
  }
};

// Pool row of token t for kv head 0; -1 if it has none (an error), -2 if the
// token lies outside the batch (a whole warp asks).
__device__ __forceinline__ int64_t find_slot(const BatchParams& b, int t, int page_shift) {
  // the search does not wait for the batch's ends
  const int begin = __ldg(b.cu_q), end = __ldg(b.cu_q + b.B);
  const int seq = warp_find_seq(b.cu_q, b.B, t);
  const int p = __ldg(b.kv_len + seq) - __ldg(b.cu_q + seq + 1) + t, w = p >> page_shift;
  if (t >= b.T || t < begin || t >= end) return -2;
  const bool report = (threadIdx.x & 31) == 0;
  if (p < 0 || w >= b.W) {
    if (report) atomicCAS(b.err, 0, kCacheBadPosition);
    return -1;
  }
  const int page = __ldg(b.table + (int64_t)seq * b.W + w);
  if (page < 0 || page >= b.num_pages) {
    if (report) atomicCAS(b.err, 0, kCacheBadPage);
    return -1;
  }
  return (((b.layer_page0 + page) * b.Hkv) << page_shift) + (p & ((1 << page_shift) - 1));
}

// L: the pairing (0, 1), or 2 to store the keys as they are. A block takes
// kTokens rows; as in rope_axes_kernel the angles of a token are computed once
// for all heads, while the first row is in flight.
// k8: four blocks per SM, 64 registers (13.7 thousand tokens with their reading back 84.6 us;
// left alone it takes 80, 89.2; five blocks spill, 110), and launched as a dependent (81.4).
template <int HD, int L, int kTokens, bool k8>
__global__ void __launch_bounds__(kThreads, k8 ? 4 : 0) cache_append_kernel(const __grid_constant__ AppendParams P) {
  constexpr int kHalf = HD / 2, kChunks = HD / 16, kRows = kThreads / kChunks / kTokens;
  static_assert(kTokens <= kThreads / 32, "a warp looks up each token");
  __shared__ float2 cs[L == 2 ? 1 : kTokens][kHalf];
  __shared__ int64_t slot[kTokens];
  const BatchParams& b = P.batch;
  const int t0 = (int)blockIdx.x * kTokens, warp = threadIdx.x >> 5;
  const int chunk = threadIdx.x % kChunks, row = threadIdx.x / kChunks;
  const int tok = row / kRows, heads = P.Hq + 2 * b.Hkv;
  const int64_t t = t0 + tok;
  auto load = [&](Pairs8<HD, L == 2 ? 0 : L>& x, int h) {
    if (t >= b.T || h >= heads) return;
    const int g = h - P.Hq;
    x.load(g < 0 ? P.q + t * P.q_stride + (int64_t)h * HD
                 : g < b.Hkv ? P.k + t * P.k_stride + (int64_t)g * HD : P.v + t * P.v_stride + (int64_t)(g - b.Hkv) * HD,
           chunk);
  };
  Pairs8<HD, L == 2 ? 0 : L> x;
  if constexpr (k8) asm volatile("griddepcontrol.wait;" ::: "memory");
  load(x, row % kRows);
  if (warp < kTokens) {
    const int64_t at = find_slot(b, t0 + warp, P.page_shift);
    if ((threadIdx.x & 31) == 0) slot[warp] = at;
  }
  if constexpr (L != 2) {
    for (int e = kThreads - 1 - (int)threadIdx.x; e < kTokens * kHalf; e += kThreads) {  // the searching warps come last
      const int at = e / kHalf, p = e % kHalf;
      if (t0 + at < b.T)
        cs[at][p] = k8 ? axes_cs_fine(P.tab, P.pos, b.T, t0 + at, p) : axes_cs(P.tab, P.pos, b.T, t0 + at, p);
    }
  }
  __syncthreads();
  const int64_t at = slot[tok];
  if (at == -2) return;
  float2 mine[8];
  if constexpr (L != 2) {
#pragma unroll
    for (int e = 0; e < 8; ++e) mine[e] = cs[tok][8 * chunk + e];
  }
  Pairs8<HD, L == 2 ? 0 : L> next;
  for (int h = row % kRows; h < heads; h += kRows) {
    if constexpr (k8) {  // quantising takes longer: the next row is in flight meanwhile
      if (h >= kRows) x = next;
      load(next, h + kRows);
    } else {
      if (h >= kRows) load(x, h);
    }
    const int g = h - P.Hq;
    if constexpr (k8) {
      if (g >= 0) {
        if (at < 0) continue;  // all lanes of a row
        Values16<HD, L == 2 ? 0 : L, L != 2> y(x);
        if constexpr (L != 2)
          if (g < b.Hkv) y.turn(mine);
        const int64_t row = at + ((int64_t)(g < b.Hkv ? g : g - b.Hkv) << P.page_shift);
        uint8_t* pages = reinterpret_cast<uint8_t*>(g < b.Hkv ? P.k_pages : P.v_pages);
        y.store(pages + row * HD, (g < b.Hkv ? P.k_scales : P.v_scales) + row, chunk);
        continue;
      }
    }
    if constexpr (L != 2)
      if (g < b.Hkv) x.turn(mine);
    if (g < 0)
      x.store(P.q_out + (t * P.Hq + h) * HD, chunk);
    else if (at >= 0)
      x.store((g < b.Hkv ? P.k_pages + (at + ((int64_t)g << P.page_shift)) * HD
                         : P.v_pages + (at + ((int64_t)(g - b.Hkv) << P.page_shift)) * HD), chunk);
  }
}

template <int HD, int L, bool k8>
cudaError_t launch_append(const AppendParams& P, cudaStream_t s) {
  if constexpr (k8)
    return P.batch.T <= kFewTokens
               ? launch_after(cache_append_kernel<HD, L, 1, k8>, dim3((unsigned)P.batch.T), kThreads, 0, s, P)
               : launch_after(cache_append_kernel<HD, L, 2, k8>, dim3((unsigned)((P.batch.T + 1) / 2)), kThreads, 0, s, P);
  if (P.batch.T <= kFewTokens)
    cache_append_kernel<HD, L, 1, k8><<<(unsigned)P.batch.T, kThreads, 0, s>>>(P);
  else
    cache_append_kernel<HD, L, 2, k8><<<(unsigned)((P.batch.T + 1) / 2), kThreads, 0, s>>>(P);
  return cudaGetLastError();
}

template <int HD, int L>
cudaError_t launch_append(const AppendParams& P, cudaStream_t s) {
  return P.k_scales ? launch_append<HD, L, true>(P, s) : launch_append<HD, L, false>(P, s);
}

// ---------------------------------------------------------------- reading back
struct ReadParams {
  BatchParams batch;
  const uint8_t *k_pages, *v_pages, *k_scales, *v_scales;
  __nv_bfloat16 *k, *v;
  int page_shift;
};

// A block takes kTokens rows of k and v; a thread 16 channels of a head. Bound by HBM
// like the append, a step's few rows by the launch.
template <int HD, int kTokens, bool k8>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const __grid_constant__ ReadParams P) {
  constexpr int kChunks = HD / 16, kRows = kThreads / kChunks / kTokens;
  __shared__ int64_t slot[kTokens];
  const BatchParams& b = P.batch;
  const int t0 = (int)blockIdx.x * kTokens, warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (warp < kTokens) {
    const int64_t at = find_slot(b, t0 + warp, P.page_shift);
    if ((threadIdx.x & 31) == 0) slot[warp] = at;
  }
  __syncthreads();
  const int chunk = threadIdx.x % kChunks, row = threadIdx.x / kChunks, tok = row / kRows;
  const int64_t at = slot[tok], t = t0 + tok;
  if (at == -2) return;
  for (int h = row % kRows; h < 2 * b.Hkv; h += kRows) {
    const int g = h < b.Hkv ? h : h - b.Hkv;
    const int64_t from = at + ((int64_t)g << P.page_shift);
    uint4* to = reinterpret_cast<uint4*>((h < b.Hkv ? P.k : P.v) + (t * b.Hkv + g) * HD + 16 * chunk);
    uint4 y[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};  // a token whose page is none
    if (at >= 0) {
      const uint8_t* pages = h < b.Hkv ? P.k_pages : P.v_pages;
      if constexpr (k8) {
        const uint4 x = *reinterpret_cast<const uint4*>(pages + from * HD + 16 * chunk);
        decode16(x, (int)(h < b.Hkv ? P.k_scales : P.v_scales)[from], y);
      } else {
        const uint4* x = reinterpret_cast<const uint4*>(pages + (from * HD + 16 * chunk) * 2);
        y[0] = x[0];
        y[1] = x[1];
      }
    }
    to[0] = y[0];
    to[1] = y[1];
  }
}

template <int HD, bool k8>
cudaError_t launch_read(const ReadParams& P, cudaStream_t s) {
  return P.batch.T <= kFewTokens
             ? launch_after(cache_read_kernel<HD, 1, k8>, dim3((unsigned)P.batch.T), kThreads, 0, s, P)
             : launch_after(cache_read_kernel<HD, 4, k8>, dim3((unsigned)((P.batch.T + 3) / 4)), kThreads, 0, s, P);
}

// The pairs of a copy travel as a kernel argument: no device memory, nothing to
// keep alive until the launch has run.
template <int N>
struct PairList {
  PagePair p[N];
};

constexpr int kCopyVecs = 4;                                // 16-byte vectors per thread
constexpr int kCopyBytes = kThreads * kCopyVecs * 16;       // bytes per block

struct CopyParams {
  uint8_t *k_pages, *v_pages;
  int64_t page_bytes, layer_bytes;
  int blocks_per_page;
  uint8_t *k_scales, *v_scales;  // 8-bit pages: copied by the first block of a page, which is never larger
  int64_t scale_bytes, scale_layer;
};

template <int N>
__global__ void __launch_bounds__(kThreads) copy_pages_kernel(const CopyParams P, const __grid_constant__ PairList<N> list) {
  const int part = (int)(blockIdx.x % P.blocks_per_page), which = (int)(blockIdx.x / P.blocks_per_page);
  const PagePair pair = list.p[blockIdx.y];
  uint8_t* pool = ((which & 1) ? P.v_pages : P.k_pages) + (int64_t)(which >> 1) * P.layer_bytes;
  const uint8_t* src = pool + pair.src * P.page_bytes;
  uint8_t* dst = pool + pair.dst * P.page_bytes;
  const int64_t at = (int64_t)part * kCopyBytes + threadIdx.x * 16;
  if (P.k_scales && part == 0) {
    uint8_t* scales = ((which & 1) ? P.v_scales : P.k_scales) + (int64_t)(which >> 1) * P.scale_layer;
    for (int64_t x = threadIdx.x * 16; x < P.scale_bytes; x += kThreads * 16)
      *reinterpret_cast<uint4*>(scales + pair.dst * P.scale_bytes + x) =
          *reinterpret_cast<const uint4*>(scales + pair.src * P.scale_bytes + x);
  }
  uint4 v[kCopyVecs];
#pragma unroll
  for (int i = 0; i < kCopyVecs; ++i)
    if (at + i * kThreads * 16 < P.page_bytes) v[i] = *reinterpret_cast<const uint4*>(src + at + i * kThreads * 16);
#pragma unroll
  for (int i = 0; i < kCopyVecs; ++i)
    if (at + i * kThreads * 16 < P.page_bytes) *reinterpret_cast<uint4*>(dst + at + i * kThreads * 16) = v[i];
}

template <int N>
cudaError_t launch_copies(const CopyParams& P, const PagePair* pairs, int n, int layers, cudaStream_t s) {
  PairList<N> list{};
  std::copy(pairs, pairs + n, list.p);
  const dim3 grid((unsigned)(P.blocks_per_page * layers * 2), (unsigned)n);
  copy_pages_kernel<N><<<grid, kThreads, 0, s>>>(P, list);
  return cudaGetLastError();
}

}  // namespace

aa_status launch_copy_pages(const aa_cache_s* c, const std::vector<PagePair>& pairs, cudaStream_t s) {
  CopyParams P;
  P.k_pages = static_cast<uint8_t*>(c->k_pages);
  P.v_pages = static_cast<uint8_t*>(c->v_pages);
  P.page_bytes = c->page_bytes();
  P.k_scales = c->k_scales;
  P.v_scales = c->v_scales;
  P.scale_bytes = (int64_t)c->cfg.num_kv_heads * c->cfg.page_size;
  P.scale_layer = P.scale_bytes * c->cfg.num_pages;
  P.layer_bytes = P.page_bytes * c->cfg.num_pages;
  P.blocks_per_page = (int)((P.page_bytes + kCopyBytes - 1) / kCopyBytes);
  const int n = (int)pairs.size();
  for (int at = 0; at < n;) {
    const int left = n - at;
    const int take = std::min(left, left <= 64 ? 64 : 1024);
    cudaError_t e = left <= 64 ? launch_copies<64>(P, pairs.data() + at, take, c->cfg.num_layers, s)
                               : launch_copies<1024>(P, pairs.data() + at, take, c->cfg.num_layers, s);
    if (e != cudaSuccess) return cuda_fail(e, "copy_pages_kernel launch");
    at += take;
  }
  return AA_OK;
}

}  // namespace aa

using namespace aa;

extern "C" aa_status aa_cache_append(aa_cache_t c, const aa_cache_batch* batch, const void* k, int64_t k_stride,
                                     const void* v, int64_t v_stride, const aa_rope_axes* rope, const int32_t* pos,
                                     const void* q, int64_t q_stride, void* q_out, int32_t q_heads,
                                     aa_stream_t stream) {
  aa_status st = check_compute_cache(c);
  if (st != AA_OK) return st;
  if ((st = check_batch(c, batch)) != AA_OK) return st;
  if (rope && !axes_valid(rope)) return fail(AA_ERR_INVALID_ARG, "rope must be filled by aa_rope_axes_init");
  const int D = c->cfg.head_dim, Hkv = c->cfg.num_kv_heads, T = batch->total_tokens;
  if (rope && rope->head_dim != D) return fail(AA_ERR_INVALID_ARG, "rope's head_dim is not the cache's");
  if (T == 0) return AA_OK;  // tensors without elements have no address
  if (q && !rope) return fail(AA_ERR_INVALID_ARG, "q is rotated: it needs rope");
  if (q ? q_heads < 1 || q_heads > 65536 : q_heads != 0)
    return fail(AA_ERR_INVALID_ARG, "q_heads must be >= 1 with q (at most 65536) and 0 without");
  if ((rope != nullptr) != (pos != nullptr)) return fail(AA_ERR_INVALID_ARG, "give both rope and pos or neither");
  if (reinterpret_cast<uintptr_t>(pos) & 3u) return fail(AA_ERR_INVALID_ARG, "pos must be a device pointer to int32");
  if ((st = check_rows("k", k, k_stride, Hkv, D)) != AA_OK || (st = check_rows("v", v, v_stride, Hkv, D)) != AA_OK ||
      (q && (st = check_turned("q", q, q_stride, q_out, q_heads, D, T)) != AA_OK))
    return st;
  if (q) {
    const size_t nq = (size_t)T * q_heads * D * 2;
    if (overlap(q_out, nq, k, rows_span(T, k_stride, Hkv, D)) || overlap(q_out, nq, v, rows_span(T, v_stride, Hkv, D)))
      return fail(AA_ERR_INVALID_ARG, "q_out overlaps k or v");
    if ((st = check_outside_pool(c, "q_out", q_out, nq)) != AA_OK) return st;
  }
  AppendParams P;
  P.tab = rope ? axes_table(rope) : AxesTable{};
  P.batch = batch_params(c, batch);
  P.pos = pos;
  P.q = static_cast<const __nv_bfloat16*>(q);
  P.k = static_cast<const __nv_bfloat16*>(k);
  P.v = static_cast<const __nv_bfloat16*>(v);
  P.q_out = static_cast<__nv_bfloat16*>(q_out);
  P.k_pages = static_cast<__nv_bfloat16*>(c->k_pages);
  P.v_pages = static_cast<__nv_bfloat16*>(c->v_pages);
  P.k_scales = c->k_scales;
  P.v_scales = c->v_scales;
  P.q_stride = q_stride;
  P.k_stride = k_stride;
  P.v_stride = v_stride;
  P.Hq = q ? q_heads : 0;
  P.page_shift = __builtin_ctz((unsigned)c->cfg.page_size);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int L = !rope ? 2 : rope->layout == AA_ROPE_ADJACENT ? 0 : 1;
  cudaError_t e;
  if (D == 128)
    e = L == 0 ? launch_append<128, 0>(P, s) : L == 1 ? launch_append<128, 1>(P, s) : launch_append<128, 2>(P, s);
  else
    e = L == 0 ? launch_append<64, 0>(P, s) : L == 1 ? launch_append<64, 1>(P, s) : launch_append<64, 2>(P, s);
  return e == cudaSuccess ? AA_OK : cuda_fail(e, "cache_append_kernel launch");
}

extern "C" aa_status aa_cache_read(aa_cache_t c, const aa_cache_batch* batch, void* k, void* v, aa_stream_t stream) {
  aa_status st = check_compute_cache(c);
  if (st != AA_OK) return st;
  if ((st = check_batch(c, batch)) != AA_OK) return st;
  const int D = c->cfg.head_dim, Hkv = c->cfg.num_kv_heads, T = batch->total_tokens;
  if (T == 0) return AA_OK;
  const size_t bytes = (size_t)T * Hkv * D * 2;
  const struct {
    const char* name;
    const void* at;
    size_t bytes;
  } read[] = {{"page_table", batch->page_table, (size_t)batch->num_seqs * batch->table_width * 4},
              {"cu_q", batch->cu_q, ((size_t)batch->num_seqs + 1) * 4},
              {"kv_len", batch->kv_len, (size_t)batch->num_seqs * 4}};
  for (const auto& [name, x] : {std::pair<const char*, const void*>{"k", k}, {"v", v}}) {
    if (!x || !aligned16(x)) return fail(AA_ERR_INVALID_ARG, std::string(name) + " must be a 16-byte aligned device pointer");
    if ((st = check_outside_pool(c, name, x, bytes)) != AA_OK) return st;
    for (const auto& y : read)
      if (overlap(x, bytes, y.at, y.bytes)) return fail(AA_ERR_INVALID_ARG, std::string(name) + " overlaps " + y.name);
  }
  if (overlap(k, bytes, v, bytes)) return fail(AA_ERR_INVALID_ARG, "k overlaps v");
  ReadParams P;
  P.batch = batch_params(c, batch);
  P.k_pages = static_cast<const uint8_t*>(c->k_pages);
  P.v_pages = static_cast<const uint8_t*>(c->v_pages);
  P.k_scales = c->k_scales;
  P.v_scales = c->v_scales;
  P.k = static_cast<__nv_bfloat16*>(k);
  P.v = static_cast<__nv_bfloat16*>(v);
  P.page_shift = __builtin_ctz((unsigned)c->cfg.page_size);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (c->fp8())
    e = D == 128 ? launch_read<128, true>(P, s) : launch_read<64, true>(P, s);
  else
    e = D == 128 ? launch_read<128, false>(P, s) : launch_read<64, false>(P, s);
  return e == cudaSuccess ? AA_OK : cuda_fail(e, "cache_read_kernel launch");
}
