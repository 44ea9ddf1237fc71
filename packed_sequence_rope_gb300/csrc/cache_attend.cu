// Attention of new tokens over the paged cache (aa_cache_attend).
//
// For new token i of sequence b, at position p = kv_len - n_b + i, and query
// head h ("When Precision Meets Position", architecture page §3.4
// "AnchorAttention: The Shared Anchor Design", "Mask construction"):
//   visible keys: [max(key_lo, 0), p], and key 0 with the anchor (p >= 0)
//   O_i = sum_j softmax_j(scale * q_i . k_j) v_j, LSE_i = ln sum_j exp(...)
// in one pass with the running maximum and sum of the softmax.
#include <algorithm>
#include <cmath>

#include "cache_attend.cuh"

namespace aa {
namespace {

// One warp per (row, query head): each lane holds HD / 32 channels, the keys
// come one after the other.
template <int HD>
__global__ void __launch_bounds__(128) attend_rows_kernel(const __grid_constant__ AttendParams P,
                                                          const __nv_bfloat16* k_pages, const __nv_bfloat16* v_pages) {
  constexpr int kPer = HD / 32;
  const BatchParams& b = P.batch;
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int t = (int)(item / P.Hq), h = (int)(item % P.Hq);
  if (t >= b.T || t < __ldg(b.cu_q) || t >= __ldg(b.cu_q + b.B)) return;
  const int seq = warp_find_seq(b.cu_q, b.B, t);
  const int p = __ldg(b.kv_len + seq) - __ldg(b.cu_q + seq + 1) + t;
  const int lo = P.key_lo ? max(__ldg(P.key_lo + t), 0) : 0;
  const int g = h / P.group;
  float q[kPer], acc[kPer] = {}, m = -INFINITY, l = 0.f;
  for (int e = 0; e < kPer; ++e) q[e] = __bfloat162float(P.q[t * P.q_stride + (int64_t)h * HD + lane * kPer + e]);
  for (int j = P.anchor ? 0 : lo; j <= p; j = j == 0 ? max(lo, 1) : j + 1) {
    const int w = j >> P.page_shift;
    if (w >= b.W) {
      if (lane == 0) atomicCAS(b.err, 0, kCacheBadPosition);
      break;
    }
    const int page = __ldg(b.table + (int64_t)seq * b.W + w);
    const bool ok = page >= 0 && page < b.num_pages;
    if (!ok && lane == 0) atomicCAS(b.err, 0, kCacheBadPage);
    const int64_t row = ((((b.layer_page0 + page) * b.Hkv + g) << P.page_shift) + (j & ((1 << P.page_shift) - 1))) * HD;
    float s = 0.f;
    for (int e = 0; e < kPer; ++e) s += ok ? q[e] * __bfloat162float(k_pages[row + lane * kPer + e]) : 0.f;
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= P.scale_log2;
    const float mn = fmaxf(m, s), f = exp2f(m - mn), w_j = exp2f(s - mn);
    m = mn;
    l = l * f + w_j;
    for (int e = 0; e < kPer; ++e)
      acc[e] = acc[e] * f + (ok ? w_j * __bfloat162float(v_pages[row + lane * kPer + e]) : 0.f);
  }
  for (int e = 0; e < kPer; ++e)
    P.o[((int64_t)t * P.Hq + h) * HD + lane * kPer + e] = __float2bfloat16(l > 0.f ? acc[e] / l : 0.f);
  if (P.lse && lane == 0) P.lse[(int64_t)h * b.T + t] = (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace
}  // namespace aa

using namespace aa;

extern "C" size_t aa_cache_attend_workspace_bytes(aa_cache_t c, int32_t num_seqs, int32_t total_tokens, int32_t max_q,
                                                  int32_t table_width, int32_t q_heads) {
  if (!c || num_seqs < 1 || total_tokens < 0 || max_q < 0 || table_width < 1 || q_heads < 1) return 0;
  return 256;
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
  if (overlap(o, (size_t)T * q_heads * D * 2, q, rows_span(T, q_stride, q_heads, D)))
    return fail(AA_ERR_INVALID_ARG, "o overlaps q");
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return fail(AA_ERR_INVALID_ARG, "workspace must be a 256-byte aligned device pointer");
  if (workspace_bytes <
      aa_cache_attend_workspace_bytes(c, batch->num_seqs, T, max_q, batch->table_width, q_heads))
    return fail(AA_ERR_INVALID_ARG, "workspace is smaller than aa_cache_attend_workspace_bytes()");
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
  if ((int64_t)std::max(max_q, 1) * P.group <= kShortRows) {
    cudaError_t e = launch_attend_short(c, P, max_q, s);
    return e == cudaSuccess ? AA_OK : cuda_fail(e, "attend_short_kernel launch");
  }
  const unsigned grid = (unsigned)(((int64_t)T * q_heads + 3) / 4);
  const auto* kp = static_cast<const __nv_bfloat16*>(c->k_pages);
  const auto* vp = static_cast<const __nv_bfloat16*>(c->v_pages);
  if (D == 128)
    attend_rows_kernel<128><<<grid, 128, 0, s>>>(P, kp, vp);
  else
    attend_rows_kernel<64><<<grid, 128, 0, s>>>(P, kp, vp);
  cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? AA_OK : cuda_fail(e, "attend_rows_kernel launch");
}
