// Rotary positions with several axes (time, height, width) for q and k in one
// launch: aa_rope_axes_init, aa_rope_axes_apply.
//
// HBM-bound: every element is read and written once. A block takes one or two
// tokens: its threads first compute the (cos, sin) of the tokens' D/2 pairs into
// shared memory, one each, which all heads of q and k then share; after that,
// eight pairs of a row per thread and head, 16-byte accesses. 64K tokens of 64
// heads of 128: 311 us a direction, 6.9 TB/s (a copy of the same bytes: 6.77).
#include <cmath>

#include "rope_axes.cuh"

namespace aa {
namespace {

constexpr int kThreads = 256;
// Up to here a block takes one token, above two. 64 tokens of 32 + 8 heads: 2.6 us
// with one, 3.0 with two; 1024 tokens: 6.6 and 5.4 us; 64K tokens, forward and
// gradient: 622 us with two, 629 with four.
constexpr int kFewTokens = 128;

struct ApplyParams {
  AxesTable tab;
  const int32_t* pos;
  const __nv_bfloat16 *q, *k;
  __nv_bfloat16 *q_out, *k_out;
  int64_t q_stride, k_stride;
  int T, Hq, Hk, inverse;
};

template <int HD, int L, int kTokens>
__global__ void __launch_bounds__(kThreads) rope_axes_kernel(const __grid_constant__ ApplyParams P) {
  constexpr int kHalf = HD / 2, kChunks = HD / 16, kRows = kThreads / kChunks / kTokens;
  __shared__ float2 cs[kTokens][kHalf];
  const int64_t t0 = (int64_t)blockIdx.x * kTokens;
  const int chunk = threadIdx.x % kChunks, row = threadIdx.x / kChunks;
  const int tok = row / kRows, heads = P.Hq + P.Hk;
  const int64_t t = t0 + tok;
  auto load = [&](Pairs8<HD, L>& x, int h) {
    if (t < P.T && h < heads)
      x.load(h < P.Hq ? P.q + t * P.q_stride + (int64_t)h * HD : P.k + t * P.k_stride + (int64_t)(h - P.Hq) * HD, chunk);
  };
  // the first row is in flight while the angles are computed
  Pairs8<HD, L> x;
  load(x, row % kRows);
  for (int e = threadIdx.x; e < kTokens * kHalf; e += kThreads) {
    const int at = e / kHalf, p = e % kHalf;
    if (t0 + at < P.T) {
      float2 v = axes_cs(P.tab, P.pos, P.T, t0 + at, p);
      if (P.inverse) v.y = -v.y;
      cs[at][p] = v;
    }
  }
  __syncthreads();
  if (t >= P.T) return;
  float2 mine[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) mine[e] = cs[tok][8 * chunk + e];
  for (int h = row % kRows; h < heads; h += kRows) {
    if (h >= kRows) load(x, h);
    x.turn(mine);
    x.store(h < P.Hq ? P.q_out + (t * P.Hq + h) * HD : P.k_out + (t * P.Hk + h - P.Hq) * HD, chunk);
  }
}

template <int HD, int L>
cudaError_t launch(const ApplyParams& P, cudaStream_t s) {
  if (P.T <= kFewTokens)
    rope_axes_kernel<HD, L, 1><<<(unsigned)P.T, kThreads, 0, s>>>(P);
  else
    rope_axes_kernel<HD, L, 2><<<(unsigned)((P.T + 1) / 2), kThreads, 0, s>>>(P);
  return cudaGetLastError();
}

}  // namespace

// [T, H, D] rows of `stride` elements: the bytes from the first element to the last
size_t rows_span(int64_t T, int64_t stride, int H, int D) { return (size_t)((T - 1) * stride + (int64_t)H * D) * 2; }

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

aa_status check_rows(const char* what, const void* x, int64_t stride, int H, int D) {
  if (!x || !aligned16(x)) return fail(AA_ERR_INVALID_ARG, std::string(what) + " must be a 16-byte aligned device pointer");
  if (stride < (int64_t)H * D || stride % 8 || stride >= (1ll << 38))
    return fail(AA_ERR_INVALID_ARG, std::string(what) + "'s token stride must be a multiple of 8 elements and >= heads * D");
  return AA_OK;
}

aa_status check_turned(const char* what, const void* x, int64_t stride, const void* out, int H, int D, int64_t T) {
  aa_status st = check_rows(what, x, stride, H, D);
  if (st != AA_OK) return st;
  if (!out || !aligned16(out))
    return fail(AA_ERR_INVALID_ARG, std::string(what) + "_out must be a 16-byte aligned device pointer");
  const bool in_place = out == x && stride == (int64_t)H * D;
  if (!in_place && overlap(x, rows_span(T, stride, H, D), out, (size_t)T * H * D * 2))
    return fail(AA_ERR_INVALID_ARG, std::string(what) + "_out overlaps " + what + " (in place needs a contiguous input)");
  return AA_OK;
}

}  // namespace aa

using namespace aa;

extern "C" aa_status aa_rope_axes_init(aa_rope_axes* r, int32_t head_dim, int32_t num_axes, int32_t layout,
                                       const int32_t* axis_of_pair, const double* theta) {
  if (!r) return fail(AA_ERR_INVALID_ARG, "rope is NULL");
  *r = aa_rope_axes{};
  if (!axis_of_pair || !theta) return fail(AA_ERR_INVALID_ARG, "axis_of_pair and theta are required");
  if (head_dim != 64 && head_dim != 128) return fail(AA_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
  if (num_axes < 1 || num_axes > 4) return fail(AA_ERR_INVALID_ARG, "num_axes must be in [1, 4]");
  if (layout != AA_ROPE_ADJACENT && layout != AA_ROPE_HALF)
    return fail(AA_ERR_INVALID_ARG, "layout must be AA_ROPE_ADJACENT or AA_ROPE_HALF");
  for (int p = 0; p < head_dim / 2; ++p) {
    if (axis_of_pair[p] < 0 || axis_of_pair[p] >= num_axes)
      return fail(AA_ERR_INVALID_ARG, "axis_of_pair[" + std::to_string(p) + "] must be in [0, num_axes)");
    if (!(theta[p] >= 0.0 && std::isfinite(theta[p])))
      return fail(AA_ERR_INVALID_ARG, "theta[" + std::to_string(p) + "] must be finite and >= 0");
  }
  r->head_dim = head_dim;
  r->num_axes = num_axes;
  r->layout = layout;
  for (int p = 0; p < head_dim / 2; ++p) {
    r->axis_of_pair[p] = axis_of_pair[p];
    const double turns = theta[p] / 6.283185307179586476925286766559;
    r->turn[p] = (uint64_t)std::ldexp(turns - std::floor(turns), 64);  // < 2^64: the fraction has 53 bits
  }
  r->ready = kAxesReady;
  return AA_OK;
}

extern "C" aa_status aa_rope_axes_apply(const aa_rope_axes* r, const int32_t* pos, int32_t T, const void* q,
                                        int64_t q_stride, void* q_out, int32_t q_heads, const void* k,
                                        int64_t k_stride, void* k_out, int32_t k_heads, int32_t inverse,
                                        aa_stream_t stream) {
  if (!axes_valid(r)) return fail(AA_ERR_INVALID_ARG, "rope must be filled by aa_rope_axes_init");
  if (T < 0 || T >= (1 << 30)) return fail(AA_ERR_INVALID_ARG, "total_tokens must be in [0, 2^30)");
  if (q_heads < 1 || k_heads < 0 || q_heads > 65536 || k_heads > 65536)
    return fail(AA_ERR_INVALID_ARG, "need q_heads >= 1 and k_heads >= 0 (at most 65536)");
  if (T == 0) return AA_OK;  // tensors without elements have no address
  if ((k_heads == 0) != (k == nullptr)) return fail(AA_ERR_INVALID_ARG, "k must be NULL exactly when k_heads is 0");
  if (!pos || (reinterpret_cast<uintptr_t>(pos) & 3u)) return fail(AA_ERR_INVALID_ARG, "pos must be a device pointer to int32");
  const int D = r->head_dim;
  aa_status st = check_turned("q", q, q_stride, q_out, q_heads, D, T);
  if (st != AA_OK) return st;
  if (k) {
    if ((st = check_turned("k", k, k_stride, k_out, k_heads, D, T)) != AA_OK) return st;
    const size_t nq = (size_t)T * q_heads * D * 2, nk = (size_t)T * k_heads * D * 2;
    if (overlap(q_out, nq, k_out, nk) || overlap(q_out, nq, k, rows_span(T, k_stride, k_heads, D)) ||
        overlap(k_out, nk, q, rows_span(T, q_stride, q_heads, D)))
      return fail(AA_ERR_INVALID_ARG, "q_out and k_out must not overlap each other or the other's input");
  }
  ApplyParams P;
  P.tab = axes_table(r);
  P.pos = pos;
  P.q = static_cast<const __nv_bfloat16*>(q);
  P.k = static_cast<const __nv_bfloat16*>(k);
  P.q_out = static_cast<__nv_bfloat16*>(q_out);
  P.k_out = static_cast<__nv_bfloat16*>(k_out);
  P.q_stride = q_stride;
  P.k_stride = k_stride;
  P.T = T;
  P.Hq = q_heads;
  P.Hk = k_heads;
  P.inverse = inverse != 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool adj = r->layout == AA_ROPE_ADJACENT;
  cudaError_t e = D == 128 ? (adj ? launch<128, 0>(P, s) : launch<128, 1>(P, s))
                           : (adj ? launch<64, 0>(P, s) : launch<64, 1>(P, s));
  return e == cudaSuccess ? AA_OK : cuda_fail(e, "rope_axes_kernel launch");
}
