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

// Four e4m3 numbers b0 .. b3 as bf16 pairs (b0, b2) and (b1, b3), exactly: sign, exponent
// and significand moved to their places in bf16 mean 2^-120 times the number (a
// subnormal one lands among bf16's subnormals); a product with `up`, a power of two, twice,
// makes that `up` * 2^-120 times. NaN codes become 480 times. (There is a conversion to f16,
// but none to bf16.)
__device__ __forceinline__ uint2 e4m3x4_to_bf16(uint32_t x, uint32_t up) {
  const uint32_t even = ((x << 4) & 0x07f007f0u) | ((x << 8) & 0x80008000u);
  const uint32_t odd = ((x >> 4) & 0x07f007f0u) | (x & 0x80008000u);
  uint2 r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r.x) : "r"(even), "r"(up));
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r.y) : "r"(odd), "r"(up));
  return r;
}

// 2^(byte - 127); NaN for 255, 0 for 0.
__device__ __forceinline__ float scale_of(uint32_t byte) {
  return __uint_as_float(byte << 23 | (byte == 255u ? 0x00400000u : 0u));
}

// The exponent that a scale's byte stands for; NaN for 255.
__device__ __forceinline__ float exponent_of(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float(0x4b000000u | byte) - 8388735.0f;  // 2^23 + byte - (2^23 + 127)
}

// What a row's codes are multiplied by, twice: e4m3x4_to_bf16's 2^120 times its scale, for a
// byte 2^(byte - 7). bf16 reaches 2^127; what is left is more_of(byte).
__device__ __forceinline__ uint32_t factor_of(int byte) {
  const uint32_t up = byte == 255 ? 0x7fc0u : (uint32_t)min(byte + 120, 254) << 7;
  return up | up << 16;
}
__device__ __forceinline__ bool has_more(int byte) { return byte > 134 && byte < 255; }
__device__ __forceinline__ uint32_t more_of(int byte) { return ((uint32_t)(byte - 7) << 7) * 0x10001u; }  // 2^(byte - 134)

// Sixteen codes as bf16, times `up`, exactly.
__device__ __forceinline__ void decode16(const uint4& x, uint32_t up, uint4 (&y)[2]) {
  const uint32_t four[4] = {x.x, x.y, x.z, x.w};
  uint32_t w[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {  // even and odd codes, then side by side
    const uint2 z = e4m3x4_to_bf16(four[e], up);
    w[2 * e] = __byte_perm(z.x, z.y, 0x5410);
    w[2 * e + 1] = __byte_perm(z.x, z.y, 0x7632);
  }
  y[0] = make_uint4(w[0], w[1], w[2], w[3]);
  y[1] = make_uint4(w[4], w[5], w[6], w[7]);
}
__device__ __forceinline__ void times16(uint4 (&y)[2], uint32_t by) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    for (uint32_t* w : {&y[i].x, &y[i].y, &y[i].z, &y[i].w}) asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(*w) : "r"(*w), "r"(by));
}
// Sixteen codes of a row whose scale has the byte `byte`.
__device__ __forceinline__ void decode16(const uint4& x, int byte, uint4 (&y)[2]) {
  decode16(x, factor_of(byte), y);
  if (has_more(byte)) times16(y, more_of(byte));
}

// Launch a kernel whose start-up may overlap the kernel before it (it waits with
// griddepcontrol.wait before it reads anything).
template <class... Params, class... Args>
cudaError_t launch_after(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
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
