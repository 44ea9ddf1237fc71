// What the kernels of aa_cache_attend share: parameters, the keys that a group
// of rows visits, and where those keys lie in the pool.
#pragma once

#include "cache_common.cuh"

namespace aa {

constexpr uint64_t kAttendWaitNs = 2000000000ull;  // limit of every wait on a copy or a product

struct AttendParams {
  BatchParams batch;
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;
  const int32_t* key_lo;
  int64_t q_stride;
  int Hq, group, anchor, page_shift;
  float scale_log2;    // softmax scale * log2 e
};

// New tokens [q0, q0 + n) of sequence b that hold kv tokens. Rows outside the
// tensors are cut off, whatever cu_q says; more tokens than the page table has
// room for are an error, and the rest is not visited.
struct SeqSpan {
  int q0, n, kv;
};
__device__ __forceinline__ SeqSpan load_seq(const BatchParams& b, int seq, int page_shift) {
  SeqSpan s;
  s.q0 = __ldg(b.cu_q + seq);
  s.n = min(__ldg(b.cu_q + seq + 1), b.T) - s.q0;
  s.kv = max(__ldg(b.kv_len + seq), 0);
  if (s.q0 < 0 || s.n < 0) s.n = 0;
  if (s.n > 0 && s.kv > b.W << page_shift) {
    atomicCAS(b.err, 0, kCacheBadPosition);
    s.kv = b.W << page_shift;
  }
  return s;
}

// The first key that row t of the batch sees (positions stay below 2^30).
__device__ __forceinline__ int first_key(const AttendParams& P, int t) {
  return P.key_lo ? min(max(__ldg(P.key_lo + t), 0), 1 << 30) : 0;
}

// Bit x: some of the tokens q_row + i (i < tokens, at positions p0 + i) sees key
// j + x, x < 64 (a whole warp asks). Together they see every key from the smallest
// first key to the last position, unless some of them see nothing.
__device__ __forceinline__ uint64_t seen_keys(const AttendParams& P, int q_row, int p0, int tokens, int j) {
  const int a = j + (threadIdx.x & 31), b = a + 32;
  bool sees_a = P.anchor && a == 0 && p0 + tokens > 0, sees_b = false;
#pragma unroll 1
  for (int i = max(j - p0, 0); i < tokens; ++i) {
    const int lo = first_key(P, q_row + i), hi = p0 + i;
    sees_a |= lo <= a && a <= hi;
    sees_b |= lo <= b && b <= hi;
  }
  return __ballot_sync(0xffffffffu, sees_a) | (uint64_t)__ballot_sync(0xffffffffu, sees_b) << 32;
}

// Four channels of a row divided by its sum, in bf16; 0 for a row that saw
// nothing (a NaN among its logits makes the sum NaN, and the row).
__device__ __forceinline__ uint2 normalised(const float4& o, float sum) {
  if (sum == 0.f) return make_uint2(0u, 0u);
  const float inv = 1.f / sum;
  return make_uint2(ptx::pack_bf16x2(o.x * inv, o.y * inv), ptx::pack_bf16x2(o.z * inv, o.w * inv));
}

// The key tiles (kKeys wide) that rows with first keys >= lo and positions <=
// hi visit: [lo, hi], and before them tile 0 if only the anchor lies there.
template <int kKeys>
struct KeyTiles {
  int first, count, anchor_tile;
  __device__ __forceinline__ KeyTiles(int lo, int hi, bool anchor) {
    first = lo / kKeys;
    const int in = lo <= hi ? hi / kKeys - first + 1 : 0;
    anchor_tile = (anchor && hi >= 0 && (in == 0 || first > 0)) ? 1 : 0;
    count = in + anchor_tile;
  }
  __device__ __forceinline__ int tile(int i) const { return i < anchor_tile ? 0 : first + i - anchor_tile; }
};

// Pool row of the page that holds position j of sequence b for head g; a row
// outside the pool (which a tensor copy fills with zeros) if there is none. j lies
// in [0, the sequence's kv).
constexpr int kNoRow = -128;
__device__ __forceinline__ int pool_row(const BatchParams& b, int seq, int g, int j, int page_shift) {
  const int page = __ldg(b.table + (int64_t)seq * b.W + (j >> page_shift));  // j < kv <= W * page size
  if (page < 0 || page >= b.num_pages) {
    atomicCAS(b.err, 0, kCacheBadPage);
    return kNoRow;
  }
  return (int)((((b.layer_page0 + page) * b.Hkv + g) << page_shift) + (j & ((1 << page_shift) - 1)));
}

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

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

// Up to so many keys per page table the chunk kernel takes whole units. Measured,
// 32 / 8 heads of 128, microseconds whole / cut: 8 sequences of 32 new tokens over
// 700 keys 17.5 / 21.5, 42 of 128 over 500 65.6 / 85.4; over 1000 keys 21.0 / 22.9
// and 99.7 / 118, but one of 32 20.0 / 15.6; over 2000 20 of 32 69.1 / 62.1.
constexpr int kWholeKeys = 768;

// Launchers (arguments already checked) and the workspaces they need.
// short: at most kShortRows rows (max_q * group) of a sequence and kv head at a time.
constexpr int kShortRows = 64;
cudaError_t launch_attend_short(const aa_cache_s* c, const AttendParams& P, int max_q, void* workspace, cudaStream_t s);
size_t short_workspace_bytes(const aa_cache_s* c, int num_seqs, int total_tokens, int max_q, int table_width, int group);
aa_status launch_attend_chunk(const aa_cache_s* c, const AttendParams& P, void* workspace, cudaStream_t s);
size_t chunk_workspace_bytes(const aa_cache_s* c, int num_seqs, int total_tokens, int table_width, int group);

}  // namespace aa
