// What the kernels of aa_cache_attend share: parameters, the keys that a group
// of rows visits, and where those keys lie in the pool.
#pragma once

#include "cache_common.cuh"

namespace aa {

constexpr uint64_t kAttendWaitNs = 2000000000ull;  // limit of every wait on a copy or a product

// A row's weights are 2^(sl2 * x - m), x its dot products, sl2 the softmax scale in log2 units: the
// product is exact in the fused operation, m is the rounded maximum. What its rounding is off by
// cancels in the weights and their sum, unless that is itself a large exponent: above this
// magnitude, in log2 units, more than 1. Over 8-bit pages such rows take a dot product off theirs
// first (1 % of a call, at 64 channels 2 %).
constexpr float kFarMax = 16777216.0f;  // 2^24

struct AttendParams {
  BatchParams batch;
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;
  const int32_t* key_lo;
  int64_t q_stride;
  int Hq, group, anchor, page_shift;
  float scale_log2;    // softmax scale * log2 e
  // 8-bit pages: a byte per token and kv head, as aa_cache_s has them
  const uint8_t *k_scales, *v_scales;
  // drafted trees: [T, tree_words] masks of the new tokens, NULL without
  const uint64_t* tree;
  int tree_words;
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

// Drafted trees: which of the keys j + x, x < 64, that are new tokens row t of the
// batch sees, the n new ones of its sequence lying at [base, base + n). Bit x. Keys
// in front of base have none.
__device__ __forceinline__ uint64_t tree_keys(const AttendParams& P, int64_t t, int base, int n, int j) {
  const int c = j - base;  // the new token that bit 0 stands for
  if (c <= -64 || c >= n) return 0;
  const uint64_t* row = P.tree + t * P.tree_words;
  const int w = c >> 6, shift = c & 63;  // c < 0: word -1 does not exist
  uint64_t bits = w >= 0 && w < P.tree_words ? __ldg(row + w) >> shift : 0;
  if (shift && w + 1 < P.tree_words) bits |= __ldg(row + w + 1) << (64 - shift);
  return n - c < 64 ? bits & ((1ull << (n - c)) - 1) : bits;
}

// Bit x: key j + x lies in [lo, hi], x < 64.
__device__ __forceinline__ uint64_t keys_between(int j, int lo, int hi) {
  const int last = hi - j, first = lo - j;
  const uint64_t upto = last < 0 ? 0ull : last >= 63 ? ~0ull : (2ull << last) - 1ull;
  return first <= 0 ? upto : first > 63 ? 0ull : upto & (~0ull << first);
}

// seen_keys() for drafted trees: bit x, some of the tokens q_row + i (i < tokens, the
// sequence's new tokens i0 + i) sees key j + x (a whole warp asks). Keys that are no new
// tokens count as seen: in front of base the rows together see all from their smallest
// first key on, and behind the last there are none.
__device__ __forceinline__ uint64_t tree_seen_keys(const AttendParams& P, int q_row, int i0, int tokens, int base, int n, int j) {
  uint64_t any = 0;
  for (int i = threadIdx.x & 31; i < tokens; i += 32)
    if (base + i0 + i >= 0) any |= tree_keys(P, q_row + i, base, n, j);
  any = (uint64_t)__reduce_or_sync(0xffffffffu, (uint32_t)(any >> 32)) << 32 | __reduce_or_sync(0xffffffffu, (uint32_t)any);
  return any | ~keys_between(j, base, base + n - 1);
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

// Up to so many keys per page table the chunk kernel takes whole units. Measured,
// 32 / 8 heads of 128, microseconds whole / cut: 8 sequences of 32 new tokens over
// 700 keys 17.5 / 21.5, 42 of 128 over 500 65.6 / 85.4; over 1000 keys 21.0 / 22.9
// and 99.7 / 118, but one of 32 20.0 / 15.6; over 2000 20 of 32 69.1 / 62.1.
constexpr int kWholeKeys = 768;

// Launchers (arguments already checked) and the workspaces they need.
// short: at most kShortRows rows (max_q * group) of a sequence and kv head at a time.
constexpr int kShortRows = 64;
cudaError_t launch_attend_short(const aa_cache_s* c, const AttendParams& P, int max_q, void* workspace, cudaStream_t s);
cudaError_t launch_attend_short_fp8(const aa_cache_s* c, const AttendParams& P, int max_q, void* workspace, cudaStream_t s);
size_t short_workspace_bytes(const aa_cache_s* c, int num_seqs, int total_tokens, int max_q, int table_width, int group);
aa_status launch_attend_chunk(const aa_cache_s* c, const AttendParams& P, void* workspace, cudaStream_t s);
aa_status launch_attend_chunk_fp8(const aa_cache_s* c, const AttendParams& P, void* workspace, cudaStream_t s);
size_t chunk_workspace_bytes(const aa_cache_s* c, int num_seqs, int total_tokens, int table_width, int group, bool from_codes);
// 8-bit pages by way of 16-bit copies of a few sequences at a time, kWideBytes at most.
constexpr size_t kWideBytes = 1ull << 30;
bool wide_fits(const aa_cache_s* c, int table_width);
size_t wide_workspace_bytes(const aa_cache_s* c, int num_seqs, int total_tokens, int table_width, int group);
aa_status launch_attend_wide(const aa_cache_s* c, const AttendParams& P, void* workspace, cudaStream_t s);

}  // namespace aa
