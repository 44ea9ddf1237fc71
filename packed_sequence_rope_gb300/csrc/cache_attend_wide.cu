// Attention of chunks over 8-bit pages by way of 16-bit copies.
//
// A chunk of many rows reads each key once per 256 rows. Making codes bf16 takes as many
// instructions as a row tile's softmax, so doing it for every unit (cache_attend_chunk.cuh)
// holds the tensor cores up; here wide_kernel does it once, into the workspace, [sequence, kv
// head, key, D] in rows, and the chunk kernel of 16-bit pages runs over that. 2048 tokens over
// 32K keys, 32 / 8 heads of 128: 799 us, of which the copies 37 (5.4 TB/s); converting in
// every unit 2200. The copies of a few sequences at a time keep the workspace small.
#include <algorithm>

#include "cache_attend_chunk.cuh"

namespace aa {
namespace {

constexpr int kWideThreads = 256, kWideKeys = 128;  // keys of a block

struct WideParams {
  AttendParams a;
  const uint8_t *k_pages, *v_pages;
  uint4 *k, *v;
  int wide_keys;
};

// Keys [kWideKeys x, kWideKeys (x + 1)) of kv head y of sequence z. Keys in front of every
// row's first one are left out.
template <int HD>
__global__ void __launch_bounds__(kWideThreads) wide_kernel(const __grid_constant__ WideParams W) {
  constexpr int kChunks = HD / 16, kRows = kWideThreads / kChunks;  // 16-byte chunks of a row, rows at a time
  const AttendParams& P = W.a;
  const BatchParams& b = P.batch;
  const int seq = (int)blockIdx.z, g = (int)blockIdx.y, j0 = (int)blockIdx.x * kWideKeys;
  const SeqSpan s = load_seq(b, seq, P.page_shift);
  if (s.n == 0 || j0 >= __ldg(b.kv_len + seq)) return;
  if (P.key_lo && !(P.anchor && j0 == 0)) {
    int lo = P.tree ? max(s.kv - s.n, 0) : INT_MAX;
    for (int i = threadIdx.x; i < s.n; i += kWideThreads) lo = min(lo, first_key(P, s.q0 + i));
    if (!__syncthreads_or(lo < j0 + kWideKeys)) return;
  }
  const int chunk = threadIdx.x % kChunks;
  // more tokens than the page table has room for: an error, and zeros
  const int end = min(j0 + kWideKeys, __ldg(b.kv_len + seq) > s.kv ? W.wide_keys : s.kv);
#pragma unroll 2
  for (int j = j0 + threadIdx.x / kChunks; j < end; j += kRows) {
    const int row = j < s.kv ? pool_row(b, seq, g, j, P.page_shift) : kNoRow;
    const int64_t to = ((int64_t)(seq * b.Hkv + g) * W.wide_keys + j) * (HD / 8) + 2 * chunk;
    uint4 yk[2], yv[2];
    const uint4 none = make_uint4(0, 0, 0, 0);  // a page that is none reads as zeros
    const int64_t at = (int64_t)row * HD + 16 * chunk;
    decode16(row < 0 ? none : __ldg(reinterpret_cast<const uint4*>(W.k_pages + at)), row < 0 ? 127 : (int)__ldg(P.k_scales + row), yk);
    decode16(row < 0 ? none : __ldg(reinterpret_cast<const uint4*>(W.v_pages + at)), row < 0 ? 127 : (int)__ldg(P.v_scales + row), yv);
    W.k[to] = yk[0];
    W.k[to + 1] = yk[1];
    W.v[to] = yv[0];
    W.v[to + 1] = yv[1];
  }
}

// Rows of a sequence and kv head in the copies: whole pieces of 64.
int64_t wide_keys(const aa_cache_s* c, int table_width) { return ((int64_t)table_width * c->cfg.page_size + 63) / 64 * 64; }
// Bytes of one sequence's copies of keys (or values).
size_t wide_bytes(const aa_cache_s* c, int table_width) {
  return (size_t)wide_keys(c, table_width) * c->cfg.num_kv_heads * c->cfg.head_dim * 2;
}
// Sequences copied at a time.
int wide_seqs(const aa_cache_s* c, int num_seqs, int table_width) {
  return (int)std::min<size_t>(num_seqs, std::min<size_t>(65535, kWideBytes / (2 * wide_bytes(c, table_width))));
}

}  // namespace

bool wide_fits(const aa_cache_s* c, int table_width) {
  return c->cfg.num_kv_heads <= 65535 && 2 * wide_bytes(c, table_width) <= kWideBytes;
}

size_t wide_workspace_bytes(const aa_cache_s* c, int num_seqs, int total_tokens, int table_width, int group) {
  const int some = wide_seqs(c, num_seqs, table_width);
  return chunk_workspace_bytes(c, some, total_tokens, table_width, group, false) + 2 * align256(some * wide_bytes(c, table_width));
}

aa_status launch_attend_wide(const aa_cache_s* c, const AttendParams& P, void* workspace, cudaStream_t s) {
  const BatchParams& b = P.batch;
  const int D = c->cfg.head_dim, some = wide_seqs(c, b.B, b.W), keys = (int)wide_keys(c, b.W);
  uint8_t* w = static_cast<uint8_t*>(workspace) + chunk_workspace_bytes(c, some, b.T, b.W, P.group, false);
  WideParams wide{P, static_cast<const uint8_t*>(c->k_pages), static_cast<const uint8_t*>(c->v_pages), nullptr, nullptr, keys};
  wide.k = reinterpret_cast<uint4*>(w);
  wide.v = reinterpret_cast<uint4*>(w + align256(some * wide_bytes(c, b.W)));
  CUtensorMap k_map, v_map;
  aa_status st = make_pool_map(&k_map, wide.k, (int64_t)some * b.Hkv * keys, D, 64);
  if (st == AA_OK) st = make_pool_map(&v_map, wide.v, (int64_t)some * b.Hkv * keys, D, 64);
  for (int first = 0; first < b.B && st == AA_OK; first += some) {
    AttendParams& A = wide.a;
    A.batch = b;
    A.batch.B = std::min(some, b.B - first);
    A.batch.table += (int64_t)first * b.W;
    A.batch.cu_q += first;
    A.batch.kv_len += first;
    const dim3 grid((unsigned)((keys + kWideKeys - 1) / kWideKeys), (unsigned)b.Hkv, (unsigned)A.batch.B);
    if (D == 128)
      wide_kernel<128><<<grid, kWideThreads, 0, s>>>(wide);
    else
      wide_kernel<64><<<grid, kWideThreads, 0, s>>>(wide);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "wide_kernel launch");
    AttendParams R = A;  // the copies are pages of 64 keys, one after the other
    R.batch.W = keys / 64;
    R.page_shift = 6;
    st = launch_chunk<kFromWide>(c, R, k_map, v_map, keys, workspace, s);
  }
  return st;
}

}  // namespace aa
