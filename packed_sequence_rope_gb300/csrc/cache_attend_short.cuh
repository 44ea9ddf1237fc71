// Attention of few new tokens per sequence (a decoding step, drafted tokens)
// over the paged cache.
//
// The work is reading K and V once: 512 bytes per key and kv head at D = 128
// for a handful of rows, so HBM bounds it and the matrix products only have to
// keep up. One cluster of CTAs takes a unit: the query heads of one kv head for
// 16 * RT rows (row = token * group + head) of one sequence, so each key is
// read once for all of them. The cluster's CTAs split the unit's 64-key tiles
// evenly; each runs
//   warp 4    the producer: page numbers from the table, tensor copies of the
//             tile's pages into a ring of stages, 128-byte swizzled
//   warps 0-3 RT row groups x 4 / RT key groups: S = Q K^T and O += P V with
//             16x8x16 products (M = 16 rows are enough; tcgen05's 128 rows would
//             leave the accumulators' way through tensor memory as the only thing
//             in the critical path), online softmax in registers
// and at the end the warps' partial results are joined in shared memory, the
// CTAs' through distributed shared memory: one launch, no workspace, and the
// same order of additions in every run. Where the units times a cluster's CTAs do
// not fill the GPU (one user with a long context), each unit gets several
// clusters; their results go to the workspace and a second kernel joins them.
//
// 8-bit pages (k8) take the same path at half of the bytes; what bounds it then is the
// work on each key. A key's 16 codes of a product step are one 16-byte row of a matrix
// load, 4 codes per lane; made f16 (one conversion for two codes, exact; to bf16 there
// is none, and its four bit operations and a product made a decoding step of 64
// sequences to 32K keys 627 us) they are the step's operand with its channels in another
// order, which the queries' operand shares. Loaded transposed, a lane's codes are two
// channels of two keys: operands of two products, for the even and the odd channels.
// The other operands are f16 then, brought into its range by powers of two. A row of
// queries is multiplied by the one that takes its maximum to 2^14: what is above 2^-21 of
// the maximum stays exact, the rest is off by at most 2^-39 of it. The keys' scales
// multiply what the products give, the logits s. A value's scale 2^e joins its weight, 2^(s + e - m) with m the
// row's running maximum of s + e, times 2^7. Weights are then below 2^15; those above 2^-21
// of the largest are rounded to 11 bits, the others are off by at most 2^-32 of it. The
// weights' sum is fp32 with a maximum of its own: scales of tokens may lie far apart.
#pragma once

#include <cfloat>
#include <type_traits>

#include "cache_attend.cuh"

namespace aa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * (kWarps + 1);
constexpr float kRescaleThreshold = 8.0f;  // log2 units: O is rescaled only when the max grows by > 2^8

constexpr float kWeightsUp = 7.0f;      // 8-bit pages: weights are 2^7 times what the maximum gives, at most 2^15
constexpr float kFarLogit = 1024.0f;    // log2 units: logits and exponents below are added with an error of 2^-14

constexpr int kSplitRanks = 4, kSplitTiles = 8;

// Results of the clusters of a unit: [split][row][query head], unnormalised O and
// (maximum in log2 units, sum).
struct ShortParts {
  int splits;
  float4* o;
  float2* ml;
};

// Keys of a tile. With 8-bit pages what a tile costs beside its keys (waits, maxima across
// lanes) counts for more: 64 sequences to 32K keys 522 us with 64 keys, 450 with 128. At 32
// rows a warp has 64 of 128 keys, which its registers do not hold: 42 sequences over 2048
// and 16K keys 90.3 and 482 us with 64, 98.1 and 466 with 128; of 64 channels 57.5 and 335,
// 69.7 and 502.
template <int RT, bool k8>
constexpr int kTileOf = k8 && RT == 1 ? 128 : 64;

template <int HD, int RT, bool k8>
struct ShortSmem {
  static constexpr int kTileKeys = kTileOf<RT, k8>;
  static constexpr int kB = k8 ? 1 : HD / 64;            // column blocks of a tile
  static constexpr int kRowBytes = k8 ? HD : 128;        // of a key in a block
  static constexpr int kStages = k8 ? (RT == 1 ? 3 : 6) : HD == 128 ? 3 : 4;
  static constexpr int kRowFloats = HD + 8;  // a warp's rows fall on different banks
  union {
    struct {
      alignas(1024) uint8_t k[kStages][kB][kTileKeys * kRowBytes];
      alignas(1024) uint8_t v[kStages][kB][kTileKeys * kRowBytes];
      alignas(16) uint8_t scales[k8 ? kStages : 1][2][k8 ? kTileKeys : 16];  // 8-bit pages: the keys', the values'
    };
    struct {  // after the last tile
      float part[kWarps][16][kRowFloats];  // each warp's O
      float merged[64][HD];                // the CTA's O, 16 * RT rows of it
    };
  };
  float m[kWarps][16], l[kWarps][16];
  float cta_m[64], cta_l[64];
  uint64_t full[kStages], empty[kStages];
};

// A converged warp waits, bounded; one lane asks for all.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int32_t* err, int site) {
  bool ok = true;
  if ((threadIdx.x & 31) == 0) ok = ptx::mbar_wait(bar, parity, kAttendWaitNs, err, site);
  return __all_sync(0xffffffffu, ok);
}

// What a call's masks need. kMaskLo: it has key_lo. Its looks for unseen keys between seen ones cost the
// other calls 1 to 4 % where they are compiled in (on the GPU: one token over 1000
// keys 6.98 us, 6.79 without them; seven tokens of eight sequences over 700, D = 64,
// 9.3 and 8.95). kMaskTree: drafted trees, with or without key_lo.
enum ShortMask { kMaskNone, kMaskLo, kMaskTree };

// The 16-byte chunk of a key's row in a tile of 8-bit pages: swizzled by 128 or 64 bytes.
template <int HD>
__device__ __forceinline__ uint32_t chunk_fp8(int key, int chunk) {
  return HD == 128 ? sw128_chunk(key, chunk) : (uint32_t)(key * 64 + ((chunk ^ (key >> 1 & 3)) << 4));
}

template <int HD, int RT, int kMask, bool k8>
__global__ void __launch_bounds__(kThreads, HD == 128 ? 2 : k8 ? 4 : 3)
    attend_short_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                        const __grid_constant__ AttendParams P, const ShortParts S) {
  using Smem = ShortSmem<HD, RT, k8>;
  constexpr bool kLo = kMask != kMaskNone, kTree = kMask == kMaskTree;
  constexpr int kTileKeys = Smem::kTileKeys, kB = Smem::kB, kRowBytes = Smem::kRowBytes, kStages = Smem::kStages;
  constexpr int kKeyGroups = kWarps / RT, kWarpKeys = kTileKeys / kKeyGroups;
  constexpr uint32_t kStageBytes = 2 * kTileKeys * kB * kRowBytes;
  static_assert(kWarpKeys <= 64, "a warp's keys are one window of bits");
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if (ptx::smem_u32(smem_raw) & 1023u) {  // swizzled tiles need a 1 KB aligned base
    if (threadIdx.x == 0) atomicCAS(P.batch.err, 0, 498);
    return;
  }
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  const BatchParams& b = P.batch;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ranks = ptx::cluster_size(), rank = ptx::cluster_rank();
  const int64_t shares = (int64_t)ranks * S.splits, share = (int64_t)ranks * blockIdx.y + rank;  // of a unit's tiles
  const int unit = (int)(blockIdx.x / ranks);
  const int g = unit % b.Hkv, seq = unit / b.Hkv;
  const int tile_tokens = 16 * RT / P.group;
  auto set_up = [&] {
    if (tid == 0) {
      ptx::tma_prefetch_desc(&tmK);
      ptx::tma_prefetch_desc(&tmV);
      for (int s = 0; s < kStages; ++s) {
        ptx::mbar_init(&sm.full[s], 1);
        ptx::mbar_init(&sm.empty[s], kWarps);
      }
      ptx::fence_mbar_init();
    }
    __syncthreads();
  };
  // 8-bit pages: launched as a dependent, whose start-up overlaps the kernel before (one token over
  // 1000 keys 10.2 us to 7.7; 7.9 with the second loop below)
  if constexpr (k8) {
    set_up();
    asm volatile("griddepcontrol.wait;" ::: "memory");
  }
  const SeqSpan span = load_seq(b, seq, P.page_shift);
  if constexpr (!k8) set_up();

  int steps = 0;  // tiles this CTA has taken so far: the ring's position
  // one pass, unless the sequence has more new tokens than max_q promised
  for (int i0 = 0; i0 < span.n; i0 += tile_tokens) {
    const int tokens = min(tile_tokens, span.n - i0), rows = tokens * P.group;
    // positions of the first and last row; the rows of a tree may see all new tokens
    const int base = span.kv - span.n, p0 = base + i0, hi = kTree ? span.kv - 1 : p0 + tokens - 1;
    const bool anchor = P.anchor && (!kTree || base > 0);
    int lo = 0;
    if constexpr (kLo) {
      lo = INT_MAX;
      for (int i = lane; i < tokens; i += 32) lo = min(lo, first_key(P, span.q0 + i0 + i));
      lo = __reduce_min_sync(0xffffffffu, lo);
      if (kTree) lo = min(lo, max(base, 0));
    }
    const KeyTiles<kTileKeys> keys(lo, hi, anchor);
    const int begin = (int)(keys.count * share / shares), end = (int)(keys.count * (share + 1) / shares);

    if (warp == kWarps) {
      // ---------------------------------------------------------- producer
      // a tile is `pages` pieces of `piece` rows, each kB column blocks of K and V
      const int piece_shift = min(P.page_shift, 6), pieces = kTileKeys >> piece_shift;
      const int copies = pieces * kB * 2;  // at most 16: one per lane
      const int at = lane & (pieces - 1), block = (lane / pieces) % kB;
      const bool is_v = lane >= pieces * kB;
      auto row_of = [&](int i) {
        const int j = keys.tile(i) * kTileKeys + (at << piece_shift);
        // pieces that no row sees are not looked up
        const bool seen = j <= hi && (j + (1 << piece_shift) > lo || (j == 0 && anchor));
        return lane < copies && i < end && seen ? pool_row(b, seq, g, j, P.page_shift) : kNoRow;
      };
      bool ok = true;
      int issued = 0, next = row_of(begin);
      for (int i = begin; i < end && ok; ++i) {
        const int n = steps + i - begin, s = n % kStages;
        const int row = next;
        next = row_of(i + 1);  // in flight while this stage is waited for
        if (n >= kStages)
          ok = warp_wait(&sm.empty[s], (n / kStages - 1) & 1, b.err, 401);
        if (!ok) break;
        if constexpr (k8) {
          // the scales of pieces that are not looked up: zeros, as their codes will be
          const bool none = lane < copies && row < 0;
          uint8_t* scales = sm.scales[s][is_v] + (at << piece_shift);
          if (none) {
            for (int x = 0; x < 1 << piece_shift; x += 16) *reinterpret_cast<uint4*>(scales + x) = make_uint4(0, 0, 0, 0);
            ptx::fence_proxy_async_smem();  // this lane's next copy to the same bytes comes after
          }
          const int scaled = __popc(__ballot_sync(0xffffffffu, lane < copies && row >= 0));
          __syncwarp();  // the zeros before the arrival
          if (lane == 0) ptx::mbar_arrive_expect_tx(&sm.full[s], kStageBytes + (uint32_t)(scaled << piece_shift));
          __syncwarp();
          if (lane < copies) {
            ptx::tma_load_2d((is_v ? sm.v[s][0] : sm.k[s][0]) + (at << piece_shift) * kRowBytes, is_v ? &tmV : &tmK,
                             &sm.full[s], 0, row);
            if (!none)
              ptx::bulk_load(scales, (is_v ? P.v_scales : P.k_scales) + row, 1u << piece_shift, &sm.full[s]);
          }
        } else {
          if (lane == 0) ptx::mbar_arrive_expect_tx(&sm.full[s], kStageBytes);
          __syncwarp();
          if (lane < copies) {
            uint8_t* dst = (is_v ? sm.v[s][block] : sm.k[s][block]) + (at << piece_shift) * 128;
            ptx::tma_load_2d(dst, is_v ? &tmV : &tmK, &sm.full[s], block * 64, row);
          }
        }
        ++issued;
      }
      // every copy lands before the stages' memory is used for anything else
      for (int n = max(steps + issued - kStages, steps); n < steps + issued; ++n)
        warp_wait(&sm.full[n % kStages], (n / kStages) & 1, b.err, 403);
    } else {
      // ---------------------------------------------------------- products and softmax
      const int rg = warp % RT, kg = warp / RT;  // row group, key group
      const int row0 = rg * 16 + (lane >> 2);
      int row_lo[2], row_hi[2];  // this lane's two rows' visible keys
      uint32_t qf[HD / 16][4];
      float sl2[2] = {P.scale_log2, P.scale_log2};  // 8-bit pages: and what takes the row's power of two off again
      bool careful = false;  // 8-bit pages: logits far from 0, see below
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = row0 + 8 * e, tok = row / P.group;
        const bool on = row < rows;
        row_lo[e] = kLo && on ? first_key(P, span.q0 + i0 + tok) : 0;
        row_hi[e] = !on ? INT_MAX : kTree ? (p0 + tok < 0 ? -1 : base - 1) : p0 + tok;
        const __nv_bfloat16* q = P.q + (int64_t)(span.q0 + i0 + tok) * P.q_stride +
                                 (int64_t)(g * P.group + row - tok * P.group) * HD + (k8 ? 4 : 2) * (lane & 3);
#pragma unroll
        for (int ks = 0; ks < HD / 16; ++ks) {
          if constexpr (k8) {
            const uint2 x = on ? __ldg(reinterpret_cast<const uint2*>(q + ks * 16)) : make_uint2(0u, 0u);
            qf[ks][e] = x.x;
            qf[ks][e + 2] = x.y;
          } else {
            qf[ks][e] = on ? __ldg(reinterpret_cast<const uint32_t*>(q + ks * 16)) : 0u;
            qf[ks][e + 2] = on ? __ldg(reinterpret_cast<const uint32_t*>(q + ks * 16 + 8)) : 0u;
          }
        }
      }
      if constexpr (k8) {
        // to f16 by the power of two that brings the row's largest finite magnitude to [2^14, 2^15)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t top = 0;
#pragma unroll
          for (int ks = 0; ks < HD / 16; ++ks)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const uint32_t u = (qf[ks][e + (x & 2)] >> (x & 1) * 16) & 0x7fffu;
              top = max(top, u < 0x7f80u ? u : 0u);
            }
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const uint32_t up = top ? min(268u - (top >> 7), 253u) : 127u;  // biased exponent of the power
          const float by = __uint_as_float(up << 23), back = __uint_as_float((254u - up) << 23);
          // A product (below 2^31) becomes a logit by way of sl2, then its key's scale (2^-124 to
          // 2^119): what stands between stays in fp32's range for queries of some 2^-100 to 2^100. Of
          // other rows a part of sl2 is left for the end.
          float rest = 1.f;
          sl2[e] *= back;
          if (sl2[e] < 0x1p-120f) {
            rest = fmaxf(P.scale_log2 * 0x1p100f * back, FLT_MIN);
            sl2[e] = 0x1p-100f;
          } else if (sl2[e] >= 0x1p90f) {
            rest = fminf(P.scale_log2 * 0x1p-60f * back, FLT_MAX);
            sl2[e] = 0x1p60f;
          }
          sm.m[warp][(lane >> 2) + 8 * e] = rest;
          sm.l[warp][(lane >> 2) + 8 * e] = 0.f;  // r, see below
          careful |= rest != 1.f;
#pragma unroll
          for (int ks = 0; ks < HD / 16; ++ks) {
            const float2 a = ptx::unpack_bf16x2(qf[ks][e]), c = ptx::unpack_bf16x2(qf[ks][e + 2]);
            qf[ks][e] = ptx::pack_f16x2(a.x * by, a.y * by);      // channels 0 and 1 of the lane's four
            qf[ks][e + 2] = ptx::pack_f16x2(c.x * by, c.y * by);  // 2 and 3
          }
        }
        careful = __any_sync(0xffffffffu, careful);
        __syncwarp();
      }
      const int all_lo = __reduce_max_sync(0xffffffffu, max(row_lo[0], row_lo[1]));
      const int all_hi = __reduce_min_sync(0xffffffffu, min(row_hi[0], row_hi[1]));
      float o[HD / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
      float lane_m[2] = {-INFINITY, -INFINITY};  // 8-bit pages: what l is relative to, each lane's own
#pragma unroll
      for (int e = 0; e < HD / 8; ++e) o[e][0] = o[e][1] = o[e][2] = o[e][3] = 0.f;

      // Tile i. 8-bit pages: a careful one multiplies what is left of sl2, and since next to a large
      // logit an exponent loses bits (from 2^24 on all of them), its logits, m and lane_m are
      // relative to a logit of the row's, r. A tile that is not gives up, before it changes anything,
      // where it meets a logit that would need it. (In one loop that is 4 to 9 % of a call at D = 64.)
      enum Outcome { kDone, kNeedsCare, kTimeout };
      auto take = [&](auto with_care, int i) __attribute__((always_inline)) {
        constexpr bool kCareful = decltype(with_care)::value;
        const int n = steps + i - begin, s = n % kStages;
        if (!warp_wait(&sm.full[s], (n / kStages) & 1, b.err, 402)) return kTimeout;
        const int j0 = keys.tile(i) * kTileKeys, jw = j0 + kg * kWarpKeys;  // the tile's, the warp's first key
        float sc[kWarpKeys / 8][4];
#pragma unroll
        for (int e = 0; e < kWarpKeys / 8; ++e) sc[e][0] = sc[e][1] = sc[e][2] = sc[e][3] = 0.f;
        if constexpr (k8) {
#pragma unroll
          for (int e = 0; e < kWarpKeys / 8; ++e) {
#pragma unroll
            for (int c = 0; c < HD / 64; ++c) {
              // matrices: four 16-channel steps of eight keys
              uint32_t kf[4];
              ptx::ldmatrix4(ptx::smem_u32(sm.k[s][0]) + chunk_fp8<HD>(kg * kWarpKeys + e * 8 + (lane & 7), c * 4 + (lane >> 3)), kf);
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                ptx::mma_16816_f16(sc[e], qf[c * 4 + x], ptx::e4m3x2_to_f16((uint16_t)kf[x]),
                                   ptx::e4m3x2_to_f16((uint16_t)(kf[x] >> 16)));
              }
            }
            const int at = kg * kWarpKeys + e * 8 + 2 * (lane & 3);
            const uint32_t of_k = *reinterpret_cast<const uint16_t*>(&sm.scales[s][0][at]);
            const float s0 = scale_of(of_k & 255u), s1 = scale_of(of_k >> 8);
#pragma unroll
            for (int x = 0; x < 4; ++x) sc[e][x] = sc[e][x] * sl2[x >> 1] * (x & 1 ? s1 : s0);
          }
        } else {
#pragma unroll
          for (int ks = 0; ks < HD / 16; ++ks) {
#pragma unroll
            for (int kp = 0; kp < kWarpKeys / 16; ++kp) {
              // matrices: keys 0-7 and 8-15 of the pair, channels 0-7 and 8-15 of the step
              const int key = kg * kWarpKeys + kp * 16 + (lane & 7) + ((lane >> 4) << 3);
              uint32_t kf[4];
              ptx::ldmatrix4(ptx::smem_u32(sm.k[s][ks >> 2]) + sw128_chunk(key, (ks & 3) * 2 + ((lane >> 3) & 1)), kf);
              ptx::mma_16816(sc[2 * kp], qf[ks], kf[0], kf[1]);
              ptx::mma_16816(sc[2 * kp + 1], qf[ks], kf[2], kf[3]);
            }
          }
        }
        const bool edge = jw < all_lo || jw + kWarpKeys - 1 > all_hi;
        if (edge) {
          uint64_t tree[2] = {0, 0};  // the lane's rows: new tokens among the warp's keys
          if constexpr (kTree) {
            if (jw + kWarpKeys > base) {
#pragma unroll
              for (int w = 0; w < 2; ++w) {
                const int row = row0 + 8 * w, tok = row / P.group;
                if (row < rows && p0 + tok >= 0)
                  tree[w] = tree_keys(P, span.q0 + i0 + tok, base, span.n, jw) >> (2 * (lane & 3));
              }
            }
          }
#pragma unroll
          for (int e = 0; e < kWarpKeys / 8; ++e)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int j = jw + e * 8 + 2 * (lane & 3) + (x & 1), w = x >> 1;
              bool seen = (j >= row_lo[w] && j <= row_hi[w]) || (j == 0 && anchor && row_hi[w] >= 0);
              if (kTree) seen |= tree[w] >> (e * 8 + (x & 1)) & 1;
              sc[e][x] = seen ? sc[e][x] : -INFINITY;
            }
          // values that no row sees: their weight is 0, but 0 * NaN is not
          constexpr int kRowChunks = kB * kRowBytes / 16;
          auto clear = [&](int key, int chunk) {
            *reinterpret_cast<uint4*>(sm.v[s][chunk / (kRowBytes / 16)] + key * kRowBytes + chunk % (kRowBytes / 16) * 16) =
                make_uint4(0, 0, 0, 0);
            if (k8 && chunk == 0) sm.scales[s][1][key] = 0;
          };
          const bool inside = jw >= lo && jw + kWarpKeys - 1 <= hi;
          if (!inside) {
            for (int x = lane; x < kWarpKeys * kRowChunks; x += 32) {
              const int key = kg * kWarpKeys + x / kRowChunks, j = j0 + key;
              if (!((j >= lo && j <= hi) || (j == 0 && anchor))) clear(key, x % kRowChunks);
            }
            ptx::fence_proxy_async_smem();  // before the next copy into this stage
            __syncwarp();
          }
          // rows that see nothing may leave their own keys unseen between seen ones
          if constexpr (kLo) {
            bool gaps = kTree && jw + kWarpKeys > base;
            if (!kTree && jw + kWarpKeys - 1 > p0)
              for (int i = lane; i < tokens; i += 32) gaps |= first_key(P, span.q0 + i0 + i) > p0 + i;
            if (__any_sync(0xffffffffu, gaps)) {
              const uint64_t some = kTree ? tree_seen_keys(P, span.q0 + i0, i0, tokens, base, span.n, jw)
                                          : seen_keys(P, span.q0 + i0, p0, tokens, jw);
              for (uint64_t none = ~some & (~0ull >> (64 - kWarpKeys)); none; none &= none - 1) {
                const int key = kg * kWarpKeys + __ffsll((long long)none) - 1;
                if (lane < kRowChunks) clear(key, lane);
              }
              ptx::fence_proxy_async_smem();
              __syncwarp();
            }
          }
        }
        uint32_t pf[kWarpKeys / 8][2];
        if constexpr (k8) {
          float mt[2] = {-INFINITY, -INFINITY}, mv[2] = {-INFINITY, -INFINITY};  // largest s, s + e
          if constexpr (kCareful) {
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const float rest = sm.m[warp][(lane >> 2) + 8 * w];
              float* at = &sm.l[warp][(lane >> 2) + 8 * w];
              float r = *at, top = -INFINITY;
#pragma unroll
              for (int e = 0; e < kWarpKeys / 8; ++e)
#pragma unroll
                for (int x = 2 * w; x < 2 * w + 2; ++x) {
                  sc[e][x] = __fmul_rn(sc[e][x], rest);  // rounded: the largest less r is to be 0
                  top = fmaxf(top, sc[e][x]);
                }
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
              const float by = top - r;
              // down only while the row has seen nothing
              if (top > -INFINITY && (by > kFarLogit / 2 || (by < -kFarLogit / 2 && m[w] == -INFINITY))) {
                m[w] -= by;
                lane_m[w] -= by;
                r = top;
              }
              __syncwarp();
              if ((lane & 3) == 0) *at = r;
#pragma unroll
              for (int e = 0; e < kWarpKeys / 8; ++e) {
                sc[e][2 * w] -= r;
                sc[e][2 * w + 1] -= r;
              }
            }
            __syncwarp();
          }
          float sv[kWarpKeys / 8][4];
#pragma unroll
          for (int e = 0; e < kWarpKeys / 8; ++e) {
            const uint32_t of_v = *reinterpret_cast<const uint16_t*>(&sm.scales[s][1][kg * kWarpKeys + e * 8 + 2 * (lane & 3)]);
            const float e0 = exponent_of(of_v & 255u), e1 = exponent_of(of_v >> 8);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              sv[e][x] = sc[e][x] + (x & 1 ? e1 : e0);
              mt[x >> 1] = fmaxf(mt[x >> 1], sc[e][x]);
              mv[x >> 1] = fmaxf(mv[x >> 1], sv[e][x]);
            }
          }
          bool need = false, large = false;
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            mv[w] = fmaxf(mv[w], __shfl_xor_sync(0xffffffffu, mv[w], 1));
            mv[w] = fmaxf(mv[w], __shfl_xor_sync(0xffffffffu, mv[w], 2));
            need |= mv[w] > m[w] + kRescaleThreshold || (m[w] == -INFINITY && mv[w] > -INFINITY);
            large |= fabsf(mt[w]) > kFarLogit && mt[w] > -INFINITY;
            if (mt[w] > lane_m[w] + kRescaleThreshold || (lane_m[w] == -INFINITY && mt[w] > -INFINITY)) {
              l[w] *= lane_m[w] == -INFINITY ? 0.f : exp2f(lane_m[w] - mt[w]);
              lane_m[w] = mt[w];
            }
          }
          if (__any_sync(0xffffffffu, need || (!kCareful && large))) {
            if (!kCareful && __any_sync(0xffffffffu, large)) return kNeedsCare;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const float mn = fmaxf(m[w], mv[w]);
              const float f = m[w] == -INFINITY ? 0.f : exp2f(m[w] - mn);
              m[w] = mn;
#pragma unroll
              for (int e = 0; e < HD / 8; ++e) {
                o[e][2 * w] *= f;
                o[e][2 * w + 1] *= f;
              }
            }
          }
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const float base = lane_m[w] == -INFINITY ? 0.f : lane_m[w];
            const float base_v = m[w] == -INFINITY ? 0.f : m[w] - kWeightsUp;
#pragma unroll
            for (int e = 0; e < kWarpKeys / 8; ++e) {
              l[w] += ptx::ex2(sc[e][2 * w] - base) + ptx::ex2(sc[e][2 * w + 1] - base);
              pf[e][w] = ptx::pack_f16x2(ptx::ex2(sv[e][2 * w] - base_v), ptx::ex2(sv[e][2 * w + 1] - base_v));
            }
          }
        } else {
          float mt[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < kWarpKeys / 8; ++e) {
            mt[0] = fmaxf(mt[0], fmaxf(sc[e][0], sc[e][1]));
            mt[1] = fmaxf(mt[1], fmaxf(sc[e][2], sc[e][3]));
          }
          bool need = false;
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            mt[w] = fmaxf(mt[w], __shfl_xor_sync(0xffffffffu, mt[w], 1));
            mt[w] = fmaxf(mt[w], __shfl_xor_sync(0xffffffffu, mt[w], 2)) * P.scale_log2;
            need |= mt[w] > m[w] + kRescaleThreshold || (m[w] == -INFINITY && mt[w] > -INFINITY);
          }
          if (__any_sync(0xffffffffu, need)) {
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const float mn = fmaxf(m[w], mt[w]);
              const float f = m[w] == -INFINITY ? 0.f : exp2f(m[w] - mn);
              l[w] *= f;
              m[w] = mn;
#pragma unroll
              for (int e = 0; e < HD / 8; ++e) {
                o[e][2 * w] *= f;
                o[e][2 * w + 1] *= f;
              }
            }
          }
          const float base[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
          for (int e = 0; e < kWarpKeys / 8; ++e)
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const float a = ptx::ex2(fmaf(sc[e][2 * w], P.scale_log2, -base[w]));
              const float c = ptx::ex2(fmaf(sc[e][2 * w + 1], P.scale_log2, -base[w]));
              l[w] += a + c;
              pf[e][w] = ptx::pack_bf16x2(a, c);  // the weights enter the product in bf16, their sum stays fp32
            }
        }
#pragma unroll
        for (int kp = 0; kp < kWarpKeys / 16; ++kp) {
          const uint32_t a[4] = {pf[2 * kp][0], pf[2 * kp][1], pf[2 * kp + 1][0], pf[2 * kp + 1][1]};
          if constexpr (k8) {
#pragma unroll
            for (int c = 0; c < HD / 32; ++c) {
              // matrices: keys 0-7 and 8-15 of 16 channels, then of the next 16
              const int key = kg * kWarpKeys + kp * 16 + (lane & 15);
              uint32_t vf[4];
              ptx::ldmatrix4_t(ptx::smem_u32(sm.v[s][0]) + chunk_fp8<HD>(key, c * 2 + (lane >> 4)), vf);
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                // a channel's two keys side by side
                const uint32_t a0 = __byte_perm(vf[2 * x], 0u, 0x3120), a1 = __byte_perm(vf[2 * x + 1], 0u, 0x3120);
                // channels 0, 2, ..., 14 of the 16; then 1, 3, ..., 15
                ptx::mma_16816_f16(o[4 * c + 2 * x], a, ptx::e4m3x2_to_f16((uint16_t)a0), ptx::e4m3x2_to_f16((uint16_t)a1));
                ptx::mma_16816_f16(o[4 * c + 2 * x + 1], a, ptx::e4m3x2_to_f16((uint16_t)(a0 >> 16)),
                                   ptx::e4m3x2_to_f16((uint16_t)(a1 >> 16)));
              }
            }
          } else {
#pragma unroll
            for (int c = 0; c < HD / 16; ++c) {
              // matrices: keys 0-7 and 8-15, channels 0-7, then channels 8-15
              const int key = kg * kWarpKeys + kp * 16 + (lane & 15);
              uint32_t vf[4];
              ptx::ldmatrix4_t(ptx::smem_u32(sm.v[s][c >> 2]) + sw128_chunk(key, (c & 3) * 2 + (lane >> 4)), vf);
              ptx::mma_16816(o[2 * c], a, vf[0], vf[1]);
              ptx::mma_16816(o[2 * c + 1], a, vf[2], vf[3]);
            }
          }
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&sm.empty[s]);
        return kDone;
      };
      int i = begin;
      Outcome last = kDone;
      if (!careful)
        for (; i < end && (last = take(std::false_type{}, i)) == kDone; ++i) {
        }
      if constexpr (k8) {
        careful |= last == kNeedsCare;
        if (careful && last != kTimeout)
          for (; i < end && take(std::true_type{}, i) == kDone; ++i) {
          }
      }
      if constexpr (k8) {  // the row's maximum of s for all four lanes, and for O
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          float mx = fmaxf(lane_m[w], __shfl_xor_sync(0xffffffffu, lane_m[w], 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          l[w] *= lane_m[w] == -INFINITY ? 0.f : exp2f(lane_m[w] - mx);
          const float f = mx == -INFINITY ? 0.f : exp2f(m[w] - kWeightsUp - mx);
          m[w] = careful ? mx + sm.l[warp][(lane >> 2) + 8 * w] : mx;
#pragma unroll
          for (int e = 0; e < HD / 8; ++e) {
            o[e][2 * w] *= f;
            o[e][2 * w + 1] *= f;
          }
        }
      }
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        l[w] += __shfl_xor_sync(0xffffffffu, l[w], 1);
        l[w] += __shfl_xor_sync(0xffffffffu, l[w], 2);
      }
      // every warp is done with the stages (and their copies have landed) before
      // their memory takes the partial results
      asm volatile("bar.sync 1, 128;" ::: "memory");
      float(*part)[Smem::kRowFloats] = sm.part[warp];
      if constexpr (k8) {
#pragma unroll
        for (int e = 0; e < HD / 8; e += 2)
#pragma unroll
          for (int w = 0; w < 2; ++w)
            *reinterpret_cast<float4*>(&part[(lane >> 2) + 8 * w][e * 8 + 4 * (lane & 3)]) =
                make_float4(o[e][2 * w], o[e + 1][2 * w], o[e][2 * w + 1], o[e + 1][2 * w + 1]);
      } else {
#pragma unroll
        for (int e = 0; e < HD / 8; ++e) {
          *reinterpret_cast<float2*>(&part[lane >> 2][e * 8 + 2 * (lane & 3)]) = make_float2(o[e][0], o[e][1]);
          *reinterpret_cast<float2*>(&part[(lane >> 2) + 8][e * 8 + 2 * (lane & 3)]) = make_float2(o[e][2], o[e][3]);
        }
      }
      if ((lane & 3) == 0) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          sm.m[warp][(lane >> 2) + 8 * w] = m[w];
          sm.l[warp][(lane >> 2) + 8 * w] = l[w];
        }
      }
    }
    steps += end - begin;
    __syncthreads();

    // ------------------------------------------------------------ join
    // the key groups of this CTA
    for (int x = tid; x < rows * (HD / 4); x += kThreads) {
      const int row = x / (HD / 4), c = (x % (HD / 4)) * 4, rg = row >> 4;
      float mx = -INFINITY, sum = 0.f;
#pragma unroll
      for (int kg = 0; kg < kKeyGroups; ++kg) mx = fmaxf(mx, sm.m[kg * RT + rg][row & 15]);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int kg = 0; kg < kKeyGroups; ++kg) {
        const int w = kg * RT + rg;
        const float mw = sm.m[w][row & 15], f = mw == -INFINITY ? 0.f : exp2f(mw - mx);
        const float4 v = *reinterpret_cast<const float4*>(&sm.part[w][row & 15][c]);
        acc.x += f * v.x;
        acc.y += f * v.y;
        acc.z += f * v.z;
        acc.w += f * v.w;
        sum += f * sm.l[w][row & 15];
      }
      *reinterpret_cast<float4*>(&sm.merged[row][c]) = acc;
      if (c == 0) {
        sm.cta_m[row] = mx;
        sm.cta_l[row] = sum;
      }
    }
    __syncthreads();
    if (ranks > 1) ptx::cluster_sync();
    // the cluster's CTAs: each takes a share of the elements
    for (int x = (int)rank * kThreads + tid; x < rows * (HD / 4); x += (int)ranks * kThreads) {
      const int row = x / (HD / 4), c = (x % (HD / 4)) * 4;
      float mx = -INFINITY, sum = 0.f;
      for (uint32_t k = 0; k < ranks; ++k)
        mx = fmaxf(mx, ptx::cluster_ld(ptx::cluster_map(ptx::smem_u32(&sm.cta_m[row]), k)));
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (uint32_t k = 0; k < ranks; ++k) {
        const float mk = ptx::cluster_ld(ptx::cluster_map(ptx::smem_u32(&sm.cta_m[row]), k));
        const float f = mk == -INFINITY ? 0.f : exp2f(mk - mx);
        const float4 v = ptx::cluster_ld4(ptx::cluster_map(ptx::smem_u32(&sm.merged[row][c]), k));
        acc.x += f * v.x;
        acc.y += f * v.y;
        acc.z += f * v.z;
        acc.w += f * v.w;
        sum += f * ptx::cluster_ld(ptx::cluster_map(ptx::smem_u32(&sm.cta_l[row]), k));
      }
      const int tok = row / P.group, h = g * P.group + row - tok * P.group;
      const int64_t t = span.q0 + i0 + tok;
      if (S.splits > 1) {
        const int64_t at = ((int64_t)blockIdx.y * b.T + t) * P.Hq + h;
        S.o[at * (HD / 4) + (c >> 2)] = acc;
        if (c == 0) S.ml[at] = make_float2(mx, sum);
        continue;
      }
      *reinterpret_cast<uint2*>(P.o + (t * P.Hq + h) * HD + c) = normalised(acc, sum);
      if (c == 0 && P.lse) P.lse[(int64_t)h * b.T + t] = (mx + log2f(sum)) * 0.69314718055994531f;
    }
    // nobody leaves (or writes its partial results again) while another reads
    __syncthreads();
    if (ranks > 1) ptx::cluster_sync();
    ptx::fence_proxy_async_smem();  // the partial results before the next pass's copies
    __syncthreads();
  }
}

// One thread per four channels of a (row, query head): the clusters' results in
// order. Rows outside the batch have none.
template <int HD>
__global__ void __launch_bounds__(256) short_join_kernel(const __grid_constant__ AttendParams P, const ShortParts S) {
  const BatchParams& b = P.batch;
  const int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x, row = x / (HD / 4);
  const int c = (int)(x % (HD / 4)), t = (int)(row / P.Hq), h = (int)(row % P.Hq);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (t >= b.T || t < max(__ldg(b.cu_q), 0) || t >= __ldg(b.cu_q + b.B)) return;
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  const int64_t step = (int64_t)b.T * P.Hq;
#pragma unroll 8
  for (int i = 0; i < S.splits; ++i) {
    const float2 ml = S.ml[row + i * step];
    const float4 v = S.o[(row + i * step) * (HD / 4) + c];
    if (ml.y == 0.f) continue;
    const float mn = fmaxf(m, ml.x), f = exp2f(m - mn), fk = exp2f(ml.x - mn);
    m = mn;
    acc.x = f * acc.x + fk * v.x;
    acc.y = f * acc.y + fk * v.y;
    acc.z = f * acc.z + fk * v.z;
    acc.w = f * acc.w + fk * v.w;
    l = f * l + fk * ml.y;
  }
  *reinterpret_cast<uint2*>(P.o + row * HD + c * 4) = normalised(acc, l);
  if (c == 0 && P.lse) P.lse[(int64_t)h * b.T + t] = (m + log2f(l)) * 0.69314718055994531f;
}

// How a call is cut: rows per tile / 16, CTAs per cluster, clusters per unit.
struct ShortShape {
  int rt, ranks, splits;
};

inline ShortShape shape_of(const aa_cache_s* c, int num_seqs, int max_q, int table_width, int group) {
  const int rows = std::max(max_q, 1) * group;
  const int64_t units = (int64_t)num_seqs * c->cfg.num_kv_heads;
  const int64_t tiles = ((int64_t)table_width * c->cfg.page_size + 63) / 64;
  ShortShape f{rows <= 16 ? 1 : rows <= 32 ? 2 : 4, 1, 1};
  // CTAs of a unit: enough to fill the SMs a few times over (ragged sequences
  // then even out), as long as each has a few tiles. Measured on 256 units of
  // up to 8K keys, 64 channels: 4 per SM 70 us, 2 per SM 72 us, 8 per SM 80 us;
  // 512 units of up to 32K keys, 128 channels: 774, 818 and 771 us.
  // With 8-bit pages a tile takes less time, a CTA's start and join do not: where most of
  // the room is taken, CTAs of less than 80 tiles of 64 keys do not get smaller (64 sequences of 8 kv
  // heads over 4000 keys of 128 channels 132 us, halved 144; 8 over 1000 10.3, halved
  // 16.8; 16 of 16 kv heads to 8K keys of 64 channels 55.9, halved 59.9).
  const int64_t at_once = (c->cfg.head_dim == 128 ? 2 : 4) * c->num_sms;
  auto enough = [&] {
    const int64_t ctas = units * f.ranks;
    return ctas >= 4 * c->num_sms || (c->fp8() && tiles < 80 * f.ranks && 2 * ctas > at_once);
  };
  while (f.ranks < 8 && !enough() && tiles >= 4 * f.ranks) f.ranks *= 2;
  // Two CTAs fit on an SM. Where clusters of 8 do not come to that many, several
  // smaller clusters per unit do, if each CTA keeps kSplitTiles tiles: the
  // second launch costs some 2 us.
  const int64_t room = 2 * c->num_sms;
  if (units * 8 < room) {
    const int64_t splits = std::min(room / (units * kSplitRanks), tiles / (kSplitRanks * kSplitTiles));
    if (splits * kSplitRanks > f.ranks) {
      f.ranks = kSplitRanks;
      f.splits = (int)splits;
    }
  }
  return f;
}

template <int HD, int RT, int kMask, bool k8>
cudaError_t launch(const aa_cache_s* c, const AttendParams& P, const ShortShape& f, const ShortParts& S, cudaStream_t s) {
  const auto kernel = attend_short_kernel<HD, RT, kMask, k8>;
  const size_t smem = sizeof(ShortSmem<HD, RT, k8>);
  static std::once_flag once[kMaxDevices];
  static cudaError_t result[kMaxDevices];
  cudaError_t e = once_per_device(once, result, c->device, [&] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((int64_t)P.batch.B * P.batch.Hkv * f.ranks), (unsigned)f.splits);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)f.ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = k8 ? 2 : 1;
  if ((e = cudaLaunchKernelEx(&cfg, kernel, c->k_map64, c->v_map64, P, S)) != cudaSuccess || f.splits == 1) return e;
  const int64_t threads = (int64_t)P.batch.T * P.Hq * (HD / 4);
  return launch_after(short_join_kernel<HD>, dim3((unsigned)((threads + 255) / 256)), 256, 0, s, P, S);
}

template <int HD, int kMask, bool k8>
cudaError_t launch(const aa_cache_s* c, const AttendParams& P, const ShortShape& f, const ShortParts& S, cudaStream_t s) {
  if constexpr (k8)  // the chunk kernel takes more than 32 rows
    return f.rt == 1 ? launch<HD, 1, kMask, k8>(c, P, f, S, s) : launch<HD, 2, kMask, k8>(c, P, f, S, s);
  else
    return f.rt == 1 ? launch<HD, 1, kMask, k8>(c, P, f, S, s)
         : f.rt == 2 ? launch<HD, 2, kMask, k8>(c, P, f, S, s)
                     : launch<HD, 4, kMask, k8>(c, P, f, S, s);
}

template <int HD, bool k8>
cudaError_t launch(const aa_cache_s* c, const AttendParams& P, const ShortShape& f, const ShortParts& S, cudaStream_t s) {
  return P.tree     ? launch<HD, kMaskTree, k8>(c, P, f, S, s)
         : P.key_lo ? launch<HD, kMaskLo, k8>(c, P, f, S, s)
                    : launch<HD, kMaskNone, k8>(c, P, f, S, s);
}

template <bool k8>
cudaError_t launch_short(const aa_cache_s* c, const AttendParams& P, int max_q, void* workspace, cudaStream_t s) {
  const ShortShape f = shape_of(c, P.batch.B, max_q, P.batch.W, P.group);
  ShortParts S{f.splits, static_cast<float4*>(workspace), nullptr};
  S.ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) +
                                   align256((size_t)f.splits * P.batch.T * P.Hq * c->cfg.head_dim * 4));
  return c->cfg.head_dim == 128 ? launch<128, k8>(c, P, f, S, s) : launch<64, k8>(c, P, f, S, s);
}

}  // namespace
}  // namespace aa
