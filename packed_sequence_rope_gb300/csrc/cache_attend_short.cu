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
#include "cache_attend.cuh"

namespace aa {
namespace {

constexpr int kTileKeys = 64;
constexpr int kWarps = 4;
constexpr int kThreads = 32 * (kWarps + 1);
constexpr float kRescaleThreshold = 8.0f;  // log2 units: O is rescaled only when the max grows by > 2^8

constexpr int kSplitRanks = 4, kSplitTiles = 8;

// Results of the clusters of a unit: [split][row][query head], unnormalised O and
// (maximum in log2 units, sum).
struct ShortParts {
  int splits;
  float4* o;
  float2* ml;
};

template <int HD>
struct ShortSmem {
  static constexpr int kB = HD / 64;
  static constexpr int kStages = HD == 128 ? 3 : 4;
  static constexpr int kRowFloats = HD + 8;  // a warp's rows fall on different banks
  union {
    struct {
      alignas(1024) uint8_t k[kStages][kB][kTileKeys * 128];
      alignas(1024) uint8_t v[kStages][kB][kTileKeys * 128];
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

// kLo: the call has key_lo. Its looks for unseen keys between seen ones cost the
// other calls 1 to 4 % where they are compiled in (on the GPU: one token over 1000
// keys 6.98 us, 6.79 without them; seven tokens of eight sequences over 700, D = 64,
// 9.3 and 8.95).
template <int HD, int RT, bool kLo>
__global__ void __launch_bounds__(kThreads, HD == 128 ? 2 : 3)
    attend_short_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                        const __grid_constant__ AttendParams P, const ShortParts S) {
  constexpr int kB = HD / 64, kStages = ShortSmem<HD>::kStages;
  constexpr int kKeyGroups = kWarps / RT, kWarpKeys = kTileKeys / kKeyGroups;
  constexpr uint32_t kStageBytes = 2 * kTileKeys * HD * 2;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if (ptx::smem_u32(smem_raw) & 1023u) {  // swizzled tiles need a 1 KB aligned base
    if (threadIdx.x == 0) atomicCAS(P.batch.err, 0, 498);
    return;
  }
  ShortSmem<HD>& sm = *reinterpret_cast<ShortSmem<HD>*>(smem_raw);
  const BatchParams& b = P.batch;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ranks = ptx::cluster_size(), rank = ptx::cluster_rank();
  const int64_t shares = (int64_t)ranks * S.splits, share = (int64_t)ranks * blockIdx.y + rank;  // of a unit's tiles
  const int unit = (int)(blockIdx.x / ranks);
  const int g = unit % b.Hkv, seq = unit / b.Hkv;
  const SeqSpan span = load_seq(b, seq, P.page_shift);
  const int tile_tokens = 16 * RT / P.group;

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

  int steps = 0;  // tiles this CTA has taken so far: the ring's position
  // one pass, unless the sequence has more new tokens than max_q promised
  for (int i0 = 0; i0 < span.n; i0 += tile_tokens) {
    const int tokens = min(tile_tokens, span.n - i0), rows = tokens * P.group;
    const int p0 = span.kv - span.n + i0, hi = p0 + tokens - 1;  // positions of the first and last row
    int lo = 0;
    if constexpr (kLo) {
      lo = INT_MAX;
      for (int i = lane; i < tokens; i += 32) lo = min(lo, first_key(P, span.q0 + i0 + i));
      lo = __reduce_min_sync(0xffffffffu, lo);
    }
    const KeyTiles<kTileKeys> keys(lo, hi, P.anchor);
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
        const bool seen = j <= hi && (j + (1 << piece_shift) > lo || (j == 0 && P.anchor));
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
        if (lane == 0) ptx::mbar_arrive_expect_tx(&sm.full[s], kStageBytes);
        __syncwarp();
        if (lane < copies) {
          uint8_t* dst = (is_v ? sm.v[s][block] : sm.k[s][block]) + (at << piece_shift) * 128;
          ptx::tma_load_2d(dst, is_v ? &tmV : &tmK, &sm.full[s], block * 64, row);
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
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = row0 + 8 * e, tok = row / P.group;
        const bool on = row < rows;
        row_lo[e] = kLo && on ? first_key(P, span.q0 + i0 + tok) : 0;
        row_hi[e] = on ? p0 + tok : INT_MAX;
        const __nv_bfloat16* q = P.q + (int64_t)(span.q0 + i0 + tok) * P.q_stride +
                                 (int64_t)(g * P.group + row - tok * P.group) * HD + 2 * (lane & 3);
#pragma unroll
        for (int ks = 0; ks < HD / 16; ++ks) {
          qf[ks][e] = on ? __ldg(reinterpret_cast<const uint32_t*>(q + ks * 16)) : 0u;
          qf[ks][e + 2] = on ? __ldg(reinterpret_cast<const uint32_t*>(q + ks * 16 + 8)) : 0u;
        }
      }
      const int all_lo = __reduce_max_sync(0xffffffffu, max(row_lo[0], row_lo[1]));
      const int all_hi = __reduce_min_sync(0xffffffffu, min(row_hi[0], row_hi[1]));
      float o[HD / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
      for (int e = 0; e < HD / 8; ++e) o[e][0] = o[e][1] = o[e][2] = o[e][3] = 0.f;

      for (int i = begin; i < end; ++i) {
        const int n = steps + i - begin, s = n % kStages;
        if (!warp_wait(&sm.full[s], (n / kStages) & 1, b.err, 402)) break;
        const int j0 = keys.tile(i) * kTileKeys, jw = j0 + kg * kWarpKeys;  // the tile's, the warp's first key
        float sc[kWarpKeys / 8][4];
#pragma unroll
        for (int e = 0; e < kWarpKeys / 8; ++e) sc[e][0] = sc[e][1] = sc[e][2] = sc[e][3] = 0.f;
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
        const bool edge = jw < all_lo || jw + kWarpKeys - 1 > all_hi;
        if (edge) {
#pragma unroll
          for (int e = 0; e < kWarpKeys / 8; ++e)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int j = jw + e * 8 + 2 * (lane & 3) + (x & 1), w = x >> 1;
              const bool seen = (j >= row_lo[w] && j <= row_hi[w]) || (j == 0 && P.anchor && row_hi[w] >= 0);
              sc[e][x] = seen ? sc[e][x] : -INFINITY;
            }
          // values that no row sees: their weight is 0, but 0 * NaN is not
          const bool inside = jw >= lo && jw + kWarpKeys - 1 <= hi;
          if (!inside) {
            for (int x = lane; x < kWarpKeys * kB * 8; x += 32) {
              const int key = kg * kWarpKeys + x / (kB * 8), j = j0 + key;
              if (!((j >= lo && j <= hi) || (j == 0 && P.anchor)))
                *reinterpret_cast<uint4*>(sm.v[s][(x >> 3) % kB] + key * 128 + (x & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
            ptx::fence_proxy_async_smem();  // before the next copy into this stage
            __syncwarp();
          }
          // rows that see nothing may leave their own keys unseen between seen ones
          if constexpr (kLo) {
            bool gaps = false;
            if (jw + kWarpKeys - 1 > p0)
              for (int i = lane; i < tokens; i += 32) gaps |= first_key(P, span.q0 + i0 + i) > p0 + i;
            if (__any_sync(0xffffffffu, gaps)) {
              for (uint64_t none = ~seen_keys(P, span.q0 + i0, p0, tokens, jw) & (~0ull >> (64 - kWarpKeys)); none;
                   none &= none - 1) {
                const int key = kg * kWarpKeys + __ffsll((long long)none) - 1;
                if (lane < kB * 8)
                  *reinterpret_cast<uint4*>(sm.v[s][lane >> 3] + key * 128 + (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
              }
              ptx::fence_proxy_async_smem();
              __syncwarp();
            }
          }
        }
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
        uint32_t pf[kWarpKeys / 8][2];
#pragma unroll
        for (int e = 0; e < kWarpKeys / 8; ++e)
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const float a = ptx::ex2(fmaf(sc[e][2 * w], P.scale_log2, -base[w]));
            const float c = ptx::ex2(fmaf(sc[e][2 * w + 1], P.scale_log2, -base[w]));
            l[w] += a + c;
            pf[e][w] = ptx::pack_bf16x2(a, c);  // the weights enter the product in bf16, their sum stays fp32
          }
#pragma unroll
        for (int kp = 0; kp < kWarpKeys / 16; ++kp) {
          const uint32_t a[4] = {pf[2 * kp][0], pf[2 * kp][1], pf[2 * kp + 1][0], pf[2 * kp + 1][1]};
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
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&sm.empty[s]);
      }
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        l[w] += __shfl_xor_sync(0xffffffffu, l[w], 1);
        l[w] += __shfl_xor_sync(0xffffffffu, l[w], 2);
      }
      // every warp is done with the stages (and their copies have landed) before
      // their memory takes the partial results
      asm volatile("bar.sync 1, 128;" ::: "memory");
      float(*part)[ShortSmem<HD>::kRowFloats] = sm.part[warp];
#pragma unroll
      for (int e = 0; e < HD / 8; ++e) {
        *reinterpret_cast<float2*>(&part[lane >> 2][e * 8 + 2 * (lane & 3)]) = make_float2(o[e][0], o[e][1]);
        *reinterpret_cast<float2*>(&part[(lane >> 2) + 8][e * 8 + 2 * (lane & 3)]) = make_float2(o[e][2], o[e][3]);
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

ShortShape shape_of(const aa_cache_s* c, int num_seqs, int max_q, int table_width, int group) {
  const int rows = std::max(max_q, 1) * group;
  const int64_t units = (int64_t)num_seqs * c->cfg.num_kv_heads;
  const int64_t tiles = ((int64_t)table_width * c->cfg.page_size + kTileKeys - 1) / kTileKeys;
  ShortShape f{rows <= 16 ? 1 : rows <= 32 ? 2 : 4, 1, 1};
  // CTAs of a unit: enough to fill the SMs a few times over (ragged sequences
  // then even out), as long as each has a few tiles. Measured on 256 units of
  // up to 8K keys, 64 channels: 4 per SM 70 us, 2 per SM 72 us, 8 per SM 80 us;
  // 512 units of up to 32K keys, 128 channels: 774, 818 and 771 us.
  while (f.ranks < 8 && units * f.ranks < 4 * c->num_sms && tiles >= 4 * f.ranks) f.ranks *= 2;
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

template <int HD, int RT, bool kLo>
cudaError_t launch(const aa_cache_s* c, const AttendParams& P, const ShortShape& f, const ShortParts& S, cudaStream_t s) {
  const auto kernel = attend_short_kernel<HD, RT, kLo>;
  const size_t smem = sizeof(ShortSmem<HD>);
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
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)f.ranks;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, kernel, c->k_map64, c->v_map64, P, S)) != cudaSuccess || f.splits == 1) return e;
  const int64_t threads = (int64_t)P.batch.T * P.Hq * (HD / 4);
  return launch_after(short_join_kernel<HD>, dim3((unsigned)((threads + 255) / 256)), 256, 0, s, P, S);
}

template <int HD, bool kLo>
cudaError_t launch(const aa_cache_s* c, const AttendParams& P, const ShortShape& f, const ShortParts& S, cudaStream_t s) {
  return f.rt == 1   ? launch<HD, 1, kLo>(c, P, f, S, s)
         : f.rt == 2 ? launch<HD, 2, kLo>(c, P, f, S, s)
                     : launch<HD, 4, kLo>(c, P, f, S, s);
}

}  // namespace

size_t short_workspace_bytes(const aa_cache_s* c, int num_seqs, int total_tokens, int max_q, int table_width, int group) {
  const ShortShape f = shape_of(c, num_seqs, max_q, table_width, group);
  const size_t rows = (size_t)total_tokens * c->cfg.num_kv_heads * group;
  return f.splits == 1 ? 256 : align256(f.splits * rows * c->cfg.head_dim * 4) + align256(f.splits * rows * 8);
}

cudaError_t launch_attend_short(const aa_cache_s* c, const AttendParams& P, int max_q, void* workspace, cudaStream_t s) {
  const ShortShape f = shape_of(c, P.batch.B, max_q, P.batch.W, P.group);
  ShortParts S{f.splits, static_cast<float4*>(workspace), nullptr};
  S.ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) +
                                   align256((size_t)f.splits * P.batch.T * P.Hq * c->cfg.head_dim * 4));
  if (c->cfg.head_dim == 128)
    return P.key_lo ? launch<128, true>(c, P, f, S, s) : launch<128, false>(c, P, f, S, s);
  return P.key_lo ? launch<64, true>(c, P, f, S, s) : launch<64, false>(c, P, f, S, s);
}

}  // namespace aa
