// Attention of chunks of new tokens over the paged cache (prompts, and any
// batch with more rows per sequence than cache_attend_short.cu takes).
//
// Rows are packed: row r of a 128-row tile is (token r / group, query head
// r % group) of one kv head, so a grouped-query layer fills the tensor cores'
// 128 rows with 128 / group tokens and reads each key once for the group. A unit
// of work is two such row tiles of one sequence and kv head; its keys come in
// tiles of 128. Three kernels:
//   chunk_plan_kernel     one CTA: each unit's key tiles and their running sum,
//                         from the lengths and key_lo on the device
//   attend_chunk_kernel   persistent, one CTA per SM. All key tiles of all
//                         units, laid end to end, are cut into equal shares, one per
//                         CTA: the SMs finish together whatever the lengths. A
//                         share's first and last unit may be cut; their partial
//                         results (fp32, with the rows' maximum and sum) go to the
//                         workspace
//   chunk_join_kernel     joins the partial results of each cut unit, in order
// The second and third are launched as programmatic dependents, so that their
// start-up overlaps the kernel before them. Where the page tables hold few keys
// a unit is short, and the second kernel alone takes whole units, without a workspace.
//
// Roles in attend_chunk_kernel (640 threads):
//   warp 0      finds the CTA's next piece of work and copies its query tiles and
//               the key tiles' pages (tensor copies, one page piece per lane)
//   warp 1      owns tensor memory and issues the products
//   warps 2, 3  clear values that no row sees (a page's unused rows)
//   warps 4-11  row tile 0: online softmax and epilogue; lane = row, two warps per
//               32 rows with half of the columns each, which exchange the rows'
//               maxima through shared memory
//   warps 12-19 the same for row tile 1
// Tensor memory: S0 [0, 128), S1 [128, 256), O0, O1 (D columns each); P replaces
// the first half of its S as packed bf16 and feeds P V from there. The issue order
// PV0(j), S0(j + 1), PV1(j), S1(j + 1) keeps the tensor cores busy with one tile
// while the other's softmax runs.
#include <algorithm>

#include "cache_attend.cuh"

namespace aa {
namespace {

constexpr int kKeys = 128;
constexpr int kSoftmaxWarps = 16;
constexpr int kThreads = 32 * (4 + kSoftmaxWarps);
constexpr int kReaders = 3 + kSoftmaxWarps;  // of a published piece: warps 1 to 3, the softmax warps
constexpr float kRescaleThreshold = 8.0f;  // log2 units: O is rescaled only when the max grows by > 2^8
constexpr uint64_t kDrainNs = 1000000000ull;
constexpr int kMinShare = 2;  // key tiles a CTA takes at least
// What a unit's queries, epilogue and start-up cost, in key tiles (some 4 us): it
// counts for so many more where the work is shared out, ahead of its tiles. 400
// units of 2 to 14 tiles: 87 us with 0, 82.4 with 1, 80.1 with 2, 79.5 with 3; one
// sequence of 128 tokens over 2K keys 20.7, 21.1, 21.0 and 21.9.
constexpr int kUnitCost = 2;

// A unit as chunk_plan_kernel describes it: tokens [i0, i0 + tokens) of a
// sequence, their positions [p0, p0 + tokens), the smallest of their first keys;
// gaps: some of them see nothing, so that keys between seen ones may be unseen.
struct Unit {
  int32_t seq, q_row, tokens, p0, lo, gaps;
};

// A cut unit, as the CTA that begins it describes it to chunk_join_kernel: its
// parts lie with the CTAs from that one to `last`. last < 0: the CTA begins none.
struct alignas(16) Cut {
  int32_t last, g, q_row, tokens;
};

struct ChunkParams {
  AttendParams a;
  int tile_tokens;     // tokens per row tile: 128 / group
  int slots;           // room for the units of one kv head
  int ctas;            // of the attention kernel, unless it takes whole units
  int whole_units;     // short contexts: CTAs take whole units, there is no plan and nothing to join
  int64_t* tiles_end;  // [slots + 1] running sum of the units' costs in key tiles; [0] = 0
  Unit* units;         // [slots]
  float4* part_o;      // [CTA][2][row tile][D / 4][128]: unnormalised O of a cut unit
  float2* part_ml;     // [CTA][2][row tile][128]: maximum (log2 units), sum
  Cut* cuts;           // [CTA]
};

// ---------------------------------------------------------------- the plan
// The unit of a slot and its number of key tiles; no tokens and 0 if the slot is
// empty (a whole warp asks). Sequence b's units start at slot
// cu_q[b] / (2 tile_tokens) + b, which leaves room for a rounded-up count and
// needs no scan over the sequences before it.
__device__ __forceinline__ Unit load_unit(const ChunkParams& C, int slot, int* count) {
  const AttendParams& P = C.a;
  const BatchParams& b = P.batch;
  const int lane = threadIdx.x & 31, unit_tokens = 2 * C.tile_tokens;
  const int seq = warp_last(b.B, [&](int i) { return __ldg(b.cu_q + i) / unit_tokens + i <= slot; });
  const SeqSpan s = load_seq(b, seq, P.page_shift);
  const int64_t i0 = (int64_t)(slot - __ldg(b.cu_q + seq) / unit_tokens - seq) * unit_tokens;
  Unit u{seq, 0, 0, 0, 0, 0};
  *count = 0;
  if (i0 >= 0 && i0 < s.n) {
    u.q_row = s.q0 + (int)i0;
    u.tokens = min(unit_tokens, s.n - (int)i0);
    u.p0 = s.kv - s.n + (int)i0;
    if (P.key_lo) {
      int lo = INT_MAX;
      bool gaps = false;
      for (int i = lane; i < u.tokens; i += 32) {
        const int first = first_key(P, u.q_row + i);
        lo = min(lo, first);
        gaps |= first > u.p0 + i;
      }
      u.lo = __reduce_min_sync(0xffffffffu, lo);
      u.gaps = __any_sync(0xffffffffu, gaps);
    }
    // rows that see nothing are written too: at least one tile
    *count = max(KeyTiles<kKeys>(u.lo, u.p0 + u.tokens - 1, P.anchor).count, 1);
  }
  return u;
}

__global__ void __launch_bounds__(1024) chunk_plan_kernel(const __grid_constant__ ChunkParams C) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int slot = warp; slot < C.slots; slot += 32) {
    int count;
    const Unit u = load_unit(C, slot, &count);
    if (lane == 0) {
      C.units[slot] = u;
      C.tiles_end[slot + 1] = count ? count + kUnitCost : 0;
    }
  }
  __syncthreads();
  __shared__ int64_t sums[32];
  int64_t carry = 0;
  if (threadIdx.x == 0) C.tiles_end[0] = 0;
  for (int base = 0; base < C.slots; base += 1024) {
    const int slot = base + (int)threadIdx.x;
    int64_t v = slot < C.slots ? C.tiles_end[slot + 1] : 0;
    for (int d = 1; d < 32; d *= 2) {
      const int64_t up = __shfl_up_sync(0xffffffffu, v, d);
      if (lane >= d) v += up;
    }
    if (lane == 31) sums[warp] = v;
    __syncthreads();
    if (warp == 0) {
      int64_t w = sums[lane];
      for (int d = 1; d < 32; d *= 2) {
        const int64_t up = __shfl_up_sync(0xffffffffu, w, d);
        if (lane >= d) w += up;
      }
      sums[lane] = w;
    }
    __syncthreads();
    v += carry + (warp ? sums[warp - 1] : 0);
    if (slot < C.slots) C.tiles_end[slot + 1] = v;
    carry += sums[31];
    __syncthreads();
  }
}

// How the key tiles of all heads are shared out, and which unit a tile belongs
// to: tile numbers run over (kv head, slot, tile of the unit).
struct Shares {
  int64_t all, share, per_head;
  Shares() = default;
  __device__ __forceinline__ Shares(const ChunkParams& C, int ctas) {
    per_head = C.tiles_end[C.slots];
    all = per_head * C.a.batch.Hkv;
    share = max((all + ctas - 1) / ctas, (int64_t)kMinShare);
  }
  // kv head, slot and first tile number of the unit that holds tile `at` (whole warp)
  __device__ __forceinline__ void find(const ChunkParams& C, int64_t at, int* g, int* slot, int64_t* begin, int* count) const {
    *g = (int)(at / per_head);
    const int64_t rem = at - *g * per_head;
    *slot = warp_last(C.slots, [&](int i) { return C.tiles_end[i] <= rem; });
    const int64_t e0 = C.tiles_end[*slot];
    *begin = *g * per_head + e0;
    *count = (int)(C.tiles_end[*slot + 1] - e0);
  }
};

// ---------------------------------------------------------------- attention
// One piece of work: key tiles [first, first + take) of a unit's `count`.
struct Piece {
  int valid, g, seq, q_row, tokens, p0, lo, gaps;
  int first, take, whole;  // whole: the unit is not cut
  int part;                // else: which of the CTA's two partial results
};

template <int HD>
struct ChunkSmem {
  static constexpr int kB = HD / 64;
  static constexpr int kStages = HD == 128 ? 2 : 4;
  // a piece's two row tiles of Q and one of the next piece: its first S product
  // does not wait for a copy
  static constexpr int kQ = 3;
  alignas(1024) uint8_t q[kQ][kB][16384];
  alignas(1024) uint8_t k[kStages][kB][16384];
  alignas(1024) uint8_t v[kStages][kB][16384];
  uint64_t q_full[kQ], q_free[kQ];
  uint64_t piece_full[2], piece_empty[2];
  uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_clean[kStages], v_empty[kStages];
  uint64_t s_full[2], p_full[2], o_full[2], drain;
  Piece piece[2];
  // Between the two warps of 32 rows, [row tile][32 rows][column half][lane]: the
  // maxima of a step, then the sums. One buffer serves all steps: a step's S is
  // issued only after both warps have handed over the last step's weights, and so
  // have read its maxima. In fp32: a base that is off by a fraction of a large
  // maximum leaves weights that underflow to 0.
  float pair[2][4][2][32];
  uint32_t tmem_base;
  int abort_flag;
};

// A converged warp waits, bounded, and gives up with the rest of the CTA. One lane
// asks for all. (A suspend-time hint on the question costs wake-up time: 871 us
// against 628 for 2048 tokens over 32K keys at D = 64.)
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int32_t* err, volatile int* abort_flag, int site) {
  bool ok = true;
  if ((threadIdx.x & 31) == 0 && !ptx::mbar_try_wait(bar, parity)) {
    const uint64_t t0 = ptx::global_timer_ns();
    for (int i = 1; ok && !ptx::mbar_try_wait(bar, parity); ++i) {
      if (i & 63) continue;
      if (*abort_flag) {
        ok = false;
      } else if (ptx::global_timer_ns() - t0 >= kAttendWaitNs) {
        atomicCAS(err, 0, site);
        *abort_flag = 1;
        ok = false;
      }
    }
  }
  return __all_sync(0xffffffffu, ok);
}

// The li-th piece of this CTA, read by a whole warp; false when there is none left.
template <class Smem>
__device__ __forceinline__ bool read_piece(Smem& sm, int li, int32_t* err, volatile int* abort_flag, int site, Piece* out) {
  if (!warp_wait(&sm.piece_full[li & 1], (li >> 1) & 1, err, abort_flag, site)) return false;
  *out = sm.piece[li & 1];
  __syncwarp();
  if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(&sm.piece_empty[li & 1]);
  return __all_sync(0xffffffffu, out->valid != 0);
}

// Bit e: key j + e lies in [lo, hi].
__device__ __forceinline__ uint32_t visible_bits(int j, int lo, int hi) {
  const int last = hi - j, first = lo - j;
  const uint32_t upto = last < 0 ? 0u : last >= 31 ? ~0u : (2u << last) - 1u;
  return first <= 0 ? upto : first > 31 ? 0u : upto & (~0u << first);
}

// Barrier phases: pieces count the piece ring; the K and V rings count the
// CTA's key tiles over all its pieces; s_full / p_full count each row tile's
// softmax steps; q_full and q_free the CTA's row tiles of Q; o_full the pieces
// in which the row tile exists. As in the packed forward every wait is bounded and its outcome made
// uniform in a warp before anything collective.
template <int HD>
__global__ void __launch_bounds__(kThreads, 1)
    attend_chunk_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const __grid_constant__ ChunkParams C) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  constexpr int kB = HD / 64, kStages = ChunkSmem<HD>::kStages, kQ = ChunkSmem<HD>::kQ, kTmemCols = 512;
  constexpr uint32_t kTileBytes = kKeys * HD * 2;
  const AttendParams& P = C.a;
  const BatchParams& b = P.batch;
  if (ptx::smem_u32(smem_raw) & 1023u) {  // swizzled tiles need a 1 KB aligned base
    if (threadIdx.x == 0) {
      atomicCAS(b.err, 0, 498);
      if (!C.whole_units) C.cuts[blockIdx.x] = Cut{-1, 0, 0, 0};
    }
    return;
  }
  ChunkSmem<HD>& sm = *reinterpret_cast<ChunkSmem<HD>*>(smem_raw);
  const int tid = threadIdx.x, warp = (int)__reduce_max_sync(0xffffffffu, (unsigned)tid >> 5), lane = tid & 31;  // uniform
  volatile int* abort_flag = &sm.abort_flag;

  if (tid == 0) {
    ptx::tma_prefetch_desc(&tmQ);
    ptx::tma_prefetch_desc(&tmK);
    ptx::tma_prefetch_desc(&tmV);
    for (int t = 0; t < 2; ++t) {
      ptx::mbar_init(&sm.s_full[t], 1);
      ptx::mbar_init(&sm.p_full[t], kSoftmaxWarps / 2);
      ptx::mbar_init(&sm.o_full[t], 1);
      ptx::mbar_init(&sm.piece_full[t], 1);
      ptx::mbar_init(&sm.piece_empty[t], kReaders);
    }
    for (int s = 0; s < kQ; ++s) {
      ptx::mbar_init(&sm.q_full[s], 1);
      ptx::mbar_init(&sm.q_free[s], 1);
    }
    for (int s = 0; s < kStages; ++s) {
      for (uint64_t* bar : {&sm.k_full[s], &sm.k_empty[s], &sm.v_full[s], &sm.v_empty[s]}) ptx::mbar_init(bar, 1);
      ptx::mbar_init(&sm.v_clean[s], 2);
    }
    ptx::mbar_init(&sm.drain, 1);
    sm.abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 1) ptx::tmem_alloc(&sm.tmem_base, kTmemCols);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = __reduce_max_sync(0xffffffffu, sm.tmem_base);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the plan, and everything before it

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    Shares shares{};
    int64_t at = blockIdx.x, end = (int64_t)C.slots * b.Hkv;  // whole units: numbers over (kv head, slot)
    if (!C.whole_units) {
      shares = Shares(C, gridDim.x);
      at = shares.share * blockIdx.x;
      end = min(at + shares.share, shares.all);
    }
    Cut cut{-1, 0, 0, 0};
    int nq = 0, ks = 0, nk = 0;  // row tiles of Q, key tiles whose V, whose K has been asked for
    bool ok = true;
    // a key tile is `pieces` page pieces, each kB column blocks of K, then of V
    const int piece_shift = min(P.page_shift, 6), pieces = kKeys >> piece_shift;
    const int copies = pieces * kB;  // at most 16: one per lane
    const int part = lane & (pieces - 1), block = (lane / pieces) % kB;
    for (int li = 0; ok; ++li) {
      if (li >= 2) ok = warp_wait(&sm.piece_empty[li & 1], ((li >> 1) - 1) & 1, b.err, abort_flag, 452);
      if (!ok) break;
      Piece w{};
      int count = 0;
      if (C.whole_units) {
        for (; at < end && count == 0; at += gridDim.x) {
          w.g = (int)(at / C.slots);
          const Unit u = load_unit(C, (int)(at % C.slots), &count);
          w.seq = u.seq;
          w.q_row = u.q_row;
          w.tokens = u.tokens;
          w.p0 = u.p0;
          w.lo = u.lo;
          w.gaps = u.gaps;
        }
        w.valid = count > 0;
        w.take = count;
        w.whole = 1;
      } else {
        for (; at < end && !w.valid;) {
          int slot;
          int64_t begin;
          shares.find(C, at, &w.g, &slot, &begin, &count);
          const Unit u = C.units[slot];
          w.seq = u.seq;
          w.q_row = u.q_row;
          w.tokens = u.tokens;
          w.p0 = u.p0;
          w.lo = u.lo;
          w.gaps = u.gaps;
          const int64_t until = min(begin + count, end);
          w.first = (int)max(at - begin - kUnitCost, (int64_t)0);
          w.take = (int)max(until - begin - kUnitCost, (int64_t)0) - w.first;
          w.valid = w.take > 0;  // else the share ends before the unit's first tile
          w.whole = w.take == count - kUnitCost;
          w.part = w.first == 0 ? 1 : 0;  // the first part of a cut unit, or a later one: at most one of each per CTA
          if (w.valid && w.first == 0 && !w.whole)
            cut = Cut{(int32_t)((begin + count - 1) / shares.share), w.g, w.q_row, w.tokens};
          at = until;
        }
      }
      if (lane == 0) {
        sm.piece[li & 1] = w;
        ptx::mbar_arrive(&sm.piece_full[li & 1]);
      }
      __syncwarp();
      if (!w.valid) break;
      const int hi = w.p0 + w.tokens - 1;
      const KeyTiles<kKeys> keys(w.lo, hi, P.anchor);
      auto row_of = [&](int i) {
        const int j = keys.tile(i) * kKeys + (part << piece_shift);
        // pieces that no row sees are not looked up (lo > hi: the rows see the anchor at most)
        const bool seen = j <= hi && ((w.lo <= hi && j + (1 << piece_shift) > w.lo) || (j == 0 && P.anchor));
        return lane < copies && i < w.first + w.take && i < keys.count && seen ? pool_row(b, w.seq, w.g, j, P.page_shift)
                                                                               : kNoRow;
      };
      int next = row_of(w.first);
      auto load_keys = [&](int i) {
        const int s = ks % kStages, row = next;
        next = row_of(i + 1);  // in flight while this stage is waited for
        // K's buffer is free one product earlier than V's, and V is wanted later
        for (int v = 0; v < 2; ++v) {
          uint64_t* full = v ? &sm.v_full[s] : &sm.k_full[s];
          if (ks >= kStages)
            ok = warp_wait(v ? &sm.v_empty[s] : &sm.k_empty[s], ((ks / kStages) - 1) & 1, b.err,
                                                       abort_flag, 451);
          if (!ok) return;
          if (lane == 0) ptx::mbar_arrive_expect_tx(full, kTileBytes);
          __syncwarp();
          if (lane < copies)
            ptx::tma_load_2d((v ? sm.v[s][block] : sm.k[s][block]) + (part << piece_shift) * 128, v ? &tmV : &tmK, full,
                             block * 64, row);
          if (v == 0) nk = ks + 1;
        }
        ++ks;
      };
      // the first key tile goes ahead of the queries, whose buffers the piece
      // before may still read
      load_keys(w.first);
      for (int t = 0; t < (w.tokens > C.tile_tokens ? 2 : 1) && ok; ++t, ++nq) {
        const int q = nq % kQ;
        if (nq >= kQ) ok = warp_wait(&sm.q_free[q], (nq / kQ - 1) & 1, b.err, abort_flag, 450);
        if (!ok) break;
        if (lane == 0) {
          ptx::mbar_arrive_expect_tx(&sm.q_full[q], (uint32_t)(C.tile_tokens * P.group * HD * 2));
          for (int c = 0; c < kB; ++c)
            ptx::tma_load_4d(sm.q[q][c], &tmQ, &sm.q_full[q], c * 64, 0, w.g, w.q_row + t * C.tile_tokens);
        }
        __syncwarp();
      }
      for (int i = w.first + 1; i < w.first + w.take && ok; ++i) load_keys(i);
    }
    if (lane == 0 && !C.whole_units) C.cuts[blockIdx.x] = cut;
    // every issued copy lands before the CTA exits
    for (int u = max(nq - kQ, 0); u < nq; ++u)
      ptx::mbar_wait(&sm.q_full[u % kQ], (u / kQ) & 1, kDrainNs, b.err, 459);
    for (int u = max(nk - kStages, 0); u < nk; ++u)
      ptx::mbar_wait(&sm.k_full[u % kStages], (u / kStages) & 1, kDrainNs, b.err, 459);
    for (int u = max(ks - kStages, 0); u < ks; ++u)
      ptx::mbar_wait(&sm.v_full[u % kStages], (u / kStages) & 1, kDrainNs, b.err, 459);
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (the whole warp, converged)
    constexpr uint32_t idesc_s = ptx::idesc_bf16_f32(128, 128, 0, 0);
    constexpr uint32_t idesc_pv = ptx::idesc_bf16_f32(128, HD, 0, 1);
    uint32_t ph_p[2] = {0, 0};
    int ks = 0, nq = 0;
    auto wait = [&](uint64_t* bar, uint32_t parity, int site) { return warp_wait(bar, parity, b.err, abort_flag, site); };
    // Descriptors of the first buffers; the others follow at kTileBytes. They are
    // made before the waits, so that nothing stands between a signal and its
    // products.
    const uint64_t q0 = ptx::smem_desc_sw128(ptx::smem_u32(sm.q[0][0]), 16, 1024);
    const uint64_t k0 = ptx::smem_desc_sw128(ptx::smem_u32(sm.k[0][0]), 16, 1024);
    const uint64_t v0 = ptx::smem_desc_sw128(ptx::smem_u32(sm.v[0][0]), 16384, 1024);
    auto issue_s = [&](int t, uint64_t qd, uint64_t kd) {
      if constexpr (HD == 128)
        ptx::mma8_ss_kk_warp(tmem + 128 * t, qd, kd, idesc_s, 0);
      else
        ptx::mma4_ss_kk_warp(tmem + 128 * t, qd, kd, idesc_s, 0);
      ptx::mma_commit_warp(&sm.s_full[t]);
    };
    bool ok = true;
    for (int li = 0; ok; ++li) {
      Piece w;
      if (!read_piece(sm, li, b.err, abort_flag, 460, &w)) break;
      // the reductions make the loops' bounds uniform for the compiler
      const int take = __reduce_max_sync(0xffffffffu, w.take);
      const int tiles = __all_sync(0xffffffffu, w.tokens > C.tile_tokens) ? 2 : 1;
      const int q[2] = {nq % kQ, (nq + 1) % kQ};
      const uint64_t qd[2] = {q0 + q[0] * (kTileBytes >> 4), q0 + q[1] * (kTileBytes >> 4)};
      // the first S products, as the piece's K and Q land
      if (!(ok = wait(&sm.k_full[ks % kStages], (ks / kStages) & 1, 463))) break;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (t >= tiles) break;
        if (!(ok = wait(&sm.q_full[q[t]], ((nq + t) / kQ) & 1, 462))) break;
        ptx::tc_fence_after();
        issue_s(t, qd[t], k0 + (ks % kStages) * (kTileBytes >> 4));
        if (take == 1) ptx::mma_commit_warp(&sm.q_free[q[t]]);
      }
      if (!ok) break;
      ptx::mma_commit_warp(&sm.k_empty[ks % kStages]);
      for (int i = 0; i < take; ++i, ++ks) {
        // waits for copies first, while the tensor cores are still busy; then
        // only the softmax's signal stands before P V and the next S of a tile
        const int s = ks % kStages, s1 = (ks + 1) % kStages;
        const bool more = i + 1 < take;
        const uint64_t vd = v0 + s * (kTileBytes >> 4), kd = k0 + s1 * (kTileBytes >> 4);
        if (!(ok = wait(&sm.v_clean[s], (ks / kStages) & 1, 464))) break;
        if (more && !(ok = wait(&sm.k_full[s1], ((ks + 1) / kStages) & 1, 463))) break;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (t >= tiles) break;
          if (!(ok = wait(&sm.p_full[t], ph_p[t], 461))) break;
          ph_p[t] ^= 1;
          ptx::tc_fence_after();
          ptx::mma8_ts_seq_warp(tmem + 256 + HD * t, tmem + 128 * t, vd, idesc_pv, i == 0 ? 0u : 1u);
          if (more)
            issue_s(t, qd[t], kd);
          else
            ptx::mma_commit_warp(&sm.o_full[t]);
          if (i + 2 == take) ptx::mma_commit_warp(&sm.q_free[q[t]]);
        }
        if (!ok) break;
        ptx::mma_commit_warp(&sm.v_empty[s]);
        if (more) ptx::mma_commit_warp(&sm.k_empty[s1]);
      }
      nq += tiles;
    }
    // every issued MMA must finish before TMEM is released
    __syncwarp();
    ptx::mma_commit_warp(&sm.drain);
    ptx::mbar_wait(&sm.drain, 0, kDrainNs, b.err, 469);
  } else if (warp < 4) {
    // ------------------------------------------------------------ clearing unseen values (warps 2 and 3)
    // The rows of V that no row of the unit sees have weight 0, but 0 * NaN is
    // not. Pieces that were not looked up hold zeros already, which leaves the
    // unseen rows of the pieces at the ends of [lo, hi], and behind the anchor (all
    // of its piece's, where no row sees another key: lo > hi). Where rows of the unit
    // see nothing, the keys at the new tokens' positions are looked at one by one.
    constexpr int kChunks = kB * 8, kRowsAtOnce = 32 / kChunks;  // 16-byte chunks of a row, rows a warp clears at once
    const int piece = 1 << min(P.page_shift, 6), chunk = lane % kChunks;
    const int first_row = (warp - 2) * kRowsAtOnce + lane / kChunks;
    int ks = 0;
    bool ok = true;
    for (int li = 0; ok; ++li) {
      Piece w;
      if (!read_piece(sm, li, b.err, abort_flag, 470, &w)) break;
      const int hi = w.p0 + w.tokens - 1;
      const KeyTiles<kKeys> keys(w.lo, hi, P.anchor);
      for (int i = w.first; i < w.first + w.take; ++i, ++ks) {
        const int s = ks % kStages;
        if (!(ok = warp_wait(&sm.v_full[s], (ks / kStages) & 1, b.err, abort_flag, 471))) break;
        const int j0 = keys.tile(i) * kKeys;
        if (j0 < w.lo || j0 + kKeys - 1 > hi) {
          auto clear = [&](int from, int to) {  // rows of the tile
            from = max(from, 0);
            to = min(to, kKeys);
#pragma unroll 4
            for (int row = from + first_row; row < to; row += 2 * kRowsAtOnce)
              *reinterpret_cast<uint4*>(sm.v[s][chunk >> 3] + row * 128 + (chunk & 7) * 16) = make_uint4(0, 0, 0, 0);
          };
          const bool anchored = P.anchor && j0 == 0 && hi >= 0 && w.lo > 0;
          const int lo_piece = w.lo & ~(piece - 1);  // its copy starts here
          if (anchored) clear(1, w.lo <= hi ? min(piece, w.lo) : piece);
          if (w.lo <= hi) {
            clear(max(lo_piece - j0, anchored ? 1 : 0), w.lo - j0);
            clear(hi + 1 - j0, (hi | (piece - 1)) + 1 - j0);
          }
          ptx::fence_proxy_async_smem();
          __syncwarp();
        }
        if (w.gaps && j0 + kKeys - 1 > w.p0) {
          const int from = (warp - 2) * 64;  // half of the tile's keys per warp
          for (uint64_t none = ~seen_keys(P, w.q_row, w.p0, w.tokens, j0 + from); none; none &= none - 1) {
            const int row = from + __ffsll((long long)none) - 1;
            if (lane < kChunks)
              *reinterpret_cast<uint4*>(sm.v[s][chunk >> 3] + row * 128 + (chunk & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          ptx::fence_proxy_async_smem();
          __syncwarp();
        }
        if (lane == 0) ptx::mbar_arrive(&sm.v_clean[s]);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int t = (warp - 4) >> 3, half = ((warp - 4) >> 2) & 1, r = (warp & 3) * 32 + lane;
    const int pair_bar = 1 + t * 4 + (warp & 3);  // named barrier of the two warps with the same rows
    auto& pair = sm.pair[t][warp & 3];
    const float sl2 = P.scale_log2;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + 128 * t + lane_off, t_o = tmem + 256 + HD * t + half * (HD / 2) + lane_off;
    uint32_t ph_s = 0;
    int nq = 0;
    // a warp that gives up still meets its partner: both leave together
    for (int li = 0;; ++li) {
      const Piece& w = sm.piece[li & 1];  // released after the epilogue
      const bool got = warp_wait(&sm.piece_full[li & 1], (li >> 1) & 1, b.err, abort_flag, 480);
      if (!ptx::bar_and(pair_bar, 64, got) || !w.valid) break;
      if (t == 1 && w.tokens <= C.tile_tokens) {
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&sm.piece_empty[li & 1]);
        continue;
      }
      const int in_tile = r / P.group;
      const bool row_valid = in_tile < C.tile_tokens && t * C.tile_tokens + in_tile < w.tokens;
      // this row's visible keys; rows that are none see all, which needs no mask
      int lo = 0, hi = INT_MAX;
      if (row_valid) {
        lo = first_key(P, w.q_row + t * C.tile_tokens + in_tile);
        hi = w.p0 + t * C.tile_tokens + in_tile;
      }
      const bool anchored = P.anchor && row_valid && hi >= 0 && half == 0;
      const int take = w.take;
      const KeyTiles<kKeys> keys(w.lo, w.p0 + w.tokens - 1, P.anchor);
      int j0 = keys.tile(w.first) * kKeys + half * 64;  // this warp's first key
      int next_j0 = keys.tile(w.first + 1) * kKeys + half * 64;
      float m = -INFINITY, l = 0.f;
      bool ok = true;
      for (int i = 0; i < take; ++i, j0 = next_j0, next_j0 += kKeys) {
        ok = warp_wait(&sm.s_full[t], ph_s, b.err, abort_flag, 482);
        if (!ok) {
          ptx::bar_and(pair_bar, 64, false);
          break;
        }
        ph_s ^= 1;
        ptx::tc_fence_after();
        // The row's maximum over both column halves, and what it changes. Also the
        // point where both warps have read their columns of S: P may overwrite them.
        auto agree = [&](float mt) {
          pair[half][lane] = mt;
          if (!ptx::bar_and(pair_bar, 64, true)) return false;
          mt = fmaxf(pair[0][lane], pair[1][lane]) * sl2;
          // TMEM access is warp-collective, so a rescale of O is decided per warp (alike
          // for both), and by rows that hold a token alone: what lies in the others
          // (the next sequence's queries, old shared memory) must not change a bit
          const bool need = row_valid && ((mt > m + kRescaleThreshold) || (m == -INFINITY && mt > -INFINITY));
          if (__any_sync(0xffffffffu, need)) {
            const float mn = fmaxf(m, mt);
            const float f = (m == -INFINITY) ? 0.f : exp2f(m - mn);
            l *= f;
            if (i > 0) {  // O holds earlier tiles: S(i) done implies their PV is done
#pragma unroll 1
              for (int c = 0; c < HD / 32; ++c) {
                float ov[16];
                ptx::tmem_ld16(t_o + c * 16, ov);
                ptx::tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) ov[e] *= f;
                ptx::tmem_st16f(t_o + c * 16, ov);
              }
            }
            m = mn;
          }
          return true;
        };
        const uint32_t t_p = t_s + half * 32;
        float sv[64];
#pragma unroll
        for (int c = 0; c < 2; ++c) ptx::tmem_ld32(t_s + half * 64 + c * 32, sv + c * 32);
        // columns that every row of the warp sees skip the per-element mask
        const bool full0 = __all_sync(0xffffffffu, lo <= j0 && j0 + 31 <= hi);
        const bool full1 = __all_sync(0xffffffffu, lo <= j0 + 32 && j0 + 63 <= hi);
        ptx::tmem_wait_ld();
        if (!full0) {
          const uint32_t bits = visible_bits(j0, lo, hi) | (j0 == 0 && anchored ? 1u : 0u);
#pragma unroll
          for (int e = 0; e < 32; ++e) sv[e] = (bits >> e) & 1u ? sv[e] : -INFINITY;
        }
        if (!full1) {
          const uint32_t bits = visible_bits(j0 + 32, lo, hi);
#pragma unroll
          for (int e = 0; e < 32; ++e) sv[32 + e] = (bits >> e) & 1u ? sv[32 + e] : -INFINITY;
        }
        float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < 64; e += 8)
#pragma unroll
          for (int x = 0; x < 4; ++x) mq[x] = fmaxf(mq[x], fmaxf(sv[e + 2 * x], sv[e + 2 * x + 1]));
        if (!(ok = agree(fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3]))))) break;
        const float mm = (m == -INFINITY) ? 0.f : m;
        const float2 sl22 = make_float2(sl2, sl2), nm2 = make_float2(-mm, -mm);
        float2 rs2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float* sc = sv + c * 32;
          uint32_t pw[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 x = __ffma2_rn(make_float2(sc[2 * e], sc[2 * e + 1]), sl22, nm2);
            const float2 pp = make_float2(ptx::ex2(x.x), ptx::ex2(x.y));
            rs2 = __fadd2_rn(rs2, pp);
            pw[e] = ptx::pack_bf16x2(pp.x, pp.y);  // the weights enter the product in bf16, their sum stays fp32
          }
          ptx::tmem_st16(t_p + c * 16, pw);
        }
        l += rs2.x + rs2.y;
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&sm.p_full[t]);
      }
      if (!ok) break;
      ok = warp_wait(&sm.o_full[t], nq & 1, b.err, abort_flag, 483);
      pair[half][lane] = l;  // the partner has read the last step's maxima: O is complete
      if (!ptx::bar_and(pair_bar, 64, ok)) break;
      l += pair[half ^ 1][lane];
      // ---- epilogue, half of the channels per warp. Its TMEM reads complete
      // (tmem_wait_ld) before this thread's next p_full arrival, which the next
      // piece's first PV of this tile (overwriting O) waits for.
      ptx::tc_fence_after();
      ++nq;
      if (w.whole) {
        const int head = w.g * P.group + r - in_tile * P.group;
        const int64_t row = w.q_row + t * C.tile_tokens + in_tile;
        const float inv_l = 1.f / l;
        if (row_valid && P.lse && half == 0) P.lse[(int64_t)head * b.T + row] = (m + log2f(l)) * 0.69314718055994531f;
        // four lanes store 64 bytes of one row together: they swap their
        // 16-byte quarters of 32 channels so that lane q holds quarter q of
        // the four rows
        const int at = row_valid ? (int)(row * P.Hq + head) : -1, q = lane & 3;
        int rows[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) rows[k] = __shfl_sync(0xffffffffu, at, (lane & ~3) + k);
#pragma unroll 1
        for (int c = 0; c < HD / 64; ++c) {
          float ov[32];
          ptx::tmem_ld32(t_o + c * 32, ov);
          ptx::tmem_wait_ld();
          uint32_t ow[4][4];  // [quarter][word]
#pragma unroll
          for (int e = 0; e < 16; ++e)
            ow[e >> 2][e & 3] = l != 0.f ? ptx::pack_bf16x2(ov[2 * e] * inv_l, ov[2 * e + 1] * inv_l) : 0u;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
#pragma unroll
            for (int d = 1; d <= 2; d *= 2)
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                if (k & d) continue;
                const uint32_t other = __shfl_xor_sync(0xffffffffu, (q & d) ? ow[k][x] : ow[k + d][x], d);
                if (q & d)
                  ow[k][x] = other;
                else
                  ow[k + d][x] = other;
              }
          }
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (rows[k] >= 0)
              *reinterpret_cast<uint4*>(P.o + (int64_t)rows[k] * HD + half * (HD / 2) + c * 32 + q * 8) =
                  make_uint4(ow[k][0], ow[k][1], ow[k][2], ow[k][3]);
        }
      } else {
        const int64_t part = ((int64_t)blockIdx.x * 2 + w.part) * 2 + t;
        float4* po = C.part_o + (part * (HD / 4) + half * (HD / 8)) * 128 + r;
#pragma unroll 1
        for (int c = 0; c < HD / 64; ++c) {
          float ov[32];
          ptx::tmem_ld32(t_o + c * 32, ov);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 8; ++e)  // hi: rows that are none leave nothing
            if (hi != INT_MAX) po[(c * 8 + e) * 128] = make_float4(ov[4 * e], ov[4 * e + 1], ov[4 * e + 2], ov[4 * e + 3]);
        }
        if (hi != INT_MAX && half == 0) C.part_ml[part * 128 + r] = make_float2(m, l);
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&sm.piece_empty[li & 1]);
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) ptx::tmem_dealloc(tmem, kTmemCols);
}

// ---------------------------------------------------------------- joining cut units
// kJoinRows rows of a cut unit at a time. With kHelp false blockIdx.y is a CTA of the
// attention kernel, and the block joins the unit that it began, if any. Contexts that
// are long for their few new tokens give few units many parts, and few rows to hide
// their latency behind: a thread keeps the loads of kAtOnce parts of its rows in
// flight, and with kHelp every block lists the cut units, up to kMaxHelp blocks take a
// share of the channels of the same rows, and the threads that this frees a share of
// the parts. Measured without / with, D = 128: 17 tokens of one sequence and kv head
// over 52K keys 66 / 26 us (138 parts), over 8K 26 / 18, over 1000 15.7 / 16.6; 64
// tokens of 8 sequences, 8 kv heads, over 1000 keys 27.0 / 30.0.
constexpr int kJoinRows = 16, kJoinThreads = 256, kAtOnce = 4, kMaxHelp = 8;
constexpr int kMaxCtas = kJoinThreads;  // a thread looks at each CTA's cut
constexpr int kJoinBlocks = 3;          // per SM
constexpr int kHelpKeys = 2048;         // blocks help with contexts above
constexpr int kHelpParts = 8;           // and where units can have so many parts

// Rows' running maximum (log2 units), sum and unnormalised O.
struct JoinState {
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  // the next N results of the row; ml.y == 0: one that saw nothing of it
  template <int N>
  __device__ __forceinline__ void add(const float2 (&ml)[N], const float4 (&v)[N]) {
    float mn = m;
#pragma unroll
    for (int x = 0; x < N; ++x) mn = fmaxf(mn, ml[x].x);
    const float f = m == -INFINITY ? 0.f : exp2f(m - mn);
    m = mn;
    l *= f;
    acc.x *= f;
    acc.y *= f;
    acc.z *= f;
    acc.w *= f;
#pragma unroll
    for (int x = 0; x < N; ++x) {
      if (ml[x].y == 0.f) continue;
      const float fk = exp2f(ml[x].x - mn);
      acc.x += fk * v[x].x;
      acc.y += fk * v[x].y;
      acc.z += fk * v[x].z;
      acc.w += fk * v[x].w;
      l += fk * ml[x].y;
    }
  }
};

template <int HD, bool kHelp>
__global__ void __launch_bounds__(kJoinThreads, kJoinBlocks) chunk_join_kernel(const __grid_constant__ ChunkParams C) {
  constexpr int kStep = kJoinThreads / (HD / 4);  // rows at a time: consecutive threads read consecutive rows
  constexpr int kMine = kJoinRows / kStep, kPieces = 256 / kJoinRows;
  const AttendParams& P = C.a;
  const int tid = threadIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  Cut u;
  int first, rows0, most = 1, share_of = 0;  // most: blocks that may share a unit's rows
  if constexpr (kHelp) {
    __shared__ Cut cuts[kMaxCtas];
    __shared__ int begins[kMaxCtas], found[kJoinThreads / 32];
    const Cut cut = tid < C.ctas ? C.cuts[tid] : Cut{-1, 0, 0, 0};
    const uint32_t here = __ballot_sync(0xffffffffu, cut.last >= 0);
    if ((tid & 31) == 0) found[tid >> 5] = __popc(here);
    __syncthreads();
    int units = 0, before = 0;
#pragma unroll
    for (int w = 0; w < kJoinThreads / 32; ++w) {
      if (w == tid >> 5) before = units;
      units += found[w];
    }
    if (cut.last >= 0) {
      before += __popc(here & ((1u << (tid & 31)) - 1u));
      cuts[before] = cut;
      begins[before] = tid;
    }
    __syncthreads();
    while (most < kMaxHelp && units * kPieces * most * 2 <= (int)gridDim.x) most *= 2;
    const int unit = (int)blockIdx.x / (kPieces * most);
    if (unit >= units) return;
    u = cuts[unit];
    first = begins[unit];
    share_of = (int)blockIdx.x / kPieces % most;
    rows0 = (int)blockIdx.x % kPieces * kJoinRows;
  } else {
    first = (int)blockIdx.y;
    u = C.cuts[first];
    if (u.last < 0) return;
    rows0 = (int)blockIdx.x * kJoinRows;
  }
  const int t = rows0 >> 7, parts = u.last - first + 1;  // row tile
  if ((rows0 & 127) >= (u.tokens - t * C.tile_tokens) * P.group) return;  // the rows hold no token
  int help = 1;
  while (help < most && parts >= 2 * help * kAtOnce) help *= 2;
  if (share_of >= help) return;
  const int columns = HD / 4 / help, group = tid / (kStep * columns);  // columns of four channels
  const int c = share_of * columns + tid / kStep % columns;
  auto row = [&](int i) { return (rows0 + tid % kStep + i * kStep) & 127; };
  JoinState mine[kMine];
  const int share = (parts + help - 1) / help, begin = first + group * share, end = min(begin + share, u.last + 1);
  for (int k0 = begin; k0 < end; k0 += kAtOnce) {
    float2 ml[kMine][kAtOnce];
    float4 v[kMine][kAtOnce];
#pragma unroll
    for (int i = 0; i < kMine; ++i)
#pragma unroll
      for (int x = 0; x < kAtOnce; ++x) {
        const int k = k0 + x;
        const int64_t part = ((int64_t)k * 2 + (k == first ? 1 : 0)) * 2 + t;
        ml[i][x] = k < end ? C.part_ml[part * 128 + row(i)] : make_float2(-INFINITY, 0.f);
        v[i][x] = k < end ? C.part_o[(part * (HD / 4) + c) * 128 + row(i)] : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
    for (int i = 0; i < kMine; ++i) mine[i].add(ml[i], v[i]);
  }
  if constexpr (kHelp) {
    if (help > 1) {  // the first group's threads take the other groups' results, in order
      __shared__ float4 group_o[kMine][kJoinThreads];
      __shared__ float2 group_ml[kMine][kJoinThreads];
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        group_o[i][tid] = mine[i].acc;
        group_ml[i][tid] = make_float2(mine[i].m, mine[i].l);
      }
      __syncthreads();
      if (group > 0) return;
      for (int g = 1; g < help; ++g)
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
          const float2 ml[1] = {group_ml[i][tid + g * kStep * columns]};
          const float4 v[1] = {group_o[i][tid + g * kStep * columns]};
          mine[i].add(ml, v);
        }
    }
  }
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int r = row(i), in_tile = r / P.group, tok = t * C.tile_tokens + in_tile;
    if (in_tile >= C.tile_tokens || tok >= u.tokens) continue;  // the row holds no token
    const int head = u.g * P.group + r - in_tile * P.group;
    const int64_t t_row = u.q_row + tok;
    *reinterpret_cast<uint2*>(P.o + (t_row * P.Hq + head) * HD + c * 4) = normalised(mine[i].acc, mine[i].l);
    if (c == 0 && P.lse) P.lse[(int64_t)head * P.batch.T + t_row] = (mine[i].m + log2f(mine[i].l)) * 0.69314718055994531f;
  }
}

// ---------------------------------------------------------------- launches
int ctas_for(const aa_cache_s* c) { return std::min(c->num_sms, kMaxCtas); }
bool whole_units(int table_width, int page_shift) { return ((int64_t)table_width << page_shift) <= kWholeKeys; }
int slots_for(int tokens, int seqs, int tile_tokens) { return tokens / (2 * tile_tokens) + seqs; }

template <int HD>
aa_status launch(const aa_cache_s* c, const AttendParams& P, void* workspace, cudaStream_t s) {
  const BatchParams& b = P.batch;
  ChunkParams C;
  C.a = P;
  C.tile_tokens = 128 / P.group;
  C.slots = slots_for(b.T, b.B, C.tile_tokens);
  C.whole_units = whole_units(b.W, P.page_shift);
  const int ctas = ctas_for(c);
  C.ctas = ctas;
  C.tiles_end = nullptr;
  C.units = nullptr;
  C.part_o = nullptr;
  C.part_ml = nullptr;
  C.cuts = nullptr;
  if (!C.whole_units) {
    uint8_t* w = static_cast<uint8_t*>(workspace);
    C.part_o = reinterpret_cast<float4*>(w);
    w += align256((size_t)ctas * 4 * 128 * HD * 4);
    C.part_ml = reinterpret_cast<float2*>(w);
    w += align256((size_t)ctas * 4 * 128 * 8);
    C.cuts = reinterpret_cast<Cut*>(w);
    w += align256((size_t)ctas * sizeof(Cut));
    C.units = reinterpret_cast<Unit*>(w);
    w += align256((size_t)C.slots * sizeof(Unit));
    C.tiles_end = reinterpret_cast<int64_t*>(w);
  }
  CUtensorMap tq;
  aa_status st = make_query_map(&tq, P.q, b.T, P.q_stride, b.Hkv, P.group, HD, C.tile_tokens);
  if (st != AA_OK) return st;
  const size_t smem = sizeof(ChunkSmem<HD>);
  static std::once_flag once[kMaxDevices];
  static cudaError_t result[kMaxDevices];
  cudaError_t e = once_per_device(once, result, c->device, [&] {
    return cudaFuncSetAttribute(attend_chunk_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  });
  if (e != cudaSuccess) return cuda_fail(e, "attend_chunk_kernel smem attribute");
  if (C.whole_units) {
    const unsigned grid = (unsigned)std::min<int64_t>((int64_t)C.slots * b.Hkv, ctas);
    e = launch_after(attend_chunk_kernel<HD>, dim3(grid), kThreads, smem, s, tq, c->k_map64, c->v_map64, C);
    return e == cudaSuccess ? AA_OK : cuda_fail(e, "attend_chunk_kernel launch");
  }
  chunk_plan_kernel<<<1, 1024, 0, s>>>(C);
  if ((e = cudaGetLastError()) != cudaSuccess) return cuda_fail(e, "chunk_plan_kernel launch");
  e = launch_after(attend_chunk_kernel<HD>, dim3((unsigned)ctas), kThreads, smem, s, tq, c->k_map64, c->v_map64, C);
  if (e != cudaSuccess) return cuda_fail(e, "attend_chunk_kernel launch");
  const bool few = (int64_t)C.slots * b.Hkv * kHelpParts <= ctas && ((int64_t)b.W << P.page_shift) > kHelpKeys;
  static_assert(256 / kJoinRows <= kHelpParts * kJoinBlocks, "a block for each piece of the few units");
  e = few ? launch_after(chunk_join_kernel<HD, true>, dim3((unsigned)(kJoinBlocks * ctas)), kJoinThreads, 0, s, C)
          : launch_after(chunk_join_kernel<HD, false>, dim3(256 / kJoinRows, (unsigned)ctas), kJoinThreads, 0, s, C);
  if (e != cudaSuccess) return cuda_fail(e, "chunk_join_kernel launch");
  return AA_OK;
}

}  // namespace

size_t chunk_workspace_bytes(const aa_cache_s* c, int num_seqs, int total_tokens, int table_width, int group) {
  if (whole_units(table_width, __builtin_ctz((unsigned)c->cfg.page_size))) return 256;  // nothing is kept
  const size_t slots = slots_for(total_tokens, num_seqs, 128 / group), ctas = ctas_for(c);
  return align256(ctas * 4 * 128 * c->cfg.head_dim * 4) + align256(ctas * 4 * 128 * 8) + align256(ctas * sizeof(Cut)) +
         align256(slots * sizeof(Unit)) + align256((slots + 1) * 8);
}

aa_status launch_attend_chunk(const aa_cache_s* c, const AttendParams& P, void* workspace, cudaStream_t s) {
  return c->cfg.head_dim == 128 ? launch<128>(c, P, workspace, s) : launch<64>(c, P, workspace, s);
}

}  // namespace aa
