/*
 * anchorattn.h — C ABI of the GB300 (sm_103a) fused RoPE + AnchorAttention
 * library (libanchorattn.so).
 *
 * The method: "When Precision Meets Position: BFloat16 Breaks Down RoPE in
 * Long-Context Training" (arXiv 2411.13476). Operation references below name
 * the page and its section:
 *   [ARCH §3.4 RoPE]    architecture page, §3.4 "Rotary Positional Embedding
 *                       (RoPE): The Theoretical Promise", Eq. 6 and Eq. 3.
 *   [ARCH §3.4 Index]   architecture page, §3.4 "Document Token Indexing"
 *                       (continuous IDs, Fig. 2 left; reset IDs, Fig. 2 middle).
 *   [ARCH §3.4 Anchor]  architecture page, §3.4 "AnchorAttention: The Shared
 *                       Anchor Design", "Core design" and "Mask construction".
 *   [ARCH §3.2]         architecture page, §3.2 "Big-Picture Architecture":
 *                       RoPE in fp32, cast to bf16, inner products in bf16.
 *   [ARCH §3.4 Diag]    architecture page, §3.4 "Diagnostic Methodology:
 *                       Measuring the Breakdown", Eq. 4 (attention difference)
 *                       and Eq. 5 (first-token logit difference).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Tensors are caller-owned, contiguous, row-major [T, H, D] bf16 (token,
 *    head, channel), 16-byte aligned device pointers. LSE/D-style per-row
 *    values are fp32 [H, T].
 *  - Q and K are passed UN-ROTATED: the library rotates them (RoPE in fp32,
 *    rounded to bf16) once per call in its own kernels; gradients are returned
 *    with respect to the un-rotated inputs (aa_bwd_from_fwd takes the
 *    forward's rotated copies instead of q and k).
 *  - Token 0 is the anchor. cu_doclens (host int32[num_docs + 1]) gives the
 *    document boundaries after it: document k occupies tokens
 *    [cu[k-1], cu[k]), with cu[0] == 1, cu[num_docs] == T, strictly increasing.
 *    In AA_MASK_CAUSAL mode cu_doclens is ignored (may be NULL).
 *  - Every call validates its arguments synchronously and returns a status
 *    without launching anything on failure. Kernel launches are asynchronous
 *    on `stream` (NULL = the legacy default stream); launch failures return
 *    AA_ERR_CUDA. Device-side waits are bounded: a wait that runs out records
 *    an error word that aa_check_device_error() turns into AA_ERR_TIMEOUT.
 *  - aa_fwd / aa_bwd / aa_rope_apply allocate no memory (scratch comes from
 *    caller workspaces sized by aa_*_workspace_bytes). aa_plan allocates the
 *    plan's device metadata; aa_plan_destroy frees it.
 *  - Compute calls may overlap on the GPU when each has its own workspace
 *    (the persistent kernels keep their work counters there); calls with one
 *    plan share its device error word, so aa_check_device_error() reports a
 *    timeout from any of them.
 *  - The compute calls enqueue only stream-ordered work (kernel launches and
 *    asynchronous memsets of their work counters), so a sequence of them may
 *    be captured in a CUDA graph and replayed while the plan, the tensors and
 *    the workspaces it names stay alive. Make one uncaptured call of each
 *    entry point per device first: the first call sets the kernels'
 *    shared-memory attributes (aa_bwd_static_workspace also looks up its
 *    array's address then).
 *  - A thread-local message describing the last failure is available from
 *    aa_last_error().
 */
#ifndef ANCHORATTN_H
#define ANCHORATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* aa_stream_t; /* identical to cudaStream_t */

typedef enum {
  AA_OK = 0,
  AA_ERR_INVALID_ARG = 1,
  AA_ERR_UNSUPPORTED = 2,
  AA_ERR_CUDA = 3,
  AA_ERR_NO_MEMORY = 4,
  AA_ERR_TIMEOUT = 5
} aa_status;

/* Which (query, key) pairs are visible. [ARCH §3.4 Anchor], [ARCH §3.4 Index]
 * CAUSAL:    j <= i over the whole packed sequence (full attention baseline).
 * INTRA_DOC: j <= i and same document; the anchor is a one-token document.
 * ANCHOR:    INTRA_DOC plus key 0 (the anchor) visible to every query; the
 *            anchor query sees only itself. */
typedef enum { AA_MASK_CAUSAL = 0, AA_MASK_INTRA_DOC = 1, AA_MASK_ANCHOR = 2 } aa_mask_mode;

/* Position IDs [ARCH §3.4 Index]. RESET: anchor 0, every document 1..N_k.
 * CONTINUOUS: 0..T-1 across documents. CAUSAL mode always uses 0..T-1. */
typedef enum { AA_POS_RESET = 0, AA_POS_CONTINUOUS = 1 } aa_pos_mode;

/* Pairing of rotated coordinates. ADJACENT = Eq. 6 of [ARCH §3.4 RoPE]
 * (pairs (2p, 2p+1)); HALF pairs (p, p + D/2); NONE disables the rotation. */
typedef enum { AA_ROPE_ADJACENT = 0, AA_ROPE_HALF = 1, AA_ROPE_NONE = 2 } aa_rope_layout;

typedef struct {
  int32_t total_tokens;  /* T >= 2, anchor included; T < 2^30                 */
  int32_t num_q_heads;   /* Hq >= 1                                            */
  int32_t num_kv_heads;  /* Hkv >= 1, Hq % Hkv == 0 (grouped-query attention)  */
  int32_t head_dim;      /* D: 64 or 128                                       */
  double rope_base;      /* theta_p = rope_base^(-2p/D); > 1                   */
  float softmax_scale;   /* <= 0 selects 1/sqrt(D)                             */
  int32_t pos_shift;     /* Delta added to every position (Eq. 3); >= 0       */
  int32_t mask_mode;     /* aa_mask_mode                                       */
  int32_t pos_mode;      /* aa_pos_mode                                        */
  int32_t rope_layout;   /* aa_rope_layout                                     */
  int32_t host_only;     /* 1: build host metadata only (no GPU needed);
                            compute calls on such a plan return
                            AA_ERR_INVALID_ARG                                 */
} aa_config;

typedef struct aa_plan_s* aa_plan_t;

/* Build the plan for one packing [ARCH §3.4 Anchor "Mask construction",
 * §3.4 Index]: per-token document and position IDs, each query row's visible
 * key interval, the live 128x128 tile lists (fully cross-document tiles are
 * dropped; the anchor column is folded in separately) in the order the
 * persistent attention kernels claim them (grouped by document, longest
 * group first: the forward's heads interleaved in each document, the
 * backward's one group per document and head; a forward item is two query
 * tiles of one head, or one query tile of two heads sharing a kv head when
 * Hq/Hkv is even), and the two-level fp32 cos/sin tables of Eq. 6 built in
 * fp64.
 * cu_doclens: host int32[num_docs + 1] (see conventions). Device metadata is
 * uploaded with copies ordered on `stream`. On success *out owns everything;
 * release it with aa_plan_destroy. */
aa_status aa_plan(const aa_config* cfg, const int32_t* cu_doclens_host, int32_t num_docs,
                  aa_stream_t stream, aa_plan_t* out);

/* aa_plan with caller-supplied rotation frequencies: theta (host double[D/2])
 * replaces Eq. 6's theta_p = rope_base^(-2p/D) for every pair p [ARCH §3.4
 * RoPE]; cfg->rope_base is then ignored. This carries the frequency tables of
 * RoPE variants such as NTK-aware scaling or YaRN, which the pages compare
 * with vanilla RoPE for 64K training (architecture page, §3.4 "Long-Context
 * Training Protocol", "Vanilla RoPE vs. NTK vs. YaRN", Table 2) without
 * defining their formulas: the caller computes the table, the library
 * rotates with it (fp64 tables, fp32 rotation, bf16 operands, as for the
 * default). The table is copied. Errors: NULL theta, or an entry that is not
 * finite and >= 0, gives AA_ERR_INVALID_ARG; otherwise as aa_plan. */
aa_status aa_plan_with_theta(const aa_config* cfg, const int32_t* cu_doclens_host, int32_t num_docs,
                             const double* theta, aa_stream_t stream, aa_plan_t* out);

/* Plan for documents given per token, possibly in interleaved chunks
 * [ARCH §3.4 Anchor "Mask construction"]; architecture page, §3.4
 * "AnchorAttention with Interleaved Chunks" (documents split into chunks that
 * are shuffled and recombined with the order inside each document kept).
 * doc_of_token: host int32[T]; token 0 is the anchor and must be 0, every
 * other token names its document with an id >= 1 (any values; chunks of one
 * document share an id, so they see each other; give each chunk its own id
 * to keep chunks apart). A token sees the anchor (ANCHOR mode) and the tokens
 * j <= i of its own document. Positions: RESET counts 1, 2, ... through the
 * document's tokens in order, CONTINUOUS is the token index; pos_shift adds.
 * cfg->mask_mode must be ANCHOR or INTRA_DOC. aa_fwd / aa_bwd /
 * aa_bwd_from_fwd / aa_bwd_static_workspace / aa_rope_apply take and return
 * tensors in the caller's token order (the library's kernels run on the
 * tokens grouped by document: the rotation passes read q and k through the
 * grouping, V is gathered once per forward (aa_bwd_from_fwd reads the
 * forward's copy), the backward's first kernel reads o, dout and lse through
 * it and keeps a grouped dout, and every output is written at its caller
 * position; the workspace sizes include those copies); aa_plan_metadata
 * returns the caller's document ids and
 * positions; aa_plan_stats / aa_plan_work count the grouped layout's tiles.
 * aa_shift_diag refuses segment plans (AA_ERR_UNSUPPORTED). Errors: NULL
 * doc_of_token, doc_of_token[0] != 0, an id < 1 after it, or the aa_plan
 * conditions give AA_ERR_INVALID_ARG. */
aa_status aa_plan_segments(const aa_config* cfg, const int32_t* doc_of_token_host, aa_stream_t stream,
                           aa_plan_t* out);

/* Free a plan (synchronises the device). NULL is accepted. */
aa_status aa_plan_destroy(aa_plan_t plan);

/* Copy the per-token document index (anchor = 0, documents 1..K; all 0 in
 * CAUSAL mode) and position ID (shift included) into caller host buffers of
 * T int32 each. Either pointer may be NULL. */
aa_status aa_plan_metadata(aa_plan_t plan, int32_t* doc_id_host, int32_t* pos_id_host);

/* unmasked_pairs: visible (query, key) pairs of the mask (the T^2/K + T count
 * of [ARCH §3.4 Anchor], "Reduction in attention computations"), anchor pairs
 * included. live_tiles: 128x128 blocks of the mask holding a visible pair.
 * causal_tiles: blocks with any j <= i (what full causal attention visits).
 * Any pointer may be NULL. */
aa_status aa_plan_stats(aa_plan_t plan, int64_t* unmasked_pairs, int64_t* live_tiles,
                        int64_t* causal_tiles);

/* Work the kernels perform: fwd_tiles = (q-tile, k-tile, head) MMA tiles of
 * the forward pass; bwd_tiles = the same count for the backward pass (one
 * tile = one 128x128 block of one query head). Any pointer may be NULL. */
aa_status aa_plan_work(aa_plan_t plan, int64_t* fwd_tiles, int64_t* bwd_tiles);

/* Rotate x [T, num_heads, D] bf16 into y (same shape; y may equal x) with the
 * plan's positions: y = R_pos x (inverse = 0) or R_pos^T x (inverse = 1),
 * fp32 arithmetic, round-to-nearest-even to bf16 [ARCH §3.4 RoPE Eq. 6,
 * ARCH §3.2]. num_heads is independent of the plan's head counts. */
aa_status aa_rope_apply(aa_plan_t plan, const void* x, void* y, int32_t num_heads,
                        int32_t inverse, aa_stream_t stream);

/* Forward [ARCH §3.4 Anchor, §3.4 RoPE]: for every query row i and head h,
 *   O_i = sum_{j visible} softmax_j(scale * (R_i q_i).(R_j k_j)) v_j,
 *   LSE_i = ln sum_{j visible} exp(scale * (R_i q_i).(R_j k_j)).
 * q [T,Hq,D], k/v [T,Hkv,D] bf16 in; o [T,Hq,D] bf16, lse [Hq,T] fp32 out.
 * Query head h reads kv head h / (Hq / Hkv). Q and K are rotated once per
 * call into `workspace` (caller-owned device memory of at least
 * aa_fwd_workspace_bytes(plan) bytes, 256-byte aligned, contents ignored),
 * which the attention kernel then reads; it also holds the kernel's work
 * counter, so forward calls with separate workspaces may overlap. */
aa_status aa_fwd(aa_plan_t plan, const void* q, const void* k, const void* v, void* o,
                 float* lse, void* workspace, size_t workspace_bytes, aa_stream_t stream);

/* Bytes of device scratch aa_fwd needs: the rotated K and Q, T*(Hkv+Hq)*D
 * bf16, which it leaves there for aa_bwd_from_fwd (none with AA_ROPE_NONE),
 * plus 256 bytes for the work counter; segment plans add a grouped copy of
 * v (read again by aa_bwd_from_fwd) and, without RoPE, of q and k. */
size_t aa_fwd_workspace_bytes(aa_plan_t plan);

/* Bytes of device scratch aa_bwd needs (rotated Q and K, fp32 dQ
 * accumulator, per-row D, anchor partial sums; segment plans add their
 * grouped copies). */
size_t aa_bwd_workspace_bytes(aa_plan_t plan);

/* Backward of aa_fwd: given dout = dL/dO, writes dq [T,Hq,D], dk/dv
 * [T,Hkv,D] bf16 = gradients with respect to the UN-ROTATED q, k and v
 * (dq = R^T dq~, dk = R^T dk~). q, k, v, o and lse must be the forward's
 * inputs and outputs. workspace: caller-owned device memory of at least
 * aa_bwd_workspace_bytes(plan) bytes, 256-byte aligned, contents ignored.
 * dK/dV of the anchor sum over every query row (and over the group's query
 * heads). dQ is accumulated with fp32 atomics, so its last bits may vary
 * between runs; every other output is run-to-run deterministic. */
aa_status aa_bwd(aa_plan_t plan, const void* q, const void* k, const void* v, const void* o,
                 const float* lse, const void* dout, void* dq, void* dk, void* dv,
                 void* workspace, size_t workspace_bytes, aa_stream_t stream);

/* aa_bwd from the forward's rotated operands (no counterpart in the paper:
 * an interface addition of this library) [ARCH §3.4 Anchor, §3.4 RoPE].
 * aa_fwd leaves the rotated Q and K (R_i q_i, R_j k_j, rounded to bf16) in
 * its workspace; a training step that keeps that workspace until the
 * backward pass, instead of q and k, passes it here as fwd_workspace and the
 * backward skips its own rotation of Q and K (two passes over them).
 *  - fwd_workspace: the workspace of an aa_fwd call with this plan and the
 *    q, k whose gradients are wanted, unchanged since that call (the library
 *    cannot check this; it is the caller's contract). Read only.
 *  - v, o, lse, dout, dq, dk, dv: as for aa_bwd; the results are the same
 *    (gradients with respect to the UN-ROTATED q, k and v): dk, dv bit for
 *    bit, dq up to the order of its fp32 atomic additions.
 *  - workspace: at least aa_bwd_from_fwd_workspace_bytes(plan) bytes,
 *    256-byte aligned, contents ignored (smaller than aa_bwd's: no rotated
 *    copies).
 *  - AA_ERR_UNSUPPORTED with AA_ROPE_NONE (aa_fwd rotates nothing; call
 *    aa_bwd); AA_ERR_INVALID_ARG for NULL or misaligned pointers or a short
 *    workspace, with nothing launched. */
aa_status aa_bwd_from_fwd(aa_plan_t plan, const void* fwd_workspace, const void* v, const void* o,
                          const float* lse, const void* dout, void* dq, void* dk, void* dv,
                          void* workspace, size_t workspace_bytes, aa_stream_t stream);

/* Bytes of device scratch aa_bwd_from_fwd needs. */
size_t aa_bwd_from_fwd_workspace_bytes(aa_plan_t plan);

/* aa_bwd without a caller-provided workspace (no counterpart in the paper:
 * an interface addition of this library).
 * Some callers cannot call cudaMalloc at the point where they run the
 * backward pass: a plugin inside a host framework whose memory planner owns
 * every device allocation, a latency-critical loop where an allocation would
 * stall or synchronise the device, or a deployment that must stay inside a
 * memory budget fixed at start-up. This entry point takes its scratch from a
 * 64 MiB array that the library reserves statically on every GPU that loads
 * it (held until the process exits) and allocates nothing itself.
 *  - Arguments and results are those of aa_bwd minus the workspace pair.
 *  - Plans whose aa_bwd_workspace_bytes() exceeds 64 MiB are rejected with
 *    AA_ERR_INVALID_ARG and a message giving both sizes; nothing is launched.
 *    aa_bwd_workspace_bytes() is the exact test. As a guide, for plans built
 *    from cu_doclens with RoPE at D = 128 a query row needs about 1 KB
 *    (rotated Q and K and the fp32 dQ accumulator) and each query head
 *    64 KB of anchor partials, so T * Hq up to about 60K query rows fit.
 *    Segment plans (aa_plan_segments) also need grouped copies of v and
 *    dout (and, without RoPE, of q and k), so somewhat fewer rows fit.
 *  - The plan's device must be current. The first call on a device looks up
 *    the array's device address (cudaGetSymbolAddress) once and keeps it for
 *    the life of the process; make that first call before any stream capture
 *    on that device. The kept address does not survive a reset of the
 *    device's primary context (cudaDeviceReset): do not call this entry point
 *    after one.
 *  - Every call on a device shares the one array, and the array keeps the
 *    last call's contents; the call overwrites all the scratch it reads, so
 *    nothing needs clearing. Calls whose executions overlap on the GPU (for
 *    instance on two streams) race on the array and give wrong results:
 *    order them on one stream or with events. */
aa_status aa_bwd_static_workspace(aa_plan_t plan, const void* q, const void* k, const void* v,
                                  const void* o, const float* lse, const void* dout, void* dq, void* dk,
                                  void* dv, aa_stream_t stream);

/* Synchronise `stream`, read and clear the plan's device error word.
 * Returns AA_ERR_TIMEOUT if a bounded device wait ran out since the last
 * check, AA_OK otherwise. */
aa_status aa_check_device_error(aa_plan_t plan, aa_stream_t stream);

/* Diagnostics: limit (nanoseconds) of every bounded device wait for this
 * plan; 0 makes each wait give up after its first poll (the kernels then
 * drain their in-flight copies and MMAs and return with the error word set).
 * The default is 2e9 ns. */
aa_status aa_set_wait_limit(aa_plan_t plan, uint64_t nanoseconds);

/* Measurement hook: when both are non-NULL CUDA events (cudaEvent_t),
 * aa_bwd and aa_bwd_from_fwd record `start` immediately before and `stop`
 * immediately after the launch of their main tile kernel, on the call's stream, so that kernel can be
 * timed on its own. NULL, NULL (the default) disables the recording. The
 * events are caller-owned and must outlive the calls that record them. */
aa_status aa_set_bwd_timing_events(aa_plan_t plan, void* start, void* stop);

/* Failure-detection self-test: launches one CTA that waits on a shared-memory
 * barrier nothing ever arrives on, bounded by the plan's wait limit
 * (aa_set_wait_limit). The wait runs out, the kernel records its site code in
 * the plan's error word and returns, leaving the context usable; the next
 * aa_check_device_error() returns AA_ERR_TIMEOUT. This is the same bounded
 * wait every attention kernel uses. */
aa_status aa_selftest_bounded_wait(aa_plan_t plan, aa_stream_t stream);

/* Shift-discrepancy diagnostics. [ARCH §3.4 Diag], [ARCH §3.4 RoPE] (Eq. 3)
 * Two plans that differ only in pos_shift (Δ1 for plan1, Δ2 for plan2) and one
 * un-rotated input q [T, Hq, D], k [T, Hkv, D] (bf16). The library rotates q
 * and k under both shifts with its own RoPE kernel (the bf16 operands its
 * attention uses) and computes, with the plans' mask:
 *   col_absdiff[h][j]         = sum_i |ATTN_ij(Δ1) - ATTN_ij(Δ2)|   (fp32 [Hq, T])
 *   first_logit_absdiff[h][i] = |A_i0(Δ1) - A_i0(Δ2)|              (fp32 [Hq, T])
 *     (0 for rows that cannot see token 0), A = scale * q~_i . k~_j the
 *     pre-softmax logit, ATTN = softmax of A over the visible keys;
 *   result (fp64, 2 + 2*Hq):  result[0] = D (Eq. 4) = sum_h sum_j
 *     col_absdiff[h][j] / n_j with n_j the rows that may attend to key j;
 *     result[1] = D_logit (Eq. 5) = (1/T) sum_h sum_i first_logit_absdiff[h][i];
 *     result[2 + 2h], result[3 + 2h] = head h's two sums.
 * Under exact arithmetic both are zero (Eq. 3); what they measure here is the
 * bf16 rounding of the rotated operands. The logits are recomputed on CUDA
 * cores in fp32 (an evaluation tool, not a training-step kernel); the column
 * sums use atomics, so their last bits can vary run to run.
 * workspace: aa_shift_diag_workspace_bytes(plan1) bytes (rotated Q and K under
 * both shifts; 0 without RoPE), 16-byte aligned device memory. Errors: plans
 * that differ in anything but pos_shift, a host-only plan, NULL or unaligned
 * pointers, or a short workspace give AA_ERR_INVALID_ARG before any launch. */
size_t aa_shift_diag_workspace_bytes(aa_plan_t plan);
aa_status aa_shift_diag(aa_plan_t plan1, aa_plan_t plan2, const void* q, const void* k, float* col_absdiff,
                        float* first_logit_absdiff, double* result, void* workspace, size_t workspace_bytes,
                        aa_stream_t stream);

/* Sharding of one packing across ranks [ARCH §3.4 Anchor] ("Mask
 * construction": documents see nothing of one another; every row sees the
 * anchor), architecture page §3.4 "AnchorContext: Implementation
 * Infrastructure" (the pages shard attention over 8 GPUs). Host only: no
 * plan, no device.
 * A piece is document `doc` (1-based, as in cu_doclens) restricted to kv
 * heads [kv_head_begin, kv_head_end) and their query heads (query head h
 * belongs to kv head h / group); `cost` = its visible pairs, (N(N+1)/2 + N)
 * per query head. Pieces go longest first to the least-loaded shard; a
 * document whose all-head cost exceeds total / num_shards is first cut into
 * ceil(cost / (total / num_shards)) kv-head ranges (at most num_kv_heads).
 * Every (document, kv head) lies in exactly one piece, so each rank runs its
 * pieces as ordinary packings (one per distinct head range, each with its
 * own copy of the anchor token) and the only exchanges are the anchor's k_0 /
 * v_0 (broadcast before the forward) and the sum of the ranks' dk_0 / dv_0
 * (all-reduce after the backward).
 *  - cu_doclens: host int32[num_docs + 1], as for aa_plan (cu[0] == 1).
 *  - group = Hq / Hkv; num_shards >= 1.
 *  - pieces: caller array of max_pieces entries, filled sorted by (shard,
 *    kv_head_begin, doc); *num_pieces receives the count. If max_pieces is
 *    too small, *num_pieces receives the count needed and AA_ERR_INVALID_ARG
 *    is returned (call with pieces = NULL, max_pieces = 0 to size the array).
 *  - shard_cost: optional int64[num_shards], each shard's summed cost. */
typedef struct {
  int32_t shard, doc, kv_head_begin, kv_head_end;
  int64_t cost;
} aa_shard_piece;
aa_status aa_shard_plan(const int32_t* cu_doclens_host, int32_t num_docs, int32_t num_kv_heads, int32_t group,
                        int32_t num_shards, aa_shard_piece* pieces, int32_t max_pieces, int32_t* num_pieces,
                        int64_t* shard_cost);

/* ------------------------------------------------------------------------
 * Rotary positions with several axes
 *
 * Tokens of images and video carry one position per axis (time, height,
 * width); text tokens carry the same number on every axis. Pair p of a head
 * belongs to one axis a(p) and turns by pos[a(p)][t] * theta_p, in the pairing
 * of `layout` (Eq. 6's 2x2 block, [ARCH §3.4 RoPE]). With one axis this is
 * Eq. 6 itself for positions that the caller gives per token.
 *
 * aa_rope_axes is a plain value that the caller owns: it holds no device
 * memory, may be copied, and serves any number of calls, threads and
 * devices. Fill it with aa_rope_axes_init; the fields are the library's. */
typedef struct {
  int32_t head_dim, num_axes, layout, ready;
  int32_t axis_of_pair[64];
  uint64_t turn[64]; /* theta_p / (2 pi) modulo 1, in units of 2^-64 */
} aa_rope_axes;

/* head_dim 64 or 128; num_axes 1..4; layout AA_ROPE_ADJACENT or AA_ROPE_HALF;
 * axis_of_pair host int32[head_dim / 2], each in [0, num_axes); theta host
 * double[head_dim / 2], finite and >= 0 (0 leaves the pair as it is). */
aa_status aa_rope_axes_init(aa_rope_axes* rope, int32_t head_dim, int32_t num_axes, int32_t layout,
                            const int32_t* axis_of_pair, const double* theta);

/* Rotate q [T, q_heads, D] and k [T, k_heads, D] (bf16) into q_out and k_out
 * (contiguous, same shapes) in one launch; inverse = 1 turns back, which is
 * also the gradient of the forward rotation.
 *  - pos: device int32 [num_axes, total_tokens], any value (negative ones
 *    turn the other way). The angle is reduced exactly in 64-bit fixed point,
 *    so it stays within 2^-20 rad for |pos| * theta_p up to 2^30.
 *  - q_stride, k_stride: elements from one token to the next, a multiple of 8
 *    and >= heads * D (a slice of a joint projection is fine); the heads of a
 *    token are contiguous. fp32 arithmetic, rounded once to bf16.
 *  - k may be NULL with k_heads = 0. q_out = q (k_out = k) rotates in place
 *    if that input is contiguous; outputs overlap nothing else.
 *  - total_tokens = 0 is an empty call; its pointers are not looked at. */
aa_status aa_rope_axes_apply(const aa_rope_axes* rope, const int32_t* pos, int32_t total_tokens, const void* q,
                             int64_t q_stride, void* q_out, int32_t q_heads, const void* k, int64_t k_stride,
                             void* k_out, int32_t k_heads, int32_t inverse, aa_stream_t stream);

/* ------------------------------------------------------------------------
 * Paged key/value cache: answering with a model that this library trained
 *
 * The pool is two caller-owned bf16 arrays, k_pages and v_pages, each
 * [num_layers, num_pages, Hkv, page_size, D]: a page holds page_size
 * consecutive tokens of one sequence, and one head's part of it is contiguous
 * (page_size * D * 2 bytes, what one copy into shared memory takes). Keys are
 * stored ROTATED, so a page needs no positions.
 *
 * 8-bit pages (aa_cache_create_fp8) hold half of the bytes: k_pages and v_pages are
 * e4m3 numbers (one byte each), and k_scales and v_scales, [num_layers, num_pages,
 * Hkv, page_size] bytes, give each token's D values of a head their power of two: the
 * values are code * 2^(byte - 127). aa_cache_append chooses the smallest exponent in
 * [-100, 119] that keeps the row's largest magnitude within 448 times it, and rounds
 * the (rotated) fp32 values once, to the nearest, ties to even: within 2^-4 of the value
 * or 2^-10 of the power, whichever is more (magnitudes above 448 * 2^119, bf16's
 * largest 14 %, become that). A row with a value that is not finite gets byte 255 and
 * is NaN as a whole. Pages that the caller fills have bytes in [3, 246], the range in which
 * bf16 holds every code times the power of two, or 255 for NaN, and no NaN codes (what
 * other bytes, 0x7f and 0xff give is not defined). All other calls are the same for both kinds.
 *
 * Two halves:
 *  - Bookkeeping on the host (aa_cache_resize, _fork, _compact, _tables,
 *    _stats): which page belongs to which sequence, with a reference count
 *    for each page, so that forked sequences share what they have in common.
 *    The handle is not thread-safe. A caller with its own scheduler leaves
 *    this half alone (max_seqs = 0) and passes its own page tables below.
 *  - Device calls (aa_cache_append, _read, _attend, _attend_tree, _tree_masks,
 *    _accept, _copy_pages): stream-ordered,
 *    no allocation, no host synchronisation. Everything that changes from
 *    step to step (page tables, lengths) is read on the device, so a step can
 *    be captured in a CUDA graph once and replayed with new contents.
 *
 * Batch layout of the device calls. B sequences; the new tokens of all of
 * them lie one after the other in [T, H, D] tensors, sequence b's in rows
 * [cu_q[b], cu_q[b + 1]) (device int32[B + 1], from 0, not decreasing; a
 * sequence may have none). kv_len[b] (device int32[B]) counts the sequence's
 * tokens INCLUDING the new ones: new token i of n_b has position
 * kv_len[b] - n_b + i. page_table: device int32 [B, table_width], entry w the
 * page of positions [w * page_size, (w + 1) * page_size); entries past a
 * sequence's last page are never read. Rows at or behind cu_q[B] are left as
 * they were.
 *
 * A page number outside [0, num_pages), or a position outside the table, is
 * never used as an address: the token is skipped (append) or reads as zeros
 * (attend), an error word is set, and aa_cache_check_error() reports it. A
 * position below 0 (kv_len[b] < n_b) is such an error for append; for attend its
 * row sees no key, which is none. */
typedef struct {
  int32_t num_layers;        /* >= 1                                             */
  int32_t num_pages;         /* >= 1; num_layers * num_pages * Hkv * page_size < 2^31 */
  int32_t page_size;         /* 16, 32, 64 or 128 tokens                         */
  int32_t num_kv_heads;      /* Hkv >= 1                                         */
  int32_t head_dim;          /* D: 64 or 128                                     */
  int32_t max_seqs;          /* sequences that the bookkeeping can hold; 0: none */
  int32_t host_only;         /* 1: bookkeeping only (no GPU needed)              */
} aa_cache_config;

typedef struct aa_cache_s* aa_cache_t;

/* k_pages, v_pages: the pool, 16-byte aligned, alive as long as the handle
 * (NULL with host_only). The handle belongs to the current device; the device
 * calls below refuse another one. Its contents need no clearing. */
aa_status aa_cache_create(const aa_cache_config* cfg, void* k_pages, void* v_pages, aa_cache_t* out);

/* A cache with 8-bit pages (see above): four caller-owned arrays, each 16-byte aligned,
 * apart from one another, alive as long as the handle (NULL with host_only). */
aa_status aa_cache_create_fp8(const aa_cache_config* cfg, void* k_pages, void* k_scales, void* v_pages, void* v_scales,
                              aa_cache_t* out);

/* Free a handle (synchronises the device). NULL is accepted. */
aa_status aa_cache_destroy(aa_cache_t cache);

/* Set the lengths of n sequences (host arrays; seqs distinct, in
 * [0, max_seqs)): lens[i] is sequence seqs[i]'s length in tokens after the
 * call. Growing takes free pages; shrinking, down to 0, gives pages back once
 * no fork shares them. Where a sequence grows into a partly filled page that
 * another one shares, the page is first copied (all layers, one launch for
 * the whole call, on `stream`): aa_cache_append after it writes only pages
 * that are the sequence's own. All or nothing: AA_ERR_NO_MEMORY if the free
 * pages do not suffice.
 * Pages given back may be handed out again at once, so the device calls
 * of one pool must be ordered with one another (one stream, or events). A
 * call that has to copy is refused while `stream` is being captured. */
aa_status aa_cache_resize(aa_cache_t cache, const int32_t* seqs, const int32_t* lens, int32_t n, aa_stream_t stream);

/* Make dst (an empty sequence) share all of src's pages and its length.
 * Nothing is copied until one of them grows into a shared page. */
aa_status aa_cache_fork(aa_cache_t cache, int32_t src, int32_t dst);

/* Move the pages in use to the front of the pool, [0, pages in use), so that
 * the rest can be handed to something else. *moved (may be NULL) receives the
 * number of pages moved; page tables taken earlier are then stale. Refused
 * while `stream` is being captured. */
aa_status aa_cache_compact(aa_cache_t cache, aa_stream_t stream, int32_t* moved);

/* Page tables and lengths of n sequences into host buffers: table
 * [n, table_width], entries past the last page -1; lens [n]. Either may be
 * NULL. AA_ERR_INVALID_ARG if a sequence has more than table_width pages. */
aa_status aa_cache_tables(aa_cache_t cache, const int32_t* seqs, int32_t n, int32_t* table_host, int32_t table_width,
                          int32_t* lens_host);

/* Pages not in use, pages that more than one sequence shares, and the most
 * pages that one sequence has. Any pointer may be NULL. */
aa_status aa_cache_stats(aa_cache_t cache, int32_t* free_pages, int32_t* shared_pages, int32_t* longest);

/* Copy page src[i] to page dst[i], all layers, keys and values (host arrays of
 * n). The pairs are checked before anything is launched and travel with the
 * launch, so they need no device memory and may be captured. Page numbers
 * must lie in the pool; no page may be the target of two pairs or both a
 * target and a source (the copies run at once), except src[i] = dst[i], which
 * is a copy of nothing. */
aa_status aa_cache_copy_pages(aa_cache_t cache, const int32_t* src, const int32_t* dst, int32_t n, aa_stream_t stream);

/* One batch of new tokens. Strides count elements from one token to the next
 * (multiples of 8, >= heads * D), so slices of a joint projection need no
 * copy. */
typedef struct {
  const int32_t* page_table; /* device [num_seqs, table_width]                    */
  const int32_t* cu_q;       /* device [num_seqs + 1]                             */
  const int32_t* kv_len;     /* device [num_seqs]                                 */
  int32_t num_seqs;          /* B >= 1                                            */
  int32_t table_width;       /* >= 1                                              */
  int32_t total_tokens;      /* T: rows of the tensors; >= cu_q[B]                */
  int32_t layer;             /* in [0, num_layers)                                */
} aa_cache_batch;

/* Write the new tokens' keys and values (k, v [T, Hkv, D]) to their pages, the
 * keys rotated by `rope` at pos (device int32 [num_axes, T]; both NULL: stored
 * as they are). With q != NULL the same launch rotates q [T, q_heads, D] into
 * q_out (contiguous; may be q if that is contiguous; not in the pool), which is
 * what aa_cache_attend takes; it needs `rope`. */
aa_status aa_cache_append(aa_cache_t cache, const aa_cache_batch* batch, const void* k, int64_t k_stride, const void* v,
                          int64_t v_stride, const aa_rope_axes* rope, const int32_t* pos, const void* q,
                          int64_t q_stride, void* q_out, int32_t q_heads, aa_stream_t stream);

/* What the pages hold of the new tokens, in bf16 (exactly; 8-bit pages decoded):
 * k, v [T, Hkv, D] contiguous, 16-byte aligned, apart from each other, the batch's
 * arrays and the pool. The keys are as stored, rotated. A token whose page number or
 * position is out of range reads as zeros. With kv_len and cu_q of the caller's
 * choice this reads any run of cached tokens that ends at kv_len. */
aa_status aa_cache_read(aa_cache_t cache, const aa_cache_batch* batch, void* k, void* v, aa_stream_t stream);

/* Attention of the new tokens over their sequences' cached keys and values
 * (the new ones included: append first). For new token i of sequence b, at
 * position p, and every query head h, over the visible keys
 *   j in [max(key_lo, 0), p], and j = 0 if anchor != 0 and p >= 0
 * (the mask of [ARCH §3.4 Anchor]: key_lo is the first token of the query's
 * document; or p - W + 1 for a sliding window):
 *   O_i = sum_j softmax_j(scale * q_i . k_j) v_j,  LSE_i = ln sum_j exp(...).
 * A row that sees no key, or whose logits are all -inf, gives O = 0 and LSE = -inf.
 * With 8-bit pages the result is that of the values that they stand for, and a key may
 * take 2^-32 of the row's largest weight times value out of it.
 * Sums are fp32: dot products that pass its range are infinite, and so may a result be whose
 * |v| times the keys that the row sees passes 2^119. With 16-bit pages logits are below 2^30.
 * Keys that no new token of their sequence sees do not reach the result, whatever
 * they hold (NaN, infinities); what a row sees makes it NaN as the formula does, and a value that
 * is not finite may reach the other rows of its sequence in the call too.
 *  - q [T, q_heads, D] bf16, ROTATED (q_stride elements from token to token);
 *    q_heads % Hkv == 0, at most 64 query heads per kv head.
 *  - max_q: the most new tokens of a sequence. It chooses the kernel, for all
 *    sequences of the call; a sequence with more is still computed, only slower.
 *    One chunk among many single tokens takes these along: two calls are faster
 *    where the contexts are long, most of all over 8-bit pages, where above 256
 *    rows every sequence's keys are first copied to 16 bits.
 *  - key_lo: device int32 [T] or NULL (0 for every row).
 *  - softmax_scale <= 0 selects 1/sqrt(D).
 *  - o [T, q_heads, D] bf16; lse [q_heads, T] fp32 or NULL. They and the workspace's
 *    bytes that the call uses overlap neither one another, nor an input or the pool.
 *  - workspace: aa_cache_attend_workspace_bytes() bytes, 256-byte aligned,
 *    contents ignored; calls that may overlap need one each.
 *  - num_seqs * Hkv < 2^27; q_heads * total_tokens < 2^31. */
aa_status aa_cache_attend(aa_cache_t cache, const aa_cache_batch* batch, const void* q, int64_t q_stride, int32_t q_heads,
                          int32_t max_q, const int32_t* key_lo, int32_t anchor, float softmax_scale, void* o, float* lse,
                          void* workspace, size_t workspace_bytes, aa_stream_t stream);

/* Drafted trees. The new tokens of a sequence are a tree of drafted continuations: all
 * lie behind its `base` = kv_len[b] - n_b cached tokens, token i in row base + i
 * of the pages, but each follows its parent only. aa_cache_attend_tree is
 * aa_cache_attend with other visible keys: new token i of sequence b sees the cached
 * j in [max(key_lo, 0), base), j = 0 if anchor != 0 and base > 0, and new token c of
 * its sequence if bit c % 64 of word c / 64 of its row of `tree` is set (device
 * uint64 [T, tree_words], 1 <= tree_words <= 2^14; bits at n_b and above are not looked at, tokens at 64 *
 * tree_words and above are not seen, by themselves neither). Any mask will do, also one where tokens see later ones.
 * Where base < 0 the tokens without a position see nothing. The workspace is
 * aa_cache_attend's. */
aa_status aa_cache_attend_tree(aa_cache_t cache, const aa_cache_batch* batch, const void* q, int64_t q_stride,
                               int32_t q_heads, int32_t max_q, const int32_t* key_lo, int32_t anchor, const uint64_t* tree,
                               int32_t tree_words, float softmax_scale, void* o, float* lse, void* workspace,
                               size_t workspace_bytes, aa_stream_t stream);

/* Masks and positions of drafted trees: parents (device int32 [T]) gives each new
 * token's parent as its index among its sequence's new tokens, smaller than its own,
 * or -1 for one that follows the cached tokens. mask (uint64 [T, tree_words]): the
 * token's ancestors and itself, as far as they lie below 64 * tree_words (which has to
 * cover the longest sequence's new tokens; no error word is set); pos (int32 [T]): kv_len - n_b + the
 * number of its ancestors, the position that it is rotated at. A parent out of range counts as -1
 * and sets the error word. Rows outside [cu_q[0], cu_q[num_seqs]) are left as they were. */
aa_status aa_cache_tree_masks(aa_cache_t cache, const int32_t* parents, const int32_t* cu_q, const int32_t* kv_len,
                              int32_t num_seqs, int32_t total_tokens, int32_t tree_words, uint64_t* mask, int32_t* pos,
                              aa_stream_t stream);

/* Keep the accepted tokens of drafted trees: path (device int32 [num_seqs, path_width])
 * lists the indices of the kept new tokens of each sequence, ascending, up to the
 * first negative entry. Their keys and values move up, path[i] to row base + i, in all
 * layers; what lies behind them is no longer of use: the sequence's length is now
 * base + the number kept (aa_cache_resize, or a caller's own kv_len). A path that does
 * not ascend or leaves its sequence's new tokens sets the error word, and nothing of
 * that sequence moves. batch->layer and total_tokens are not used. The pages written
 * to are the sequences' own (aa_cache_resize has seen to it). */
aa_status aa_cache_accept(aa_cache_t cache, const aa_cache_batch* batch, const int32_t* path, int32_t path_width,
                          aa_stream_t stream);

/* Bytes of device scratch aa_cache_attend needs for a batch of these sizes
 * (partial results of keys that are split among CTAs). Chunks: 20 MB at D = 64, 40 at
 * 128, and 32 bytes per sequence and per 256 rows of a kv head more (over 8-bit pages
 * with up to 256 rows of a sequence: per 128). Few new tokens over long contexts: the
 * results of up to 76 splits, 4 * D + 8 bytes per row and split. 256 bytes where nothing
 * is split. Chunks over 8-bit pages whose sequences have more than 256 rows (max_q times
 * the query heads of a kv head): 16-bit copies of a few sequences' keys and values more,
 * 4 * D * Hkv bytes per position of their tables, up to 1 GiB; a smaller max_q asks for
 * less, at the price of time. A smaller batch may need more. 0 for invalid sizes. */
size_t aa_cache_attend_workspace_bytes(aa_cache_t cache, int32_t num_seqs, int32_t total_tokens, int32_t max_q,
                                       int32_t table_width, int32_t q_heads);

/* Synchronise `stream`, read and clear the cache's device error word:
 * AA_ERR_INVALID_ARG if a device call met a page number or a position outside
 * its range, a parent or a path of drafted tokens that is none, since the last check, AA_ERR_TIMEOUT if a bounded device wait ran
 * out, AA_OK otherwise. */
aa_status aa_cache_check_error(aa_cache_t cache, aa_stream_t stream);

const char* aa_status_string(aa_status status);
const char* aa_last_error(void);

#ifdef __cplusplus
}
#endif
#endif /* ANCHORATTN_H */
