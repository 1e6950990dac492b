/*
 * gdn.h - C ABI of the MI355X (gfx950) Gated DeltaNet engine (libgdn.so).
 *
 * The library implements the data-parallel hot path of a Gated DeltaNet (GDN)
 * layer on one GPU: chunked prefill with explicit initial/final state, the
 * per-token recurrent step with compact state-update capture, replay of the
 * captured updates, and immutable state snapshots.
 *
 * The method (the gated delta rule; value head h reads key/query head
 * h / (Hv/Hq), "inverse-GQA" key sharing):
 *
 *     alpha_t = exp(g_t)
 *     delta_t = beta_t * (v_t - (alpha_t S_{t-1})^T k_t)
 *     S_t     = alpha_t S_{t-1} + k_t delta_t^T          (S is [dk x dv], fp32)
 *     o_t     = scale * S_t^T q_t
 *
 * Sources: [onnxruntime PR 32767, "[WebGPU EP] adds state update capacity
 * support for GatedDeltaNet", sections "Changes", "Test Coverage", "DFlash2
 * Prerequisite"] for capture, the active flag, replay S = decay*S +
 * outer(key, delta) and shared-key heads; [executorch issue 23097, "Enable the
 * native Kev example on NVIDIA GPUs ...", "Work to cover"] for the chunked
 * prefill with explicit initial/final state and FP32 recurrence under 16-bit
 * weights; [executorch issue 23099, "Enable the native Kev example on the
 * WebGPU backend", "Work to cover"] for the prefix snapshot that repeated
 * evaluations must leave unchanged.
 *
 * Conventions common to every entry point
 * ---------------------------------------
 *  - All pointers are DEVICE pointers (hipMalloc'd or torch-allocated on the
 *    current device) unless stated otherwise; the caller owns every buffer.
 *    The library allocates nothing and keeps no pointer after returning.
 *  - Every call is asynchronous on `stream` (a hipStream_t; NULL = the null
 *    stream).  Buffers must stay alive until the queued work has finished.
 *  - Arguments are validated on the host before anything is enqueued.  A status
 *    other than GDN_OK means nothing was enqueued; gdn_last_error() returns a
 *    thread-local message.  Nothing aborts.
 *  - Layouts are contiguous row-major (last index fastest):
 *        q, k        [T_total, Hq, dk]   dtype = shape.dtype
 *        v, o        [T_total, Hv, dv]   dtype = shape.dtype
 *        g, beta     [T_total, Hv]       fp32 (g = log of the decay alpha)
 *        states      [N, Hv, dk, dv]     fp32 (dv fastest)
 *    T_total = B*T for dense input (B rows of T tokens) or T for packed ragged
 *    input given by cu_seqlens (int32 [N+1], device, 0 = cu[0] <= ... <=
 *    cu[N] = T; empty sequences allowed).  cu_seqlens is not read on the host;
 *    kernels clamp every range to [0, T] and cap the chunk count at the
 *    workspace size, so malformed values give unspecified results, never an
 *    out-of-bounds access.
 *  - Supported sizes: dk, dv in {16, 32, 64, 128}; Hv % Hq == 0; pointers
 *    16-byte aligned; fp32 data for fp32 inputs is computed in fp32, fp16/bf16
 *    inputs use 16-bit matrix-core products with fp32 accumulation and an fp32
 *    state, and o is rounded to the input dtype (round to nearest even).
 */
#ifndef GDN_H
#define GDN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { GDN_F32 = 0, GDN_F16 = 1, GDN_BF16 = 2 } gdn_dtype;

typedef enum {
  GDN_OK = 0,
  GDN_ERR_INVALID_ARG = 1, /* bad pointer, size, alignment, aliasing */
  GDN_ERR_UNSUPPORTED = 2, /* valid but outside the compiled set (dk, dv, chunk) */
  GDN_ERR_HIP = 3          /* a HIP launch or runtime call failed */
} gdn_status;

/* Problem description shared by prefill and recurrent step. */
typedef struct {
  int32_t B;     /* dense: rows; ragged: number of sequences N (cu_seqlens has B+1 entries) */
  int32_t T;     /* dense: tokens per row; ragged: total packed tokens */
  int32_t Hq;    /* query/key heads */
  int32_t Hv;    /* value heads, a multiple of Hq */
  int32_t dk;    /* key/query head dim */
  int32_t dv;    /* value head dim */
  float scale;   /* o = scale * S^T q (usually dk^-1/2) */
  int32_t dtype; /* gdn_dtype of q, k, v, o */
} gdn_shape;

/*
 * Optional input prologue, applied inside the kernels of the *_ex entry points
 * [executorch issue 23097, "Work to cover": reusing a GDN prefill means adapting
 * its gate and scaling conventions].  The pages give no formulas; these are the
 * common ones, each switched on separately.  A zeroed struct (or NULL) is the
 * identity: q, k, g and beta are used as given.
 *
 *  qk_l2norm      nonzero: every q_t and k_t (per key head) is replaced by
 *                 x * (sum_i x_i^2 + qk_l2norm_eps)^(-1/2), computed in fp32
 *                 from the input-dtype values.  eps = 0 is allowed; an all-zero
 *                 row then gives non-finite results.
 *  qk_l2norm_eps  finite, >= 0 (read only when qk_l2norm is set).
 *  beta_is_logit  nonzero: beta = 1 / (1 + exp(-b)) of the `beta` input.
 *  gate_A_log     NULL: `g` holds the log decay.  Otherwise fp32 [Hv] on the
 *                 device, and the log decay of value head h is
 *                 -exp(gate_A_log[h]) * softplus(g + gate_dt_bias[h]),
 *                 softplus(x) = log(1 + exp(x)).
 *  gate_dt_bias   fp32 [Hv] on the device, or NULL (zeros); only with gate_A_log.
 * Captured records hold the prologue's results: decay = exp of the gated log
 * decay, key = the normalised fp32 key, delta with the sigmoid beta.
 */
typedef struct {
  int32_t qk_l2norm;
  float qk_l2norm_eps;
  int32_t beta_is_logit;
  const float* gate_A_log;
  const float* gate_dt_bias;
} gdn_prologue;

/* Version of this ABI (bumped on any signature change). */
int32_t gdn_abi_version(void);

/* Bytes of device workspace gdn_prefill_chunked needs for `shape`,
 * `chunk_size` and the input form (`ragged` nonzero when cu_seqlens will be
 * passed, so shape->T is the packed total); 0 if the arguments are invalid.
 * Host only, no HIP call. */
size_t gdn_prefill_workspace_bytes(const gdn_shape* shape, int32_t chunk_size, int32_t ragged);

/*
 * Chunked prefill [executorch issue 23097, "Work to cover": chunked GDN prefill
 * with explicit initial/final state and FP32 recurrence].
 *
 * Computes o for every token and (optionally) the state after each sequence's
 * last token, processing each sequence in chunks of `chunk_size` tokens
 * (16, 32 or 64; chunks restart at each sequence start, the last one may be
 * partial).  The result equals the token-by-token recurrence up to rounding.
 *
 * Precondition on g: every g <= 0 (decay alpha = exp(g) <= 1), the usual case
 * of a forgetting gate.  The chunked form then only forms decay ratios
 * exp(G_i - G_j) with j <= i, exp(G_i) and exp(G_last - G_j) (G = in-chunk
 * cumulative sum of g), all <= 1, which keeps its 16-bit matrix operands in
 * range.  With some g > 0 those factors exceed 1 and can overflow 16-bit
 * operands, so o and final_state are unspecified (the call still completes
 * and accesses only the buffers given).  The precondition is not checked (g is
 * not read on the host); gdn_recurrent_step accepts any finite g.
 *
 *  initial_state   [N, Hv, dk, dv] fp32 or NULL (zeros).  Sequence s reads
 *                  initial_state + s * initial_state_batch_stride (elements);
 *                  stride 0 broadcasts one state to all sequences (snapshot
 *                  reuse).  Never written unless it is also `final_state`.
 *  final_state     [N, Hv, dk, dv] fp32 or NULL (not written).  May equal
 *                  initial_state only with stride Hv*dk*dv (in-place update).
 *  workspace       device scratch of gdn_prefill_workspace_bytes() bytes,
 *                  16-byte aligned; contents on entry are ignored.
 */
gdn_status gdn_prefill_chunked(const gdn_shape* shape, const void* q, const void* k,
                               const void* v, const float* g, const float* beta,
                               const float* initial_state, int64_t initial_state_batch_stride,
                               const int32_t* cu_seqlens, int32_t chunk_size, void* o,
                               float* final_state, void* workspace, size_t workspace_bytes,
                               void* stream);

/*
 * Chunked prefill that also emits the state at every chunk boundary
 * [executorch issue 23097, "Work to cover": GDN chunk boundaries, prefix
 * snapshots retained in device memory and reused; executorch issue 23099,
 * "Work to cover": the reused prefix stays unchanged].  A boundary state is a
 * ready-made snapshot of the prefix that ends there: passing it as
 * `initial_state` of a later call continues the sequence from that point.
 *
 * Same arguments, results and errors as gdn_prefill_chunked, plus
 *  chunk_states           [num_chunks, Hv, dk, dv] fp32, device, 16-byte
 *                         aligned, not NULL.  Sequence s has
 *                         n_s = ceil(L_s / chunk_size) chunks (0 when empty);
 *                         its chunk j has index sum_{s' < s} n_s' + j (dense
 *                         input: s * ceil(T / chunk_size) + j) and receives the
 *                         state after the first min((j+1)*chunk_size, L_s)
 *                         tokens of s, so each sequence's last entry equals its
 *                         final state.  Must not overlap any other buffer.
 *  chunk_states_capacity  entries available (>= 0); chunks with an index at
 *                         or beyond it are not written (size it to
 *                         sum_s n_s to receive them all).
 * Costs one extra fp32 state write per (chunk, value head).
 */
gdn_status gdn_prefill_chunked_states(const gdn_shape* shape, const void* q, const void* k,
                                      const void* v, const float* g, const float* beta,
                                      const float* initial_state, int64_t initial_state_batch_stride,
                                      const int32_t* cu_seqlens, int32_t chunk_size, void* o,
                                      float* final_state, float* chunk_states,
                                      int64_t chunk_states_capacity, void* workspace,
                                      size_t workspace_bytes, void* stream);

/*
 * gdn_prefill_chunked / gdn_prefill_chunked_states with the input prologue:
 * `prologue` may be NULL (identity) and `chunk_states` may be NULL (no
 * boundary states; chunk_states_capacity is then ignored).  Same layouts,
 * results and errors otherwise.
 */
gdn_status gdn_prefill_chunked_ex(const gdn_shape* shape, const gdn_prologue* prologue, const void* q,
                                  const void* k, const void* v, const float* g, const float* beta,
                                  const float* initial_state, int64_t initial_state_batch_stride,
                                  const int32_t* cu_seqlens, int32_t chunk_size, void* o,
                                  float* final_state, float* chunk_states, int64_t chunk_states_capacity,
                                  void* workspace, size_t workspace_bytes, void* stream);

/*
 * gdn_prefill_chunked without a workspace argument, for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc).  The entry point itself allocates nothing:
 * its workspace is a fixed device array of GDN_NOALLOC_SCRATCH_BYTES inside the
 * library, one per GPU, held from the first call on that GPU until the process
 * ends.  The caller still passes every input and output.
 *
 * Same arguments (minus workspace), layouts, results and errors as
 * gdn_prefill_chunked, plus GDN_ERR_UNSUPPORTED when the problem needs more
 * workspace than the array holds (gdn_prefill_workspace_bytes() >
 * GDN_NOALLOC_SCRATCH_BYTES; at 16-bit inputs and chunk 64 that is about
 * 10,000 (chunk, value head) pairs, e.g. 20,000 tokens at 32 value heads).
 * The array keeps the last call's contents; every call writes each part of
 * it that it reads, so nothing needs clearing.  All calls on one GPU share
 * the array: calls that overlap in time on one GPU (other streams, other host
 * threads) race and give unspecified results, so order them on one stream.
 * The first call on a device looks up the array's address (no allocation).
 */
#define GDN_NOALLOC_SCRATCH_BYTES (128u * 1024u * 1024u)
gdn_status gdn_prefill_chunked_noalloc(const gdn_shape* shape, const void* q, const void* k,
                                       const void* v, const float* g, const float* beta,
                                       const float* initial_state, int64_t initial_state_batch_stride,
                                       const int32_t* cu_seqlens, int32_t chunk_size, void* o,
                                       float* final_state, void* stream);

/*
 * Recurrent step with compact state-update capture [onnxruntime PR 32767,
 * "Changes": state_update_capacity, the required [batch] capture_count input,
 * the packed float32 state_update output, clamped per-row prefix capture,
 * state_update_active = 0 clears the whole output].
 *
 * Runs the recurrence token by token over each row (dense rows of T tokens or
 * ragged rows through cu_seqlens), writing o and (optionally) final_state; the
 * argument rules for initial_state / final_state are those of prefill.
 *
 * Capture (state_update_capacity > 0):
 *  capture_count   int32 [B] device, required.  Row b captures its first
 *                  n_b = min(max(capture_count[b], 0), capacity, L_b) tokens.
 *  state_update    fp32 [B, capacity, R], R = Hv + Hq*dk + Hv*dv, required.
 *                  Record c of row b (token c of the row) is
 *                  [decay: alpha per value head (Hv) | key: fp32 k per key head
 *                  (Hq*dk) | delta: delta per value head (Hv*dv)], so that
 *                  replaying it applies S = decay*S + outer(key, delta).
 *  state_update_active
 *                  nonzero: records c < n_b are written, all other entries are
 *                  left untouched (their content is unspecified);
 *                  0: the whole state_update buffer is zero-filled and no
 *                  record is written (o and final_state are still computed).
 * capacity == 0 disables capture (capture_count, state_update may be NULL);
 * capacity < 0 is GDN_ERR_INVALID_ARG.
 */
gdn_status gdn_recurrent_step(const gdn_shape* shape, const void* q, const void* k,
                              const void* v, const float* g, const float* beta,
                              const float* initial_state, int64_t initial_state_batch_stride,
                              const int32_t* cu_seqlens, void* o, float* final_state,
                              int32_t state_update_capacity, const int32_t* capture_count,
                              int32_t state_update_active, float* state_update, void* stream);

/* gdn_recurrent_step with the input prologue (`prologue` may be NULL). */
gdn_status gdn_recurrent_step_ex(const gdn_shape* shape, const gdn_prologue* prologue, const void* q,
                                 const void* k, const void* v, const float* g, const float* beta,
                                 const float* initial_state, int64_t initial_state_batch_stride,
                                 const int32_t* cu_seqlens, void* o, float* final_state,
                                 int32_t state_update_capacity, const int32_t* capture_count,
                                 int32_t state_update_active, float* state_update, void* stream);

/*
 * Replay of captured state updates [onnxruntime PR 32767, "Changes" and
 * "DFlash2 Prerequisite": compact-state replay after partial acceptance].
 *
 * For each row b and each record c < m_b = min(max(replay_count[b], 0),
 * capacity), in order: S[b,h] = decay_c[h] * S[b,h] + outer(key_c[h/(Hv/Hq)],
 * delta_c[h]).  `state` [B, Hv, dk, dv] fp32 is updated in place (normally the
 * pre-step state); `state_update` is the buffer gdn_recurrent_step filled with
 * the same B, Hq, Hv, dk, dv, capacity and is only read.  The caller keeps
 * m_b <= n_b of the capture (records beyond n_b are unspecified).
 */
gdn_status gdn_replay_state_updates(int32_t B, int32_t Hq, int32_t Hv, int32_t dk, int32_t dv,
                                    int32_t state_update_capacity, const float* state_update,
                                    const int32_t* replay_count, float* state, void* stream);

/*
 * Immutable state snapshot [executorch issue 23099 / 23097, "Work to cover":
 * a prefix snapshot reused across question batches; repeated evaluations must
 * leave the prefix unchanged].
 *
 * Copies num_states * Hv * dk * dv fp32 values from src to dst (bitwise),
 * ordered on `stream`.  src and dst must not overlap.  No entry point ever
 * writes a buffer that is passed to it only as initial_state, so a snapshot
 * used as initial_state stays bit-identical across any number of calls.
 */
gdn_status gdn_state_snapshot(const float* src, float* dst, int64_t num_states, int32_t Hv,
                              int32_t dk, int32_t dv, void* stream);

/*
 * ---------------------------------------------------------------------------
 * Linear attention with a decay for each head (no delta rule)
 * ---------------------------------------------------------------------------
 *
 *     alpha_t = exp(g_t)
 *     S_t     = alpha_t S_{t-1} + k_t v_t^T          (S is [dk x dv], fp32)
 *     o_t     = scale * S_t^T q_t
 *
 * with the shapes, layouts, head map, state and cu_seqlens rules of the gated
 * delta rule above (up to 2^30 tokens); there is no beta.  `g` holds log decays in fp32:
 * g_token_stride = Hv for one value per token and value head ([T_total, Hv]),
 * or 0 for one value per value head ([Hv], the same at every token).
 *
 * Precision: o is rounded once to the input dtype; for 16-bit inputs the
 * products with the state and with the in-chunk scores use those in two parts of
 * the input type (2^-16 of a term for bf16, 2^-22 for fp16), and the final state is
 * summed from terms of fp32 accuracy (fp16: of 2^-22, but no finer than 2^-38 of the
 * largest decayed v of the same column in the same chunk).
 *
 * Infinities and NaN touch later tokens only: one in v makes its column of o NaN or
 * infinite from its token on and that column of the state, one in k the outputs
 * from its token on and its row of the state, one in q its token's outputs.
 *
 * Precondition of the prefill: g <= 0 (g = -infinity forgets everything before
 * the token).  The step takes g of any sign.
 */

/* Bytes of device workspace gdn_linear_prefill needs for `shape` and the input
 * form (`ragged` nonzero when cu_seqlens will be passed); 0 is a valid answer
 * (no workspace needed), (size_t)-1 if the arguments are invalid.  Host only. */
size_t gdn_linear_workspace_bytes(const gdn_shape* shape, int32_t ragged);

/*
 * Prefill over whole sequences, in chunks.  initial_state,
 * initial_state_batch_stride, cu_seqlens, o and final_state as in
 * gdn_prefill_chunked.  Few, long sequences are split into segments whose
 * states are computed side by side in `workspace` (16-byte aligned, contents on
 * entry ignored; may be NULL when gdn_linear_workspace_bytes() is 0).
 */
gdn_status gdn_linear_prefill(const gdn_shape* shape, const void* q, const void* k, const void* v,
                              const float* g, int64_t g_token_stride, const float* initial_state,
                              int64_t initial_state_batch_stride, const int32_t* cu_seqlens, void* o,
                              float* final_state, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Token by token over each row, with the arguments of gdn_recurrent_step.
 * Capture (state_update_capacity > 0): row b writes its first
 * min(max(capture_count[b], 0), capacity, L_b) records
 * [alpha (Hv) | k (Hq*dk) | v (Hv*dv)] in fp32 into state_update [B, capacity, R];
 * other entries are left untouched.  gdn_replay_state_updates applies them
 * (S = alpha*S + outer(k, v)), bit-identical to this step.
 */
gdn_status gdn_linear_step(const gdn_shape* shape, const void* q, const void* k, const void* v,
                           const float* g, int64_t g_token_stride, const float* initial_state,
                           int64_t initial_state_batch_stride, const int32_t* cu_seqlens, void* o,
                           float* final_state, int32_t state_update_capacity, const int32_t* capture_count,
                           float* state_update, void* stream);

/*
 * Verification of drafted tokens against the target's probabilities, from
 * given uniform random numbers (speculative sampling).  For row b with
 * n_b = min(draft_count[b], K) drafts (K without draft_count; < 0: idle row):
 *
 *   draft i = 0, 1, ... is accepted while  u[b,i] * q_i[x_i] < p_i[x_i],
 *   p_i = target_probs[b,i,:], q_i = draft_probs[b,i,:], x_i = draft_tokens[b,i];
 *   a = number of accepted drafts (the first refusal ends the row).
 *   One more token is drawn with weights w over the vocabulary:
 *     a < n_b:  w = max(p_a - q_a, 0); if all of these are 0, w = p_a
 *     a == n_b: w = p_a
 *   as the lowest index v with  sum_{j <= v} w_j > u[b,K] * sum_j w_j
 *   (the last v with w_v > 0 if rounding leaves none).
 *
 * Products, differences and sums are taken in 64 bits; the sums' order, which goes
 * by the sizes, moves them by at most about 2^-47 of the total, and a draw nearer
 * than that to the border between two tokens may give either.  draft_probs NULL: the drafts are
 * deterministic (q_i is 1 at x_i and 0 elsewhere).  A draft token outside
 * [0, V) is refused, with q_a = 0 everywhere if draft_probs is NULL.  Weights
 * that are NaN, infinite or not positive count as 0; a row whose weights are all 0 draws
 * the token -1.  An idle row (draft_count[b] < 0) emits nothing: emit_count[b] = 0,
 * its tokens -1.
 *
 *  target_probs  [B, K+1, V] dtype, row r = b*(K+1)+i at target_row_stride * r
 *  draft_probs   [B, K, V] dtype or NULL, row r = b*K+i at draft_row_stride * r
 *  draft_tokens  int32 [B, K]      uniforms  fp32 [B, K+1], in [0, 1)
 *  draft_count   int32 [B] or NULL
 *  tokens        int32 [B, K+1]: the accepted drafts, the drawn token, then -1
 *  emit_count    int32 [B]: a + 1, the number of tokens emitted.  Where a row
 *                is the last emitted token followed by the drafts, this is also
 *                the number of its tokens whose state updates are to be kept,
 *                i.e. the replay_count of gdn_replay_state_updates.
 *  workspace     gdn_verify_workspace_bytes() bytes, 16-byte aligned, contents
 *                on entry ignored; may be NULL where that is 0.
 * K >= 0 (K = 0 is plain sampling), V >= 1; the probabilities need only the
 * alignment of their type.
 */
typedef struct {
  int32_t B;                 /* rows */
  int32_t K;                 /* drafted tokens per row (capacity) */
  int32_t V;                 /* vocabulary */
  int32_t dtype;             /* gdn_dtype of target_probs and draft_probs */
  int64_t target_row_stride; /* elements between probability rows, >= V */
  int64_t draft_row_stride;
} gdn_verify_shape;

size_t gdn_verify_workspace_bytes(const gdn_verify_shape* shape);   /* (size_t)-1 if invalid */

gdn_status gdn_verify_drafts(const gdn_verify_shape* shape, const void* target_probs, const void* draft_probs,
                             const int32_t* draft_tokens, const float* uniforms, const int32_t* draft_count,
                             int32_t* tokens, int32_t* emit_count, void* workspace, size_t workspace_bytes,
                             void* stream);

/*
 * The norms after and before a block, fused with its gate, residual and scale.
 * For each token (row of D values made of D/group groups):
 *
 *   n = y * (mean_group(y^2) + eps)^(-1/2) * post_weight     (n = y without post_weight)
 *   m = n * act(gate)                                        (m = n with GDN_ACT_NONE)
 *   h = residual + residual_scale * m                        (no residual: 0)
 *   normed = h * (mean_D(h^2) + eps)^(-1/2) * next_weight    (only with next_weight)
 *
 * everything in fp32, h and normed rounded once to `dtype` (normed is computed
 * from the unrounded h).  With group = dv, D = Hv*dv and GDN_ACT_SILU this is the
 * gated output norm of a GDN layer; with group = D it ends a block and
 * prepares the next one's input.
 *
 *  y, gate, residual, h, normed  [T, D] dtype; gate required unless
 *      GDN_ACT_NONE; residual, post_weight, next_weight may be NULL; normed is
 *      required exactly with next_weight.
 *  post_weight [group] dtype, next_weight [D] dtype.
 *  h may be residual itself or y itself (in place); no other overlap.
 * group is D, or one of 16, 32, 64, 128 dividing D; D <= 16384.  Rows need only
 * the alignment of their type.
 */
typedef enum { GDN_ACT_NONE = 0, GDN_ACT_SILU = 1, GDN_ACT_SIGMOID = 2 } gdn_act;

typedef struct {
  int64_t T;            /* tokens */
  int32_t D;            /* width */
  int32_t group;        /* group width of the norm after the block */
  int32_t dtype;        /* gdn_dtype */
  int32_t gate_act;     /* gdn_act */
  float residual_scale;
  float eps;            /* finite, >= 0 */
} gdn_norm_shape;

gdn_status gdn_block_norm(const gdn_norm_shape* shape, const void* y, const void* gate, const void* residual,
                          const void* post_weight, const void* next_weight, void* h, void* normed,
                          void* stream);

/*
 * ---------------------------------------------------------------------------
 * Attention layers between the delta-rule blocks: keys and values in pages
 * ---------------------------------------------------------------------------
 *
 * k_cache, v_cache  [num_pages, Hkv, page_size, d] dtype: the page_size rows of one
 *                   head in one page are contiguous.
 * block_table       int32 [N, max_pages]: key j of sequence s is row j % page_size of
 *                   page block_table[s, j / page_size].  A number outside
 *                   [0, num_pages) is no page: what is appended there is dropped, and
 *                   the keys there are absent (masked).
 * cache_lens        int32 [N]: keys of each sequence, its new tokens included.  New
 *                   token i of the L_s of sequence s has the place
 *                   cache_lens[s] - L_s + i.
 * cu_seqlens        int32 [N+1] as above (packed rows; those behind cu_seqlens[N] are
 *                   neither read nor written), or NULL: T tokens for each of N rows.
 * Offsets that decrease or overlap leave the outputs of these rows unspecified; nothing
 * out of range is read or written.
 * d in {32, 64, 128, 256}; page_size a multiple of 16 up to 1024; max_pages * page_size
 * up to 2^26; N up to 2^20; Hq/Hkv up to 256; all pointers 16-byte aligned, token strides multiples of 16 bytes
 * (cu_seqlens, cache_lens, block_table, positions, pair_axis, inv_freq: 4-byte).
 */
typedef struct {
  int32_t N;            /* sequences */
  int32_t T;            /* tokens per sequence, or with cu_seqlens the number of packed rows */
  int32_t Hq, Hkv;      /* query heads, a multiple of the key/value heads */
  int32_t d;            /* head dim of queries, keys and values */
  int32_t dtype;        /* gdn_dtype of all of them */
  int32_t page_size;
  int32_t num_pages;
  int32_t max_pages;    /* columns of block_table */
} gdn_cache_shape;

/*
 * Appends new keys and values to their pages, the keys (and the queries, into
 * q_out) rotated by their positions on the way:
 *
 *   a_j = position * inv_freq[j],  j = 0 .. rotary/2 - 1
 *   (x1, x2) -> (x1 cos a_j - x2 sin a_j, x1 sin a_j + x2 cos a_j)
 *   x1, x2 = elements j, j + rotary/2, or with `interleaved` 2j, 2j + 1;
 *   the elements from `rotary` on stay as they are.
 *
 * The angle is reduced in 64 bits, its sine and cosine and the rotation are taken
 * in 32, rounded once.
 *
 *  k, v       [tokens, Hkv, d] at their token strides (elements), as slices of one
 *             projection's rows have them; q [tokens, Hq, d] or NULL.
 *  q_out      [tokens, Hq, d] contiguous, required exactly with q; may be q itself
 *             where q is contiguous.
 *  inv_freq   fp32 [rotary/2], or NULL (rotary = 0): keys are appended as they are.
 *  positions  int32 [axes, tokens], or NULL: the token's place in the cache.
 *  pair_axis  int32 [rotary/2]: the axis (time, height, width, ...) whose position
 *             turns pair j, clamped to [0, axes); NULL: axis 0.
 * rotary is even, 0 <= rotary <= d.  Tokens whose place is outside of the table or
 * on no page are not appended (their q_out is written).  Two tokens on one place:
 * unspecified which stays.
 */
typedef struct {
  int64_t q_token_stride, k_token_stride, v_token_stride;
  int32_t rotary;
  int32_t interleaved;
  int32_t axes;         /* rows of positions, 1 .. 8 */
} gdn_append_shape;

gdn_status gdn_cache_append(const gdn_cache_shape* shape, const gdn_append_shape* append, const void* q,
                            const void* k, const void* v, const float* inv_freq, const int32_t* positions,
                            const int32_t* pair_axis, const int32_t* block_table, const int32_t* cache_lens,
                            const int32_t* cu_seqlens, void* q_out, void* k_cache, void* v_cache, void* stream);

/*
 * Attention of the new tokens over the cache, causal:
 *
 *   o_i = sum_j w_ij v_j / sum_j w_ij,  w_ij = exp(scale * q_i . k_j)
 *   over the keys j of the sequence with  p_i - window < j <= p_i  (window > 0) or
 *   j <= p_i (window = 0), p_i the token's place; query head h reads key head
 *   h / (Hq/Hkv).
 *
 * A token that sees no key, and one whose weights are all 0, gets 0.  What lies in
 * masked places (infinities, NaN, pages never written) touches nothing.
 *
 * Precision: scores, the running maximum and all sums in fp32, o rounded once; for
 * 16-bit inputs the weights are rounded to the input type (against a running
 * maximum, at most 2^8) as operands of their product with v, and summed as rounded,
 * two at a time in steps that were seen to be off by at most 1.4 units of fp32's last
 * place (or 2^-37; the largest weight is at least 1).
 * fp16 keeps weights down to 2^-31 of the row's largest, each off by 2^-32 of that at
 * most where it is below 2^-21 of it.  Scores times log2(e) beyond 2^24, where fp32 has
 * no fractions for them, may give NaN.
 *
 *  q, o       [tokens, Hq, d]; q at q_token_stride (elements), o contiguous.
 *  scale      > 0; scale * log2(e) finite.
 *  workspace  gdn_cache_attention_workspace_bytes() bytes, 16-byte aligned, contents
 *             on entry ignored; may be NULL where that is 0.  Long sequences are split
 *             over their keys; the parts are joined in a fixed order.
 */
size_t gdn_cache_attention_workspace_bytes(const gdn_cache_shape* shape, int32_t ragged);   /* (size_t)-1 if invalid */

gdn_status gdn_cache_attention(const gdn_cache_shape* shape, const void* q, int64_t q_token_stride,
                               const void* k_cache, const void* v_cache, const int32_t* block_table,
                               const int32_t* cache_lens, const int32_t* cu_seqlens, float scale, int32_t window,
                               void* o, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Beam search: the K best continuations of W beams for each of B searches.
 *
 *   c(w, v) = scores[b,w] + logits[b,w,v] - log sum_u exp(logits[b,w,u])
 *
 * of an unfinished beam w and every token v; a finished beam has one continuation,
 * pad_token, with its score unchanged.  The K largest in descending order, ties to
 * the lowest w, then the lowest v.
 *
 * exp in fp32 (2^-22 of a term near the maximum), sums, logarithm and scores in 64 bits; new_scores
 * rounded once to fp32.  Two continuations of different beams nearer than about
 * 2^-24 may change places.  Logits of -infinity are no continuations.  A beam counts
 * as absent if its score is not finite, or (unfinished) a logit is NaN or +infinity,
 * or all are -infinity.  Places that are left have token -1, parent -1, score
 * -infinity and count as finished.
 *
 *  logits        [B, W, V] dtype, row r = b*W+w at row_stride * r (the alignment of
 *                their type is enough)
 *  scores        fp32 [B, W]            finished  uint8 [B, W] or NULL (none)
 *  tokens, parents  int32 [B, K]        new_scores  fp32 [B, K]
 *  new_finished  uint8 [B, K]: finished[parent], or token == eos_token (-1: none)
 *  workspace     gdn_beam_workspace_bytes() bytes, 16-byte aligned, contents on entry
 *                ignored
 * 1 <= W <= 64, 1 <= K <= 64, V <= 2^24; new_scores and new_finished must not be
 * scores and finished.
 */
typedef struct {
  int32_t B, W, K, V;
  int32_t dtype;
  int32_t eos_token, pad_token;   /* pad_token in [0, V) */
  int64_t row_stride;             /* >= V */
} gdn_beam_shape;

size_t gdn_beam_workspace_bytes(const gdn_beam_shape* shape);   /* (size_t)-1 if invalid */

gdn_status gdn_beam_select(const gdn_beam_shape* shape, const void* logits, const float* scores,
                           const uint8_t* finished, int32_t* tokens, int32_t* parents, float* new_scores,
                           uint8_t* new_finished, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Moves rows (states, convolution windows, pages) after a beam selection:
 *
 *   dst[l, d] = src[l, s]  for every layer l and every entry (g, j) of G groups of W
 *   s = src_index[g, j] (+ g * src_group),  d = dst_index[g, j], or g * W + j without
 *
 * Bitwise.  Within a group all reads come before all writes, so dst may be src: the
 * rows of one group may be permuted, repeated and dropped in place.  A row that one
 * group writes must not be read or written by another, and no row is written twice.
 * Entries whose index is outside of [0, src_group) (src_group > 0), or whose row is
 * outside of [0, src_rows) or [0, dst_rows), write nothing.
 *
 *  src, dst     layers at their strides in bytes (multiples of 16, also negative), rows of
 *               row_bytes (a multiple of 16); 16-byte aligned.  dst is src (with equal
 *               strides) or apart from it.
 *  src_index, dst_index  int32 [G, W], W <= 64
 */
typedef struct {
  int64_t layers, src_layer_stride, dst_layer_stride;
  int64_t src_rows, dst_rows, row_bytes;
  int64_t src_group;    /* rows from one group's index 0 to the next's; 0: indexes count from the first row */
  int32_t G, W;
} gdn_reorder_shape;

gdn_status gdn_state_reorder(const gdn_reorder_shape* shape, const void* src, void* dst, const int32_t* src_index,
                             const int32_t* dst_index, void* stream);

/*
 * Measurement support (not part of the method).  gdn_profile_enable(1) makes
 * every entry point bracket each kernel it launches with a pair of hipEvents
 * recorded on the launch stream; gdn_profile_collect() waits for all pending
 * events, reports per kernel the number of launches and their summed duration
 * in milliseconds (up to max_kernels entries; names are static strings), and
 * clears the record.  Returns the number of distinct kernels seen.  Disabled by
 * default; costs nothing measurable when disabled.
 */
gdn_status gdn_profile_enable(int32_t on);
int32_t gdn_profile_collect(const char** names, double* total_ms, int32_t* launches, int32_t max_kernels);

/* Static description of a status code. */
const char* gdn_status_string(gdn_status status);

/* Thread-local detail about the last non-OK status returned on this thread. */
const char* gdn_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H */
