/*
 * gdr.h -- C ABI of the GB300 (sm_103a) gated delta rule forward library
 * (libgdr.so).
 *
 * The operation (Gated DeltaNet forward, one value-head h, state S in
 * R^{V x K} held V-major as S[v][k] in fp32):
 *
 *   S~  = exp(g_t) S_{t-1}        (per-key-channel gate: S_{t-1} diag(exp(gk_t)))
 *   n_t = beta_t (v_t - S~ k_t)
 *   S_t = S~ + n_t k_t^T
 *   o_t = scale * S_t q_t         (read after the update)
 *
 * The step order, the raw (not cumulative) gate and the post-update read are
 * those of FlashQLA PR #1 ("Fused recurrent GDN decode + SGLang DFlash verify
 * kernel"), core decode-kernel commit.  Value-head h reads key/query head
 * h / (Hv / Hk) (same page, review commit: grouped-value attention mapping).
 *
 * Conventions for every entry point
 *   - All tensor pointers are DEVICE pointers unless stated otherwise, dense,
 *     row-major, in the layouts given, 16-byte aligned.
 *   - Token-major packed layout: the batch is folded into the token axis and
 *     sequence b owns tokens [cu_seqlens[b], cu_seqlens[b+1]).
 *   - dtype GDR_BF16 or GDR_F32 applies to q, k, v, beta and o.  Gates (g, gk)
 *     are always fp32; prefill states are always fp32.
 *   - The caller owns every buffer, including the workspace.  No entry point
 *     allocates, frees or synchronises the device (except
 *     gdr_get_device_status and GDR_VALIDATE, which say so), so calls can be
 *     captured in a CUDA graph.  Work is enqueued on `stream` (NULL = legacy
 *     default stream).
 *   - Inputs are never written.  Outputs must not alias inputs.
 *   - Return value: GDR_OK or a gdr_status error code; on error nothing was
 *     launched and gdr_last_error() describes the problem (thread-local).
 *     Argument and shape checks happen on the host before any launch.
 *   - Empty work (T_total == 0 or N == 0) returns GDR_OK without a launch (but
 *     for final states, which are then the initial ones).  A prefill or its
 *     backward with T_total > 0 and N == 0 is refused.
 */
#ifndef GDR_H_
#define GDR_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define GDR_API __attribute__((visibility("default")))
#else
#define GDR_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t. */
typedef struct CUstream_st* gdr_stream_t;

typedef enum gdr_status {
    GDR_OK = 0,
    GDR_ERR_INVALID_ARG = 1,    /* null pointer, bad size, misaligned pointer  */
    GDR_ERR_UNSUPPORTED = 2,    /* shape / dtype / device not supported        */
    GDR_ERR_WORKSPACE = 3,      /* workspace missing or too small              */
    GDR_ERR_LAUNCH = 4,         /* a CUDA launch or runtime call failed        */
    GDR_ERR_DEVICE_TIMEOUT = 5, /* a bounded device-side wait gave up          */
    GDR_ERR_VALIDATION = 6      /* GDR_VALIDATE found bad input content        */
} gdr_status;

typedef enum gdr_dtype {
    GDR_BF16 = 0,
    GDR_F32 = 1,
    GDR_E4M3 = 2 /* gdr_rmsnorm_fwd's y only: 8-bit codes with fp32 scales */
} gdr_dtype;

typedef enum gdr_gate_kind {
    GDR_GATE_SCALAR = 0,  /* g  [T, Hv]     one log-decay per token and value-head */
    GDR_GATE_CHANNEL = 1  /* gk [T, Hv, K]  one log-decay per key channel (KDA)    */
} gdr_gate_kind;

/* flags (bitwise or) */
#define GDR_QK_L2NORM  0x1 /* normalise q and k rows in-library: x * rsqrt(sum x^2 + 1e-6) */
#define GDR_NEG_EIGVAL 0x2 /* gdr_gating_fwd: beta = 2 * sigmoid(b)                         */
#define GDR_COMMIT     0x4 /* gdr_recurrent_fwd: write the final state back to the pool     */
#define GDR_VALIDATE   0x8 /* check input contents on the device first (synchronises).
                              * The findings land in one library-wide device word:
                              * validated calls from different host threads must be
                              * serialised by the caller, or one call's reset of the
                              * word can hide the other's findings.  (The gdr_linrec_*
                              * calls have a word of their own and take turns.)      */
#define GDR_CHANNEL_GATE 0x10 /* gdr_recurrent_fwd: g is per key channel, [T_total, Hv, K]  */
#define GDR_CHUNK_SCAN 0x20   /* gdr_chunk_fwd: chunk-parallel state scan (long sequences)     */

/* Chunk length of the chunked prefill (tokens).  The pages' kernels use 64. */
#define GDR_CHUNK 64

/*
 * gdr_chunk_workspace_size -- bytes of device workspace gdr_chunk_fwd needs.
 * Host only; depends on sizes, never on cu_seqlens contents (the chunk count
 * is bounded by ceil(T_total / 64) + N, the "capacity" of attention-gym
 * PR #344's inter-chunk state kernel).  Returns GDR_OK and sets *bytes.
 */
GDR_API int gdr_chunk_workspace_size(int N, int64_t T_total, int Hk, int Hv, int K, int V,
                             int gate_kind, int dtype, int flags, size_t* bytes);

/*
 * gdr_chunk_fwd -- chunked (WY, 64-token chunks) prefill over packed
 * variable-length sequences.  Computes exactly the recurrence above; the
 * chunked form is an implementation choice (FlashQLA PR #1 names the
 * chunked-prefill pieces cumsum / A / kkt-solve; attention-gym PR #344 gives
 * the inter-chunk state kernel with its per-chunk state h and v_new).
 *
 *   q, k           [T_total, Hk, K]   dtype
 *   v              [T_total, Hv, V]   dtype
 *   g              [T_total, Hv] fp32 log-decay (<= 0), or NULL
 *   gk             [T_total, Hv, K] fp32 per-key-channel log-decay, or NULL;
 *                  exactly one of g / gk is non-NULL
 *   beta           [T_total, Hv]      dtype, in [0, 1] (or [0, 2])
 *   initial_state  [N, Hv, V, K] fp32, or NULL for zeros
 *   cu_seqlens     [N+1] int32 device, cu[0] = 0, non-decreasing,
 *                  cu[N] = T_total; every sequence non-empty.  A cu_seqlens
 *                  that breaks the first three rules is found on the device
 *                  and nothing is written (the call still returns GDR_OK;
 *                  GDR_VALIDATE turns it into GDR_ERR_VALIDATION)
 *   scale          read scale (usually 1/sqrt(K))
 *   o              [T_total, Hv, V]   dtype (written)
 *   final_state    [N, Hv, V, K] fp32 (written), or NULL
 *   workspace      device scratch of at least gdr_chunk_workspace_size bytes,
 *                  256-byte aligned; contents need no initialisation
 * Supported: Hv % Hk == 0, K == V, K in {64, 128}.  bf16 inputs run on the
 * tensor cores at both sizes (a 64-channel head as a 128-channel tile whose
 * upper channels are zero), fp32 inputs on the CUDA cores.  Any finite g <= 0 is
 * accepted: every exponential formed is of an in-chunk difference
 * exp(gam_i - gam_j), i >= j (cuLA PR #113 review on exp(-prefix) overflow).
 *
 * GDR_CHUNK_SCAN (bf16, K = V = 128; ignored otherwise, with the same
 * results): the serial chain over a sequence's chunks is cut into segments.
 * The state map of a segment is affine in its start state,
 * S_end = S_start P + B, with P [K, K] and B [V, K]; in one parallel pass
 * the first segment of each sequence runs from the initial state (writing
 * its part of o) while the others form their B (and P, but for the last),
 * a scan composes them into every segment's start state, and the later
 * segments then run in parallel again to write o.  It pays for long
 * sequences with few value heads: the plain chain runs Hv * K / 32 CTAs per
 * sequence, 64 tokens per step, and the scan costs about three chain passes
 * of work instead of one, so it wins while 12 * Hv * N is well under the
 * GPU's SM count (measured on GB300 with one 32768-token sequence: 5x at
 * Hv = 1, 2.5x at Hv = 4, 1.5x at Hv = 8, a loss at Hv = 16).  The caller
 * decides; the flag always takes the scan where it applies.  The workspace
 * grows by about
 * 2 * (ceil(T_total / 64 / G) + N + 1) * Hv * K * K * 4 bytes, G the segment
 * length in chunks (at least 4 where sequences allow) that the library derives
 * from N, T_total and Hv.
 */
GDR_API int gdr_chunk_fwd(const void* q, const void* k, const void* v, const float* g,
                  const float* gk, const void* beta, const float* initial_state,
                  const int32_t* cu_seqlens, int N, int64_t T_total, int Hk, int Hv,
                  int K, int V, float scale, int dtype, int flags, void* o,
                  float* final_state, void* workspace, size_t ws_bytes,
                  gdr_stream_t stream);

/*
 * gdr_chunk_fwd_noalloc -- gdr_chunk_fwd without a caller workspace.  There is
 * no counterpart on the reference pages; it exists for callers that cannot
 * allocate device memory (a serving engine whose arena already owns all device
 * memory, a plugin host that exposes no allocator, a decode loop that cannot
 * afford cudaMalloc's implicit synchronisation).
 *   Same arguments and results as gdr_chunk_fwd, minus workspace / ws_bytes.
 *   Scratch comes from an array of GDR_NOALLOC_WORKSPACE_BYTES compiled into
 *   the library; every GPU that loads the library holds it until exit.  A
 *   problem whose gdr_chunk_workspace_size exceeds it is rejected with
 *   GDR_ERR_WORKSPACE before anything runs.
 *   Every call looks up the array's device address in the context current on
 *   the calling thread (the address belongs to the context, so it stays right
 *   after cudaDeviceReset or with another context current on the device).
 *   The first call in a context may load the library's device code there:
 *   make it before any stream capture.
 *   Nothing is allocated or freed, by the library or any routine it calls.
 *   All calls share the one array and it keeps the previous call's contents
 *   (nothing in it has to start at zero): calls whose work overlaps on the
 *   GPU -- on different streams, or from different host threads -- race on it
 *   and must be serialised by the caller.
 */
#define GDR_NOALLOC_WORKSPACE_BYTES (64ull << 20)
GDR_API int gdr_chunk_fwd_noalloc(const void* q, const void* k, const void* v, const float* g,
                                  const float* gk, const void* beta, const float* initial_state,
                                  const int32_t* cu_seqlens, int N, int64_t T_total, int Hk, int Hv,
                                  int K, int V, float scale, int dtype, int flags, void* o,
                                  float* final_state, gdr_stream_t stream);

/*
 * gdr_recurrent_fwd -- slot-indexed recurrent decode / multi-step verify
 * (FlashQLA PR #1, paged verify commit and deployment-facts commit).
 *
 *   q, k           [T_total, Hk, K] dtype;   v [T_total, Hv, V] dtype
 *   g              [T_total, Hv] fp32 raw log-decay, or with GDR_CHANNEL_GATE
 *                  [T_total, Hv, K] fp32 per-key-channel log-decay (column c
 *                  of the state scaled by e^{g[t,h,c]}: the per-channel decode
 *                  of tokenspeed PR #834);  beta [T_total, Hv] dtype
 *   state_pool     [num_slots, Hv, V, K] (V-major), pool_dtype GDR_F32 or
 *                  GDR_BF16; read, and written in place only with GDR_COMMIT
 *   state_indices  [N] int32 device: pool slot of sequence b; -1 (any value
 *                  < 0) is padding: nothing of sequence b is read or written
 *                  (its o rows, pool slot and ibuf row stay untouched); slot 0
 *                  is a valid slot; valid slots must be unique and < num_slots
 *   cu_seqlens     [N+1] int32 device (decode: 0..N); a sequence may be empty
 *   o              [T_total, Hv, V] dtype (written for non-padding sequences)
 *   intermediate_states  [rows >= N, steps, Hv, V, K] pool dtype, or NULL:
 *                  row b, step t receives the state after token t of
 *                  sequence b (t < L_b), rounded to the pool dtype; rows of
 *                  padding sequences and steps >= L_b are untouched.  Requires
 *                  L_b <= steps (checked under GDR_VALIDATE).
 * The carried state stays fp32 between tokens; only stores round.
 */
GDR_API int gdr_recurrent_fwd(const void* q, const void* k, const void* v, const float* g,
                      const void* beta, void* state_pool, int pool_dtype, int num_slots,
                      const int32_t* state_indices, const int32_t* cu_seqlens, int N,
                      int64_t T_total, int Hk, int Hv, int K, int V, float scale, int dtype,
                      int flags, void* o, void* intermediate_states, int steps,
                      gdr_stream_t stream);

/*
 * gdr_recurrent_fwd_norm -- gdr_recurrent_fwd with the gated RMSNorm output
 * epilogue fused (tokenspeed PR #834, fused gated-norm epilogue commit): every
 * value row x = o[t,h,:] of the recurrence output is written as
 *   x / sqrt(mean_v(x^2) + eps) * norm_weight[v] * sigmoid(norm_gate[t,h,v])
 * norm_weight [V] fp32 device; norm_gate [T_total, Hv, V] dtype device;
 * eps >= 0.  The normalisation uses the fp32 output before any rounding (one
 * bf16 round trip fewer than a separate norm kernel).  Every other argument,
 * flag and guarantee is gdr_recurrent_fwd's.
 */
GDR_API int gdr_recurrent_fwd_norm(const void* q, const void* k, const void* v, const float* g,
                      const void* beta, void* state_pool, int pool_dtype, int num_slots,
                      const int32_t* state_indices, const int32_t* cu_seqlens, int N,
                      int64_t T_total, int Hk, int Hv, int K, int V, float scale, int dtype,
                      int flags, const float* norm_weight, const void* norm_gate, float eps,
                      void* o, void* intermediate_states, int steps, gdr_stream_t stream);

/*
 * gdr_recurrent_fwd_gated -- gdr_recurrent_fwd with the gates formed inside the
 * kernel from the raw projections (FlashQLA PR #1, in-kernel gating commit):
 *   g[t,h]    = -exp(A_log[h]) * softplus(a[t,h] + dt_bias[h])
 *               (softplus beta 1, threshold 20, as gdr_gating_fwd)
 *   beta[t,h] = sigmoid(b[t,h]), times 2 with GDR_NEG_EIGVAL
 *   a, b [T_total, Hv] dtype; A_log, dt_bias [Hv] fp32 device.
 * beta is kept in fp32 (it is not rounded to dtype as gdr_gating_fwd's output
 * is).  Every other argument, flag (GDR_QK_L2NORM, GDR_COMMIT, GDR_VALIDATE)
 * and guarantee is gdr_recurrent_fwd's; GDR_CHANNEL_GATE is not accepted.
 */
GDR_API int gdr_recurrent_fwd_gated(const void* q, const void* k, const void* v, const void* a,
                      const void* b, const float* A_log, const float* dt_bias, void* state_pool,
                      int pool_dtype, int num_slots, const int32_t* state_indices,
                      const int32_t* cu_seqlens, int N, int64_t T_total, int Hk, int Hv, int K,
                      int V, float scale, int dtype, int flags, void* o, void* intermediate_states,
                      int steps, gdr_stream_t stream);

/*
 * gdr_gating_fwd -- gate preparation from raw projections (FlashQLA PR #1,
 * host-gating and in-kernel-gating commits):
 *   g[t,h]    = -exp(A_log[h]) * softplus(a[t,h] + dt_bias[h])
 *               (softplus beta 1, threshold 20)
 *   beta[t,h] = sigmoid(b[t,h]), times 2 with GDR_NEG_EIGVAL
 *   a, b [T, Hv] dtype; dt_bias, A_log [Hv] fp32; g [T, Hv] fp32 (written);
 *   beta [T, Hv] dtype (written).
 */
GDR_API int gdr_gating_fwd(const void* a, const float* dt_bias, const float* A_log, const void* b,
                   int64_t T, int Hv, int dtype, int flags, float* g, void* beta,
                   gdr_stream_t stream);

/*
 * The gated linear recurrence: per channel c of sequence n, with the
 * natural-log decay g <= 0 (-inf, a reset, is allowed),
 *
 *   h_t = exp(g_t) h_{t-1} + x_t,   h before the first token = initial_state[n]
 *
 * over the packed tokens cu_seqlens[n] .. cu_seqlens[n+1]-1.  The state is
 * carried in fp32 whatever the tensors' types.
 *
 * Conventions of gdr_linrec_fwd, gdr_linrec_bwd and gdr_linrec_step, where
 * they go beyond the library's:
 *   - Token tensors are [T_total, D] with a row stride in elements of their
 *     own (so they can be column blocks of a wider matrix): D or more for
 *     tensors that are written, any stride >= 0 for those that are only read
 *     (0: one row for every token).  They need their element's alignment only;
 *     16-byte aligned rows (8 elements of the type) with D and the strides
 *     multiples of 8 take the fast path.
 *   - dtype (GDR_BF16 or GDR_F32) is that of x, y and their gradients,
 *     gate_dtype (GDR_BF16 or GDR_F32) that of g and dg.  Prefill states are
 *     fp32 [N, D], dense; the one that is written overlaps none that is read.
 *   - cu_seqlens [N+1] int32 device, cu[0] = 0, non-decreasing; sequences may
 *     be empty.  cu[N] may be less than T_total (a padded batch): rows from
 *     cu[N] on are neither read nor written.  A cu_seqlens that breaks these
 *     rules never causes an access outside the tensors, but what is written
 *     is then unspecified; GDR_VALIDATE (the only flag of fwd and bwd) turns
 *     it, and a gate that is NaN or > 0, into GDR_ERR_VALIDATION.
 *   - A NaN or infinity stays within its sequence and channel.
 *   - Results do not depend on scheduling: equal inputs give equal bits.
 *   - A tile of a long call waits for the state that reaches it from the tiles
 *     before it, which are running by then.  Every wait is bounded (one second):
 *     one that gives up is reported by gdr_get_device_status, and what the call
 *     has not written by then stays unwritten.
 *   - D up to 2^24, T_total up to 2^31 - 512.
 *
 * gdr_linrec_workspace_size -- bytes of device workspace that gdr_linrec_fwd
 * and gdr_linrec_bwd need (the same for both; may be 0).  Host only.
 */
GDR_API int gdr_linrec_workspace_size(int N, int64_t T_total, int D, int dtype, int gate_dtype,
                                      size_t* bytes);

/*
 * gdr_linrec_fwd -- the recurrence over packed sequences (prefill, training
 * forward).
 *   x              [T_total, D] dtype, row stride x_stride
 *   g              [T_total, D] gate_dtype, row stride g_stride
 *   initial_state  [N, D] fp32, or NULL for zeros
 *   y              [T_total, D] dtype, row stride y_stride (written): y_t = h_t
 *   final_state    [N, D] fp32 (written: the last h, the initial state where
 *                  a sequence is empty), or NULL
 *   workspace      device scratch of gdr_linrec_workspace_size bytes, 256-byte
 *                  aligned (NULL where that is 0); needs no initialisation.
 *                  Calls whose work may overlap on the GPU need one each.
 */
GDR_API int gdr_linrec_fwd(const void* x, int64_t x_stride, const void* g, int64_t g_stride,
                           const float* initial_state, const int32_t* cu_seqlens, int N,
                           int64_t T_total, int D, int dtype, int gate_dtype, int flags, void* y,
                           int64_t y_stride, float* final_state, void* workspace, size_t ws_bytes,
                           gdr_stream_t stream);

/*
 * gdr_linrec_bwd -- gradients of gdr_linrec_fwd from the gradient dy of y and
 * d_final_state [N, D] fp32 (NULL for zeros) of the final state.  With mu
 * after a sequence's last token = d_final_state[n],
 *
 *   lam_t = dy_t + mu_{t+1},  mu_t = exp(g_t) lam_t
 *   dx_t = lam_t,   dg_t = mu_t h_{t-1},   d_initial_state[n] = mu of the first token
 *
 * h_{t-1} is read from y, the forward's output as stored (initial_state, or 0,
 * before the first token).
 *   dx  [T_total, D] dtype, dg [T_total, D] gate_dtype (written)
 *   d_initial_state [N, D] fp32 (written; d_final_state's row where a sequence
 *                   is empty), or NULL
 */
GDR_API int gdr_linrec_bwd(const void* dy, int64_t dy_stride, const void* g, int64_t g_stride,
                           const void* y, int64_t y_stride, const float* initial_state,
                           const float* d_final_state, const int32_t* cu_seqlens, int N,
                           int64_t T_total, int D, int dtype, int gate_dtype, int flags, void* dx,
                           int64_t dx_stride, void* dg, int64_t dg_stride, float* d_initial_state,
                           void* workspace, size_t ws_bytes, gdr_stream_t stream);

/*
 * gdr_linrec_step -- the recurrence over a few tokens of each sequence, from
 * and to a slot-indexed state pool: decode and multi-step verify, with
 * gdr_recurrent_fwd's rules.
 *   state_pool     [num_slots, D] pool_dtype (GDR_F32 or GDR_BF16), dense; read,
 *                  and written in place only with GDR_COMMIT
 *   state_indices  [N] int32 device: the slot of each sequence; a value < 0 is
 *                  padding (nothing of that sequence is read or written, its
 *                  gates are not checked; nor for a value >= num_slots, an
 *                  error that GDR_VALIDATE reports).  With GDR_COMMIT valid slots must be unique.
 *   intermediate_states  [rows >= N, steps, D] pool dtype, dense, or NULL: row
 *                  b, step t receives the state after token t of sequence b;
 *                  steps >= L_b and padding rows are untouched.  L_b <= steps
 *                  (checked under GDR_VALIDATE; later tokens' states are
 *                  dropped otherwise).
 * Flags: GDR_COMMIT, GDR_VALIDATE.
 */
GDR_API int gdr_linrec_step(const void* x, int64_t x_stride, const void* g, int64_t g_stride,
                            void* state_pool, int pool_dtype, int num_slots,
                            const int32_t* state_indices, const int32_t* cu_seqlens, int N,
                            int64_t T_total, int D, int dtype, int gate_dtype, int flags, void* y,
                            int64_t y_stride, void* intermediate_states, int steps,
                            gdr_stream_t stream);

/*
 * gdr_rmsnorm_fwd -- root-mean-square norm of every row, with the residual's
 * addition before it:
 *
 *   s = round(x + residual)  (x without a residual)
 *   y = s / sqrt(mean(s^2) + eps) * weight
 *
 * The sum is rounded to dtype first, so that y is the norm of the residual
 * stream as it is stored.
 *   x, residual    [M, D] dtype (GDR_BF16 or GDR_F32), row strides in elements
 *                  (any >= 0); residual may be NULL
 *   weight         [D] fp32
 *   residual_out   [M, D] dtype: s (written).  Given if and only if residual
 *                  is.  It may be residual or x itself (the same pointer and
 *                  stride): the addition is then in place.
 *   y              [M, D] y_dtype (written): dtype, or GDR_E4M3 with scales
 *   scales         [M, ceil(D / group)] fp32, dense (written), with GDR_E4M3
 *                  only: for each group of scale_group consecutive elements of
 *                  a row (32, 64 or 128; 0: the whole row), with a the larger of
 *                  max |y| and 1e-12, scale = a / 448 and the stored code is
 *                  y / scale (both quotients rounded to fp32) rounded to the
 *                  nearest e4m3 value, half-way to the even code, so that
 *                  code * scale stands for y.  y is fp32, not rounded before.
 *                  A NaN in a group makes its scale and all its codes NaN; an
 *                  infinity makes the scale infinite, its own code NaN and the
 *                  group's finite values' 0.
 * D up to GDR_RMSNORM_MAX_D.  Rows need their element's alignment only; rows
 * of 8 aligned elements, with D and the strides multiples of 8, take the fast
 * path.  Sums are fp32: a row whose sum of squares passes fp32's range
 * (elements above about 1e19) gives 0 for its finite elements; with eps = 0 one
 * whose squares fall below it (elements under about 1e-19) loses precision, and
 * one whose squares vanish gives infinities and NaN.
 * The codes are for a caller's own products: no entry point of the library reads
 * them, and the scales are plain fp32 in row order, not a layout of block-scaled
 * matrix instructions.
 */
#define GDR_RMSNORM_MAX_D 32768
GDR_API int gdr_rmsnorm_fwd(const void* x, int64_t x_stride, const void* residual,
                            int64_t residual_stride, const float* weight, int64_t M, int D,
                            float eps, int dtype, void* residual_out, int64_t residual_out_stride,
                            void* y, int64_t y_stride, int y_dtype, float* scales, int scale_group,
                            gdr_stream_t stream);

/* gdr_rmsnorm_bwd_workspace_size -- bytes of device workspace gdr_rmsnorm_bwd
 * needs.  Host only. */
GDR_API int gdr_rmsnorm_bwd_workspace_size(int64_t M, int D, size_t* bytes);

/*
 * gdr_rmsnorm_bwd -- gradients of gdr_rmsnorm_fwd from dy, the gradient of y
 * (for GDR_E4M3: of the values its codes stand for, the rounding taken as the
 * identity), and d_residual_out, the gradient that arrives at s along the
 * residual stream (NULL for zeros).  With r = 1 / sqrt(mean(s^2) + eps) and
 * z = weight * dy,
 *
 *   dx = r z - r^3 s mean(s z) + d_residual_out   (of x and of residual alike)
 *   dweight = sum over rows of r dy s
 *
 *   dy, s, d_residual_out  [M, D] dtype, row strides in elements (any >= 0); s
 *                          is the forward's residual_out (or x)
 *   dx                     [M, D] dtype (written); may be dy or d_residual_out
 *                          itself (the same pointer and stride)
 *   dweight                [D] fp32 (written, not accumulated into), or NULL
 *   workspace              gdr_rmsnorm_bwd_workspace_size bytes, 256-byte
 *                          aligned; needs no initialisation; may be NULL with
 *                          dweight NULL
 * The rows are summed in a fixed order: equal inputs give equal bits.  Rows
 * come by copies whose waits are bounded (one second): one that gives up is
 * reported by gdr_get_device_status; dx rows that the call has not written by
 * then stay unwritten, and dweight is then NaN.
 */
GDR_API int gdr_rmsnorm_bwd(const void* dy, int64_t dy_stride, const void* s, int64_t s_stride,
                            const float* weight, const void* d_residual_out,
                            int64_t d_residual_out_stride, int64_t M, int D, float eps, int dtype,
                            void* dx, int64_t dx_stride, float* dweight, void* workspace,
                            size_t ws_bytes, gdr_stream_t stream);

/* Description of the last error on the calling thread ("" if none). */
GDR_API const char* gdr_last_error(void);

/*
 * gdr_get_device_status -- synchronises `stream`, then reads and clears the
 * library's device error word of the current device (set by a bounded device
 * wait that gave up).  *word receives the raw word (0 = clean).  Returns
 * GDR_OK if the word was 0, GDR_ERR_DEVICE_TIMEOUT otherwise.  Diagnostic only.
 */
GDR_API int gdr_get_device_status(gdr_stream_t stream, int* word);

/*
 * gdr_selftest_bounded_wait -- diagnostic for the failure path (no counterpart
 * on the pages): enqueues on `stream` one small kernel that waits on an
 * mbarrier nothing ever completes, using the same bounded wait as the
 * tensor-core kernels (about one second of %globaltimer); it then sets bit
 * 0x100 of the device error word and returns.  A following
 * gdr_get_device_status reports GDR_ERR_DEVICE_TIMEOUT, and the context stays
 * usable.  Nothing faults, traps or spins without a limit.
 */
GDR_API int gdr_selftest_bounded_wait(gdr_stream_t stream);

/*
 * gdr_selftest_linrec_lost_copy -- the same for gdr_linrec_fwd's way out: the
 * recurrence over dense fp32 tensors, from zero states, in which the tiles of
 * row `lost_row` (counted along the tokens, 160 or 320 a row) wait for bytes
 * that nothing copies.  After two or three seconds bit 0x200 of the device error
 * word is set; y and final_state hold the recurrence's values or are unwritten.
 */
GDR_API int gdr_selftest_linrec_lost_copy(const float* x, const float* g, const int32_t* cu_seqlens,
                                          int N, int64_t T_total, int D, int lost_row, float* y,
                                          float* final_state, void* workspace, size_t ws_bytes,
                                          gdr_stream_t stream);

/*
 * gdr_selftest_rmsnorm_lost_copy -- the same for gdr_rmsnorm_bwd's way out, on
 * dense bf16 rows of 512 to 4096 elements with eps 1e-6: row `lost_row` waits
 * for bytes that nothing copies.  Bit 0x400 of the device error word is set; dx
 * holds the gradients or is unwritten, and dweight is NaN.
 */
GDR_API int gdr_selftest_rmsnorm_lost_copy(const void* dy, const void* s, const float* weight, int64_t M,
                                           int D, int64_t lost_row, void* dx, float* dweight,
                                           void* workspace, size_t ws_bytes, gdr_stream_t stream);

/*
 * Kernel timing for diagnostics (no counterpart on the pages; measurement
 * support).  gdr_profile_enable(1): from then on every kernel the library
 * launches is bracketed by two CUDA events on its stream (not capturable:
 * leave it off under stream capture).  gdr_profile_read: waits for the
 * recorded events, then reports per kernel name (sorted) the summed device
 * time in ms and the launch count since the previous read, and clears them.
 *   names      receives "name1,name2,...," (truncated to name_cap bytes)
 *   total_ms, launches  arrays of max_kernels entries
 *   *n_kernels number of entries filled
 */
GDR_API int gdr_profile_enable(int on);
GDR_API int gdr_profile_read(int max_kernels, char* names, size_t name_cap, double* total_ms,
                             int* launches, int* n_kernels);

/* Library version (major * 10000 + minor * 100 + patch). */
GDR_API int gdr_version(void);

#ifdef __cplusplus
}
#endif
#endif /* GDR_H_ */
