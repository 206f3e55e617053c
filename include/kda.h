/*
 * kda.h -- C ABI of libkda, the GB300 (sm_103a) Kimi Delta Attention core.
 *
 * The library computes the gated delta rule with a per-key-channel decay, the
 * mixer core of the Kimi-Linear / Kimi-K3 KDA layers, for every independent
 * (sequence, head) unit:
 *
 *     q^ = q / sqrt(|q|^2 + 1e-6),  k^ = k / sqrt(|k|^2 + 1e-6)     (if use_qk_l2norm)
 *     S_t = (I - beta_t k^_t k^_t^T) Diag(exp g_t) S_{t-1} + beta_t k^_t v_t^T
 *     o_t = scale * S_t^T q^_t
 *
 * optionally followed by the head-wise sigmoid-gated RMSNorm
 *
 *     y = o / sqrt(mean_v(o^2) + eps) * w * sigmoid(gate)
 *
 * Sources (page title, section):
 *   nnterp encyclopedia "Kimi-Linear": section 02 "support()" (the kernel's
 *   arguments attention_queries/keys/values, decays, betas, state_input and its
 *   outputs attention_head_outputs, state_output, with their layouts); section 03
 *   "Kimi Delta Attention decays each key channel" (g per key channel, fp32,
 *   non-positive; beta = sigmoid(b_proj); L2 norm and 1/sqrt(key_dim) applied in
 *   the kernel; state [batch, heads, key_dim, value_dim]); section 03 "Loading"
 *   (a prompt runs a chunked kernel that carries the state from one 64-token
 *   chunk to the next, a decode step the token-by-token kernel); section 04
 *   "From the family module" (the state decays channel by channel before each
 *   delta-rule update; call contract (query, key, value, g=, beta=,
 *   initial_state=) -> (core_attn_out, last_recurrent_state)).
 *   Kimi-K3 atlas "gate-project (decode, P = 1000)": sections "Parameters" (the
 *   gated RMSNorm holds 128 weights shared by the 96 heads) and "Code" (o_norm(o,
 *   gate) with activation 'sigmoid', heads then flattened to heads * head_dim).
 *
 * Conventions for every entry point:
 *   - Every tensor pointer is a DEVICE pointer (cudaMalloc, or any memory the
 *     GPU can address) unless its name ends in _host.  Tensors are dense,
 *     row-major, contiguous, 16-byte aligned.  The caller owns every buffer; the
 *     library allocates no device memory and keeps no pointer after the call.
 *   - Work is enqueued on `stream` (a cudaStream_t; NULL = the legacy default
 *     stream) and returns without synchronising.  Outputs are valid once the
 *     stream reaches that point.
 *   - Arguments are validated on the host before anything is launched.  A bad
 *     argument returns KDA_ERR_INVALID_ARG, an unsupported but well-formed
 *     request KDA_ERR_UNSUPPORTED, a CUDA launch/runtime error KDA_ERR_CUDA;
 *     nothing is launched in the first two cases.  kda_last_error() then holds a
 *     message for the calling thread.  No C++ exception crosses the ABI.
 *   - Precondition (not checked on the device): g lies in [-5, 0] (the layer's
 *     gate_lower_bound is -5), beta in [0, 1].  Out-of-range values give
 *     numerically meaningless but memory-safe results.
 */
#ifndef KDA_H
#define KDA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum kda_status {
    KDA_OK = 0,
    KDA_ERR_INVALID_ARG = 1,  /* null pointer, bad size, misalignment, bad cu_seqlens */
    KDA_ERR_UNSUPPORTED = 2,  /* well-formed but not built (dims, dtype, chunk, mode) */
    KDA_ERR_CUDA = 3,         /* a CUDA runtime / launch error */
    KDA_ERR_TIMEOUT = 4       /* a bounded device wait gave up (returned by kda_device_status) */
} kda_status;

typedef enum kda_dtype {
    KDA_BF16 = 0,
    KDA_F32 = 1
} kda_dtype;

typedef enum kda_mode {
    KDA_MODE_AUTO = 0,    /* tensor-core path where supported, else the fp32 path */
    KDA_MODE_TENSOR = 1,  /* tcgen05 path only (K = V = 128, chunk = 64); else UNSUPPORTED */
    KDA_MODE_FP32 = 2,    /* CUDA-core fp32 chunked path (any supported K, V, chunk) */
    KDA_MODE_SPLIT = 3    /* tcgen05 path, the two-kernel split form (needs a workspace) */
} kda_mode;

/* Library version (major * 10000 + minor * 100 + patch). */
int kda_version(void);

/* Message describing the last failed call on this thread ("" if none). */
const char *kda_last_error(void);

/* Static name of a status code. */
const char *kda_status_string(int status);

/* Number of kernels this library has launched in this process (all threads). */
uint64_t kda_launch_count(void);

/*
 * kda_device_status -- failures detected on the device since the last call.
 *
 * Every wait inside the kernels (on a bulk or TMA copy, or on the tensor core) is
 * bounded.  A CTA whose wait gives up lets the copies it started land, writes NaN
 * into every output it was responsible for (the state, o and y of its (sequence,
 * head) units, or the y and state rows of its convolution tiles; a decode CTA also
 * poisons every later unit it owned), and counts the event in a device-side counter.
 * (An attention CTA poisons the rows that it had not written yet.)
 * The compute calls are asynchronous and cannot see this, so this call synchronises
 * `stream` (a cudaStream_t; NULL = the legacy default stream), reads the counters of
 * the current device and clears them.  Returns KDA_ERR_TIMEOUT if any wait gave up
 * (kda_last_error() names the kernels and counts), KDA_ERR_CUDA if the stream or a
 * counter read failed, KDA_OK otherwise.  The counters are shared by all streams of
 * the device: call it when the work to be checked has been enqueued on `stream` or
 * has finished.  No counterpart on the pages: it is the library's failure detection.
 */
kda_status kda_device_status(void *stream);

/*
 * kda_set_wait_limit -- bound on the first-line waits on copies from global memory.
 *
 * The decode step's copy waits (kda_recurrent_step, kda_recurrent_step_logits with
 * K = V = 128), the short convolution's tile waits (kda_short_conv_fwd over a prompt)
 * and the fused tensor-core prefill's tile and blob waits (kda_chunk_fwd,
 * kda_chunk_fwd_logits without a workspace or with one in the concurrent form) and the
 * attention kernels' tile waits (kda_attn_decode, kda_attn_prompt) poll their mbarrier at
 * most this many times before they give up, for the calls made after this one
 * (process-wide).  polls < 0 restores the default (2^26; the attention kernels never poll
 * more than 2^21 times); 0 makes every such wait give up at once, which tests of the failure
 * handling use (kda_device_status then reports KDA_ERR_TIMEOUT and the outputs hold NaN).  The waits that let copies in
 * flight land before a CTA exits, the tensor-core waits, and the split form's kernels
 * always keep their full bound.  Returns KDA_OK, or
 * KDA_ERR_INVALID_ARG above 2^32 - 1.  No counterpart on the pages.
 */
kda_status kda_set_wait_limit(int64_t polls);

/*
 * kda_chunk_prepass_hits -- how many chunks of the concurrent form (kda_chunk_fwd with a
 * workspace) took their state-independent operands from the pre-pass rather than
 * forming them in the fused kernel, since the last call (a diagnostic of how much
 * of the work the idle SMs took over).  Synchronises `stream`, reads the current
 * device's counter into *chunks and clears it.  KDA_ERR_INVALID_ARG for a NULL
 * chunks, KDA_ERR_CUDA if the stream or the read failed.  No counterpart on the pages.
 */
kda_status kda_chunk_prepass_hits(void *stream, uint64_t *chunks);

/*
 * kda_chunk_fwd -- chunked prefill over whole prompts.
 *
 * Pages: nnterp "Kimi-Linear" section 03 "Loading" (the chunked kernel carries
 * the state from one 64-token chunk to the next and never holds it per token),
 * section 02 (argument and output layouts), section 04 (call contract).
 *
 * Dense mode (cu_seqlens == NULL): N = B sequences of T tokens.
 *   q, k   [B, T, H, K]  qkv_dtype          v [B, T, H, V] qkv_dtype
 *   g      [B, T, H, K]  float, log decay    beta [B, T, H] float
 *   initial_state [N, H, K, V] float or NULL (zero state)
 *   final_state   [N, H, K, V] float or NULL; may be the same buffer as
 *                 initial_state (updated in place)
 *   o      [B, T, H, V]  o_dtype, the per-head outputs (head outputs before the
 *                        gated norm); may be NULL when y is given
 * Varlen mode (cu_seqlens != NULL): B must be 1, T is the packed token count and
 *   sequence n covers tokens [cu_seqlens[n], cu_seqlens[n+1]), n < n_seqs;
 *   initial_state / final_state are [n_seqs, H, K, V].  cu_seqlens is a device
 *   int32 array of n_seqs + 1 entries.  cu_seqlens_host, if not NULL, is a host
 *   copy of it: it is checked (starts at 0, non-decreasing, ends at T) and used to
 *   start the longest sequences first.  Without it the device array is trusted;
 *   kernels still clamp every sequence to [0, T] so a bad array cannot make them
 *   read or write out of bounds.
 * Gated norm (gate != NULL): gate [B, T, H, V] gate_dtype, norm_w [V] float,
 *   eps > 0, y [B, T, H * V] o_dtype, y = RMSNorm_v(o) * norm_w * sigmoid(gate).
 * chunk: tokens per chunk, 16, 32 or 64 (the tensor path needs 64).
 * scale: applied to q^ (1/sqrt(K) for the layer).  use_qk_l2norm: 0 or 1.
 * Supported K, V: 32, 64, 128 (fp32 path); 128 (tensor path).
 * workspace: caller-owned device scratch of workspace_bytes, or NULL.  With NULL
 *   the tensor path runs one fused kernel per (sequence, head).  A workspace of at
 *   least kda_chunk_workspace_size(B, T, H, n_seqs) bytes lets it use the SMs that
 *   kernel leaves idle (N * H below the SM count): a pre-pass kernel on a stream the
 *   call creates forms chunks' state-independent operands (grams, UT transform) ahead
 *   of the fused kernel, which takes each one that is ready when it gets there and
 *   forms the rest itself, never waiting (the concurrent form; the caller's stream
 *   covers both kernels).  With mode KDA_MODE_SPLIT the pre-pass instead forms every
 *   chunk's operands first, then one CTA per (sequence, head) runs the state through
 *   the chunks (the split form).  All forms give the same bits.  A workspace that is
 *   too small, misaligned or overlaps a tensor of the call is KDA_ERR_INVALID_ARG; the
 *   fp32 path ignores it.  Its contents are scratch: overwritten by the call,
 *   meaningless after it.  Calls that may overlap on the GPU need workspaces of
 *   their own.
 * mode: a kda_mode.  Returns a kda_status.
 */
kda_status kda_chunk_fwd(const void *q, const void *k, const void *v, kda_dtype qkv_dtype,
                         const float *g, const float *beta, const float *initial_state,
                         float *final_state, void *o, kda_dtype o_dtype,
                         const int32_t *cu_seqlens, const int32_t *cu_seqlens_host, int n_seqs,
                         int B, int T, int H, int K, int V, int chunk, float scale,
                         int use_qk_l2norm, const void *gate, kda_dtype gate_dtype,
                         const float *norm_w, float eps, void *y, void *workspace,
                         size_t workspace_bytes, int mode, void *stream);

/*
 * kda_chunk_workspace_size -- bytes of the workspace kda_chunk_fwd and
 * kda_chunk_fwd_logits take for the concurrent and split tensor-core forms: 32 KiB per
 * (chunk slot, head) for (ceil(B * T / 64) + N) slots, N = n_seqs in varlen mode
 * (n_seqs > 0), else B, then a 4-byte flag per (slot, head) and a 4-byte progress
 * word per (sequence, head), each array 256-byte aligned.  0 for arguments no call
 * accepts.  Host only; launches nothing.
 */
size_t kda_chunk_workspace_size(int B, int T, int H, int n_seqs);

/*
 * kda_chunk_fwd_noalloc -- kda_chunk_fwd for callers that cannot allocate device memory.
 *
 * The concurrent and split tensor-core prefill forms keep chunks' state-independent
 * operands in scratch memory between their two kernels, and kda_chunk_fwd takes that
 * scratch from the caller as a workspace.  Some callers have no way to provide one: code behind a
 * fixed operator or plugin interface that passes only input and output tensors, and
 * code that runs where device allocation is not allowed or not possible (a memory
 * pool owned by another component, a latency-critical path that must not allocate).
 * This entry point takes the same arguments as kda_chunk_fwd without the workspace
 * and uses a fixed 64 MiB array in the library's own device memory instead.  It makes
 * no allocation of any kind: no cudaMalloc, no cudaFree, no allocating library routine.
 *
 *   - Limit: a call may need at most 64 MiB of scratch, i.e. 2048 (chunk slot, head)
 *     blobs of 32 KiB (kda_chunk_workspace_size gives a call's need); for example one
 *     prompt of up to 1280 tokens at 96 heads.  A larger call returns
 *     KDA_ERR_UNSUPPORTED with a message giving both sizes, and launches nothing.
 *   - The array exists on every GPU that loads the library and stays there until the
 *     process exits.  The first call on a device, with that device current, looks up
 *     the array's device address (cudaGetSymbolAddress, once per device); make that
 *     first call before any stream capture.
 *   - Every call shares the one array and leaves its contents behind.  Nothing in it
 *     needs to start at zero: a call clears the flags it uses itself and writes every
 *     other byte before reading it.  Calls whose work can overlap on the GPU
 *     (different streams, different host threads) race on the array and must be
 *     ordered by the caller.
 *   - Results are identical to kda_chunk_fwd with a workspace (the same kernels).
 * No counterpart on the pages: it is an interface for a class of callers.
 */
kda_status kda_chunk_fwd_noalloc(const void *q, const void *k, const void *v, kda_dtype qkv_dtype,
                                 const float *g, const float *beta, const float *initial_state,
                                 float *final_state, void *o, kda_dtype o_dtype,
                                 const int32_t *cu_seqlens, const int32_t *cu_seqlens_host, int n_seqs,
                                 int B, int T, int H, int K, int V, int chunk, float scale,
                                 int use_qk_l2norm, const void *gate, kda_dtype gate_dtype,
                                 const float *norm_w, float eps, void *y, int mode, void *stream);

/*
 * kda_chunk_fwd_logits -- kda_chunk_fwd with the decay and the write strength
 * computed inside the kernels from the logits the layer's projections produce,
 * instead of read as fp32 g and beta (halves the g traffic with bf16 logits).
 *
 * Pages: Kimi-K3 atlas "gate-project (decode, P = 1000)", section "Code" (the
 * layer holds A_log = log U(1, 16) per head, f_a_proj / f_b_proj producing one
 * decay logit per key channel of each head, dt_bias with one bias per such logit,
 * b_proj with one write-strength logit per head, gate_lower_bound); nnterp
 * encyclopedia "Kimi-Linear", section 03 (g per key channel, fp32, non-positive;
 * beta = sigmoid(b_proj)).  The line combining them is not on the pages; this
 * library reads it as
 *     g[t][h][c] = max(g_lower_bound, -exp(A_log[h]) * softplus(g_logits[t][h][c] + dt_bias[h][c]))
 *     beta[t][h] = sigmoid(beta_logits[t][h])
 *
 *   g_logits    [B, T, H, K] g_logits_dtype     A_log [H] float
 *   dt_bias     [H, K] float or NULL (zero)     g_lower_bound <= 0; -INFINITY for none
 *   beta_logits [B, T, H] beta_logits_dtype
 * Everything else as kda_chunk_fwd.
 */
kda_status kda_chunk_fwd_logits(const void *q, const void *k, const void *v, kda_dtype qkv_dtype,
                                const void *g_logits, kda_dtype g_logits_dtype, const float *A_log,
                                const float *dt_bias, float g_lower_bound, const void *beta_logits,
                                kda_dtype beta_logits_dtype, const float *initial_state, float *final_state,
                                void *o, kda_dtype o_dtype, const int32_t *cu_seqlens,
                                const int32_t *cu_seqlens_host, int n_seqs, int B, int T, int H, int K, int V,
                                int chunk, float scale, int use_qk_l2norm, const void *gate,
                                kda_dtype gate_dtype, const float *norm_w, float eps, void *y, void *workspace,
                                size_t workspace_bytes, int mode, void *stream);

/*
 * kda_chunk_fwd_host / kda_chunk_fwd_logits_host -- kda_chunk_fwd (_logits) for a
 * caller whose tensors are in HOST memory: a dense prompt (B sequences of T tokens)
 * streamed through the device in segments of `segment` tokens.
 *
 * Page: nnterp encyclopedia "Kimi-Linear", section 03 "Loading" (the chunked kernel
 * carries the state from one 64-token chunk to the next; a segment boundary is a
 * chunk boundary, so the outputs equal those of one kda_chunk_fwd call on device
 * copies of the same tensors, bit for bit).
 *
 * Every tensor argument -- q, k, v, g, beta (or g_logits, beta_logits, A_log,
 * dt_bias), initial_state, final_state, o, gate, norm_w, y -- is a HOST pointer with
 * the layout of kda_chunk_fwd (dense only: no cu_seqlens).  Page-locked memory
 * (cudaHostAlloc / cudaHostRegister) lets the copies overlap the kernels; pageable
 * memory works, with copies that do not overlap.  Outputs must not overlap inputs.
 *
 *   segment    tokens per segment, a multiple of 64; 0 = 1024.
 *   workspace  DEVICE memory of at least kda_chunk_fwd_host_workspace_size(B, H, K,
 *              V, segment) bytes, 256-byte aligned: the state, two buffers of each
 *              tensor's segment, the small parameters.  Owned by the caller; in use
 *              until `stream` reaches the end of the call.
 *   stream     the caller's stream: the kernels run on it, the copies on two streams
 *              the call creates and destroys, and `stream` waits for the last copy, so
 *              the outputs are in host memory once `stream` has completed
 *              (cudaStreamSynchronize).  The host buffers must stay valid until then.
 * Other arguments and errors as kda_chunk_fwd.
 */
size_t kda_chunk_fwd_host_workspace_size(int B, int H, int K, int V, int segment);

kda_status kda_chunk_fwd_host(const void *q, const void *k, const void *v, kda_dtype qkv_dtype, const float *g,
                              const float *beta, const float *initial_state, float *final_state, void *o,
                              kda_dtype o_dtype, int B, int T, int H, int K, int V, int chunk, float scale,
                              int use_qk_l2norm, const void *gate, kda_dtype gate_dtype, const float *norm_w,
                              float eps, void *y, int segment, void *workspace, size_t workspace_bytes, int mode,
                              void *stream);

kda_status kda_chunk_fwd_logits_host(const void *q, const void *k, const void *v, kda_dtype qkv_dtype,
                                     const void *g_logits, kda_dtype g_logits_dtype, const float *A_log,
                                     const float *dt_bias, float g_lower_bound, const void *beta_logits,
                                     kda_dtype beta_logits_dtype, const float *initial_state, float *final_state,
                                     void *o, kda_dtype o_dtype, int B, int T, int H, int K, int V, int chunk,
                                     float scale, int use_qk_l2norm, const void *gate, kda_dtype gate_dtype,
                                     const float *norm_w, float eps, void *y, int segment, void *workspace,
                                     size_t workspace_bytes, int mode, void *stream);

/*
 * kda_recurrent_fwd -- the token-by-token form over T tokens (fp32 arithmetic).
 *
 * Pages: nnterp "Kimi-Linear" section 03 "Loading" (the token-by-token kernel;
 * the per-token `states` readout needs it) and section 02 (`state` / `states`
 * [batch seq heads key_dim value_dim]).
 *
 * Same arguments and layouts as kda_chunk_fwd, without chunk and mode, plus
 *   states [B, T, H, K, V] float or NULL: the state after every token (varlen:
 *          [1, T, H, K, V] indexed by packed token).
 */
kda_status kda_recurrent_fwd(const void *q, const void *k, const void *v, kda_dtype qkv_dtype,
                             const float *g, const float *beta, const float *initial_state,
                             float *final_state, void *o, kda_dtype o_dtype, float *states,
                             const int32_t *cu_seqlens, const int32_t *cu_seqlens_host,
                             int n_seqs, int B, int T, int H, int K, int V, float scale,
                             int use_qk_l2norm, const void *gate, kda_dtype gate_dtype,
                             const float *norm_w, float eps, void *y, void *stream);

/*
 * kda_recurrent_step -- one decode token per sequence, gated norm fused.
 *
 * Pages: nnterp "Kimi-Linear" section 03 "Loading" (a decode step runs the
 * token-by-token kernel); Kimi-K3 atlas "gate-project (decode, P = 1000)"
 * (decode shapes [B, 96, 1, 128] in, [B, 1, 12288] after the flatten).
 *
 *   q, k  [B, H, K] qkv_dtype     v [B, H, V] qkv_dtype
 *   g     [B, H, K] float         beta [B, H] float
 *   state_in  [B, H, K, V] float or NULL (zero state)
 *   state_out [B, H, K, V] float; may be the same buffer as state_in (in place)
 *   o     [B, H, V] o_dtype or NULL when y is given
 *   gate  [B, H, V] gate_dtype or NULL; norm_w [V]; eps; y [B, H * V] o_dtype
 * Supported K, V: 32, 64, 128.
 */
kda_status kda_recurrent_step(const void *q, const void *k, const void *v, kda_dtype qkv_dtype,
                              const float *g, const float *beta, const float *state_in,
                              float *state_out, void *o, kda_dtype o_dtype, int B, int H, int K,
                              int V, float scale, int use_qk_l2norm, const void *gate,
                              kda_dtype gate_dtype, const float *norm_w, float eps, void *y,
                              void *stream);

/*
 * kda_recurrent_step_logits -- kda_recurrent_step with g and beta computed from
 * their logits, as kda_chunk_fwd_logits defines them:
 *   g_logits [B, H, K] g_logits_dtype, A_log [H], dt_bias [H, K] or NULL,
 *   g_lower_bound, beta_logits [B, H] beta_logits_dtype.
 */
kda_status kda_recurrent_step_logits(const void *q, const void *k, const void *v, kda_dtype qkv_dtype,
                                     const void *g_logits, kda_dtype g_logits_dtype, const float *A_log,
                                     const float *dt_bias, float g_lower_bound, const void *beta_logits,
                                     kda_dtype beta_logits_dtype, const float *state_in, float *state_out,
                                     void *o, kda_dtype o_dtype, int B, int H, int K, int V, float scale,
                                     int use_qk_l2norm, const void *gate, kda_dtype gate_dtype,
                                     const float *norm_w, float eps, void *y, void *stream);

/*
 * kda_recurrent_step_conv -- the decode step with the q, k and v short
 * convolutions (+ SiLU) fused ahead of it, in one kernel.
 *
 * Pages: nnterp encyclopedia "Kimi-Linear", section 03 "Kimi Delta Attention
 * decays each key channel" (a width-4 convolution before the delta rule, whose
 * last inputs are carried outside the recurrent state) and section "Printout"
 * (depthwise Conv1d, kernel 4, padding 3, no bias); Kimi-K3 atlas "gate-project
 * (decode, P = 1000)", section "Code" (q_conv1d, k_conv1d, v_conv1d =
 * ShortConvolution(..., activation='silu') applied to the projections).
 *
 * As kda_recurrent_step (or kda_recurrent_step_logits: give exactly one of the
 * pairs g, beta / g_logits, beta_logits with A_log; the other pointers NULL), but
 *   q, k  [B, H, K] qkv_dtype, v [B, H, V] qkv_dtype are the RAW projections of
 *         this token; the step uses silu(conv(.)) of each, then (optionally) the
 *         L2 norm of q and k, as the layer does.
 *   conv_weight[f]    [H*128, W] float: f = 0 for q, 1 for k, 2 for v (the Conv1d
 *                     weight [D, 1, W] without its middle axis); no bias.
 *   conv_state_in[f]  [B, W-1, H*128] float: the W-1 raw inputs before this token,
 *                     oldest first, as kda_short_conv_fwd keeps them; the array
 *                     pointer NULL (or all three entries NULL) = zero history.
 *   conv_state_out[f] [B, W-1, H*128] float, required: the new history (the old
 *                     one shifted by this token).  Each may be conv_state_in[f]
 *                     itself (in place); no other overlap is allowed.
 * conv_weight, conv_state_in and conv_state_out are HOST arrays of three device
 * pointers, read during the call only.  The convolution output stays in fp32 in
 * the kernel (no rounding to qkv_dtype between the two steps).  Supported: K = V =
 * 128, W in {2, 3, 4}; other shapes return KDA_ERR_UNSUPPORTED.  Returns a kda_status.
 */
kda_status kda_recurrent_step_conv(const void *q, const void *k, const void *v, kda_dtype qkv_dtype,
                                   const float *const conv_weight[3], int W,
                                   const float *const conv_state_in[3], float *const conv_state_out[3],
                                   const float *g, const float *beta,
                                   const void *g_logits, kda_dtype g_logits_dtype, const float *A_log,
                                   const float *dt_bias, float g_lower_bound, const void *beta_logits,
                                   kda_dtype beta_logits_dtype, const float *state_in, float *state_out,
                                   void *o, kda_dtype o_dtype, int B, int H, int K, int V, float scale,
                                   int use_qk_l2norm, const void *gate, kda_dtype gate_dtype,
                                   const float *norm_w, float eps, void *y, void *stream);

/*
 * kda_gated_rmsnorm -- the head-wise sigmoid-gated RMSNorm on its own.
 *
 * Page: Kimi-K3 atlas "gate-project (decode, P = 1000)", sections "Parameters"
 * and "Code".
 *   o    [rows, H, V] o_dtype       gate [rows, H, V] gate_dtype
 *   w    [V] float                  y    [rows, H * V] y_dtype
 *   y = o / sqrt(mean_v(o^2) + eps) * w * sigmoid(gate); rows may be 0.
 * Supported V: 32, 64, 128.
 */
kda_status kda_gated_rmsnorm(const void *o, kda_dtype o_dtype, const void *gate,
                             kda_dtype gate_dtype, const float *w, float eps, void *y,
                             kda_dtype y_dtype, int64_t rows, int H, int V, void *stream);

/*
 * kda_short_conv_fwd -- causal depthwise short convolution along the sequence,
 * with an optional SiLU: the preprocessing of q, k and v before the delta rule.
 *
 * Pages: nnterp encyclopedia "Kimi-Linear", section "Printout" (the layer's conv1d
 * is Conv1d(12288, 12288, kernel_size=(4,), padding=(3,), groups=12288,
 * bias=False): one filter per channel, padded by 3 before the first token, the
 * first T outputs kept); Kimi-K3 atlas "gate-project (decode, P = 1000)", section
 * "Code" (q_conv1d, k_conv1d, v_conv1d = ShortConvolution(hidden_size,
 * kernel_size=short_conv_kernel_size = 4, activation='silu')).
 *
 *   y[t][c] = act( bias[c] + sum_{w<W} weight[c][w] * x[t - (W-1) + w][c] )
 *
 * Positions before a sequence read its conv state (the W-1 inputs before it,
 * oldest first) or zero; act is SiLU (z / (1 + e^-z)) when activation = 1, the
 * identity when 0.
 *
 * Dense mode (cu_seqlens == NULL): N = B sequences of T tokens.
 *   x       [B, T, D] x_dtype      y [B, T, D] y_dtype (must not overlap x)
 *   weight  [D, W] float (the Conv1d weight [D, 1, W] without its middle axis)
 *   bias    [D] float or NULL
 *   conv_state_in  [N, W-1, D] float or NULL (zero history)
 *   conv_state_out [N, W-1, D] float or NULL: the last W-1 inputs of each
 *                  sequence, oldest first (a sequence shorter than W-1 keeps part
 *                  of its old state).  It may be the same buffer as
 *                  conv_state_in only for a decode step (dense, T = 1); otherwise
 *                  the two must not overlap.
 * Varlen mode: as kda_chunk_fwd (B = 1, T packed, cu_seqlens device int32
 *   [n_seqs + 1], optional host copy cu_seqlens_host, which is then checked).
 * A decode step is T = 1 with both states given.  Supported: W in {2, 3, 4},
 * D a multiple of 8, B * T <= INT32_MAX.  Returns a kda_status.
 */
kda_status kda_short_conv_fwd(const void *x, kda_dtype x_dtype, const float *weight, const float *bias,
                              const float *conv_state_in, float *conv_state_out, void *y,
                              kda_dtype y_dtype, const int32_t *cu_seqlens,
                              const int32_t *cu_seqlens_host, int n_seqs, int B, int T, int D, int W,
                              int activation, void *stream);

/*
 * kda_o_proj -- the layer's output projection applied to the gated-norm output y.
 *
 * Page: Kimi-K3 atlas "gate-project (decode, P = 1000)", sections "Parameters"
 * (output projection: 88,080,384 weights = 12288 inputs x 7168 outputs) and "Code"
 * (o = o_proj(o) after o_norm and the heads flattened to heads * head_dim).
 *
 *   out[r][n] = sum_c y[r][c] * w_o[n][c]            (nn.Linear, no bias)
 *
 *   y     [rows, in_features] bf16 (the y of kda_chunk_fwd / kda_recurrent_step with a
 *         bf16 output dtype)
 *   w_o   [out_features, in_features] bf16 (the nn.Linear weight layout)
 *   out   [rows, out_features] out_dtype; must not overlap y or w_o
 * A dense GEMM on the tensor cores (this library's own tcgen05 kernel, bf16 operands,
 * fp32 accumulation, one rounding to out_dtype).  in_features must be a multiple of
 * 64 and out_features of 128 (KDA_ERR_UNSUPPORTED otherwise); rows may be 0.  Keeps
 * no state between calls.
 */
kda_status kda_o_proj(const void *y, const void *w_o, void *out, kda_dtype out_dtype, int64_t rows,
                      int in_features, int out_features, void *stream);

/*
 * Full attention.  The hybrid stacks interleave KDA layers with layers of full attention
 * (nnterp encyclopedia "Kimi-Linear", section 03: one block in four; Kimi-K3 atlas
 * "final-block-state", the layer-type schedule).  The four calls below serve such layers
 * of hybrid stacks with grouped heads: positions, a paged 8-bit key/value cache, the decode
 * step's attention over that cache and the prompt's attention.  The pages give no kernels
 * for these; the formulas are stated here.  Of Kimi-Linear's own full-attention layers,
 * which have no rotary positions, keys of 192 channels and values of 128, only the
 * prompt's attention takes the widths; the cache has one width, 64 or 128, for both.
 *
 * Rows of q, k and v may lie a stride apart (slices of a fused projection): a stride is the
 * distance of one token's row to the next in elements, at least heads * dim and a multiple
 * of 16 bytes; within a row the heads are dense.  Index arrays and scales need only the
 * alignment of their type, so slices of larger arrays are used as they lie.
 */

typedef enum kda_rotary_layout {
    KDA_ROTARY_HALF = 0,        /* pairs (i, i + rotary_dim / 2) */
    KDA_ROTARY_INTERLEAVED = 1  /* pairs (2i, 2i + 1) */
} kda_rotary_layout;

/*
 * kda_rotary -- rotary positions: the first rotary_dim channels of every head turned in
 * pairs (a, b) by the angle w = positions[t] * inv_freq[i],
 *     (a, b) -> magnitude * (a cos w - b sin w, a sin w + b cos w),
 * the other channels copied.
 *
 *   x, out     [tokens, heads, dim] dtype, x_stride / out_stride apart; out may be x itself
 *              (same pointer, same stride), no other overlap
 *   positions  [tokens] int32, any values: angles are formed and reduced in integers, within
 *              positions * 2^-64 turns; cos and sin carry fp32's relative precision
 *   inv_freq   [rotary_dim / 2] double, finite, radians per position (scaled for long contexts by
 *              the caller), magnitude the factor that such a scaling puts on the rotated part
 *   inverse    1: the transposed rotation (angles negated), which undoes a rotation of
 *              magnitude 1 and is the gradient of any
 * rotary_dim a multiple of 16, at most dim; dim a multiple of 8, at most 256
 * (KDA_ERR_UNSUPPORTED otherwise).  tokens may be 0.
 */
kda_status kda_rotary(const void *x, kda_dtype dtype, int64_t x_stride, const int32_t *positions,
                      const double *inv_freq, float magnitude, int rotary_dim, int layout, int inverse, void *out,
                      int64_t out_stride, int64_t tokens, int heads, int dim, void *stream);

/*
 * kda_kv_append -- appends new tokens' keys and values to a paged 8-bit cache, the keys
 * rotated on the way, and rotates the same tokens' queries.
 *
 * The cache: k_cache, v_cache [num_pages, kv_heads, page_size, dim] e4m3 codes, k_scale,
 * v_scale [num_pages, kv_heads] float; a value is code * scale.  Scales are powers of two
 * 2^e, -100 <= e <= 100, the smallest that holds a block's largest finite value within 448.
 * Token j of sequence n lies at place j % page_size of page block_table[n][j / page_size].
 * A page whose place 0 is written by the call gets a new scale; a page that holds earlier
 * tokens keeps its scale or, if a new value needs it, takes a larger one, its codes then
 * moving to it (an exponent shift, rounded where it ends among the subnormals).  Places
 * behind the last token are left as they are.  Infinities and NaN are stored as NaN and
 * do not count for the scale.
 *
 *   k, v         [tokens, kv_heads, dim] bf16, k_stride / v_stride apart
 *   context_lens [n_seqs] int32: tokens in the cache before the call (not changed)
 *   cu_seqlens   [n_seqs + 1] int32: sequence n's new tokens are rows
 *                [cu_seqlens[n], cu_seqlens[n + 1]) (clamped to [0, tokens]); NULL: one new
 *                token per sequence, tokens == n_seqs
 *   block_table  [n_seqs, max_blocks] int32.  A token whose page is negative, not below
 *                num_pages, or behind the table is not stored (padding).
 *   inv_freq     as kda_rotary, the position being the token's place in its sequence;
 *                NULL: nothing is rotated (rotary_dim 0)
 *   q, q_out     [tokens, q_heads, dim] bf16, q q_stride apart, q_out dense; both or neither
 *   k_out        [tokens, kv_heads, dim] bf16, dense, or NULL: the rotated keys
 * Rows of q_out and k_out that belong to no sequence are left as they are.
 * dim 64 or 128; page_size 16, 32, 64 or 128; at most 65535 sequences and 65535 cache heads;
 * num_pages * kv_heads * page_size below 2^31 - 256 (KDA_ERR_UNSUPPORTED otherwise).
 * No page may be written for two sequences, or for two places of one, in one call (pages that
 * are only read, full ones of a shared beginning, may stand in several rows of block_table).
 */
kda_status kda_kv_append(const void *k, int64_t k_stride, const void *v, int64_t v_stride, int64_t tokens,
                         int kv_heads, int dim, void *k_cache, void *v_cache, float *k_scale, float *v_scale,
                         int num_pages, int page_size, const int32_t *block_table, int max_blocks,
                         const int32_t *context_lens, const int32_t *cu_seqlens, int n_seqs, const double *inv_freq,
                         float magnitude, int rotary_dim, int layout, const void *q, int64_t q_stride, int q_heads,
                         void *q_out, void *k_out, void *stream);

/*
 * kda_attn_decode -- one query token per sequence over the paged 8-bit cache.
 *
 *     o[n][i] = sum_j softmax_j(scale * q[n][i] . K_j) V_j,   j < seq_lens[n],
 * K_j and V_j the cached (code * scale) rows of head i / (q_heads / kv_heads).
 *
 *   q         [n_seqs, q_heads, dim] bf16, q_stride apart; q_heads a multiple of kv_heads
 *   cache     as kda_kv_append; scales may be any positive floats, value scales from 2^-126 to
 *             2^120
 *   seq_lens  [n_seqs] int32: tokens to attend to (with the new one), clamped to
 *             [0, max_blocks * page_size].  0 gives a zero row and lse -INFINITY.
 *   o         [n_seqs, q_heads, dim] o_dtype
 *   lse       [n_seqs, q_heads] float or NULL: log(sum_j e^(scale q . K_j))
 *   workspace device scratch of kda_attn_decode_workspace_size(n_seqs, q_heads, kv_heads,
 *             dim, max_blocks * page_size) bytes, 16-byte aligned; calls that may overlap on
 *             the GPU (two captured graphs among them) need workspaces of their own.  Where the
 *             size is 0 it may be NULL.
 * Scores, their maxima and all sums are fp32; the weights are rounded to f16 for the product with
 * the values: a relative error of 2^-12 each, of the largest and the smallest alike, or in all at
 * most 2^-9 (half a step of bf16) of the largest sum of weights times |values| among 8 or 16
 * channels, which is reached only by codes of 448 throughout.
 * What lies in a page behind a sequence's last token is not read into the result, whatever
 * it is.  A sequence with a page number out of [0, num_pages) gives NaN rows.
 * dim 64 or 128; page_size 16, 32, 64 or 128; limits as kda_kv_append.  Results do not
 * depend on timing.  Whether sequences are cut into pieces, which takes the workspace, goes by
 * the block table's width, not by the lengths on the device: a table no wider than the
 * sequences need serves short ones faster, in other last bits.
 */
size_t kda_attn_decode_workspace_size(int n_seqs, int q_heads, int kv_heads, int dim, int64_t max_tokens);

kda_status kda_attn_decode(const void *q, int64_t q_stride, const void *k_cache, const void *v_cache,
                           const float *k_scale, const float *v_scale, int num_pages, int page_size,
                           const int32_t *block_table, int max_blocks, const int32_t *seq_lens, int n_seqs,
                           int q_heads, int kv_heads, int dim, float scale, void *o, kda_dtype o_dtype, float *lse,
                           void *workspace, size_t workspace_bytes, void *stream);

/*
 * kda_attn_prompt -- causal attention over whole prompts, on the tensor cores.
 *
 *     o[i] = sum_{j < seen_i} softmax_j(scale * q_i . k_j) v_j,   seen_i = i + 1 + (keys - queries),
 * for every query row i of a sequence; query head h reads key/value head
 * h / (q_heads / kv_heads).  A sequence with more keys than queries continues a context whose
 * rows come first; a row that sees nothing (more queries than keys) gives zero and lse
 * -INFINITY.
 *
 *   q   [q_rows, q_heads, dim], k [k_rows, kv_heads, dim], v [k_rows, kv_heads, dim_v], bf16,
 *       q_stride / k_stride / v_stride apart
 *   o   [q_rows, q_heads, dim_v] o_dtype         lse [q_rows, q_heads] float or NULL:
 *       log(sum_j e^(scale q_i . k_j))
 *   cu_seqlens   [n_seqs + 1] int32: sequence n's queries are rows
 *       [cu_seqlens[n], cu_seqlens[n + 1]) (clamped to [0, q_rows]); rows of no sequence are
 *       left as they are.  NULL: n_seqs sequences of q_rows / n_seqs rows each.
 *   cu_seqlens_k [n_seqs + 1] int32: the same for the keys.  NULL: as cu_seqlens where that is
 *       given (k_rows == q_rows), else n_seqs sequences of k_rows / n_seqs rows.
 * (dim, dim_v) one of (64, 64), (128, 128), (192, 128) (KDA_ERR_UNSUPPORTED otherwise); q_heads a
 * multiple of kv_heads; at most 2^30 rows, 65535 heads and 16384 sequences; scale finite and not 0.  Nothing a row does not see enters its result,
 * be it infinite or NaN.  The weights are rounded to bf16 for the product with v.
 *
 *   workspace    device scratch of kda_attn_prompt_workspace_size(...) bytes, 16-byte aligned, for
 *                this call alone, or NULL.  With few rows and heads for the GPU's SMs the size is
 *                not 0, and a call with the workspace divides each row's keys among several
 *                CTAs and joins their sums (rounded differently than in one go).
 */
size_t kda_attn_prompt_workspace_size(int64_t q_rows, int64_t k_rows, int q_heads, int kv_heads, int dim_v, int n_seqs);

kda_status kda_attn_prompt(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                           int64_t v_stride, int64_t q_rows, int64_t k_rows, int q_heads, int kv_heads, int dim,
                           int dim_v, const int32_t *cu_seqlens, const int32_t *cu_seqlens_k, int n_seqs, float scale,
                           void *o, kda_dtype o_dtype, float *lse, void *workspace, size_t workspace_bytes,
                           void *stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H */
