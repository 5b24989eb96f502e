/*
 * gdn2.h -- C ABI of the MI355X (gfx950) Gated DeltaNet-2 core library, libgdn2.so.
 *
 * The method (burn-gdn2 0.1.5 docs page, section "Architecture"): per sequence and per
 * value head, a matrix state S in R^{d_k x d_v} follows
 *
 *     S_t = (I - k_t (b_t . k_t)^T) diag(alpha_t) S_{t-1} + k_t (w_t . v_t)^T
 *     o_t = q_t^T S_t
 *
 * with alpha_t the channel-wise decay and b_t the erase gate on the key axis, and w_t the
 * write gate on the value axis. The same page names two ways to run it, and this library
 * exports one call for each:
 *   - gdn2_chunk_fwd       the chunked WY-decomposition forward ("Chunk" mode, training and
 *                          prefill; chunk_size defaults to 64 on that page);
 *   - gdn2_recurrent_step  one fused token-by-token step ("FusedRecurrent" mode, decode),
 *                          which reads and writes a persistent state in place as the
 *                          GDN decode verify page (LocalAI mirror), section 2, describes.
 * Around them (each declared below with its own description):
 *   - gdn2_recurrent_fwd        several tokens per call against a pool of fp32 or bf16
 *                               states, with optional fused prologue and epilogue;
 *   - gdn2_chunk_bwd, gdn2_chunk_bwd_states
 *                               the gradients of the chunked forward (recomputing the
 *                               chunk states, or from those a training forward saved);
 *   - gdn2_map_gates, gdn2_map_gates_bwd
 *                               the inputs of other delta-rule variants (KDA, GDN,
 *                               FG2-GDN, FG2-GDN+) mapped onto these, and their gradients
 *                               mapped back;
 *   - gdn2_chunk_fwd_noalloc    the chunked forward on a static device workspace, for
 *                               callers that cannot allocate;
 *   - gdn2_short_conv_fwd, gdn2_short_conv_bwd, gdn2_short_conv_step
 *                               the short causal convolution before the recurrence, over
 *                               prompts, its gradients, and for single tokens;
 *   - gdn2_selective_scan_fwd, gdn2_selective_scan_bwd, gdn2_selective_scan_step
 *                               the selective state space scan, the other linear recurrence
 *                               of hybrid layers (a decay per channel and state), over
 *                               prompts, its gradients, and for single tokens;
 *   - gdn2_block_norm_fwd, gdn2_block_norm_bwd
 *                               the norms after and before a block, fused with its gate, the
 *                               residual and its scale, and their gradients;
 *   - gdn2_qk_rotary_fwd, gdn2_qk_rotary_bwd, gdn2_qk_rotary_append
 *                               the attention layer that hybrid stacks put beside the recurrent
 *                               ones: norms of queries and keys per head with the rotation by
 *                               position, their gradients, and into the pages of a cache;
 *   - gdn2_paged_attention_step the attention of new tokens over that cache;
 *   - gdn2_pool_copy            slots of pools copied: pages of a cache, states of sequences.
 * Calls added since version 9 of the ABI change none of its calls, so the number stays.
 *
 * Conventions (the pages are silent on these; this is the reading the library implements):
 *   - o_t reads the state AFTER the update of token t.
 *   - The decay argument carries log(alpha) <= 0, in the input dtype; the kernels take exp.
 *   - No query scaling (a caller wanting 1/sqrt(d_k) pre-scales q; o is linear in q).
 *   - Grouped value attention: value head h reads key head h / (h_v / h_k)
 *     (burn-gdn2 "num_v_heads"; the llama.cpp notes' 48 value heads over 16 key groups).
 *   - The negative-eigenvalue option of burn-gdn2 (allow_neg_eigval, "b x 2") is the
 *     caller's b in (0,2); the library has no flag for it.
 *
 * Layouts (all contiguous, last dimension fastest):
 *   q, k          [B, T, h_k, d_k]      input dtype
 *   v, w, o       [B, T, h_v, d_v]      input dtype (o is written in the input dtype)
 *   log_alpha, b  [B, T, h_v, d_k]      input dtype
 *   S0, S_T, S    [N, h_v, d_k, d_v]    fp32 always, d_v fastest
 * A packed (variable-length) batch uses B = 1, T = total tokens and cu_seqlens (int32,
 * N + 1 offsets, device memory): sequence n owns tokens cu_seqlens[n] .. cu_seqlens[n+1]-1.
 * Without cu_seqlens the batch is dense: N = B sequences of T tokens each.
 *
 * Ownership: the caller allocates every buffer (inputs, outputs, workspace, state). The
 * library allocates no device memory and keeps no state between calls apart from the
 * thread-local error message.
 *
 * Streams: every call only enqueues work on `stream` (a hipStream_t; NULL is the default
 * stream) and returns without synchronising. No call reads device memory on the host.
 * The work enqueued is kernel launches only (no allocation, copy, fill or host
 * synchronisation), so a caller may capture the calls into a HIP graph and replay it; a
 * replay reads and writes the buffers given at capture time.
 *
 * Errors: arguments are validated on the host before anything is enqueued; a failed check
 * returns a status code and launches nothing. A failed launch returns GDN2_ERR_HIP. A short
 * message for the last failure of the calling thread is available from gdn2_last_error().
 * Device-side contents (cu_seqlens values, NaN/Inf in the data) are not checked: NaN and
 * Inf propagate into the affected (sequence, head) outputs.
 */
#ifndef GDN2_H
#define GDN2_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define GDN2_ABI_VERSION 9

typedef enum gdn2_status {
    GDN2_OK = 0,
    GDN2_ERR_NULL_ARG = 1,      /* a required pointer is NULL */
    GDN2_ERR_BAD_SHAPE = 2,     /* a dimension is out of range or inconsistent */
    GDN2_ERR_UNSUPPORTED = 3,   /* valid but not built: head dims, chunk size, dtype */
    GDN2_ERR_WORKSPACE = 4,     /* workspace missing or smaller than required */
    GDN2_ERR_HIP = 5            /* the HIP runtime reported an error */
} gdn2_status;

typedef enum gdn2_dtype {
    GDN2_F32 = 0,               /* fp32 inputs and o; fp32 arithmetic throughout */
    GDN2_BF16 = 1               /* bf16 inputs and o; bf16 matrix-core operands, fp32
                                   accumulation, fp32 state */
} gdn2_dtype;

typedef enum gdn2_state_dtype {
    GDN2_STATE_F32 = 0,         /* fp32 recurrent state */
    GDN2_STATE_BF16 = 1         /* bf16 recurrent state: widened to fp32 for the update inside
                                   a call, rounded to nearest even when written back */
} gdn2_state_dtype;

/*
 * Optional fusions of the stages the burn-gdn2 page (section "Architecture") draws around
 * the recurrence: the L2-Norm of q and k before it, and the Gated RMS Norm with a SiLU
 * gate after it (its Configuration table gives norm_eps = 1e-5). Pass NULL for none.
 *
 *   qk_l2norm    nonzero: every q and k vector (one token of one key head, d_k values) is
 *                replaced by x / sqrt(sum_c x_c^2 + l2norm_eps) before it is used
 *   l2norm_eps   >= 0 (1e-6 is a usual choice; with 0 an all-zero vector gives NaN)
 *   gate         NULL, or a device tensor shaped like o ([.., h_v, d_v], input dtype): the
 *                output becomes  o / sqrt(mean_c o_c^2 + norm_eps) * norm_weight * silu(gate)
 *                per (token, value head), silu(g) = g / (1 + exp(-g)); must not alias o
 *   norm_weight  device fp32 [d_v], required with a gate (shared by all value heads)
 *   norm_eps     >= 0
 *
 * gdn2_recurrent_fwd only: the short causal depthwise convolution that the same diagram
 * puts before the L2-Norm (burn-gdn2 use_short_conv; the GDN decode verify page, section 1,
 * give its kernel width 4, and section 2 its state of the last 3 inputs per channel, kept
 * in the recurrent cache and read and written back every step). The convolved channels are
 * q, k and v, C = 2 h_k d_k + h_v d_v of them in that order (q of key head 0..h_k-1, then
 * k likewise, then v of value head 0..h_v-1, each head's d values contiguous):
 *   conv_weight  NULL: no convolution. Else device fp32 [C][4]; tap 3 multiplies the
 *                current token, tap 0 the input three tokens back
 *   conv_state   device fp32 [num_slots][3][C], the last three inputs of each channel
 *                (oldest first), on the same slots as the recurrent state; read and updated
 *                in place
 *   conv_silu    nonzero: y = silu(conv(x)); zero: y = conv(x)
 * The convolved q and k are what the L2-norm (if on) and the recurrence see.
 *
 *   gate_mode    0: b and w are the GDN-2 gates. A gdn2_gate_mode (see gdn2_map_gates):
 *                the call runs that variant with its gate mapping fused into the kernels,
 *                reading the variant's own gates (no mapping pass, no mapped tensors):
 *                  GDN2_GATES_KDA       b = beta [.., h_v]; w unused (may be NULL)
 *                  GDN2_GATES_GDN       as KDA, and log_alpha [.., h_v] (one per head)
 *                  GDN2_GATES_FG2       b = beta [.., h_v, d_k], d_v = d_k; w unused
 *                  GDN2_GATES_FG2_PLUS  b = beta [.., h_v, d_k], w = beta_v [.., h_v, d_v]
 *                The FG2 modes scale the keys by sqrt(beta) inside the kernels, so they
 *                take neither qk_l2norm nor the short convolution (GDN2_ERR_UNSUPPORTED).
 *
 * gdn2_chunk_fwd only (the recurrent calls return GDN2_ERR_UNSUPPORTED when it is set):
 *   chunk_states NULL, or device fp32 [num_chunks][h_v][d_k][d_v]: the state entering
 *                every chunk of every sequence, the quantity the chunked form hands from one
 *                chunk to the next (burn-gdn2 docs page, "Architecture", Chunk WY mode): a
 *                training backward recomputes each chunk from it, and a serving cache can
 *                resume any sequence at a chunk boundary from it. Chunk j of sequence n is
 *                entry n * ceil(T / chunk_size) + j of a dense batch, and entry
 *                sum_{m < n} ceil(len_m / chunk_size) + j of a packed one (len_m =
 *                cu_seqlens[m+1] - cu_seqlens[m]); entry j holds the state after the first
 *                j * chunk_size tokens of the sequence (entry 0: S0, or zeros). The caller
 *                owns it; it must not overlap any input, output or the workspace.
 */
typedef struct gdn2_fusion {
    int32_t qk_l2norm;
    float l2norm_eps;
    const void *gate;
    const float *norm_weight;
    float norm_eps;
    const float *conv_weight;
    float *conv_state;
    int32_t conv_silu;
    int32_t gate_mode;
    float *chunk_states;
} gdn2_fusion;

typedef struct gdn2_dims {
    int32_t batch;      /* dense: number of sequences B. packed: must be 1.
                           recurrent step: number of sequences N. */
    int32_t seqlen;     /* dense: tokens per sequence T (>= 0). packed: total tokens.
                           recurrent step: must be 1. */
    int32_t num_seqs;   /* packed: N, the number of sequences (cu_seqlens has N+1 entries).
                           dense and recurrent step: ignored. */
    int32_t h_k;        /* key/query heads (>= 1) */
    int32_t h_v;        /* value heads, a multiple of h_k */
    int32_t d_k;        /* key head dim: 64 or 128 */
    int32_t d_v;        /* value head dim: 64 or 128 */
    int32_t dtype;      /* gdn2_dtype */
} gdn2_dims;

/* Library ABI version (GDN2_ABI_VERSION of the build). */
int32_t gdn2_abi_version(void);

/* Static text for a status code. */
const char *gdn2_status_string(int32_t status);

/* Message of the last failing call made by this thread ("" if none). */
const char *gdn2_last_error(void);

/*
 * Bytes of device workspace gdn2_chunk_fwd needs for these dims and chunk size, or 0 if
 * the dims or the chunk size are invalid. For a packed batch the size uses the upper bound
 * ceil(T / chunk_size) + N on the number of chunks, so it depends only on the dims.
 */
size_t gdn2_chunk_fwd_workspace_bytes(const gdn2_dims *dims, int32_t chunk_size);

/*
 * Chunked WY forward over a whole batch (burn-gdn2 docs page, "Chunk" mode of the
 * Architecture section; chunk_size as in its Configuration table).
 *
 *   q, k, v, log_alpha, b, w   device inputs in the layouts above (dims->dtype)
 *   S0          device fp32 [N, h_v, d_k, d_v] initial states, or NULL for zero states
 *   cu_seqlens  device int32 [N+1] for a packed batch, or NULL for a dense batch.
 *               Precondition (not checked on the device): cu_seqlens[0] = 0,
 *               non-decreasing, cu_seqlens[N] = T. Zero-length sequences are allowed and
 *               return S_T = S0 (or zeros).
 *   chunk_size  32, 64 or 128 tokens per chunk of the WY form (results do not depend on
 *               it beyond rounding). Every dtype and head-dim pair is built at every size.
 *   o           device output [B, T, h_v, d_v] in the input dtype; must not alias inputs
 *   S_T         device fp32 [N, h_v, d_k, d_v] final states, or NULL to skip them. S_T may
 *               be the same buffer as S0 (in-place continuation); no other aliasing.
 *   workspace   device buffer of at least gdn2_chunk_fwd_workspace_bytes() bytes, 256-byte
 *               aligned; its contents on entry are ignored and are clobbered.
 *   fusion      NULL, or the optional q/k L2-norm and gated output norm (gdn2_fusion);
 *               the gate is [B, T, h_v, d_v]. A short convolution is not built for this
 *               call (GDN2_ERR_UNSUPPORTED)
 *   stream      hipStream_t the work is enqueued on
 * Returns GDN2_OK or an error status (nothing is enqueued on a validation error).
 */
gdn2_status gdn2_chunk_fwd(const void *q, const void *k, const void *v,
                           const void *log_alpha, const void *b, const void *w,
                           const float *S0, const int32_t *cu_seqlens, int32_t chunk_size,
                           void *o, float *S_T, const gdn2_dims *dims,
                           void *workspace, size_t workspace_bytes,
                           const gdn2_fusion *fusion, void *stream);

/*
 * For callers that cannot allocate device memory: code under HIP graph capture, tight
 * serving loops, harnesses that forbid hipMalloc. gdn2_chunk_fwd with the same arguments
 * minus the workspace, which comes instead from a static device array of
 * GDN2_STATIC_WORKSPACE_BYTES (128 MiB) that the library holds on every GPU it runs on
 * until the process ends. The call allocates nothing (no hipMalloc, no allocating library
 * routine); the caller still allocates the inputs and outputs.
 *   - Calls whose gdn2_chunk_fwd_workspace_bytes() exceeds GDN2_STATIC_WORKSPACE_BYTES
 *     return GDN2_ERR_WORKSPACE and enqueue nothing (128 MiB holds, for instance, a bf16
 *     batch of 4,096 tokens x 16 heads at d = 128 with chunk_size 64).
 *   - Every call on one GPU uses that GPU's one array, and the array keeps the last call's
 *     contents (none of which a later call reads). Calls that can overlap in time on one
 *     GPU -- issued to different streams with no ordering between them -- race on the
 *     array and give undefined results; order them on one stream (or with events).
 *   - The device is the stream's (the current device for a NULL stream). The first call on
 *     a device looks the array's address up once (hipGetSymbolAddress); later calls reuse it.
 * Results are those of gdn2_chunk_fwd (the same kernels run).
 */
#define GDN2_STATIC_WORKSPACE_BYTES ((size_t)128 << 20)

gdn2_status gdn2_chunk_fwd_noalloc(const void *q, const void *k, const void *v,
                                   const void *log_alpha, const void *b, const void *w,
                                   const float *S0, const int32_t *cu_seqlens,
                                   int32_t chunk_size, void *o, float *S_T,
                                   const gdn2_dims *dims, const gdn2_fusion *fusion,
                                   void *stream);

/*
 * Bytes of device workspace gdn2_chunk_bwd needs for these dims and chunk size, or 0 if
 * the dims are invalid (same upper bound on the chunks of a packed batch as the forward).
 */
size_t gdn2_chunk_bwd_workspace_bytes(const gdn2_dims *dims, int32_t chunk_size);

/*
 * Gradients of gdn2_chunk_fwd (without fusion options, GDN-2 gates) with respect to every
 * input and the initial state, taken through the chunked form of the burn-gdn2 docs page
 * ("Architecture", Chunk mode; its Chunk WY training path): the forward is re-run to store
 * the state entering every chunk, then one pass runs the state gradient backward over the
 * chunks, and one pass per chunk forms the input gradients. Built for bf16 inputs (bf16
 * matrix-core products, fp32 accumulation) and fp32 inputs (fp32 products) at every
 * supported head-dim pair.
 *
 *   q .. w, S0, cu_seqlens, dims   as for gdn2_chunk_fwd
 *   chunk_size  32, 64 or 128: the chunk size of the forward call whose gradients these are.
 *               The chunked form computes the same function at every chunk size, so the
 *               gradients do not depend on it; all three are computed with 64-token chunks
 *               (the same bits). Other values return GDN2_ERR_UNSUPPORTED.
 *   dO          device [B, T, h_v, d_v] in the input dtype: dL/do
 *   dS_T        device fp32 [N, h_v, d_k, d_v]: dL/dS_T, or NULL for zero
 *   dq, dk      device fp32 [B, T, h_k, d_k]   (value heads that share a key head add up,
 *               with fp32 atomics: when h_v > h_k the summation order, and so the last bits,
 *               may differ between runs; with h_v == h_k they are stored, and every call
 *               gives the same bits)
 *   dv, dw      device fp32 [B, T, h_v, d_v]
 *   dlog_alpha, db   device fp32 [B, T, h_v, d_k]
 *   dS0         device fp32 [N, h_v, d_k, d_v]: dL/dS0 (written also when S0 is NULL)
 *   workspace   at least gdn2_chunk_bwd_workspace_bytes() bytes, 256-byte aligned
 * Outputs must not alias inputs or each other. Every output is overwritten.
 * Returns GDN2_OK or an error status (nothing is enqueued on a validation error).
 */
gdn2_status gdn2_chunk_bwd(const void *q, const void *k, const void *v,
                           const void *log_alpha, const void *b, const void *w,
                           const float *S0, const int32_t *cu_seqlens, int32_t chunk_size,
                           const void *dO, const float *dS_T, float *dq, float *dk, float *dv,
                           float *dw, float *dlog_alpha, float *db, float *dS0,
                           const gdn2_dims *dims, void *workspace, size_t workspace_bytes,
                           void *stream);

/*
 * gdn2_chunk_bwd for a forward that saved the state entering every chunk (its
 * gdn2_fusion.chunk_states, taken with chunk_size 64 on the same inputs, S0 and layout):
 * the chunked form hands exactly that state from one chunk to the next (burn-gdn2 docs page,
 * "Architecture", Chunk WY training path), so the backward uses it instead of re-running
 * the serial pass over the chunks. Gradients equal gdn2_chunk_bwd's (the same bits when no
 * value heads share a key head). chunk_size must be 64 (GDN2_ERR_UNSUPPORTED otherwise);
 * with fp32 inputs the states are recomputed and chunk_states is only checked.
 *
 *   chunk_states  device fp32 [num_chunks][h_v][d_k][d_v], the layout of
 *                 gdn2_fusion.chunk_states; read only; must not alias an output
 *   other arguments, the workspace size and the error behaviour as for gdn2_chunk_bwd
 */
gdn2_status gdn2_chunk_bwd_states(const void *q, const void *k, const void *v,
                                  const void *log_alpha, const void *b, const void *w,
                                  const float *S0, const int32_t *cu_seqlens, int32_t chunk_size,
                                  const float *chunk_states, const void *dO, const float *dS_T,
                                  float *dq, float *dk, float *dv, float *dw, float *dlog_alpha,
                                  float *db, float *dS0, const gdn2_dims *dims, void *workspace,
                                  size_t workspace_bytes, void *stream);

/*
 * One decode step for N sequences, one token each (burn-gdn2 "FusedRecurrent" mode; the
 * GDN decode verify page, section 2, describes the same fused state read-update-write).
 *
 *   q, k          device [N, h_k, d_k]   (dims->batch = N, dims->seqlen = 1)
 *   v, w          device [N, h_v, d_v]
 *   log_alpha, b  device [N, h_v, d_k]
 *   S             device fp32 [N, h_v, d_k, d_v], read and updated in place
 *   o             device [N, h_v, d_v] in the input dtype; must not alias any input or S
 *   stream        hipStream_t
 * Each state is read from memory once and written once.
 */
gdn2_status gdn2_recurrent_step(const void *q, const void *k, const void *v,
                                const void *log_alpha, const void *b, const void *w,
                                float *S, void *o, const gdn2_dims *dims, void *stream);

/*
 * Multi-token recurrent forward against a state cache (burn-gdn2 "FusedRecurrent" mode run
 * over T tokens). The GDN decode verify page (LocalAI mirror) describes, in section 2, the
 * recurrent cache whose slots hold one state per sequence and are read and written back
 * every step, and a fused kernel that keeps its share of a state in registers across the
 * tokens of the call; section 4 names a bf16 state as the way to cut the state traffic.
 * T > 1 serves short multi-token steps (draft tokens of speculative decoding, short
 * prefills) at the state traffic of one step.
 *
 * Sequence n runs tokens 0..T-1 in order, starting from the state in its slot, and the
 * slot holds the state after token T-1 on return. Every state is read from memory once and
 * written once per call, whatever T is.
 *
 *   q, k          device [N, T, h_k, d_k]   (dims->batch = N >= 0, dims->seqlen = T >= 1)
 *   v, w          device [N, T, h_v, d_v]
 *   log_alpha, b  device [N, T, h_v, d_k]   (input dtype dims->dtype for all six)
 *   state         device [num_slots, h_v, d_k, d_v] in state_dtype (gdn2_state_dtype),
 *                 read and updated in place
 *   state_idx     device int32 [N]: the slot of sequence n; or NULL, meaning slot n (then
 *                 num_slots must be >= N). An entry outside [0, num_slots) marks a padding
 *                 sequence: its slot is neither read nor written and its o rows are zeros.
 *                 Precondition (not checked on the device): the valid entries are
 *                 distinct; two sequences on one slot race.
 *   o             device [N, T, h_v, d_v] in the input dtype; must not alias an input or
 *                 the state
 *   fusion        NULL, or the optional short convolution, q/k L2-norm and gated output
 *                 norm (gdn2_fusion); the gate is [N, T, h_v, d_v]. Padding sequences still
 *                 get zero o rows, and their conv state is untouched.
 *   stream        hipStream_t
 * With T = 1, state_idx = NULL and an fp32 state this is gdn2_recurrent_step.
 */
gdn2_status gdn2_recurrent_fwd(const void *q, const void *k, const void *v,
                               const void *log_alpha, const void *b, const void *w,
                               void *state, int32_t state_dtype, const int32_t *state_idx,
                               int32_t num_slots, void *o, const gdn2_dims *dims,
                               const gdn2_fusion *fusion, void *stream);

/*
 * Gate mappings: other members of the gated delta-rule family as GDN-2 inputs. The
 * burn-gdn2 page ("Architecture") introduces the channel-wise b_t and w_t as the
 * replacement of the scalar gate of Kimi Delta Attention; the FG2-GDN page (section 2)
 * writes its update with keys and values scaled by sqrt(beta). Each mode below is exactly
 * GDN-2 with mapped inputs (per value head h, key head h / (h_v / h_k)):
 *
 *   GDN2_GATES_KDA       S = (I - beta k k^T) diag(alpha) S + beta k v^T
 *                        beta  [rows, h_v] (one value per token and value head)
 *                        -> b_out [rows, h_v, d_k] = beta, w_out [rows, h_v, d_v] = beta;
 *                        q, k, v and log_alpha are used as they are
 *   GDN2_GATES_GDN       as KDA with a scalar decay: log_alpha [rows, h_v]
 *                        -> also log_alpha_out [rows, h_v, d_k] = log_alpha
 *   GDN2_GATES_FG2       S = (I - k~ k~^T) diag(alpha) S + k~ v~^T, k~ = sqrt(beta) . k,
 *                        v~ = sqrt(beta) . v; beta [rows, h_v, d_k]; needs d_v = d_k
 *                        -> k_out [rows, h_v, d_k] = k~, v_out [rows, h_v, d_v] = v~,
 *                           b_out = w_out = 1
 *   GDN2_GATES_FG2_PLUS  as FG2 with the erase scale beta [rows, h_v, d_k] on the keys and
 *                        the write scale beta_v [rows, h_v, d_v] on the values:
 *                        S = (I - k~ k~^T) diag(alpha) S + k~ (sqrt(beta_v) . v)^T
 *                        -> k_out = sqrt(beta) . k, b_out = 1, w_out = sqrt(beta_v);
 *                           v is used as it is
 *
 * rows = dims->batch x dims->seqlen tokens in the layout of the call that follows (dense,
 * packed or recurrent); dims is that call's dims. In the FG2 modes k_out is per value head,
 * so the follow-up call takes h_k = h_v, with q_out [rows, h_v, d_k] (q replicated per
 * value head) in place of q; q_out is required when h_v > h_k and may be NULL (q used as it
 * is) when h_v = h_k. All tensors are in dims->dtype. Pointers a mode does not use are
 * ignored. The outputs a mode writes must not alias its inputs or each other. An
 * elementwise pass on `stream` (HBM-bound); nothing else is computed.
 */
typedef enum gdn2_gate_mode {
    GDN2_GATES_KDA = 1,
    GDN2_GATES_FG2 = 2,
    GDN2_GATES_FG2_PLUS = 3,
    GDN2_GATES_GDN = 4
} gdn2_gate_mode;

gdn2_status gdn2_map_gates(int32_t mode, const gdn2_dims *dims, const void *q, const void *k,
                           const void *v, const void *log_alpha, const void *beta,
                           const void *beta_v, void *q_out, void *k_out, void *v_out,
                           void *log_alpha_out, void *b_out, void *w_out, void *stream);

/*
 * Gradients through gdn2_map_gates: the chain rule of its mapping (the mappings are those
 * of gdn2_map_gates, after the burn-gdn2 "Architecture" section and the FG2-GDN summary,
 * section 2). Given the gradients of a loss with respect to the GDN-2 inputs the mapping
 * wrote (for instance from gdn2_chunk_bwd run on them), it writes the gradients with
 * respect to the variant's own inputs. Only the gradients the mapping changes are written;
 * every other gradient of the variant is the mapped one itself:
 *   GDN2_GATES_KDA       dbeta [rows, h_v] = sum over d_k of db_m + sum over d_v of dw_m;
 *                        dq, dk, dv, dlog_alpha are dq_m, dk_m, dv_m, dla_m
 *   GDN2_GATES_GDN       as KDA, and dlog_alpha [rows, h_v] = sum over d_k of dla_m
 *   GDN2_GATES_FG2       dk [rows, h_k, d_k] = sum over the key head's value heads of
 *                        sqrt(beta) . dk_m; dv [rows, h_v, d_v] = sqrt(beta) . dv_m;
 *                        dbeta [rows, h_v, d_k] = (dk_m . k + dv_m . v) / (2 sqrt(beta));
 *                        dq [rows, h_k, d_k] = sum over the value heads of dq_m when
 *                        h_v > h_k (when h_v = h_k, dq is dq_m); dlog_alpha is dla_m;
 *                        db_m and dw_m are not read (b = w = 1 are constants)
 *   GDN2_GATES_FG2_PLUS  dk and dq as FG2; dbeta = dk_m . k / (2 sqrt(beta));
 *                        dbeta_v [rows, h_v, d_v] = dw_m / (2 sqrt(beta_v)); dv and
 *                        dlog_alpha are dv_m and dla_m
 *
 *   mode, dims          as for gdn2_map_gates (rows = dims->batch x dims->seqlen)
 *   k, v, beta, beta_v  the forward's inputs of gdn2_map_gates, device, dims->dtype
 *   dq_m, dk_m          device fp32 [rows, h', d_k]: dL/dq', dL/dk' of the mapped inputs
 *                       (h' = h_v in the FG2 modes, whose mapped keys are per value head)
 *   dv_m, dw_m          device fp32 [rows, h_v, d_v];  dla_m, db_m  device fp32 [rows, h_v, d_k]
 *   dq .. dbeta_v       device fp32 outputs, in the shapes listed above
 * Pointers a mode does not read or write are ignored. In the FG2 modes beta (and beta_v)
 * must be > 0 (the derivative of the square root); a zero gives inf or NaN there. Outputs
 * must not alias the inputs or each other. One elementwise pass on `stream` (HBM-bound).
 */
gdn2_status gdn2_map_gates_bwd(int32_t mode, const gdn2_dims *dims, const void *k,
                               const void *v, const void *beta, const void *beta_v,
                               const float *dq_m, const float *dk_m, const float *dv_m,
                               const float *dla_m, const float *db_m, const float *dw_m,
                               float *dq, float *dk, float *dv, float *dlog_alpha,
                               float *dbeta, float *dbeta_v, void *stream);

/*
 * ---- Around the recurrence ---------------------------------------------------------------
 *
 * The calls below share these conventions on top of those at the head of this file:
 *   - Token tensors are [B, T, ...] (dense) or [1, T, ...] with cu_seqlens (packed). A packed
 *     batch may end before T (cu_seqlens[N] <= T): rows behind the last sequence are neither
 *     read nor written. Offsets are held inside [0, T] on the device, so a wrong table gives
 *     wrong results but no access outside the tensors; it has to be non-decreasing. Empty
 *     sequences are allowed and hand their initial state on.
 *   - A stride field gives the elements from one token to the next of an input that is a column
 *     slice of a wider tensor (a projection's output); 0 means contiguous. The sequences of a
 *     dense batch follow each other at seqlen times that stride. Outputs are contiguous.
 *   - grad_dtype is the type of the token gradients that go in and come out: GDN2_F32, or the
 *     call's dtype. Gradients of parameters and states are fp32.
 *   - All sums, states and statistics are held in fp32. Every call gives the same bits for the
 *     same arguments (no atomics).
 *   - At most 2^30 tokens and 2^20 channels; no tensor may reach over more than 2^40 elements,
 *     strides included. Outputs must not overlap inputs, the workspace or
 *     each other (the same pointer twice is refused).
 */

/*
 * The short causal depthwise convolution that the burn-gdn2 diagram ("Architecture",
 * use_short_conv) puts before the recurrence, over whole prompts; gdn2_fusion.conv_weight is
 * its form inside gdn2_recurrent_fwd, with the same weights and states. With W = width taps:
 *     a_t[c] = bias[c] + sum_{j < W} weight[c][j] x_{t - W + 1 + j}[c],   y_t = silu(a_t) or a_t
 * where the W - 1 inputs before a sequence are its rows of state0 (oldest first), or zeros.
 */
typedef struct gdn2_conv_dims {
    int32_t batch, seqlen, num_seqs;   /* as in gdn2_dims */
    int32_t channels;                  /* C >= 1 */
    int32_t width;                     /* W: 2, 3 or 4 taps */
    int32_t dtype;                     /* gdn2_dtype of x and y */
    int32_t grad_dtype;                /* of dy and dx (backward only) */
    int32_t silu;                      /* nonzero: y = silu(a) */
    int64_t x_stride;                  /* elements between tokens of x, >= C, or 0 */
} gdn2_conv_dims;

/*
 *   x           device [B, T, C]
 *   weight      device fp32 [C][W];  bias  device fp32 [C], or NULL
 *   state0      device fp32 [N][W-1][C], the inputs before each sequence, or NULL for zeros
 *   cu_seqlens  device int32 [N+1] for a packed batch, or NULL
 *   y           device [B, T, C]
 *   state_T     device fp32 [N][W-1][C], the last W-1 inputs of each sequence (of state0 and x
 *               together, where it is shorter), or NULL. A row of a conv_state pool has this
 *               layout, so decoding goes on from it.
 */
gdn2_status gdn2_short_conv_fwd(const void *x, const float *weight, const float *bias,
                                const float *state0, const int32_t *cu_seqlens, void *y,
                                float *state_T, const gdn2_conv_dims *dims, void *stream);

/* Bytes of device workspace gdn2_short_conv_bwd needs, or 0 if the dims are invalid. */
size_t gdn2_short_conv_bwd_workspace_bytes(const gdn2_conv_dims *dims);

/*
 * Gradients of gdn2_short_conv_fwd, which is formed again from its inputs.
 *   dy          device [B, T, C] (grad_dtype): dL/dy
 *   dstate_T    device fp32 [N][W-1][C]: dL/dstate_T, or NULL for zero
 *   dx          device [B, T, C] (grad_dtype)
 *   dweight     device fp32 [C][W];  dbias  device fp32 [C], required with a bias
 *   dstate0     device fp32 [N][W-1][C], or NULL to skip it
 *   workspace   at least gdn2_short_conv_bwd_workspace_bytes() bytes, 256-byte aligned
 */
gdn2_status gdn2_short_conv_bwd(const void *x, const float *weight, const float *bias,
                                const float *state0, const int32_t *cu_seqlens, const void *dy,
                                const float *dstate_T, void *dx, float *dweight, float *dbias,
                                float *dstate0, const gdn2_conv_dims *dims, void *workspace,
                                size_t workspace_bytes, void *stream);

/*
 * The convolution of T tokens (seqlen >= 1) of each of N sequences (batch >= 0) against a pool
 * of conv states, as gdn2_recurrent_fwd runs the recurrence against its pool.
 *   x, y        device [N, T, C]
 *   conv_state  device fp32 [num_slots][W-1][C], read and updated in place
 *   state_idx   device int32 [N], the slot of each sequence, or NULL (slot n). An entry outside
 *               [0, num_slots) marks a padding sequence: zero y rows, no state touched. The
 *               valid entries must be distinct.
 */
gdn2_status gdn2_short_conv_step(const void *x, const float *weight, const float *bias,
                                 float *conv_state, const int32_t *state_idx, int32_t num_slots,
                                 void *y, const gdn2_conv_dims *dims, void *stream);

/*
 * The selective state space scan. Where the delta rule keeps a matrix per head, it keeps
 * d_state values per channel, each with a decay of its own that follows the token's step:
 *     dt_t[d]   = softplus(dt[t][d] + dt_bias[d])         (or the sum alone)
 *     h_t[d][n] = exp(dt_t[d] A[d][n]) h_{t-1}[d][n] + dt_t[d] B_t[g][n] x_t[d]
 *     y_t[d]    = sum_n C_t[g][n] h_t[d][n] + D[d] x_t[d]
 *     o_t[d]    = y_t[d] silu(gate_t[d])                  (without a gate: y_t)
 * Channel d reads group g = d / (channels / groups) of B and C.
 */
typedef struct gdn2_scan_dims {
    int32_t batch, seqlen, num_seqs;   /* as in gdn2_dims */
    int32_t channels;                  /* >= 1 */
    int32_t d_state;                   /* states per channel: 1 .. 128 */
    int32_t groups;                    /* of B and C; channels is a multiple of it */
    int32_t dtype;                     /* gdn2_dtype of x, dt, B, C, gate and o */
    int32_t grad_dtype;                /* of the token gradients (backward only) */
    int32_t dt_softplus;               /* nonzero: softplus of dt + dt_bias */
    /* elements between tokens, or 0: */
    int64_t x_stride, dt_stride, b_stride, c_stride, gate_stride;
} gdn2_scan_dims;

/*
 * Bytes of device workspace gdn2_selective_scan_fwd needs for these dims (0 too where it needs
 * none, and if the dims are invalid).
 */
size_t gdn2_selective_scan_fwd_workspace_bytes(const gdn2_scan_dims *dims);

/*
 *   x, dt, gate  device [B, T, channels];  gate may be NULL
 *   A            device fp32 [channels][d_state], the rates (<= 0 for a stable state)
 *   B, C         device [B, T, groups, d_state]
 *   D, dt_bias   device fp32 [channels], each may be NULL (zero)
 *   S0           device fp32 [N][channels][d_state] initial states, or NULL for zeros
 *   cu_seqlens   device int32 [N+1] for a packed batch, or NULL
 *   o            device [B, T, channels]
 *   S_T          device fp32 [N][channels][d_state] final states, or NULL. Not S0's buffer.
 *   workspace    at least gdn2_selective_scan_fwd_workspace_bytes() bytes, 256-byte aligned
 */
gdn2_status gdn2_selective_scan_fwd(const void *x, const void *dt, const float *A, const void *B,
                                    const void *C, const float *D, const void *gate,
                                    const float *dt_bias, const float *S0, const int32_t *cu_seqlens,
                                    void *o, float *S_T, const gdn2_scan_dims *dims, void *workspace,
                                    size_t workspace_bytes, void *stream);

/*
 * Bytes of device workspace gdn2_selective_scan_bwd needs, or 0 if the dims are invalid. About, with
 * c = channels and s = d_state: c (s + 1) / 2 bytes per token for the state before every eighth one;
 * 8 c (s + 1) bytes per tile of 8 to 64 tokens; and 8 s bytes per token and workgroup of channels,
 * of which a group has one per 256, 128, 64, 32 or 16 channels at up to 8, 16, 32, 64 or 128 states
 * (4,096 tokens x 4,096 x 16: 0.2 GB; 16,384 x 8,192 x 128: 19.4 GB).
 */
size_t gdn2_selective_scan_bwd_workspace_bytes(const gdn2_scan_dims *dims);

/*
 * Gradients of gdn2_selective_scan_fwd, which is formed again from its inputs.
 *   x .. cu_seqlens   the forward's inputs
 *   dO           device [B, T, channels] (grad_dtype): dL/do
 *   dS_T         device fp32 [N][channels][d_state]: dL/dS_T, or NULL for zero
 *   dx, ddt      device [B, T, channels] (grad_dtype); ddt is of dt as given, before dt_bias
 *   dgate        device [B, T, channels] (grad_dtype), required with a gate
 *   dB, dC       device [B, T, groups, d_state] (grad_dtype), contiguous
 *   dA           device fp32 [channels][d_state]
 *   dD, ddt_bias device fp32 [channels], each required with its input
 *   dS0          device fp32 [N][channels][d_state], or NULL to skip it
 *   workspace    at least gdn2_selective_scan_bwd_workspace_bytes() bytes, 256-byte aligned
 */
gdn2_status gdn2_selective_scan_bwd(const void *x, const void *dt, const float *A, const void *B,
                                    const void *C, const float *D, const void *gate,
                                    const float *dt_bias, const float *S0, const int32_t *cu_seqlens,
                                    const void *dO, const float *dS_T, void *dx, void *ddt, float *dA,
                                    void *dB, void *dC, float *dD, void *dgate, float *ddt_bias,
                                    float *dS0, const gdn2_scan_dims *dims, void *workspace,
                                    size_t workspace_bytes, void *stream);

/*
 * The scan of T tokens (seqlen >= 1) of each of N sequences (batch >= 0) against a pool of
 * states, as gdn2_recurrent_fwd runs the delta rule against its pool.
 *   state        device [num_slots][channels][d_state] in state_dtype (gdn2_state_dtype), read
 *                once and written once per call
 *   state_idx    device int32 [N], the slot of each sequence, or NULL (slot n). An entry outside
 *                [0, num_slots) marks a padding sequence: zero o rows, no state touched. The
 *                valid entries must be distinct.
 *   o            device [N, T, channels]
 */
gdn2_status gdn2_selective_scan_step(const void *x, const void *dt, const float *A, const void *B,
                                     const void *C, const float *D, const void *gate,
                                     const float *dt_bias, void *state, int32_t state_dtype,
                                     const int32_t *state_idx, int32_t num_slots, void *o,
                                     const gdn2_scan_dims *dims, void *stream);

/*
 * The norms after and before a block, fused with the block's gate, the residual and its scale.
 * Per row, rms(v) = v / sqrt(mean(v^2) + eps), and each stage but the last only where its
 * argument is given:
 *     p = rms(x) norm_weight,  u = p silu(gate),  h = residual + scale u,  y = rms(h) next_weight
 * With norm_weight and gate alone this is the gated output norm that gdn2_fusion.gate fuses
 * into the recurrence (x its o, one row per token and value head), with gradients; with all of
 * them it is the whole boundary between two blocks. Both norms are taken of fp32 values (y of h
 * before it is rounded to its type).
 */
typedef struct gdn2_norm_dims {
    int64_t rows;                      /* 0 .. 2^31-1 */
    int32_t d;                         /* columns: 1 .. 16384 */
    int32_t dtype;                     /* gdn2_dtype of x, gate and y */
    int32_t residual_dtype;            /* of residual and h: GDN2_F32 or dtype */
    int32_t grad_dtype;                /* of dy, dx, dgate (backward only). dh and dresidual have
                                          it too, and GDN2_F32 with a GDN2_F32 residual */
    float eps;                         /* >= 0; with 0 a row of zeros gives NaN */
    int64_t x_stride, gate_stride;     /* elements between rows, >= d, or 0 */
} gdn2_norm_dims;

/*
 *   x, gate, residual                 device [rows, d];  gate and residual may be NULL
 *   norm_weight, scale, next_weight   device fp32 [d], each may be NULL
 *   h            device [rows, d]; may be residual's own buffer
 *   y            device [rows, d], written (and required) with next_weight only
 */
gdn2_status gdn2_block_norm_fwd(const void *x, const void *gate, const void *residual,
                                const float *norm_weight, const float *scale,
                                const float *next_weight, void *h, void *y,
                                const gdn2_norm_dims *dims, void *stream);

/* Bytes of device workspace gdn2_block_norm_bwd needs, or 0 if the dims are invalid. */
size_t gdn2_block_norm_bwd_workspace_bytes(const gdn2_norm_dims *dims);

/*
 * Gradients of gdn2_block_norm_fwd, which is formed again from its inputs.
 *   x .. next_weight    the forward's inputs
 *   dh           device [rows, d]: dL/dh, or NULL for zero (with next_weight only)
 *   dy           device [rows, d]: dL/dy, required with next_weight
 *   dx, dgate, dresidual              device [rows, d], the last two for a gate, a residual
 *   dnorm_weight, dscale, dnext_weight   device fp32 [d], each required with its input
 *   workspace    at least gdn2_block_norm_bwd_workspace_bytes() bytes, 256-byte aligned; not
 *                needed without norm_weight, scale and next_weight
 */
gdn2_status gdn2_block_norm_bwd(const void *x, const void *gate, const void *residual,
                                const float *norm_weight, const float *scale,
                                const float *next_weight, const void *dh, const void *dy, void *dx,
                                void *dgate, void *dresidual, float *dnorm_weight, float *dscale,
                                float *dnext_weight, const gdn2_norm_dims *dims, void *workspace,
                                size_t workspace_bytes, void *stream);

/*
 * ---- The attention layer of hybrid stacks ------------------------------------------------
 *
 * Stacks of recurrent layers keep a softmax attention layer every few layers. The calls below
 * are what such a layer needs beside its projections: its queries and keys normed per head and
 * rotated by position, in training and in front of a cache; the attention of new tokens over the
 * cache; and copies of slots, for the cache's pages and for the state pools of the recurrent
 * layers. Layouts:
 *   q, q_out, o        [B, T, h_q, d];   k, v  [B, T, h_k, d]      (q head j reads k head j / (h_q / h_k))
 *   k_pages, v_pages   [num_pages][h_k][page_size][d]: a page holds page_size consecutive tokens of
 *                      one sequence, each head's rows contiguous. Place `slot` of a pool of pages is
 *                      row slot % page_size of page slot / page_size.
 * Strides, types, sums, sizes and overlaps are as around the recurrence above: token strides of
 * column slices (0: contiguous), fp32 sums and statistics, the same bits at every call (no
 * atomics), outputs that overlap nothing else.
 */

typedef struct gdn2_rotary_dims {
    int32_t batch, seqlen;             /* B, T >= 0 */
    int32_t h_q, h_k;                  /* heads, h_q >= 1; h_k = 0: no keys (fwd and bwd) */
    int32_t d;                         /* values per head: even, 2 .. 512 */
    int32_t d_rot;                     /* the first d_rot of them are rotated: even, 0 .. d */
    int32_t interleaved;               /* 0: pairs (i, i + d_rot/2); nonzero: pairs (2i, 2i + 1) */
    int32_t num_positions;             /* rows of cos_sin, >= 1 (>= 0 with d_rot = 0) */
    int32_t dtype;                     /* gdn2_dtype of q, k, v, their outputs and the pages */
    int32_t grad_dtype;                /* of dq_out, dk_out, dq, dk (backward only) */
    float eps;                         /* >= 0; with 0 a row of zeros gives NaN */
    int64_t q_stride, k_stride, v_stride;   /* elements between tokens, or 0 */
} gdn2_rotary_dims;

/*
 * Per token and head: y = x / sqrt(mean(x^2) + eps) weight (without a weight y = x), then pair i
 * of the first d_rot values turns by the angle of the token's position p,
 *     y_a' = y_a cos[p][i] - y_b sin[p][i],   y_b' = y_b cos[p][i] + y_a sin[p][i],
 * all in fp32 and rounded once.
 *   q            device [B, T, h_q, d];  k  device [B, T, h_k, d], or NULL with h_k = 0
 *   cos_sin      device fp32 [num_positions][d_rot]: d_rot/2 cosines, then d_rot/2 sines (NULL with
 *                d_rot = 0)
 *   positions    device int32 [B, T], or NULL: token t of each sequence is at position t. A position
 *                outside [0, num_positions) marks a padding token: zero rows come out. (With
 *                d_rot = 0 only negative ones do.)
 *   q_weight, k_weight   device fp32 [d], each may be NULL
 *   q_out, k_out contiguous. May be q's and k's own buffers, if those are contiguous.
 */
gdn2_status gdn2_qk_rotary_fwd(const void *q, const void *k, const float *cos_sin,
                               const int32_t *positions, const float *q_weight, const float *k_weight,
                               void *q_out, void *k_out, const gdn2_rotary_dims *dims, void *stream);

/* Bytes of device workspace gdn2_qk_rotary_bwd needs, or 0 if the dims are invalid. */
size_t gdn2_qk_rotary_bwd_workspace_bytes(const gdn2_rotary_dims *dims);

/*
 * Gradients of gdn2_qk_rotary_fwd, which is formed again from its inputs.
 *   dq_out, dk_out   device, contiguous (grad_dtype): dL/dq_out, dL/dk_out
 *   dq, dk           device, contiguous (grad_dtype); rows of padding tokens come out zero, and give
 *                    nothing to the weights' gradients
 *   dq_weight, dk_weight   device fp32 [d], each required with its weight. With h_k = 0, dk_weight is
 *                    zeros, or may be NULL
 *   workspace        at least gdn2_qk_rotary_bwd_workspace_bytes() bytes, 256-byte aligned; not
 *                    needed without weights
 */
gdn2_status gdn2_qk_rotary_bwd(const void *q, const void *k, const float *cos_sin,
                               const int32_t *positions, const float *q_weight, const float *k_weight,
                               const void *dq_out, const void *dk_out, void *dq, void *dk,
                               float *dq_weight, float *dk_weight, const gdn2_rotary_dims *dims,
                               void *workspace, size_t workspace_bytes, void *stream);

/*
 * gdn2_qk_rotary_fwd in front of a cache: q_out is written as there, the keys and the values (as
 * they are) go to the pages. For whole prompts, packed or not, and for single tokens: a token's
 * place is given by its slot.
 *   positions        device int32 [B, T], required
 *   slots            device int32 [B, T]: the place of each token in the pages, distinct. Outside
 *                    [0, num_pages * page_size): the token is not put anywhere (its q row is
 *                    written all the same). A padding token (by its position) is not put anywhere
 *                    either.
 *   q_out            contiguous. May be q's own buffer, if that is contiguous.
 *   k_pages, v_pages num_pages * page_size <= 2^31 - 1
 */
gdn2_status gdn2_qk_rotary_append(const void *q, const void *k, const void *v, const float *cos_sin,
                                  const int32_t *positions, const float *q_weight,
                                  const float *k_weight, const int32_t *slots, void *q_out,
                                  void *k_pages, void *v_pages, int32_t num_pages, int32_t page_size,
                                  const gdn2_rotary_dims *dims, void *stream);

typedef struct gdn2_attention_dims {
    int32_t num_seqs;                  /* N >= 0 */
    int32_t new_tokens;                /* T >= 1: query tokens per sequence */
    int32_t h_q, h_k;                  /* h_q a multiple of h_k */
    int32_t d;                         /* 64, 128 or 256 */
    int32_t num_pages, page_size;      /* num_pages * h_k * page_size <= 2^31 - 1 */
    int32_t max_pages;                 /* columns of page_table; max_pages * page_size <= 2^29 */
    int32_t window;                    /* a query sees this many keys at most, its own among them;
                                          0: all before it */
    int32_t dtype;                     /* gdn2_dtype of q, the pages and o */
    float scale;                       /* of the products of queries and keys; finite */
    int64_t q_stride;                  /* elements between tokens of q, or 0 */
} gdn2_attention_dims;

/*
 * Bytes of device workspace gdn2_paged_attention_step needs for these dims (0 too where it needs
 * none, and if the dims are invalid). They do not depend on the lengths. With window = 0 they grow with
 * num_seqs and are enough for any window; with a window more sequences may need less than fewer.
 */
size_t gdn2_paged_attention_step_workspace_bytes(const gdn2_attention_dims *dims);

/*
 * The last T tokens of each of N sequences attend to the sequence's cached tokens, themselves among
 * them (gdn2_qk_rotary_append puts them there first). Token t of sequence n stands at place
 * p = seq_lens[n] - T + t and sees the places j <= p, with a window those with j > p - window:
 *     s_j = scale q . k_j,   o = sum_j softmax(s)_j v_j,   lse = log sum_j e^(s_j)
 * A token that sees nothing (an empty sequence; more new tokens than the sequence has) gives o = 0
 * and lse = -inf, and so does one all of whose products are -inf. A key whose scaled product is -inf
 * takes no part beside others, whatever the scale's sign. What lies in the pages at places that a
 * token does not see is not used for it, NaN included; of those that it sees, an infinite value gives
 * inf or NaN in its element of o. Weights (1 for the largest) and values are summed in fp32 and divided
 * at the end, so finite values whose sum leaves fp32 give inf.
 *   q            device [N, T, h_q, d]
 *   k_pages, v_pages   device [num_pages][h_k][page_size][d], 16-byte aligned
 *   page_table   device int32 [N][max_pages]: the page of each page_size tokens of a sequence. Only
 *                entries of places that are seen are used; held inside [0, num_pages). Sequences may
 *                share pages.
 *   seq_lens     device int32 [N], the cached tokens of each sequence with the new ones; held inside
 *                [0, max_pages * page_size]
 *   o            device [N, T, h_q, d], contiguous, 16-byte aligned
 *   lse          device fp32 [N, T, h_q], or NULL
 *   workspace    at least gdn2_paged_attention_step_workspace_bytes() bytes, 256-byte aligned; nothing
 *                is kept in it from one call to the next, but two calls at once need one each
 */
gdn2_status gdn2_paged_attention_step(const void *q, const void *k_pages, const void *v_pages,
                                      const int32_t *page_table, const int32_t *seq_lens, void *o,
                                      float *lse, const gdn2_attention_dims *dims, void *workspace,
                                      size_t workspace_bytes, void *stream);

/*
 * Copies slots inside each of several pools: slot dst[i] takes the bytes of slot src[i], for every
 * i < count and every pool. The pages of a cache are slots of two pools per layer, a recurrent
 * layer's states, conv states and scan states slots of one each; a forked sequence, or a pool
 * whose sequences are moved together, is one call over all layers.
 *   pools        HOST array of num_pools device pointers, pool p being [num_slots] slots of
 *                slot_bytes[p] bytes (HOST array, each >= 1)
 *   src, dst     device int32 [count]. A pair with an entry outside [0, num_slots) is skipped. One
 *                source may have many destinations. The destinations have to be distinct, and none
 *                may be the source of another pair.
 */
gdn2_status gdn2_pool_copy(void *const *pools, const int64_t *slot_bytes, int32_t num_pools,
                           int32_t num_slots, const int32_t *src, const int32_t *dst, int32_t count,
                           void *stream);

/*
 * Host helper: checks a HOST copy of cu_seqlens (N+1 entries) against total tokens T.
 * Returns GDN2_OK when cu[0] = 0, cu is non-decreasing and cu[N] = T, else
 * GDN2_ERR_BAD_SHAPE (GDN2_ERR_NULL_ARG for a NULL pointer). Touches no device.
 */
gdn2_status gdn2_check_cu_seqlens(const int32_t *cu_seqlens_host, int32_t num_seqs,
                                  int32_t total_tokens);

#ifdef __cplusplus
}
#endif

#endif /* GDN2_H */
