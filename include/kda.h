/*
 * kda.h — C ABI of libkda.so: the Kimi Delta Attention (KDA) gated delta rule on
 * NVIDIA B200 (sm_100a).
 *
 * The operation (one head; dk x dv fp32 state S; per token t):
 *     S_t = (I - beta_t k_t k_t^T) Diag(exp g_t) S_{t-1} + beta_t k_t v_t^T
 *     o_t = S_t^T q_t
 * i.e. the state is decayed per key channel by exp(g_t) (g_t <= 0), corrected by
 * the delta rule with strength beta_t along k_t, written with k_t v_t^T and read
 * with q_t after the write.  The query scale is 1.  Sources: the open-model-atlas
 * page "Kimi-K3 ?inspect=blocks" (self.layers: 69 KDA layers keep a state of fixed
 * size between calls) and maxtext PR #5548's review, item 2 (KDA tensors A_log,
 * dt_bias, conv weights and o_norm kept in F32; exp(A_log) drives the decay).
 *
 * Entry points
 *   kda_forward_chunked          chunked prefill: outputs and final state
 *   kda_forward_chunked_varlen   the same over N packed sequences (cu_seqlens)
 *   kda_decode_step              one token per sequence, state in place
 *   kda_layer_forward            the layer core (conv + SiLU, L2-norm, gate, beta,
 *                                recurrence, RMSNorm x sigmoid gate); _noalloc and
 *                                _varlen variants
 *   kda_layer_decode_step        one decode step of the layer core with a conv cache
 *   kda_backward_chunked         gradients of the recurrence's inputs
 *   kda_gdr_forward              the recurrence with one gate per value head and value heads
 *                                that share key heads; states dense or in cache pages
 *   kda_gdr_backward             its gradients
 *   kda_gdr_decode               the same for one or a few tokens a sequence, on cache pages
 *   kda_pages_fork, _copy, _free, _compact   pages of a state cache
 *   kda_*_workspace_size, kda_check_device_error, kda_status_string, kda_abi_version
 *   kda_set_wait_test_hooks      wait limit and failure injection for the failure path
 *
 * Conventions for every entry point
 *   - Pointers are DEVICE pointers unless a comment says otherwise; the caller owns
 *     and allocates every buffer.  The library allocates no device memory in any call
 *     (kda_layer_forward_noalloc uses a fixed array the library holds from load time).
 *   - Layouts are dense and row-major (last index fastest):
 *       q, k, g : [B, T, H, dk]      v, out : [B, T, H, dv]      beta : [B, T, H]
 *       state   : [B, H, dk, dv] fp32
 *   - Every tensor pointer must be 16-byte aligned (KDA_ERR_MISALIGNED otherwise).
 *   - Calls are asynchronous on `stream` and never synchronise it.  KDA_OK means the
 *     arguments were valid and the kernels were launched.  Arguments are validated
 *     before anything is launched; on any error nothing is launched and no output
 *     is touched.  Faults inside kernels and bounded-wait timeouts surface through
 *     kda_check_device_error() (which synchronises the stream).
 *   - The library never aborts, exits or prints.  It is reentrant; concurrent calls
 *     on different streams must not share output buffers.
 */
#ifndef KDA_H
#define KDA_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same underlying type as cudaStream_t; NULL is the legacy default stream. */
typedef struct CUstream_st *kda_stream_t;

typedef enum {
    KDA_OK = 0,
    KDA_ERR_INVALID_ARG = 1,  /* null required pointer, non-positive size, bad enum  */
    KDA_ERR_UNSUPPORTED = 2,  /* valid but not built: head dims, chunk size, dtype    */
    KDA_ERR_MISALIGNED = 3,   /* a tensor pointer is not 16-byte aligned              */
    KDA_ERR_CUDA = 4,         /* a CUDA runtime call failed (launch, attribute, ...)  */
    KDA_ERR_TIMEOUT = 5,      /* a kernel's bounded wait gave up (device error word)  */
    KDA_ERR_WORKSPACE = 6,    /* workspace missing or smaller than required           */
    KDA_ERR_INDEX = 7         /* a page index out of range, not live, or named twice  */
} kda_status_t;

typedef enum {
    KDA_F32 = 0,  /* q, k, v, g, beta, out (and the layer's raw inputs) are float32  */
    KDA_BF16 = 1  /* ... are bfloat16; the state is always float32                   */
} kda_dtype_t;

/* Static, NUL-terminated description of a status code (never NULL). */
const char *kda_status_string(kda_status_t status);

/* Version of this ABI (major * 100 + minor). */
int kda_abi_version(void);

/*
 * Chunked prefill (chunkwise-parallel form of the recurrence; results equal the
 * token-by-token recurrence up to rounding).
 *   q, k, g       [B, T, H, dk]   io dtype; g is the per-channel log-decay (<= 0)
 *   v             [B, T, H, dv]   io dtype
 *   beta          [B, T, H]       io dtype, the delta-rule strength in [0, 1]
 *   initial_state [B, H, dk, dv]  fp32, or NULL for a zero initial state
 *   out           [B, T, H, dv]   io dtype (written)
 *   final_state   [B, H, dk, dv]  fp32, or NULL to skip; may equal initial_state
 *                                 (in-place state passing)
 *   chunk         must be 64.
 * Supported: dk, dv in {64, 128} in either io dtype.  io KDA_BF16 with dk = dv = 128 runs
 * on the tcgen05 tensor-core kernel only: on a device or driver where that kernel cannot
 * run the call returns KDA_ERR_UNSUPPORTED (no slower kernel is substituted).  io KDA_F32
 * and the other bf16 head-dim pairs run exact fp32 CUDA-core kernels.  T = 0 is valid: out
 * is untouched and final_state receives initial_state (or zeros).
 */
kda_status_t kda_forward_chunked(const void *q, const void *k, const void *v, const void *g,
                                 const void *beta, const float *initial_state, void *out,
                                 float *final_state, int B, int T, int H, int dk, int dv,
                                 int chunk, kda_dtype_t io, kda_stream_t stream);

/*
 * Bytes of device workspace kda_backward_chunked needs: for every 16-token chunk, the fp32
 * state at its start (d * d floats) and the chunk's forward quantities U and X = V - K^ S
 * (2 * 16 * d floats) and its three 16 x 16 matrices, so
 * B * H * ceil(T / 16) * (d * d + 32 * d + 768) * 4 with d = dk.  dk must equal dv
 * (KDA_ERR_UNSUPPORTED otherwise).  *bytes is written on KDA_OK.
 */
kda_status_t kda_backward_workspace_size(int B, int T, int H, int dk, int dv, kda_dtype_t io,
                                         size_t *bytes);

/*
 * kda_backward_chunked — gradients of the recurrence of kda_forward_chunked (training;
 * the pages' runs differentiate the KDA layer: maxtext PR #5550, its jax.grad test and the
 * C4 training steps).  Given d_out = dL/dout and d_final_state = dL/dS_T, writes dL/d of
 * every input.  Computed in fp32 from the io-dtype inputs: a forward sweep stores each
 * 16-token chunk's start state and forward quantities in `workspace`, then a reverse sweep
 * reloads them and applies the chain rule (pairwise decays exp(G_i - G_j), j <= i, so no
 * gate overflows).
 *   q, k, g, v, beta, initial_state   as kda_forward_chunked (inputs, unchanged)
 *   d_out          [B, T, H, dv] io dtype
 *   d_final_state  [B, H, dk, dv] fp32 or NULL (zero)
 *   d_q, d_k, d_g  [B, T, H, dk] io dtype (written; d_g is the gradient of the log-decay g)
 *   d_v            [B, T, H, dv] io dtype (written)
 *   d_beta         [B, T, H] io dtype (written)
 *   d_initial_state [B, H, dk, dv] fp32 (written) or NULL; may equal d_final_state
 *   workspace      device buffer of kda_backward_workspace_size() bytes, 256-byte aligned
 * Supported: dk = dv in {64, 128}, both dtypes.  T = 0: d_initial_state receives
 * d_final_state (or zeros).
 */
kda_status_t kda_backward_chunked(const void *q, const void *k, const void *v, const void *g,
                                  const void *beta, const float *initial_state, const void *d_out,
                                  const float *d_final_state, void *d_q, void *d_k, void *d_v,
                                  void *d_g, void *d_beta, float *d_initial_state, void *workspace,
                                  size_t workspace_bytes, int B, int T, int H, int dk, int dv,
                                  kda_dtype_t io, kda_stream_t stream);

/*
 * kda_forward_chunked_varlen — chunked prefill of N packed sequences of different lengths
 * (the variable-length batches that segment ids or a padding mask describe; the MaxText
 * port of the Kimi-K3 model rejects packing for KDA).  Each sequence runs the recurrence
 * from its own initial state; no state crosses a sequence boundary.
 *   q, k, g       [T_total, H, dk]  io dtype, the sequences' tokens back to back
 *   v             [T_total, H, dv]  io dtype
 *   beta          [T_total, H]      io dtype
 *   cu_seqlens    [N + 1] int32, DEVICE memory: sequence n is tokens cu_seqlens[n] ..
 *                 cu_seqlens[n + 1] - 1.  Expected non-decreasing from 0 to T_total.  The
 *                 values are read on the device only and are not checked; every offset is
 *                 clamped into [0, T_total] (and each end to at least its start), so no
 *                 access leaves the buffers, but other malformed arrays give unspecified
 *                 results.  A zero-length sequence passes its initial state through.
 *   initial_state [N, H, dk, dv]  fp32 or NULL (zeros)
 *   out           [T_total, H, dv]  io dtype (written at every token of the N sequences)
 *   final_state   [N, H, dk, dv]  fp32 or NULL; may equal initial_state
 *   chunk         must be 64.
 * Supported: as kda_forward_chunked.  T_total = 0: final_state receives initial_state.
 */
kda_status_t kda_forward_chunked_varlen(const void *q, const void *k, const void *v, const void *g,
                                        const void *beta, const float *initial_state, void *out,
                                        float *final_state, const int *cu_seqlens, int N,
                                        int T_total, int H, int dk, int dv, int chunk,
                                        kda_dtype_t io, kda_stream_t stream);

/*
 * One decode step: the recurrence for a single new token per sequence, with the
 * state updated in place (read once, written once).
 *   q, k, g [B, H, dk] io dtype; v, out [B, H, dv] io dtype; beta [B, H] io dtype;
 *   state [B, H, dk, dv] fp32, read and overwritten.
 * Supported: dk, dv in {64, 128}, both dtypes.
 */
kda_status_t kda_decode_step(const void *q, const void *k, const void *v, const void *g,
                             const void *beta, float *state, void *out, int B, int H, int dk,
                             int dv, kda_dtype_t io, kda_stream_t stream);

/*
 * Bytes of device workspace kda_layer_forward needs for these sizes.  0 for bf16 at
 * dk = dv = 128, whose prologue, chunked step and epilogue run as one tensor-core kernel;
 * otherwise the fp32 prologue outputs and the chunked step's output (q, k, g, v, beta, o in
 * fp32, each rounded up to 256 bytes).  *bytes is written on KDA_OK.
 */
kda_status_t kda_layer_workspace_size(int B, int T, int H, int dk, int dv, kda_dtype_t io,
                                      size_t *bytes);

/*
 * KDA layer core: prologue -> chunked gated delta rule -> epilogue.
 *   prologue  q = l2norm(SiLU(conv_q * q_raw)), k = l2norm(SiLU(conv_k * k_raw)),
 *             v = SiLU(conv_v * v_raw)   (depthwise causal conv, kernel 4, zero history,
 *                                          PyTorch Conv1d tap order; l2norm eps 1e-6)
 *             g = max(-exp(A_log[h]) * softplus(g_raw + dt_bias), gate_lower_bound),
 *             beta = sigmoid(b_raw)
 *   epilogue  out = o_norm_w * cast_io(o * rsqrt(mean_dv(o^2) + norm_eps)) * sigmoid(o_gate_raw)
 * (open-model-atlas "Kimi-K3" linear_attn_config: short_conv_kernel_size 4;
 *  atlas.klimoza.dev KimiRMSNorm excerpt; maxtext PR #5543 sigmoid output gate.)
 *   q_raw, k_raw  [B, T, H*dk]  io dtype      v_raw       [B, T, H*dv]  io dtype
 *   conv_q, conv_k [H*dk, 4] fp32             conv_v      [H*dv, 4]     fp32
 *   g_raw         [B, T, H, dk] io dtype      A_log       [H]           fp32
 *   dt_bias       [H*dk] fp32 or NULL (zero)  b_raw       [B, T, H]     io dtype
 *   gate_lower_bound  a lower bound on every log-decay g, <= 0; -INFINITY for none.  (The
 *                 Kimi-K3 linear-attention config sets gate_lower_bound = -5.0 and gives no
 *                 formula; it is read as a bound on g itself, so that no token decays the
 *                 state by more than exp(bound) per channel.)  NaN or > 0: KDA_ERR_INVALID_ARG.
 *   o_gate_raw    [B, T, H, dv] io dtype      o_norm_w    [dv] fp32 or NULL (ones)
 *   initial_state / final_state as in kda_forward_chunked.
 *   out           [B, T, H, dv] io dtype (written)
 *   workspace     device buffer of at least kda_layer_workspace_size() bytes, 256-byte
 *                 aligned (may be NULL when that size is 0).
 * Supported: dk, dv in {64, 128}, both dtypes (as kda_forward_chunked).
 */
kda_status_t kda_layer_forward(const void *q_raw, const void *k_raw, const void *v_raw,
                               const float *conv_q, const float *conv_k, const float *conv_v,
                               const void *g_raw, const float *A_log, const float *dt_bias,
                               float gate_lower_bound, const void *b_raw, const void *o_gate_raw,
                               const float *o_norm_w, float norm_eps, const float *initial_state,
                               void *out, float *final_state, void *workspace, size_t workspace_bytes,
                               int B, int T, int H, int dk, int dv, kda_dtype_t io,
                               kda_stream_t stream);

/*
 * kda_layer_forward_varlen — kda_layer_forward over N packed sequences of different lengths
 * (the padding-mask / segment-id case; see kda_forward_chunked_varlen).  Every raw tensor is
 * token-major over T_total tokens ([T_total, H*dk], [T_total, H, dk], [T_total, H], ...);
 * states are [N, H, dk, dv]; cu_seqlens is the device int32 [N + 1] offsets array (same
 * rules as kda_forward_chunked_varlen).  The short conv's history is zero before each
 * sequence's first token, so no input of one sequence reaches another's outputs.
 * Workspace: kda_layer_workspace_size(1, T_total, H, dk, dv, io) bytes.
 */
kda_status_t kda_layer_forward_varlen(const void *q_raw, const void *k_raw, const void *v_raw,
                                      const float *conv_q, const float *conv_k, const float *conv_v,
                                      const void *g_raw, const float *A_log, const float *dt_bias,
                                      float gate_lower_bound, const void *b_raw, const void *o_gate_raw,
                                      const float *o_norm_w, float norm_eps, const float *initial_state,
                                      void *out, float *final_state, const int *cu_seqlens, void *workspace,
                                      size_t workspace_bytes, int N, int T_total, int H, int dk, int dv,
                                      kda_dtype_t io, kda_stream_t stream);

/* Size in bytes of the built-in scratch that kda_layer_forward_noalloc uses (64 MiB). */
#define KDA_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)

/*
 * kda_layer_forward_noalloc — kda_layer_forward for callers that cannot allocate device
 * memory on their call path: a serving loop whose device memory is planned once at
 * start-up, a plugin or callback interface that provides no allocator, or code that
 * cannot pay for cudaMalloc (which may synchronise the device).  The paper has no
 * counterpart to this entry point; it exists for those callers only.
 *   Arguments, layouts and results are those of kda_layer_forward without the workspace
 *   pair.  The caller still owns and passes every input and output.
 *   Scratch: a library-owned device array of KDA_NOALLOC_SCRATCH_BYTES, held by every GPU
 *   that loads the library until the process exits.  Sizes whose workspace
 *   (kda_layer_workspace_size) exceeds it are rejected with KDA_ERR_WORKSPACE before
 *   anything runs.  All calls share the array and it keeps the last call's contents;
 *   each call writes every scratch byte it reads, so nothing needs clearing.  Calls that
 *   overlap on the GPU (other streams or host threads) race on it and must be serialised
 *   by the caller.
 *   The first call on each device looks up the array's device address (with that device
 *   current); make that first call before any stream capture begins.
 */
kda_status_t kda_layer_forward_noalloc(const void *q_raw, const void *k_raw, const void *v_raw,
                                       const float *conv_q, const float *conv_k,
                                       const float *conv_v, const void *g_raw, const float *A_log,
                                       const float *dt_bias, float gate_lower_bound, const void *b_raw,
                                       const void *o_gate_raw, const float *o_norm_w,
                                       float norm_eps, const float *initial_state, void *out,
                                       float *final_state, int B, int T, int H, int dk, int dv,
                                       kda_dtype_t io, kda_stream_t stream);

/*
 * kda_layer_decode_step — one decode step of the layer core for B sequences: the prologue,
 * the gated delta rule and the epilogue of kda_layer_forward for the single new token t,
 * with the conv history kept in a cache instead of recomputed.
 *   y = SiLU(w[c,0] x[t-3] + w[c,1] x[t-2] + w[c,2] x[t-1] + w[c,3] x[t])  per channel, for q,
 *   k and v, x[t-3..t-1] read from the cache, which then shifts in x[t]; then as
 *   kda_layer_forward: q, k L2-normalised, g, beta, the state update
 *   S <- (I - beta k k^T) Diag(exp g) S + beta k v^T, o = S^T q, RMSNorm x gain x sigmoid gate.
 * (The Kimi-K3 linear-attention config's short conv of kernel 4; the pages note that KDA
 *  decode with a cached state is not yet implemented in the MaxText port.)
 *   q_raw, k_raw  [B, H*dk] io dtype         v_raw        [B, H*dv] io dtype
 *   cache_q, cache_k [B, 3, H*dk] io dtype   cache_v      [B, 3, H*dv] io dtype
 *                 updated in place; tap 0 is the oldest token (t-3); zeros = empty history
 *   conv_q, conv_k [H*dk, 4] fp32            conv_v       [H*dv, 4] fp32
 *   g_raw         [B, H, dk] io dtype        A_log        [H] fp32
 *   dt_bias       [H*dk] fp32 or NULL        b_raw        [B, H] io dtype
 *   gate_lower_bound  as in kda_layer_forward (-INFINITY for none)
 *   o_gate_raw    [B, H, dv] io dtype        o_norm_w     [dv] fp32 or NULL (ones)
 *   state         [B, H, dk, dv] fp32, updated in place
 *   out           [B, H, dv] io dtype (written)
 * Supported: dk = dv = 128 (KDA_ERR_UNSUPPORTED otherwise), both dtypes.  Every pointer
 * 16-byte aligned.  n calls from an empty cache and state give the outputs of
 * kda_layer_forward over the same n tokens.
 */
kda_status_t kda_layer_decode_step(const void *q_raw, const void *k_raw, const void *v_raw,
                                   const float *conv_q, const float *conv_k, const float *conv_v,
                                   void *cache_q, void *cache_k, void *cache_v, const void *g_raw,
                                   const float *A_log, const float *dt_bias, float gate_lower_bound,
                                   const void *b_raw, const void *o_gate_raw, const float *o_norm_w,
                                   float norm_eps, float *state, void *out, int B, int H, int dk, int dv,
                                   kda_dtype_t io, kda_stream_t stream);

/*
 * ---- The gated delta rule with one gate per value head and grouped heads ("gdr") ----
 *
 * Hv value heads share Hk key heads (Hv a multiple of Hk): value head h reads q and k of key
 * head h / (Hv / Hk).  Per value head, with a dk x dv fp32 state S and, per token, a
 * log-decay g (one number, expected <= 0) and a strength beta in [0, 1]:
 *     S' = exp(g) S;   u = beta (v - S'^T k);   S <- S' + k u^T;   o = S^T q
 *   q, k       [T_total, Hk, dk]  io dtype     v, out  [T_total, Hv, dv]  io dtype
 *   g, beta    [T_total, Hv]      io dtype     states  [.., Hv, dk, dv]   fp32
 *   cu_seqlens [N + 1] int32 device offsets of N packed sequences, as
 *              kda_forward_chunked_varlen; or NULL for N sequences of T_total / N tokens each
 *              (T_total a multiple of N).
 * Any head counts, dk and dv in {64, 128} (all four pairs), both io dtypes.  bf16 at
 * dk = dv = 128 runs on tcgen05 kernels (KDA_ERR_UNSUPPORTED where they cannot run); its
 * products read the state, its corrections and their gradients as bf16 hi + lo pairs with
 * fp32 sums, so states and out carry about 2^-16 relative error before out's own rounding.
 * The other shapes run to fp32 accuracy: products as split tf32 on the tensor cores (a factor within
 * 2^-23, the product of the low parts, at most 2^-24, left out; within 2^-21 in the chunk's inverse),
 * summed in fp32.  A g below -128 (-inf among them) acts as
 * a full reset, which exp(g) = 0 is; NaN inputs reach their own head's values and no other's.
 * A buffer that is written shares no memory with another argument unless it says so here (the
 * same pointer is refused: KDA_ERR_INVALID_ARG).
 */

/*
 * Bytes of device workspace of kda_gdr_forward (backward = 0) or kda_gdr_backward
 * (backward = 1): per 64-token chunk and value head, the chunk's matrices M and P M (32 KiB),
 * for the backward pass also the chunk's states, corrections and their gradients, for the
 * forward pass also the states of up to 148 sequences and heads.  More sequences, tokens or value
 * heads never need less, so a workspace of the largest call does for all.  A call needs it only
 * while it runs; calls that overlap on the GPU need one each (two captured graphs that may run
 * at once among them).
 */
kda_status_t kda_gdr_workspace_size(int N, int T_total, int Hk, int Hv, int dk, int dv, kda_dtype_t io,
                                    int backward, size_t *bytes);

/*
 * kda_gdr_forward — outputs and final states of N sequences.
 *   initial_state  [N, Hv, dk, dv] fp32, or with initial_index [pages, Hv, dk, dv]; NULL: zeros
 *   initial_index  [N] int32 device: the page each sequence starts from, -1 for zeros; several
 *                  sequences may start from one page.  NULL: sequence n starts from page n.
 *   final_state    as initial_state (may be the same buffer), NULL: not kept
 *   final_index    [N] int32 device: the page each final state goes to, -1: not kept; NULL: n.
 *                  Pages that no sequence names are left as they were.
 *   pages          pages of the two buffers, where an index is given (else ignored)
 *   out            written at every token of the N sequences; rows behind the last are left alone
 *   workspace      kda_gdr_workspace_size(.., 0) bytes, 256-byte aligned
 * Index values are checked on the device: an index out of range counts as -1; of sequences with
 * the same final page the first keeps its state there, and a final page that another sequence
 * starts from (in the same buffer) is not written.  Each sets the device error word
 * (KDA_ERR_INDEX from kda_check_device_error).  A sequence of length 0 passes its state through.
 * A sequence and head whose bounded wait runs out (KDA_ERR_TIMEOUT) leaves its final state as it was.
 */
kda_status_t kda_gdr_forward(const void *q, const void *k, const void *v, const void *g, const void *beta,
                             const float *initial_state, const int *initial_index, void *out, float *final_state,
                             const int *final_index, int pages, const int *cu_seqlens, void *workspace,
                             size_t workspace_bytes, int N, int T_total, int Hk, int Hv, int dk, int dv,
                             kda_dtype_t io, kda_stream_t stream);

/*
 * kda_gdr_backward — gradients of kda_gdr_forward's inputs, given d_out = dL/d out and
 * d_final_state = dL/d final_state (dense [N, Hv, dk, dv] fp32, or NULL for zeros).  The
 * forward pass is recomputed from the inputs; nothing of it need be kept.
 *   initial_state   [N, Hv, dk, dv] fp32 or NULL (zeros)
 *   d_q, d_k        [T_total, Hk, dk] io dtype (written; summed over the value heads of the group)
 *   d_v             [T_total, Hv, dv] io dtype (written)     d_g, d_beta  [T_total, Hv] io dtype (written)
 *   d_initial_state [N, Hv, dk, dv] fp32 (written) or NULL; may be d_final_state
 * Rows of no sequence (behind the last, where T_total is larger than its end) are left as they were.
 *   workspace       kda_gdr_workspace_size(.., 1) bytes, 256-byte aligned
 * No atomics: the same inputs give the same bits.
 */
kda_status_t kda_gdr_backward(const void *q, const void *k, const void *v, const void *g, const void *beta,
                              const float *initial_state, const int *cu_seqlens, const void *d_out,
                              const float *d_final_state, void *d_q, void *d_k, void *d_v, void *d_g, void *d_beta,
                              float *d_initial_state, void *workspace, size_t workspace_bytes, int N, int T_total,
                              int Hk, int Hv, int dk, int dv, kda_dtype_t io, kda_stream_t stream);

/*
 * kda_gdr_decode — T >= 1 tokens of N sequences, token by token, states updated in place (read
 * and written once per call, whatever T).
 *   q, k [N, T, Hk, dk]; v, out [N, T, Hv, dv]; g, beta [N, T, Hv], io dtype
 *   state [N, Hv, dk, dv] fp32, or with index [pages, Hv, dk, dv]
 *   index [N] int32 device: each sequence's page; -1: an idle row, whose out is left alone.  A
 *         page out of range, or one that an earlier row names, makes its row idle and sets the
 *         device error word (KDA_ERR_INDEX).  NULL: sequence n's state is n.
 * Exact fp32 arithmetic in every dtype.  dk, dv in {64, 128}.
 */
kda_status_t kda_gdr_decode(const void *q, const void *k, const void *v, const void *g, const void *beta,
                            float *state, const int *index, int pages, void *out, int N, int T, int Hk, int Hv,
                            int dk, int dv, kda_dtype_t io, kda_stream_t stream);

/*
 * ---- Pages of a state cache ----
 *
 * cache is [layers, pages, page_bytes] of any contents (the states of kda_gdr_decode, or of
 * kda_decode_step with one page a sequence), page_bytes a multiple of 16; refs [pages] int32
 * (device) counts the holders of each page, 0 for a free one.  Everything is decided on the
 * device, so every call can be captured in a graph; bad indices are left out and set the
 * device error word (KDA_ERR_INDEX).
 *
 * kda_pages_fork: for each i < n a free page, lowest first, with the contents of page
 * parents[i] in every layer (zeros for parents[i] = -1); children[i] receives its number and its
 * refs becomes 1.  children[i] = -1 where parents[i] is not a live page (its free page stays
 * free), and, without an error, where no free page is left.  children may not overlap parents.
 */
kda_status_t kda_pages_fork(void *cache, size_t page_bytes, int layers, int pages, int *refs, const int *parents,
                            int *children, int n, kda_stream_t stream);

/*
 * kda_pages_copy: page dst[i] <- page src[i] in every layer (zeros for src[i] = -1; dst[i] = -1:
 * nothing).  A pair is left out, with the error word set, where an index is out of range, where
 * an earlier pair has the same destination, or where its source is another pair's destination.
 */
kda_status_t kda_pages_copy(void *cache, size_t page_bytes, int layers, int pages, const int *src, const int *dst,
                            int n, kda_stream_t stream);

/* kda_pages_free: refs[ids[i]] -= 1 (-1: nothing).  A page that nobody holds is left at 0. */
kda_status_t kda_pages_free(int *refs, int pages, const int *ids, int n, kda_stream_t stream);

/* Bytes of device workspace of kda_pages_compact (at most 8 (pages + 1)). */
kda_status_t kda_pages_workspace_size(int pages, size_t *bytes);

/*
 * kda_pages_compact: moves the m live pages to pages 0 .. m - 1.  Live pages below m stay; the
 * k-th live page at or above m moves to the k-th free page below it, its refs with it.  table
 * [n] int32 (NULL with n = 0) holds page numbers and is renumbered in place (-1 stays; a number
 * of no live page becomes -1 and sets the error word).  live [1] int32 or NULL receives m.
 */
kda_status_t kda_pages_compact(void *cache, size_t page_bytes, int layers, int pages, int *refs, int *table, int n,
                               int *live, void *workspace, size_t workspace_bytes, kda_stream_t stream);

/*
 * kda_set_wait_test_hooks — the failure path of the tensor-core kernels, made testable
 * without a GPU fault.  Those kernels wait on their own mbarriers (tile loads, MMA
 * completion) with a time limit; a wait that runs out sets the device error word, makes
 * the whole CTA stop, wait for everything it already issued (loads, MMAs, copies, stores),
 * free its tensor memory and return, so the context stays usable and the next
 * kda_check_device_error returns KDA_ERR_TIMEOUT.  The paper has no counterpart to this
 * entry point.
 *   wait_limit_ns    limit of each such wait, in ns of %globaltimer; 0 restores the
 *                    default of 2 s
 *   skip_load_chunk  >= 0: in every later launch, the tile load of that chunk index is
 *                    never issued, so the wait for it runs out after the limit (the
 *                    kernel's outputs from that chunk on are then unspecified); -1: off; c <= -2:
 *                    that of chunk -2 - c, in the launch before the walks of kda_gdr_forward and
 *                    kda_gdr_backward alone
 * The settings are process-wide and read at each launch of those kernels; change them only
 * while no call is being made from another host thread.  Always returns KDA_OK.
 */
kda_status_t kda_set_wait_test_hooks(unsigned long long wait_limit_ns, int skip_load_chunk);

/*
 * Synchronises `stream`, then reports and clears the library's device error word
 * (set by a kernel whose bounded wait gave up) and any sticky CUDA error.
 * Returns KDA_OK, KDA_ERR_TIMEOUT, KDA_ERR_INDEX or KDA_ERR_CUDA.
 */
kda_status_t kda_check_device_error(kda_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H */
