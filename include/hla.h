/*
 * hla.h — C ABI of libhla, the GB300 (sm_103a) hybrid linear-attention layer.
 *
 * The layer replaces softmax attention in a frozen LLaMA/Qwen backbone, as in
 * "The Key to Going Linear: Analysis-Driven Transformer Linearization"
 * (summary page "迈向线性的关键：分析驱动的 Transformer 线性化"):
 *   - exact softmax over a fixed cache budget of n_sinks sink tokens plus a
 *     sliding window (section 填补近似缺口的实用设计);
 *   - a Gated DeltaNet state S (d x d, fp32, one per query head) that absorbs
 *     every non-sink token when it leaves the window (GDN equation, section
 *     线性注意力替换机制, with a scalar gate alpha = exp(g));
 *   - keys and queries of the linear branch go RoPE -> causal depthwise
 *     short conv (width 8) -> L2 norm (section 实践建议, item 3);
 *   - o_t = softmax_{j in sinks U window}(q_t k_j / sqrt(d)) V
 *           + lambda_h * qhat_t^T S_t,
 *     the inference-time weighting of the two branches of "Untangling
 *     Component Imbalance in Hybrid Linear Attention Conversion", section
 *     关键设计 (1).
 *
 * Conventions for every entry point:
 *   - All tensor pointers are DEVICE pointers unless marked "host".  The
 *     caller owns every buffer; the library allocates no device memory and
 *     never synchronises the stream, except hla_check_device_error.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default).
 *     Every kernel of a call runs on it, some with programmatic dependent
 *     launch; the library creates no stream or event of its own.
 *   - Argument errors are detected on the host, before any launch, and return
 *     HLA_ERR_INVALID_ARG / HLA_ERR_UNSUPPORTED without touching the GPU.
 *   - A failed launch returns HLA_ERR_CUDA (the CUDA error is consumed).
 *   - Problems found on the device (malformed cu_seqlens, a bounded wait that
 *     ran out) are recorded in a device error word and read back with
 *     hla_check_device_error / hla_check_workspace_error.
 *   - Results are deterministic: fixed reduction order, no atomics in the
 *     numeric path.
 *   - Tensors are dense and row-major; every pointer must be 16-byte aligned.
 *   - Positions restart at 0 at the start of every sequence.
 */
#ifndef HLA_H
#define HLA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define HLA_API __attribute__((visibility("default")))

/* status codes */
#define HLA_OK 0
#define HLA_ERR_INVALID_ARG 1 /* bad pointer, size, alignment or parameter */
#define HLA_ERR_UNSUPPORTED 2 /* valid but not implemented (e.g. head_dim 96) */
#define HLA_ERR_STATE 3       /* decode state inconsistent (device error word) */
#define HLA_ERR_CUDA 4        /* a CUDA call or launch failed */
#define HLA_ERR_TIMEOUT 5     /* a bounded device-side wait ran out */
#define HLA_ERR_WORKSPACE 6   /* workspace smaller than hla_prefill_workspace_bytes */

/* element type of q, k, v, out and of the KV ring */
#define HLA_DTYPE_F32 0
#define HLA_DTYPE_BF16 1

/* flags */
#define HLA_FLAG_L2NORM_Q 0x1u       /* qhat = L2(conv(RoPE q)); set by default */
#define HLA_FLAG_SOFTMAX_OFF 0x2u    /* test hook: drop the softmax branch */
#define HLA_FLAG_LINEAR_OFF 0x4u     /* test hook: drop the linear branch */
#define HLA_FLAG_GDN_RECURRENT 0x8u  /* use the token-serial fp32 GDN kernel in
                                        place of the chunked tensor-core one */
#define HLA_FLAG_GLA 0x10u           /* gated linear attention in place of the
                                        delta rule: S <- alpha S + khat vhat^T
                                        (no erase term, beta unused), the other
                                        update of section 线性注意力替换机制 */
#define HLA_FLAG_GDN_SCAN 0x40u      /* token-serial GDN path (fp32 layers, head
                                        dim 64, or with HLA_FLAG_GDN_RECURRENT)
                                        in its context-parallel form: each
                                        sequence's absorptions are cut into
                                        parts; every part's state map
                                        S -> P S + R is formed at once, a scan
                                        over the parts gives their start
                                        states, then all parts run at once.
                                        Three times the work on many more
                                        SMs: for long sequences with few
                                        (sequence, head) units.  No effect on
                                        the tensor-core path. */
#define HLA_FLAG_TEST_STALL 0x20u    /* test hook (tensor-core path): the GDN
                                        state kernel loads nothing, so its
                                        bounded waits run out after about a
                                        millisecond; the call completes and the
                                        workspace error word reads back
                                        HLA_ERR_TIMEOUT.  Outputs are then
                                        undefined. */

/* Layer shape.  n_q_heads must be a multiple of n_kv_heads (grouped-query
 * attention: q-head h reads kv-head h / (n_q_heads / n_kv_heads)).
 * head_dim: 64 or 128.  n_sinks >= 0, window >= 1 (the window includes the
 * current token).  conv_width: 8.  rope_base: RoPE base (rotate-half pairs
 * (i, i + d/2), angle p * base^(-2i/d)).  flags: HLA_FLAG_*. */
typedef struct hla_params {
    int n_q_heads;
    int n_kv_heads;
    int head_dim;
    int n_sinks;
    int window;
    int conv_width;
    float rope_base;
    int dtype;
    unsigned flags;
} hla_params;

/* Decode state of n_seqs sequences: caller-owned device buffers.
 *   S         fp32  [N, Hq, d, d]     GDN state, S[n][h][i][j], i = key dim
 *   k_ring    dtype [N, Hkv, n_sinks + window, d]  RoPE'd keys: slot p for a
 *             sink p < n_sinks, slot n_sinks + (p - n_sinks) % window otherwise
 *   v_ring    dtype [N, Hkv, n_sinks + window, d]  raw values, same slots
 *   pend_k    fp32  [N, Hkv, window + 1, d]  khat of tokens still in the window,
 *             slot p % (window + 1)
 *   pend_v    fp32  [N, Hkv, window + 1, d]  vhat, same slots
 *   pend_g    fp32  [N, Hq, window + 1]      log-gate g of those tokens
 *   pend_beta fp32  [N, Hq, window + 1]      beta of those tokens
 *   conv_q    fp32  [N, 7, Hq, d]   RoPE'd q of positions p-7 .. p-1
 *   conv_k    fp32  [N, 7, Hkv, d]  RoPE'd k of positions p-7 .. p-1
 *   conv_v    fp32  [N, 7, Hkv, d]  raw v of positions p-7 .. p-1
 *   pos       int64 [N]  next position of each sequence
 *   err       int32 [4]  device error word (0 = fine)
 *   scratch   per-step temporaries of hla_decode_step (size from
 *             hla_state_bytes); dead between calls, not part of the state
 * Every buffer but scratch is the resumable state: copying them out and back
 * in resumes decoding exactly. */
typedef struct hla_state {
    float* S;
    void* k_ring;
    void* v_ring;
    float* pend_k;
    float* pend_v;
    float* pend_g;
    float* pend_beta;
    float* conv_q;
    float* conv_k;
    float* conv_v;
    int64_t* pos;
    int32_t* err;
    void* scratch;
} hla_state;

/* byte sizes of the hla_state buffers, in struct order */
typedef struct hla_state_sizes {
    size_t S, k_ring, v_ring, pend_k, pend_v, pend_g, pend_beta, conv_q, conv_k, conv_v, pos, err, scratch;
} hla_state_sizes;

/* Human-readable name of a status code (static string). */
HLA_API const char* hla_status_string(int status);

/* Sizes of the decode-state buffers for n_seqs sequences (host only). */
HLA_API int hla_state_bytes(const hla_params* params, int n_seqs, hla_state_sizes* out);

/* Workspace bytes hla_prefill needs for total_tokens tokens in n_seqs
 * sequences (host only).  The workspace holds the feature-path outputs and
 * the linear-branch output between kernels. */
HLA_API int hla_prefill_workspace_bytes(const hla_params* params, int64_t total_tokens, int n_seqs,
                                        size_t* bytes);

/* Zeroes every buffer of `st` (positions 0, empty state, empty caches).
 * Asynchronous on `stream`. */
HLA_API int hla_state_init(const hla_params* params, int n_seqs, const hla_state* st, void* stream);

/* Prefill: runs the layer over n_seqs packed sequences.
 *   q [total, Hq, d], k, v [total, Hkv, d]  pre-RoPE, in params->dtype
 *   g, beta [total, Hq] fp32      log alpha (<= 0) and beta in (0, 1), per
 *                                 token and query head
 *   lambda [Hq] fp32              weight of the linear branch per query head
 *   conv_wq [Hq*d, 8], conv_wk [Hkv*d, 8], conv_wv [Hkv*d, 8] fp32  depthwise
 *                                 filters, tap 7 on the current token
 *   cu_seqlens int32 [n_seqs + 1] (device) sequence offsets: 0 = c_0 <= c_1
 *                                 <= ... <= c_n = total_tokens
 *   out [total, Hq, d]            params->dtype
 *   st                            NULL, or a state freshly set up by
 *                                 hla_state_init for n_seqs sequences: it
 *                                 receives everything decoding needs.  A
 *                                 state with a position other than 0 is
 *                                 not fresh: the first kernel flags it in
 *                                 the state's error word (then
 *                                 hla_check_device_error returns
 *                                 HLA_ERR_STATE) and its contents are
 *                                 undefined; `out` is unaffected
 *   ws, ws_bytes                  workspace of at least
 *                                 hla_prefill_workspace_bytes bytes
 * With total_tokens == 0 the per-token pointers may be NULL.
 * Asynchronous; no allocation, no synchronisation.  Malformed cu_seqlens are
 * clamped on the device (no out-of-range access) and flagged in the workspace
 * error word. */
HLA_API int hla_prefill(const hla_params* params, const void* q, const void* k, const void* v,
                        const float* g, const float* beta, const float* lambda,
                        const float* conv_wq, const float* conv_wk, const float* conv_wv,
                        const int32_t* cu_seqlens, int n_seqs, int64_t total_tokens, void* out,
                        const hla_state* st, void* ws, size_t ws_bytes, void* stream);

/* hla_prefill without a caller-supplied workspace.  The paper has no
 * counterpart: this entry point exists for callers that cannot call
 * cudaMalloc, for instance a plugin inside a host framework that owns every
 * byte of device memory through its own pool and gives the plugin no
 * allocator, or a latency-critical caller that cannot afford the implicit
 * device-wide synchronisation of cudaMalloc/cudaFree.
 * Arguments and results are those of hla_prefill; the scratch memory comes
 * from a 64 MiB buffer inside the library.  That buffer is device memory of
 * every process that loads libhla.so, on every GPU where the library's
 * device code gets loaded (at context creation under eager module loading;
 * under lazy loading, the CUDA default, once this entry point first runs on
 * that GPU), whether or not the process ever calls hla_prefill_noalloc, and
 * it is held until the process exits.  Prefills whose
 * hla_prefill_workspace_bytes exceeds 64 MiB (about 1,300 tokens of a
 * 32 q / 8 kv head, head_dim 128 bf16 layer) return HLA_ERR_WORKSPACE before
 * any GPU work.
 * The first call on each device (and the first after that device's context
 * was reset) looks up the buffer's device address, a host-side set-up step;
 * make that first call before any stream capture.
 * It allocates nothing: no cudaMalloc, no cudaFree.
 * All calls share the one buffer and each overwrites what the last left in
 * it: calls that overlap on the GPU (other streams, other threads) race, so
 * order them on one stream.  Problems found on the device (malformed
 * cu_seqlens, a bounded wait that ran out) land in the buffer's error word:
 * read it with hla_prefill_noalloc_check_error. */
HLA_API int hla_prefill_noalloc(const hla_params* params, const void* q, const void* k,
                                const void* v, const float* g, const float* beta,
                                const float* lambda, const float* conv_wq, const float* conv_wk,
                                const float* conv_wv, const int32_t* cu_seqlens, int n_seqs,
                                int64_t total_tokens, void* out, const hla_state* st, void* stream);

/* The device error word of hla_prefill_noalloc's buffer on the current
 * device, as hla_check_workspace_error reads a workspace's: synchronises
 * `stream`, stores the word in *code (may be NULL), clears it, and returns
 * HLA_OK if it was zero, else the matching HLA_ERR_* status.  Allocates
 * nothing. */
HLA_API int hla_prefill_noalloc_check_error(void* stream, int32_t* code);

/* One decode step for every sequence of `st`: token pos[n] of sequence n.
 *   q [N, Hq, d], k, v [N, Hkv, d]  (params->dtype), g, beta [N, Hq] fp32,
 *   lambda and conv filters as for hla_prefill, out [N, Hq, d].
 * The token leaving the window (position pos - window, if not a sink) is
 * absorbed into S first; then the new token's output is formed; pos += 1.
 * At most 8 query heads per kv head (else HLA_ERR_UNSUPPORTED).  A sequence
 * whose pos is negative (no prefill or decode step leaves one) is left as it
 * is, its output row is undefined, and the state's error word reports
 * HLA_ERR_STATE.  Asynchronous. */
HLA_API int hla_decode_step(const hla_params* params, int n_seqs, const void* q, const void* k,
                            const void* v, const float* g, const float* beta, const float* lambda,
                            const float* conv_wq, const float* conv_wk, const float* conv_wv,
                            const hla_state* st, void* out, void* stream);

/* Prefill that continues from a decode state: appends the tokens of each
 * sequence to the context st already holds (after hla_prefill with a state,
 * hla_decode_step, or an earlier call of this one), the first at position
 * st->pos[n].  Arguments as for hla_prefill, except that st is required and
 * is read and advanced: the conv histories, the window keys and values, the
 * tokens still waiting to be absorbed and S carry across the boundary, and
 * pos[n] grows by the sequence's token count.  The outputs and the state
 * afterwards are those of one prefill over the whole sequence (equivalently,
 * of decoding the new tokens one at a time).  A state that never passed
 * through hla_state_init starts from whatever its buffers hold; pos < 0 is
 * flagged in the state's error word (HLA_ERR_STATE) and that sequence is left
 * as it is (its output rows are undefined).  ws, ws_bytes: a workspace of at
 * least hla_prefill_continue_workspace_bytes bytes (its error word as for
 * hla_prefill).  On the tensor-core path (bf16, head_dim 128, 1, 2, 4 or 8
 * query heads per kv head) each sequence's cached sinks and window are laid
 * in front of its new tokens, the positions between them left out, and the
 * prefill's softmax and chunked GDN kernels run on these rows from the cached
 * S; the other layers take a token-serial path (one CTA per query head).
 * There, a sequence table whose sequences overlap (cu_seqlens decreasing once
 * clamped to [0, total_tokens]) is flagged in the state's error word (the
 * sequence-table code, 1) and the outputs and the state are undefined; every
 * write still stays inside ws, out and the state.
 * Asynchronous; no allocation. */
HLA_API int hla_prefill_continue(const hla_params* params, const void* q, const void* k, const void* v,
                                 const float* g, const float* beta, const float* lambda,
                                 const float* conv_wq, const float* conv_wk, const float* conv_wv,
                                 const int32_t* cu_seqlens, int n_seqs, int64_t total_tokens, void* out,
                                 const hla_state* st, void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes hla_prefill_continue needs for total_tokens new tokens in
 * n_seqs sequences (host only): on the tensor-core path the prefill's
 * workspace for the new tokens plus every sequence's n_sinks + window cached
 * rows, and the extended rows' v, g, beta and output. */
HLA_API int hla_prefill_continue_workspace_bytes(const hla_params* params, int64_t total_tokens, int n_seqs,
                                                 size_t* bytes);

/* Component-usage diagnostics of a prefill (synthetic analysis; not part of
 * the layer's output path).  Arguments as for hla_prefill, without a decode
 * state, plus:
 *   out [total, Hq, d]      params->dtype, scratch for the branch outputs:
 *                           afterwards it holds lambda_h o_lin (the linear
 *                           branch alone)
 *   branch_sq [n_seqs, Hq, 2] fp32: per sequence and q-head, the sums over
 *                           its positions of |o_sm|^2 (index 0) and of
 *                           |lambda_h o_lin|^2 (index 1), from the rounded
 *                           branch outputs: how much each branch carries
 *                           ("Untangling Component Imbalance in Hybrid Linear
 *                           Attention Conversion", sections 摘要, 方法详解)
 *   key_stats [total, Hkv, 2] fp32: per position p and kv head, with u_i the
 *                           RoPE'd key i scaled to unit length and m_p the mean
 *                           of u_0..u_p within the sequence: the key
 *                           concentration |m_p| (index 0) and the projection
 *                           residual |u_p - (mhat_p . u_p) mhat_p| (index 1;
 *                           1 where m_p = 0), the quantities of the analysis in
 *                           "迈向线性的关键：分析驱动的 Transformer 线性化",
 *                           sections 从 softmax 到 delta 规则的一阶近似 (Lemma 2)
 *                           and 填补近似缺口的实用设计
 *   ws, ws_bytes            as for hla_prefill
 * Runs the prefill twice (each branch alone; HLA_FLAG_SOFTMAX_OFF and
 * HLA_FLAG_LINEAR_OFF in params are overridden) and three reduction kernels.
 * Asynchronous; no allocation. */
HLA_API int hla_prefill_diagnostics(const hla_params* params, const void* q, const void* k, const void* v,
                                    const float* g, const float* beta, const float* lambda,
                                    const float* conv_wq, const float* conv_wk, const float* conv_wv,
                                    const int32_t* cu_seqlens, int n_seqs, int64_t total_tokens, void* out,
                                    float* branch_sq, float* key_stats, void* ws, size_t ws_bytes,
                                    void* stream);

/* Workspace bytes hla_backward needs for total_tokens tokens in n_seqs
 * sequences (host only).  fp32 throughout: the recomputed features and the
 * per-head gradients before the kv-group sums (about 10 T Hq d + 6 T Hkv d
 * floats for T tokens), the softmax rows' max, sum and D (3 T Hq), the GDN
 * state every 64 absorptions ((T / 64 + n_seqs + 1) Hq d^2), the states of
 * one 64-absorption block per sequence and q-head (n_seqs Hq 8 d^2 for d 128,
 * 4 d^2 for d 64), and the sink keys' partial sums per 64-query block
 * (2 (T / 64 + n_seqs) Hq n_sinks d). */
HLA_API int hla_backward_workspace_bytes(const hla_params* params, int64_t total_tokens, int n_seqs,
                                         size_t* bytes);

/* Backward of the layer: the gradients of sum(dout . o) with respect to every
 * input of hla_prefill, for the training of the layer's new parameters (the
 * gates, beta, lambda and the conv filters) on a frozen backbone ("迈向线性的
 * 关键：分析驱动的 Transformer 线性化", section 实践建议).  Arguments q .. n_seqs,
 * total_tokens as for hla_prefill, plus:
 *   dout [total, Hq, d]        params->dtype, the gradient of the output
 *   dq [total, Hq, d], dk, dv [total, Hkv, d]   fp32 (a kv head's gradient
 *                              sums over the q-heads that read it)
 *   dg, dbeta [total, Hq]      fp32 (zero for tokens no state absorbs: the
 *                              sinks and the last `window` positions)
 *   dlambda [Hq]               fp32
 *   dconv_wq [Hq*d, 8], dconv_wk, dconv_wv [Hkv*d, 8]   fp32
 *   ws, ws_bytes               workspace of at least
 *                              hla_backward_workspace_bytes bytes
 * Every output is overwritten.  The forward is recomputed inside (the
 * features, the softmax row statistics, the GDN states), in fp32 from the
 * stored inputs, whatever the forward path (the tensor-core prefill's bf16 and
 * fp16 operands are not reproduced).  GDN: per sequence and q-head a cluster
 * of 8 CTAs, each with d / 8 value columns of S; a forward pass stores the
 * state every 64 absorptions, then per 64-absorption block (last first) the
 * states every 8 (d 128) or 16 (d 64) absorptions are recomputed, and per such
 * stage its states are held in registers while the read-out and absorption
 * steps run backwards.  Softmax: 64 x 64 fp32 tiles, per query block then per
 * key block.  HLA_FLAG_GLA differentiates the GLA update;
 * HLA_FLAG_SOFTMAX_OFF / HLA_FLAG_LINEAR_OFF the layer without that branch;
 * HLA_FLAG_GDN_RECURRENT and HLA_FLAG_GDN_SCAN have no effect; HLA_FLAG_TEST_STALL is rejected
 * (HLA_ERR_INVALID_ARG).  Deterministic (fixed reduction order, no atomics).
 * Malformed cu_seqlens are clamped on the device and flagged in the
 * workspace's error word (hla_check_workspace_error).  With total_tokens == 0
 * the per-token pointers may be NULL and the parameter gradients are zeroed.
 * Asynchronous; no allocation. */
HLA_API int hla_backward(const hla_params* params, const void* q, const void* k, const void* v,
                         const float* g, const float* beta, const float* lambda,
                         const float* conv_wq, const float* conv_wk, const float* conv_wv,
                         const int32_t* cu_seqlens, int n_seqs, int64_t total_tokens, const void* dout,
                         float* dq, float* dk, float* dv, float* dg, float* dbeta, float* dlambda,
                         float* dconv_wq, float* dconv_wk, float* dconv_wv, void* ws, size_t ws_bytes,
                         void* stream);

/* ---------------------------------------------------------------------------
 * The full softmax layers beside the hybrid ones: a linearised backbone keeps
 * some of its layers (and its teacher all of them) as plain causal attention.
 * Rotary positions, attention over packed prompts with its gradient, a paged
 * key / value cache kept in 8 bits, and the decode step over that cache.
 * ------------------------------------------------------------------------- */

/* element type of a cache (hla_cache_params.cache_dtype): 8-bit floats (4
 * exponent, 3 mantissa bits, largest 448) with one power of two per row */
#define HLA_DTYPE_E4M3 2

/* which elements of a head form a rotated pair (r = rot_dim) */
#define HLA_ROPE_HALF 0        /* (i, i + r/2) */
#define HLA_ROPE_INTERLEAVED 1 /* (2i, 2i + 1) */

/* how the angle per position w_i = base^(-2i/r) is scaled for long contexts */
#define HLA_ROPE_SCALE_NONE 0
#define HLA_ROPE_SCALE_LINEAR 1 /* w_i / factor */
#define HLA_ROPE_SCALE_BANDS 2  /* by t_i = original_len w_i / (2 pi), the turns of the original context: t_i <= low
                                   gives w_i / factor, t_i >= high gives w_i, linear in t_i between */
#define HLA_ROPE_SCALE_YARN 3   /* by index: with x(t) = r ln(original_len / (2 pi t)) / (2 ln base), pairs below
                                   floor(x(high)) keep w_i, above ceil(x(low)) get w_i / factor, linear in i between
                                   (both ends clamped to [0, r - 1]); rotated values times 0.1 ln(factor) + 1 */

/* Rotary positions of q and k.  head_dim: even, 2 to 256.  rot_dim: even, 2 to
 * head_dim; the elements past it are copied.  n_q_heads or n_kv_heads may be 0
 * when that tensor is absent.  low, high: the band edges in turns (read with
 * BANDS and YARN; 0 for both = 1 and 4 for BANDS, 1 and 32 for YARN).
 * q_stride, k_stride: elements from a token to the next in q and k (0: dense;
 * otherwise at least heads * head_dim: the slices of a fused projection).  The
 * outputs are dense; or, given the address of the input, take its stride. */
typedef struct hla_rope_params {
    int n_q_heads;
    int n_kv_heads;
    int head_dim;
    int rot_dim;
    int layout;
    int scaling;
    int dtype;
    int original_len;
    double base;
    double factor;
    double low;
    double high;
    int64_t q_stride;
    int64_t k_stride;
} hla_rope_params;

/* Host only: the scaled angle per position of every pair (w, rot_dim / 2
 * doubles) and the factor on the rotated values. */
HLA_API int hla_rope_frequencies(const hla_rope_params* params, double* w, double* gain);

/* Rotates q [total, Hq, d] and k [total, Hkv, d] (params->dtype; either may be
 * NULL, with its output) to the positions given per token (int64, device, any
 * value): a pair (a, b) at angle t becomes gain (a cos t - b sin t, b cos t +
 * a sin t).  In place where an output is its input's address.  Angles are
 * formed as 64-bit fractions of a turn: exact products with frequencies of
 * double precision, off by about 2^-53 of p w_i at any position p.
 * The outputs must not overlap the inputs in any other way.  Asynchronous. */
HLA_API int hla_rope(const hla_rope_params* params, const void* q, const void* k, const int64_t* positions,
                     int64_t total_tokens, void* q_out, void* k_out, void* stream);

/* Its gradient: rotates back, times gain (dq_out, dk_out are the gradients of
 * hla_rope's outputs, with q_stride and k_stride; dq, dk those of its inputs). */
HLA_API int hla_rope_backward(const hla_rope_params* params, const void* dq_out, const void* dk_out,
                              const int64_t* positions, int64_t total_tokens, void* dq, void* dk, void* stream);

/* Softmax attention.  n_q_heads a multiple of n_kv_heads; head_dim 64 or 128;
 * dtype of q, k, v, out and the gradients; scale: on the scores (0: 1 /
 * sqrt(head_dim)).  q_stride, k_stride, v_stride: elements from a token to the
 * next (0: dense; otherwise at least heads * head_dim and a multiple of 16
 * bytes).  out, dout and the gradients are dense. */
typedef struct hla_attn_params {
    int n_q_heads;
    int n_kv_heads;
    int head_dim;
    int dtype;
    float scale;
    int reserved; /* 0 */
    int64_t q_stride;
    int64_t k_stride;
    int64_t v_stride;
} hla_attn_params;

/* Workspace bytes of hla_attention, or (backward != 0) of
 * hla_attention_backward: for few rows over many keys, and for few heads, more
 * than for large calls, since such work is cut into parts whose results lie in
 * the workspace.  With less than that, a call takes as many parts as there is
 * room for (slower; the bits of a result depend on the number of parts); the
 * least is 256 bytes, and for the gradient what one part needs, which grows
 * with total_q, total_k and n_seqs: the workspace of the largest call serves
 * every smaller one.
 * Below that a call returns HLA_ERR_WORKSPACE.  The first 16 bytes are the error
 * word: zero them before the first use; calls only ever set it,
 * hla_check_workspace_error reads and clears it.  Two calls that may run at the
 * same time need a workspace each. */
HLA_API int hla_attention_workspace_bytes(const hla_attn_params* params, int64_t total_q, int64_t total_k,
                                          int n_seqs, int backward, size_t* bytes);

/* Causal attention over n_seqs packed sequences.
 *   q [total_q, Hq, d], k, v [total_k, Hkv, d]
 *   cu_seqlens_q, cu_seqlens_k int32 [n_seqs + 1] (device): offsets of each
 *       sequence's query and key rows, 0 = c_0 <= ... <= c_n <= total;
 *       cu_seqlens_k NULL: the same as cu_seqlens_q (total_k = total_q).  Row
 *       i of a sequence with Lq queries and Lk keys sees keys j <= i + Lk - Lq
 *       (whole prompts: Lk = Lq; a prompt's next chunk behind its earlier
 *       keys: Lk > Lq).
 *   out [total_q, Hq, d], lse fp32 [total_q, Hq]: the natural log of the sum
 *       of exponentials (what hla_attention_backward needs)
 * A row that sees no key has out 0 and lse -infinity.  What a row does not see
 * does not reach it, infinities and NaN included (the padding of a batch may
 * hold anything).  Rows at and past c_n are left as they were.  A malformed
 * table is clamped on the device (no access out of range) and flagged in the
 * workspace's error word.  Outputs must not overlap inputs.  bf16 layers run on
 * the tensor cores: fp32 scores and sums, probabilities rounded to bf16 for
 * their product with v.  Asynchronous; deterministic (for a workspace size). */
HLA_API int hla_attention(const hla_attn_params* params, const void* q, const void* k, const void* v,
                          const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int n_seqs, int64_t total_q,
                          int64_t total_k, void* out, float* lse, void* ws, size_t ws_bytes, void* stream);

/* Gradients of sum(dout . out) from hla_attention's inputs, out and lse:
 * dq [total_q, Hq, d], dk, dv [total_k, Hkv, d] (a kv head's sums over the
 * query heads that read it), in params->dtype from fp32 sums.  Keys that no
 * row sees have gradients 0; rows at and past c_n are left as they were.
 * bf16 layers: P and dS rounded to bf16 for their products; dq and dk where
 * dS nearly cancels are not left with the rounding of `out` (dq to about
 * 4 x 2^-8 of its size).
 * Infinities and NaN of keys do not reach dq of rows before them; those of a
 * row's dout and q may reach dk and dv of keys up to 127 after it in its own
 * sequence (bf16 layers).  Outputs must not overlap inputs or each other.
 * Asynchronous; deterministic (fixed order of sums, no atomics). */
HLA_API int hla_attention_backward(const hla_attn_params* params, const void* q, const void* k, const void* v,
                                   const void* out, const float* lse, const void* dout,
                                   const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int n_seqs,
                                   int64_t total_q, int64_t total_k, void* dq, void* dk, void* dv, void* ws,
                                   size_t ws_bytes, void* stream);

/* A paged key / value cache.  dtype: of the rows written and read (F32 or
 * BF16); cache_dtype: HLA_DTYPE_E4M3, or dtype itself (kept as it is).
 * page_size: tokens per page, a multiple of 16; n_pages: pages in the pool;
 * max_pages: entries per sequence in the page table. */
typedef struct hla_cache_params {
    int n_kv_heads;
    int head_dim;
    int dtype;
    int cache_dtype;
    int page_size;
    int n_pages;
    int max_pages;
    int reserved; /* 0 */
} hla_cache_params;

/* Caller-owned device buffers (every pointer 16-byte aligned):
 *   k, v          cache_dtype [n_pages, Hkv, page_size, d]
 *   k_exp, v_exp  uint8 [n_pages, Hkv, page_size] (E4M3 only, else NULL): the
 *                 row's value is its 8-bit floats times 2^(byte - 127)
 *   page_table    int32 [n_seqs, max_pages]: position p of a sequence is row
 *                 p % page_size of page page_table[n][p / page_size]
 *   err           int32 [4], the error word: zero it before the first use; set
 *                 by a position or page number out of range (HLA_ERR_STATE) */
typedef struct hla_cache {
    void* k;
    void* v;
    uint8_t* k_exp;
    uint8_t* v_exp;
    const int32_t* page_table;
    int32_t* err;
} hla_cache;

/* Bytes of k (and of v), and of k_exp (and of v_exp; 0 if not E4M3). */
HLA_API int hla_cache_bytes(const hla_cache_params* params, size_t* rows, size_t* exponents);

/* Writes k, v [total, Hkv, d] (packed sequences, cu_seqlens as for
 * hla_attention) into the cache: row i of sequence n at position start[n] + i
 * (start: int64, device).  E4M3: the row's power of two is the smallest 2^e
 * with max |x| <= 448 2^e (e >= -127; over the row's finite values), and each
 * value is rounded once, to the nearest 8-bit float of x 2^-e (infinities to
 * the largest, NaN stays NaN).  A row whose position or page is out of range
 * is skipped and flagged.  No two rows may be the same place.  Asynchronous. */
HLA_API int hla_cache_write(const hla_cache_params* params, const hla_cache* cache, const void* k, const void* v,
                            const int32_t* cu_seqlens, const int64_t* start, int n_seqs, int64_t total_tokens,
                            void* stream);

/* Reads rows back in params->dtype: the positions start[n] + i into k, v
 * [total, Hkv, d], as hla_cache_write takes them (exact but for values below
 * the type's smallest normal).  A row out of range reads as zeros and is
 * flagged; rows at and past cu_seqlens[n_seqs] are left as they were. */
HLA_API int hla_cache_read(const hla_cache_params* params, const hla_cache* cache, const int32_t* cu_seqlens,
                           const int64_t* start, int n_seqs, int64_t total_tokens, void* k, void* v, void* stream);

/* Workspace bytes of hla_attention_decode (no error word: flags go to the
 * cache's).  Two calls that may run at the same time need one each. */
HLA_API int hla_attention_decode_workspace_bytes(const hla_attn_params* params, const hla_cache_params* cache_params,
                                                 size_t* bytes);

/* One query token per sequence over the cache: q [n_seqs, Hq, d] (q_stride
 * applies) attends to positions 0 .. lens[n] - 1 (int64, device; the token's
 * own key and value written before), into out [n_seqs, Hq, d].  A sequence
 * with no keys has out 0.  Keys whose page is out of range, and positions past
 * max_pages * page_size, are left out and flagged; a negative length counts as
 * 0 and is flagged.  A cache of more than 2^32 - 2 rows is HLA_ERR_UNSUPPORTED
 * here.  The heads, head_dim and dtype of both parameter sets must
 * agree.  Asynchronous; deterministic. */
HLA_API int hla_attention_decode(const hla_attn_params* params, const hla_cache_params* cache_params,
                                 const hla_cache* cache, const void* q, const int64_t* lens, int n_seqs, void* out,
                                 void* ws, size_t ws_bytes, void* stream);

/* As hla_check_device_error, for a cache's error word. */
HLA_API int hla_check_cache_error(const hla_cache* cache, void* stream, int32_t* code);

/* ---------------------------------------------------------------------------
 * What stands around a layer's mixing: the norm in front of it (or of its
 * heads) with the residual's addition, the frozen projections in 4 bits, and a
 * gated linear recurrence as the mixing of layers that keep a vector of state.
 * ------------------------------------------------------------------------- */

/* Root-mean-square norm of rows of n_cols values, n_heads of them per token (1:
 * the hidden rows; more: every head of q or k).  dtype of x, residual, weight,
 * sum; out_dtype: dtype, or HLA_DTYPE_E4M3 (8-bit floats with one power of two
 * per `group` values: 32, 128 (n_cols a multiple of it) or 0, the whole row
 * (n_cols a multiple of 16); then x, residual, weight, sum start on 16 bytes and
 * the strides are multiples of 16 bytes).  offset: added to the weight (some
 * backbones keep weight - 1).  x_stride, residual_stride: elements from a token
 * to the next (0: dense; otherwise at least n_heads * n_cols).  Outputs are
 * dense.  n_cols up to 2^20. */
typedef struct hla_norm_params {
    int n_cols;
    int n_heads;
    int dtype;
    int out_dtype;
    int group;
    float eps;
    float offset;
    int reserved; /* 0 */
    int64_t x_stride;
    int64_t residual_stride;
} hla_norm_params;

/* s = x + residual, rounded to dtype; out = s / sqrt(mean(s^2) + eps) * (offset +
 * weight), from fp32 sums: a row whose sum of squares passes 2^128 (values of
 * 1.8e19 / sqrt(n_cols)) has an infinite mean and finite values become 0; without
 * eps a row needs a mean of 2^-126 at least (values of 1.1e-19).
 *   x, residual [tokens, n_heads, n_cols]   residual may be NULL (s = x)
 *   weight [n_cols]          NULL: out = s / sqrt(mean(s^2) + eps)
 *   out [tokens, n_heads, n_cols]           out_dtype
 *   exp uint8 [tokens, n_heads, n_cols / group] (1 for group 0; E4M3, else NULL):
 *       a value is its 8-bit float times 2^(byte - 127), the smallest power that
 *       keeps the group's finite values within 448 (infinities become the
 *       largest, NaN stays NaN)
 *   sum [tokens, n_heads, n_cols]           s; needed with a residual, else NULL
 * sum (or out, of type dtype) may be x or the residual itself where that is dense;
 * outputs must not overlap anything in another way.  Asynchronous;
 * deterministic. */
HLA_API int hla_rms_norm(const hla_norm_params* params, const void* x, const void* residual, const void* weight,
                         int64_t tokens, void* out, uint8_t* exp, void* sum, void* stream);

/* Workspace bytes of hla_rms_norm_backward with a weight (no error word; they
 * depend on n_cols alone).  Two calls that may run at the same time need one
 * each. */
HLA_API int hla_rms_norm_backward_workspace_bytes(const hla_norm_params* params, size_t* bytes);

/* Gradients of sum(dout . out) (+ sum(dsum . sum), dsum may be NULL) with respect
 * to s (the gradient of x and of the residual alike) and the weight: s is
 * hla_rms_norm's `sum` (or x, without a residual; x_stride applies), dout, dsum
 * and dx [tokens, n_heads, n_cols] dense in dtype, dweight fp32 [n_cols] (NULL:
 * not wanted; it needs the weight).  Of 8-bit outputs, dout is the gradient of the
 * values that they stand for.  dx may be dout or dsum.  ws may be NULL without
 * dweight.  Asynchronous; deterministic. */
HLA_API int hla_rms_norm_backward(const hla_norm_params* params, const void* s, const void* weight, const void* dout,
                                  const void* dsum, int64_t tokens, void* dx, float* dweight, void* ws,
                                  size_t ws_bytes, void* stream);

/* Gated linear recurrence h_t = exp(g_t) h_{t-1} + x_t of n_channels values,
 * states in fp32.  gate_dim: channels in a row that share a gate (1, or 64 or 128
 * of a head; n_channels a multiple of it).  dtype of x and out (and their
 * gradients), gate_dtype of g: F32 or BF16 each.  x_stride, g_stride: elements
 * from a token to the next (0: dense; otherwise at least n_channels, n_channels /
 * gate_dim, and below 2^32).  out, dout and the gradients are dense. */
typedef struct hla_recurrence_params {
    int n_channels;
    int gate_dim;
    int dtype;
    int gate_dtype;
    int64_t x_stride;
    int64_t g_stride;
} hla_recurrence_params;

/* Workspace bytes of hla_recurrence and hla_recurrence_backward; that of the
 * largest call serves every smaller one of the same params.  The first 16 bytes
 * are the error word, as in hla_attention_workspace_bytes.  Two calls that may
 * run at the same time need a workspace each. */
HLA_API int hla_recurrence_workspace_bytes(const hla_recurrence_params* params, int64_t total_tokens, size_t* bytes);

/* The recurrence over n_seqs packed sequences (cu_seqlens as for hla_attention).
 *   g [total, n_channels / gate_dim]   the logarithms of the gates (0 or less in a
 *                      layer that forgets; -infinity: the state starts anew)
 *   x [total, n_channels]
 *   h0 fp32 [n_seqs, n_channels]       the states in front; NULL: zeros
 *   out [total, n_channels]            h_t, rounded to dtype
 *   h_last fp32 [n_seqs, n_channels]   the states behind each sequence's last row (h0
 *                      of a sequence without rows); may be NULL, may be h0 itself
 *   states fp32 [ceil(total / 64), n_channels]: for hla_recurrence_backward, the
 *                      state in front of every 64th row; may be NULL
 * An infinity or NaN makes later rows of its own channel and sequence NaN or
 * infinite, and no others (of a gate that channels share: of those channels).
 * A gate whose exponential passes fp32's range (g above 88.7) is an infinity.
 * Rows at and past c_n are left as they were.  A malformed table is clamped on
 * the device and flagged in the workspace's error word; rows whose place it
 * leaves open are undefined.  A wait for earlier rows that runs out is flagged
 * there too and leaves NaN in the rows and states behind them (and in
 * hla_recurrence_backward's gradients of the rows in front).  Outputs must not
 * overlap inputs otherwise.  Asynchronous; deterministic. */
HLA_API int hla_recurrence(const hla_recurrence_params* params, const void* g, const void* x, const float* h0,
                           const int32_t* cu_seqlens, int n_seqs, int64_t total_tokens, void* out, float* h_last,
                           float* states, void* ws, size_t ws_bytes, void* stream);

/* Gradients of sum(dout . h) + sum(dh_last . h_last) (h before its rounding to
 * dtype; dh_last may be NULL) with respect to g (dg, gate_dtype: sums over the
 * channels that share a gate), x (dx) and h0 (dh0 fp32, may be NULL; may be
 * dh_last itself), from the inputs and the states that hla_recurrence kept.
 * Asynchronous; deterministic. */
HLA_API int hla_recurrence_backward(const hla_recurrence_params* params, const void* g, const void* x, const float* h0,
                                    const float* states, const int32_t* cu_seqlens, int n_seqs, int64_t total_tokens,
                                    const void* dout, const float* dh_last, void* dg, void* dx, float* dh0, void* ws,
                                    size_t ws_bytes, void* stream);

/* One token per sequence: h [n_seqs, n_channels] fp32 becomes exp(g) h + x, and
 * out [n_seqs, n_channels] is h rounded to dtype.  g, x as above, one row per
 * sequence.  Asynchronous. */
HLA_API int hla_recurrence_step(const hla_recurrence_params* params, const void* g, const void* x, float* h, int n_seqs,
                                void* out, void* stream);

/* Products with frozen weights in 4 bits.  W [n_out, n_in]: W[n][k] = scale (q - 8)
 * + offset, q in 0 .. 15, with a scale (and offset) per row n and group of inputs.
 * group: 32, 64 or 128; n_in a multiple of it.  dtype of out, scales, offsets.
 * x_dtype: dtype, or HLA_DTYPE_E4M3 with a power of two per x_group inputs (32,
 * 128 or 0, the whole row), as hla_rms_norm writes them.  x_stride: elements from
 * a token to the next (0: dense; otherwise at least n_in). */
typedef struct hla_linear4_params {
    int n_in;
    int n_out;
    int group;
    int dtype;
    int x_dtype;
    int x_group;
    int64_t x_stride;
} hla_linear4_params;

/* Workspace bytes of hla_linear4 (no error word; grows with tokens): rows that are
 * not bf16 on 16-byte boundaries, a multiple of 16 bytes apart, are laid out
 * there.  (It is asked for whatever the number of tokens; up to 16 of them are not
 * laid out.)  Two calls that may run at the same time need one each. */
HLA_API int hla_linear4_workspace_bytes(const hla_linear4_params* params, int64_t tokens, size_t* bytes);

/* out [tokens, n_out] = x W^T, from fp32 sums.  A group's products with q - 8 (and
 * with offsets its values) are summed before the scale: |x| has to be below 2^118
 * (3.3e35).  Larger values, infinities and NaN make outputs of their own token
 * infinite or NaN, also where x W^T is not, and no others.
 *   x [tokens, n_in], x_exp uint8 [tokens, n_in / x_group] (E4M3, else NULL)
 *   w uint8 [n_out, n_in / 2]: inputs 2i (low half) and 2i + 1
 *   scales, offsets [n_out, n_in / group]   offsets may be NULL (0)
 * Meant for the tokens of a decode step: the weights are read once per 64 tokens.
 * Asynchronous; deterministic. */
HLA_API int hla_linear4(const hla_linear4_params* params, const void* x, const uint8_t* x_exp, const uint8_t* w,
                        const void* scales, const void* offsets, int64_t tokens, void* out, void* ws, size_t ws_bytes,
                        void* stream);

/* Weights [n_out, n_in] (dtype, dense, finite) to 4 bits.  offsets NULL: scale =
 * max |w| / 7 of the group, q = 1 .. 15; else scale = (max - min) / 15, offset =
 * min + 8 scale, q = 0 .. 15; scale and offset rounded to dtype, then q to the
 * nearest.  Asynchronous. */
HLA_API int hla_linear4_quantize(const hla_linear4_params* params, const void* weight, uint8_t* w, void* scales,
                                 void* offsets, void* stream);

/* Synchronises `stream`, reads the state's device error word into *code
 * (may be NULL), clears it, and returns HLA_OK if it was zero, else the
 * matching HLA_ERR_* status. */
HLA_API int hla_check_device_error(const hla_state* st, void* stream, int32_t* code);

/* Same for the error word at the head of a prefill workspace. */
HLA_API int hla_check_workspace_error(void* ws, void* stream, int32_t* code);

/* Measurement hook (not part of the layer): for the calling thread, makes
 * hla_prefill record events[i] (cudaEvent_t handles owned by the caller) on
 * its stream at stage boundaries.  Tensor-core path (bf16, head_dim 128):
 * 0 before the first kernel, 1 after the feature path, 2 after the softmax
 * branch, 6 after the decode-state hand-off.  The linear branch runs in up to
 * four parts of the chunk slots, each a chunk-local launch and a state launch
 * (which also combines the two branches), all on the caller's stream: for
 * part p, 7 + 4p before and 8 + 4p after its chunk-local launch, 9 + 4p
 * before and 10 + 4p after its state launch.  Without the hook each
 * chunk-local launch runs beside the launch before it (the softmax, or the
 * previous part's state launch); with the hook on, every launch runs alone,
 * so each interval times one launch.  3 = 4 = 2; marks of parts not run are
 * recorded together after the last state launch, 5 after it.
 * Token-serial path: 0, 1 as above, 2 = 3 = 1, 4 after the GDN kernel, 5
 * after the softmax + combine, 6 after the hand-off (7 to 22 not recorded).
 * hla_backward, with the hook on, records 0 before its first kernel and
 * i = 1 .. 8 after its i-th stage (RoPE rows, conv and L2 features, GDN
 * backward, softmax backward, L2 backward, conv and RoPE backward, filter
 * partial sums + their reduction as one, lambda reduction); the L2, conv and
 * RoPE backward are one launch, so 5 = 4; its launches run one after another
 * either way.
 * Entries beyond n_events, or NULL entries, are skipped; n_events = 0
 * switches the hook off.  The array must stay valid while the hook is on. */
HLA_API int hla_prefill_stage_events(void** events, int n_events);

/* Measurement hook (not part of the layer): *out = the number of kernels one
 * hla_prefill call with these params launches (with_state != 0: with a
 * decode state to fill).  Memsets and event records are not counted.  Returns
 * the params check's status. */
HLA_API int hla_prefill_launch_count(const hla_params* params, int with_state, int* out);

#ifdef __cplusplus
}
#endif

#endif /* HLA_H */
