/*
 * bi_model.h -- C ABI of the batch-invariant layers of the policy model: the bf16 GEMM of a linear
 * layer, RMSNorm, and the attention layer's parts: the norm of each query and key head with its
 * rotation, and softmax attention, both with their backward passes.  Same library
 * (libbi_isloss.so), status codes and conventions as bi_isloss.h.
 *
 * Sources (page titles and sections):
 *   "Zero Mismatch, Simple Async RL", section "Only one probability gap comes from old weights":
 *       kernel selection by batch shape, reduction order and different prefill/decode arithmetic
 *       change logprobs although the parameters are the same.
 *   "Zero Mismatch, Simple Async RL", section "Large-model validation exposes concrete failure
 *       mechanisms": shape-selected library kernels are a source of batch variance.
 *   "REINFORCE Zero: 为什么内核对齐后...", the paragraph before Fig. 2: trainer-inference invariance
 *       removes the kernel-mismatch term with batch-invariant kernels and a matched forward pass.
 *
 * Batch invariance: every output row depends only on its own input row and the weights.  The same
 * kernel serves every M (one row alone, as in decode, or 10^5 packed rows, as in prefill or the
 * learner): one tile shape, a fixed reduction order, no split of the reduction across CTAs, no
 * atomics.  Rows are therefore bit-identical whatever batch they sit in and wherever they sit.
 *
 * Conventions: device pointers owned by the caller, bf16 passed as uint16_t bit patterns,
 * row-major; work is enqueued on `stream` (a cudaStream_t; NULL = legacy default stream) without
 * synchronising; the library allocates nothing.  The return value reports host-visible errors
 * (nothing is launched unless it is BI_OK); *dev_status (device int32) is set to BI_OK and raised
 * by the kernel to BI_ERR_TIMEOUT if a bounded wait ran out (outputs then undefined).  Kernels
 * never trap.
 */
#ifndef BI_MODEL_H
#define BI_MODEL_H

#include "bi_isloss.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Y = X W^T: the linear layer y_m = W x_m.
 *   x   [M, K] bf16   input rows                       16-byte aligned
 *   w   [N, K] bf16   weight, one row per output        16-byte aligned
 *   y   [M, N] bf16   output, fp32 accumulation rounded to nearest even; overwritten
 *   M   >= 0 and <= 2^31 - 256 (M = 0 launches nothing and leaves *dev_status = BI_OK)
 *   N   > 0, a multiple of 8 and < 2^31;  K > 0, a multiple of 8 and < 2^31
 * Tiling: 256 x 256 output tiles on CTA pairs (tcgen05 M = 256 instructions), K in chunks of 64
 * taken in increasing order; the same for every M.
 * Returns BI_ERR_INVALID_ARG for a NULL or misaligned pointer, BI_ERR_UNSUPPORTED_SHAPE for N or
 * K outside the rules above, BI_ERR_CUDA when the device set-up or the launch fails.
 */
BI_API bi_status bi_gemm_bf16(const uint16_t* x, const uint16_t* w, uint16_t* y, int64_t M, int32_t N, int32_t K,
                              int32_t* dev_status, void* stream);

/*
 * RMSNorm: y_m = x_m / sqrt(mean_j x_mj^2 + eps) * g, row by row.
 *   x   [M, H] bf16   16-byte aligned;   g [H] bf16 gain, 16-byte aligned
 *   y   [M, H] bf16   output (may not alias x), 16-byte aligned
 *   eps >= 0 and finite;  M >= 0;  H > 0 and a multiple of 8
 * Arithmetic: fp32; the sum of squares of a row in a fixed order (a fixed per-lane order, then a
 * fixed shuffle tree whose lane-0 total the whole row uses), r = rsqrt(ss / H + eps),
 * y = bf16((x r) g).
 * Returns BI_ERR_INVALID_ARG for a NULL or misaligned pointer, aliasing x and y, or a negative or
 * non-finite eps; BI_ERR_UNSUPPORTED_SHAPE for H; BI_ERR_CUDA when the launch fails.
 */
BI_API bi_status bi_rmsnorm(const uint16_t* x, const uint16_t* g, float eps, uint16_t* y, int64_t M, int32_t H,
                            int32_t* dev_status, void* stream);

/*
 * RMS norm of each query and key head, and the rotation of its position, in one pass.  With x one
 * head's D values, y = x / sqrt(mean(x^2) + eps) * g (gq for q's heads, gk for k's), and for i < R/2
 * and the angle a_i = position * inv_freq_i:
 *   z_i         = y_i cos a_i - y_{i+R/2} sin a_i
 *   z_{i + R/2} = y_{i+R/2} cos a_i + y_i sin a_i
 * and z = y past R.  gq = gk = NULL: y = x (rotation only).
 *   q [T][Hq][D], k [T][Hkv][D] bf16: heads are D apart, tokens q_ld and k_ld elements (slices of one
 *     projection's output are fine); 16-byte aligned, q_ld >= Hq D and k_ld >= Hkv D multiples of 8
 *   gq, gk [D] bf16, 16-byte aligned;  positions [T] int32 (any value);  inv_freq [R / 2] float
 *   q_out, k_out: the same layouts with their own token strides; may not overlap q or k
 *   0 <= T < 2^31;  Hq, Hkv in 1..4096;  D a multiple of 16 and <= 256;  R a multiple of 16, 0 < R <= D
 * Arithmetic: fp32, one rounding to bf16; the angles in turns in fp64, so that far positions keep
 * their phase.  A head's output depends on its own input, position and gains only.
 * Returns BI_ERR_INVALID_ARG for a NULL, misaligned or aliased pointer, a bad stride, or a negative or
 * non-finite eps; BI_ERR_UNSUPPORTED_SHAPE for Hq, Hkv, D or R; BI_ERR_CUDA when the launch fails.
 */
BI_API bi_status bi_qk_norm_rope(const uint16_t* q, const uint16_t* k, int64_t q_ld, int64_t k_ld, const uint16_t* gq,
                                 const uint16_t* gk, const int32_t* positions, const float* inv_freq, float eps,
                                 int64_t T, int32_t Hq, int32_t Hkv, int32_t D, int32_t R, uint16_t* q_out,
                                 uint16_t* k_out, int64_t q_out_ld, int64_t k_out_ld, int32_t* dev_status,
                                 void* stream);

/*
 * Its gradient: dq, dk (bf16, laid out like q, k with their own token strides) and, with gains,
 * dgq, dgk [D] float, overwritten (zeros for T = 0).  dq_out, dk_out: gradients of q_out and k_out;
 * q, k: the inputs (not read without gains, and may then be NULL).  dq and dk may not overlap an input.
 * The gains' gradients are added up in a fixed order for a given T (no atomics): the same call gives
 * the same bits.  ws: bi_qk_norm_rope_bwd_workspace_bytes(D) bytes, 256-byte aligned (gains only).
 */
BI_API size_t bi_qk_norm_rope_bwd_workspace_bytes(int32_t D);
BI_API bi_status bi_qk_norm_rope_bwd(const uint16_t* dq_out, const uint16_t* dk_out, int64_t dq_out_ld,
                                     int64_t dk_out_ld, const uint16_t* q, const uint16_t* k, int64_t q_ld,
                                     int64_t k_ld, const uint16_t* gq, const uint16_t* gk, const int32_t* positions,
                                     const float* inv_freq, float eps, int64_t T, int32_t Hq, int32_t Hkv, int32_t D,
                                     int32_t R, uint16_t* dq, uint16_t* dk, int64_t dq_ld, int64_t dk_ld, float* dgq,
                                     float* dgk, int32_t* dev_status, void* ws, size_t ws_bytes, void* stream);

/*
 * Softmax attention over S sequences: out_i = sum_j p_ij v_j with p_i = softmax_j(scale q_i . k_j)
 * over the keys that query i sees, and lse_i = log sum_j exp(scale q_i . k_j).
 *   q [Tq][Hq][D], k, v [Tk][Hkv][D] bf16: heads are D apart, tokens q_ld, k_ld, v_ld elements
 *     (slices of one projection's output, or caches); 16-byte aligned, strides multiples of 8.
 *     Query head h reads key/value head h / (Hq / Hkv).
 *   q_offsets, k_offsets [S + 1] int64 (device): sequence s has the query rows
 *     q_offsets[s] .. q_offsets[s+1] - 1 and the key rows from k_offsets[s] on; k_lens [S] int32
 *     (device) how many of the rows up to k_offsets[s+1] are keys (a cache with room behind them),
 *     NULL for all.  For packed self-attention pass the same offsets twice.
 *   causal != 0: the queries are the last ones of their sequence's positions: query i of n sees the keys
 *     j <= i + (keys - n).  A decode step is one query a sequence over its cache.
 *   out [Tq][Hq][D] bf16, lse [Hq][Tq] float.  A query that sees no key gets zeros and -infinity.  Rows
 *     in no sequence are left as they were; key rows in none are not used, whatever they hold.
 *   scale > 0, finite;  D 64 or 128;  Hq a multiple of Hkv, Hq / Hkv <= 128, Hkv <= 4096;
 *   0 <= Tq, Tk < 2^31 - 512;  0 <= S, and S + Tq / floor(128 Hkv / Hq) and S + Tk / 128 below 2^31 - 2^20
 * A row's result has the same bits in any batch and whether it is computed among its sequence's other
 * queries (prefill) or alone over a cache (decode).  A NaN or infinity in a key or value row of a sequence
 * reaches every query of that sequence that shares a 128-row tile with one that sees it.
 * The terms of the softmax are rounded to bf16 for the product with v; sums, maxima and lse are fp32.
 * out may not overlap an input.  ws belongs to the call until its kernels end: calls (and graphs) that may
 * run at the same time need one each.
 * Device status: BI_ERR_BAD_OFFSETS (offsets that decrease or leave the tensors, k_lens below 0 or past the
 * next offset): nothing is written then.  Returns BI_ERR_WORKSPACE for a ws below
 * bi_attn_fwd_workspace_bytes(...) bytes or not 256-byte aligned, and the codes of the entry points above.
 */
BI_API size_t bi_attn_fwd_workspace_bytes(int64_t Tq, int64_t Tk, int32_t S, int32_t Hq, int32_t Hkv, int32_t D);
BI_API bi_status bi_attn_fwd(const uint16_t* q, const uint16_t* k, const uint16_t* v, int64_t q_ld, int64_t k_ld,
                             int64_t v_ld, const int64_t* q_offsets, const int64_t* k_offsets, const int32_t* k_lens,
                             int32_t S, int64_t Tq, int64_t Tk, int32_t Hq, int32_t Hkv, int32_t D, int32_t causal,
                             float scale, uint16_t* out, float* lse, int32_t* dev_status, void* ws, size_t ws_bytes,
                             void* stream);

/*
 * Its gradient: dq [Tq][Hq][D], dk, dv [Tk][Hkv][D] bf16 (tokens dq_ld, dk_ld, dv_ld elements apart, so they
 * may be slices of one buffer) of sum(out * dout), overwritten.  q, k, v, the offsets, causal and scale as in
 * the forward, out and lse its results; dout [Tq][Hq][D] bf16 with dout_ld elements between tokens.  The
 * probabilities are recomputed: p_ij = exp(scale q_i . k_j - lse_i); with delta_i = dout_i . out_i and
 * ds_ij = p_ij (dout_i . v_j - delta_i),
 *   dv_j = sum_i p_ij dout_i,   dk_j = scale sum_i ds_ij q_i,   dq_i = scale sum_j ds_ij k_j,
 * the sums over i running over all query heads of the key/value head.  p and ds are rounded to bf16 for
 * their products, sums are fp32 in an order that depends on the places in the sequence only: no atomics, and
 * a sequence's gradients have the same bits in any batch.  A query that sees no key, and a key that no query
 * sees, get zeros; rows in no sequence (and cache rows behind k_lens) are left as they were.
 * dq, dk and dv may overlap neither each other nor an input.  A NaN or infinity in a row of a sequence
 * stays in that sequence.  Errors as in the forward, for a ws of bi_attn_bwd_workspace_bytes(...).
 */
BI_API size_t bi_attn_bwd_workspace_bytes(int64_t Tq, int64_t Tk, int32_t S, int32_t Hq, int32_t Hkv, int32_t D);
BI_API bi_status bi_attn_bwd(const uint16_t* dout, int64_t dout_ld, const uint16_t* q, const uint16_t* k,
                             const uint16_t* v, int64_t q_ld, int64_t k_ld, int64_t v_ld, const uint16_t* out,
                             const float* lse, const int64_t* q_offsets, const int64_t* k_offsets,
                             const int32_t* k_lens, int32_t S, int64_t Tq, int64_t Tk, int32_t Hq, int32_t Hkv,
                             int32_t D, int32_t causal, float scale, uint16_t* dq, uint16_t* dk, uint16_t* dv,
                             int64_t dq_ld, int64_t dk_ld, int64_t dv_ld, int32_t* dev_status, void* ws,
                             size_t ws_bytes, void* stream);

/* Test hook, not for production use: the next bi_attn_fwd or bi_attn_bwd on this host thread that launches
 * kernels gives each of their waits this limit in nanoseconds, in place of 4 s and 40 ns a key and query row.
 * 0 disables the hook. */
BI_API void bi_debug_attn_wait_limit_once(uint64_t limit_ns);

#ifdef __cplusplus
}
#endif

#endif /* BI_MODEL_H */
