/*
 * emu_operators.h -- C ABI of the operators that stand before and after the
 * FP8 product of emu_fp8gemm.h in a language model, in the same library:
 *
 *  - emu_add_rms_norm_quant: the residual's addition, the root-mean-square
 *    norm and the 8-bit codes (with scales) that the next product takes, and
 *    emu_add_rms_norm_backward, the norm's gradient;
 *  - emu_int8_scaled_mm: the product of 8-bit integers with a scale for each
 *    row of either operand, accumulated exactly;
 *  - emu_token_logprobs: log probabilities of given tokens, the
 *    distribution's entropy and its most likely tokens, and
 *    emu_token_logprobs_backward, their gradient with respect to the logits.
 *
 * Conventions are those of emu_fp8gemm.h: device pointers owned by the
 * caller; every call only enqueues kernels on `stream`, never synchronises
 * and never allocates; arguments are checked on the host before anything is
 * enqueued, and a status other than EMU_OK means that nothing was written.
 * Matrices are row-major with a leading dimension in elements; elements are
 * aligned to their own size, and no more is asked of pointers or leading
 * dimensions.  Results are deterministic: they depend on the order of no
 * atomic operation.
 * Outputs must not overlap inputs unless a call says so.  Sums, statistics
 * and products are held in binary32 (int32 for int8 products) and rounded
 * once, to nearest even, where they are stored.
 */
#ifndef EMU_OPERATORS_H
#define EMU_OPERATORS_H

#include "emu_fp8gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types; the first five are emu_out_dtype's. */
typedef enum {
    EMU_DT_BF16 = 0,
    EMU_DT_FP16 = 1,
    EMU_DT_FP32 = 2,
    EMU_DT_E4M3FN = 3,
    EMU_DT_E5M2 = 4,
    EMU_DT_INT8 = 5
} emu_dtype;

/*
 * v = x + residual;  y = v / sqrt(mean(v^2) + eps) * weight;
 * q = round(clamp(y / scale, -Q, Q)), row by row.
 *
 * x [T, n] (bf16, fp16 or fp32); weight [n], of x's type or fp32; residual
 * NULL, or [T, n] of x's type or fp32.  q [T, n] of q_dtype: e4m3fn (Q = 448),
 * e5m2 (57344) or int8 (127, so that codes are symmetric); ties go to even.
 * scale: NULL, or one binary32 value on the device for all rows.  Where it is
 * NULL each row's own scale max(max|y| / Q, 2^-126) is used and written to
 * row_scales [T].  h_out: NULL, or (with a residual) [T, n] of the
 * residual's type that takes v; it may be the residual itself.
 * A NaN in a row's y gives that row the scale NaN (scale == NULL) and NaN
 * codes, 0 for int8, which has none; an infinity in v makes y NaN.
 * The squares of v are summed in binary32, in which values beyond 1.8e19
 * overflow: such a row counts as one with an infinite mean (y = 0).  Those of
 * values under 1e-19 lose digits and vanish under 4e-23, which shows where eps
 * is below some 1e-31.
 * n = 0 with T > 0 is refused; T = 0 does nothing.
 */
EMU_API emu_status emu_add_rms_norm_quant(const void *x, emu_dtype x_dtype, int64_t ldx,
                                          const void *weight, emu_dtype w_dtype,
                                          const void *residual, emu_dtype res_dtype, int64_t ldres,
                                          int64_t T, int64_t n, float eps,
                                          void *q, emu_dtype q_dtype, int64_t ldq,
                                          const float *scale, float *row_scales,
                                          void *h_out, int64_t ldh, hipStream_t stream);

/*
 * The norm's gradient.  With h [T, n] the norm's input (what h_out took, or
 * x where there was no residual), r = 1 / sqrt(mean(h^2) + eps), n_i = h_i r,
 * g [T, n] the gradient of y (of the codes times their scale, where the
 * rounding to 8 bits is passed straight through) and u = g * weight:
 *   grad_in = r (u - n mean(u n)) + grad_h;   grad_weight = sum over rows g n.
 * grad_in [T, n] of g's type is the gradient of x and of the residual alike.
 * h is of g's type or fp32, weight of g's type or fp32, grad_h NULL or of
 * g's type or fp32; grad_in may be g or (of its type) grad_h itself.
 * grad_weight [n] of weight's type; T = 0 writes zeros to it.  workspace:
 * emu_add_rms_norm_backward_workspace(T, n) bytes, 16-byte aligned, contents
 * on entry and return do not matter.  The sums are binary32's: where a row's
 * sum of squares overflows, r is 0 as in the forward call, and where that of
 * u h does as well, its grad_in is NaN.
 */
EMU_API emu_status emu_add_rms_norm_backward(const void *g, emu_dtype g_dtype, int64_t ldg,
                                             const void *h, emu_dtype h_dtype, int64_t ldh,
                                             const void *weight, emu_dtype w_dtype,
                                             const void *grad_h, emu_dtype gh_dtype, int64_t ldgh,
                                             int64_t T, int64_t n, float eps,
                                             void *grad_in, int64_t ldgi, void *grad_weight,
                                             void *workspace, size_t workspace_bytes, hipStream_t stream);
EMU_API size_t emu_add_rms_norm_backward_workspace(int64_t T, int64_t n);

/*
 * out = (a @ w.T) * scale_a * scale_w + bias.
 *
 * a [M, K] and w [N, K] int8 (all 256 codes), the sum exact in int32
 * (K <= 131071, so that no sum can pass it); out [M, N] bf16, fp16 or fp32:
 * RN(RN32(RN32(RN32(sum) * scale_a) * scale_w) + bias).  scale_a: M binary32
 * values if a_per_row, else one; scale_w: N if w_per_row, else one.  bias:
 * NULL, or [N] of out's type or fp32.  K = 0 gives bias (or 0).
 * workspace: emu_int8_scaled_mm_workspace(...) bytes, 16-byte aligned; NULL
 * where that is 0.  It depends on the pointers' alignment and the leading
 * dimensions besides the sizes: `aligned` says that a, w, lda and ldw are all
 * multiples of 16 and the last two at most EMU_INT8_MAX_ALIGNED_LD.
 */
#define EMU_INT8_MAX_ALIGNED_LD (INT64_C(1) << 22)
EMU_API emu_status emu_int8_scaled_mm(const int8_t *a, int64_t lda, const int8_t *w, int64_t ldw,
                                      int64_t M, int64_t N, int64_t K,
                                      const float *scale_a, int a_per_row, const float *scale_w, int w_per_row,
                                      const void *bias, emu_dtype bias_dtype,
                                      void *out, emu_dtype out_dtype, int64_t ldo,
                                      void *workspace, size_t workspace_bytes, hipStream_t stream);
EMU_API size_t emu_int8_scaled_mm_workspace(int64_t M, int64_t N, int64_t K, int aligned);

/* The most alternatives a call of emu_token_logprobs can ask for. */
#define EMU_MAX_TOP_TOKENS 64

/*
 * With lse_t = log sum_v exp(z[t, v]) and lp[t, v] = z[t, v] - lse_t:
 *   logprobs[t, c] = lp[t, tokens[t, c]];  entropy[t] = -sum_v exp(lp) lp;
 *   top_tokens[t, i], top_logprobs[t, i]: the top_k largest lp in falling
 *   order, equal logits by rising token.
 *
 * logits [T, V] bf16, fp16 or fp32; tokens [T, C] int64 (dense), C >= 0; the
 * outputs are dense binary32 (top_tokens int64).  top_k <= min(V,
 * EMU_MAX_TOP_TOKENS); V <= 2^31 - 1 - 4096.
 * A token below 0 stands for none: its log probability is 0.  One of V or
 * more is out of the vocabulary: NaN.  A logit of -inf has probability 0 and
 * adds nothing to the entropy.  A row of nothing but -inf: lse and every log
 * probability are -inf and the entropy is 0.  A row with +inf: lse, the entropy
 * and every log probability are NaN.  A row with a NaN: the same, and its
 * top_tokens are -1.
 * workspace: emu_token_logprobs_workspace(T, V, top_k) bytes, 16-byte
 * aligned; NULL where that is 0.
 */
EMU_API emu_status emu_token_logprobs(const void *logits, emu_dtype z_dtype, int64_t ldz,
                                      int64_t T, int64_t V, const int64_t *tokens, int64_t C, int64_t top_k,
                                      float *logprobs, float *entropy, float *lse,
                                      float *top_logprobs, int64_t *top_tokens,
                                      void *workspace, size_t workspace_bytes, hipStream_t stream);
EMU_API size_t emu_token_logprobs_workspace(int64_t T, int64_t V, int64_t top_k);

/* The most tokens and alternatives that a row's gradient can come from. */
#define EMU_MAX_GRAD_TOKENS 1024

/*
 * The gradient of a loss that reads emu_token_logprobs's outputs: with
 * g [T, C] that of logprobs, g_entropy [T] that of the entropy and g_top
 * [T, top_k] that of top_logprobs (each NULL: zero),
 *   grad[t, v] = sum_c g [v = token c] + sum_i g_top [v = top i]
 *                - p (sum_c g + sum_i g_top) - g_entropy p (lp + entropy),
 * p = exp(lp), over the tokens that are not below 0.  The gradient of lse
 * itself is not taken.  lse and entropy are the forward call's.  grad [T, V]
 * is of the logits' type and may be the logits themselves.  Where a logit is
 * -inf its p and p lp are 0.  A row whose lse is -inf gets zeros.  A token or
 * top token of V or more, as a NaN in lse, gives its row NaN (also one whose
 * lse is -inf).  C (if g is given) and top_k (if g_top is) are at most
 * EMU_MAX_GRAD_TOKENS together; the forward call takes any C.
 */
EMU_API emu_status emu_token_logprobs_backward(const void *logits, emu_dtype z_dtype, int64_t ldz,
                                               int64_t T, int64_t V, const int64_t *tokens, int64_t C,
                                               const float *lse, const float *entropy,
                                               const float *g, const float *g_entropy,
                                               const int64_t *top_tokens, const float *g_top, int64_t top_k,
                                               void *grad, int64_t ldgrad, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* EMU_OPERATORS_H */
