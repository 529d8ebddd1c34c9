/*
 * emu_block_operators.h -- C ABI of the operators on 8-bit floating point
 * codes with a scale for each block of 128, in the same library:
 *
 *  - emu_block_quant: the codes and scales of activations (blocks of 1 x 128)
 *    or of weights (128 x 128);
 *  - emu_swiglu_block_quant: the gated activation silu(gate) * up with its
 *    codes and, to be kept for the gradient, those of gate and up, and
 *    emu_swiglu_block_backward, the gradient from what was kept;
 *  - emu_block_scaled_mm: the product of such codes, and
 *    emu_grouped_block_scaled_mm, the same by groups of rows, each with
 *    weights of its own (experts);
 *  - emu_block_weight_grad: the gradient of a product's weights, from the
 *    codes that its input was kept in.
 *
 * Conventions are those of emu_operators.h: device pointers owned by the
 * caller, calls only enqueue kernels on `stream`, arguments are checked on the
 * host first, elements are aligned to their own size and no more is asked,
 * results are deterministic, outputs must not overlap inputs.
 *
 * Codes are e4m3fn (largest value Q = 448) or e5m2 (57344).  A value's code
 * times the scale of its block stands for the value; along an axis of n values
 * there are (n + 127) / 128 blocks, the last of which may be shorter.  Scales
 * are binary32, or e8m0: one byte b for the power of two 2^(b - 127), 255
 * for NaN.
 */
#ifndef EMU_BLOCK_OPERATORS_H
#define EMU_BLOCK_OPERATORS_H

#include "emu_operators.h"

#ifdef __cplusplus
extern "C" {
#endif

#define EMU_BLOCK 128

typedef enum {
    EMU_SCALE_FP32 = 0,
    EMU_SCALE_E8M0 = 1
} emu_scale_type;

/*
 * Codes and scales of x [E, T, n] (bf16, fp16 or fp32; rows ldx and matrices
 * x_stride elements apart).  block_rows is 1 (a scale for 128 values of a row)
 * or 128 (one for 128 x 128 values of a matrix).  With m the largest magnitude
 * of a block its scale is max(RN32(m / Q), 2^-126), or for e8m0 the least
 * power of two s >= 2^-126 with m <= s Q; codes are the nearest to x / s, ties
 * to even.  A block with an infinity or a NaN has the scale NaN and NaN codes.
 * q [E, T, n] dense; scales [E, (T + block_rows - 1) / block_rows, blocks of
 * n] dense.  Where a block's m is below 2^-100 a code of fp32 scales may be
 * that of x / s rounded twice.
 */
EMU_API emu_status emu_block_quant(const void *x, emu_dtype x_dtype, int64_t ldx, int64_t x_stride,
                                   int64_t E, int64_t T, int64_t n, int block_rows,
                                   void *q, emu_dtype q_dtype, void *scales, emu_scale_type s_type,
                                   hipStream_t stream);

/*
 * h = gate / (1 + exp(-gate)) * up, in binary32, as codes q [T, F] and scales
 * [T, blocks of F] of 1 x 128, as emu_block_quant makes them.  gate and up
 * [T, F] of one type (bf16, fp16 or fp32).  kept: NULL, or [T, 2 F] for the
 * codes of gate, then those of up, in each row; kept_scales [T, 2 (blocks of
 * F)] likewise, each half with blocks of its own.  All of them dense, of
 * q_dtype and s_type.
 */
EMU_API emu_status emu_swiglu_block_quant(const void *gate, int64_t ldgate, const void *up, int64_t ldup,
                                          emu_dtype dtype, int64_t T, int64_t F,
                                          void *q, emu_dtype q_dtype, void *scales, emu_scale_type s_type,
                                          void *kept, void *kept_scales, hipStream_t stream);

/*
 * The gradient of h above from what was kept (dense): with a and b the values
 * that gate's and up's codes stand for and p = 1 / (1 + exp(-a)),
 *   grad[t, i] = g b p (1 + a (1 - p));  grad[t, F + i] = g a p.
 * g [T, F] bf16, fp16 or fp32; grad [T, 2 F] of g's type.
 */
EMU_API emu_status emu_swiglu_block_backward(const void *g, emu_dtype g_dtype, int64_t ldg,
                                             const void *kept, emu_dtype q_dtype,
                                             const void *kept_scales, emu_scale_type s_type,
                                             int64_t T, int64_t F, void *grad, int64_t ldgrad, hipStream_t stream);

/*
 * out = a @ w.T + bias of what codes and scales stand for:
 *   out[m, n] = sum over blocks b of K of
 *     sa[m, b] sw[n / 128, b] (sum over k in b of a[m, k] w[n, k]) + bias[n].
 *
 * a [M, K] and w [N, K] of e4m3fn or e5m2 each; scales of one type, with any
 * strides (in elements): that of row m of a and block b at m sa_row +
 * b sa_block, that of rows 128 j .. 128 j + 127 of w and block b at j sw_row +
 * b sw_block.  out [M, N] bf16, fp16 or fp32; bias NULL, or [N] of out's type
 * or fp32.  K = 0 gives the bias (or 0).
 * Blocks' sums are added in binary32.  Within one, for outputs of 16 bits, the
 * matrix instruction adds each 8 products of consecutive k (from a multiple of 8
 * on) beside the largest exponent sum of the 8 to 13 fraction bits, each cut
 * toward zero, and these sums in binary32: some 1.5e-5 of a sum of normal
 * codes.  For outputs in fp32 all products are added in binary32.  fp32 scales
 * are multiplied first (RN32(sa sw)); so are e8m0 ones for outputs in fp32.
 * An infinity or a NaN among a's, w's or the scales' values gives what IEEE
 * arithmetic gives.
 * workspace: emu_block_scaled_mm_workspace(...) bytes, 16-byte aligned; NULL
 * where that is 0.  `aligned` says of an operand that its pointer, leading
 * dimension and stride between matrices are multiples of 16 and the second at
 * most EMU_BLOCK_MAX_ALIGNED_LD.
 * K up to EMU_BLOCK_MAX_ALIGNED_LD, sa_row and sw_row up to 2^20.
 */
#define EMU_BLOCK_MAX_ALIGNED_LD (INT64_C(1) << 22)
EMU_API emu_status emu_block_scaled_mm(const void *a, emu_dtype a_dtype, int64_t lda,
                                       const void *w, emu_dtype w_dtype, int64_t ldw,
                                       int64_t M, int64_t N, int64_t K,
                                       const void *scale_a, int64_t sa_row, int64_t sa_block,
                                       const void *scale_w, int64_t sw_row, int64_t sw_block, emu_scale_type s_type,
                                       const void *bias, emu_dtype bias_dtype,
                                       void *out, emu_dtype out_dtype, int64_t ldo,
                                       void *workspace, size_t workspace_bytes, hipStream_t stream);
EMU_API size_t emu_block_scaled_mm_workspace(int64_t M, int64_t N, int64_t K, emu_dtype out_dtype,
                                             int a_aligned, int w_aligned);

/*
 * The same by groups of a's rows: group e has the rows from ends[e - 1] (0 for
 * the first) to ends[e] and the weights w[e] [N, K], w_stride and sw_stride
 * elements from those before.  ends [E] is on the device, int32 or int64
 * (ends_bits 32 or 64), and read by the kernels alone: an end below the one
 * before counts as that one, one above T as T.  A group may have no rows.
 * Rows behind the last group's are left as they are, or become 0 where
 * zero_rest is not 0; without groups those are all rows, and no operand is
 * read.  T up to 2^24, E up to 65536.
 */
EMU_API emu_status emu_grouped_block_scaled_mm(const void *a, emu_dtype a_dtype, int64_t lda,
                                               const void *w, emu_dtype w_dtype, int64_t ldw, int64_t w_stride,
                                               int64_t T, int64_t E, int64_t N, int64_t K,
                                               const void *scale_a, int64_t sa_row, int64_t sa_block,
                                               const void *scale_w, int64_t sw_row, int64_t sw_block,
                                               int64_t sw_stride, emu_scale_type s_type,
                                               const void *ends, int ends_bits, int zero_rest,
                                               void *out, emu_dtype out_dtype, int64_t ldo,
                                               void *workspace, size_t workspace_bytes, hipStream_t stream);
EMU_API size_t emu_grouped_block_scaled_mm_workspace(int64_t T, int64_t E, int64_t N, int64_t K, emu_dtype out_dtype,
                                                     int a_aligned, int w_aligned);

/*
 * The gradient of a product's weights from the codes that its input was kept
 * in: out[n, k] = sum over rows t of g[t, n] x[t, k], x what codes and scales
 * stand for, in bf16 (which holds it exactly, but for values below 2^-133 or
 * beyond the type's largest).
 *
 * g [T, N] bf16, fp16 or fp32; codes [T, K] e4m3fn or e5m2, blocks of 1 x 128
 * with e8m0 scales, that of row t and block b at t s_row + b s_block; out of
 * any of g's types.  Products are exact (those of fp16 and fp32 g as two and
 * three parts; for outputs of 16 bits those of fp32 g as two, within 2^-17; what
 * of g lies below 2^-133 counts as 0) and added in binary32; an out of no rows
 * is 0.
 * ends NULL: one sum over all rows, out [N, K].  Else E sums by groups of
 * rows, as in emu_grouped_block_scaled_mm: out [E, N, K], out_stride elements
 * between matrices, which lie one after the other or row by row beside each
 * other, and rows behind the last group's take no part.
 * workspace: emu_block_weight_grad_workspace(...) bytes, 16-byte aligned (E =
 * 0: no groups); `aligned` says that the pointer and the rows' distance in
 * bytes are multiples of 16 and the leading dimension is at most
 * EMU_BLOCK_MAX_ALIGNED_LD.
 * T up to 2^30, N and K to EMU_BLOCK_MAX_ALIGNED_LD, E to 65536, and at most
 * 2^23 tiles of 128 x 128 in all.
 */
EMU_API emu_status emu_block_weight_grad(const void *g, emu_dtype g_dtype, int64_t ldg,
                                         const void *codes, emu_dtype c_dtype, int64_t ldc,
                                         const void *scales, int64_t s_row, int64_t s_block,
                                         int64_t T, int64_t N, int64_t K,
                                         const void *ends, int ends_bits, int64_t E,
                                         void *out, emu_dtype out_dtype, int64_t ldo, int64_t out_stride,
                                         void *workspace, size_t workspace_bytes, hipStream_t stream);
EMU_API size_t emu_block_weight_grad_workspace(int64_t T, int64_t E, int64_t N, int64_t K, emu_dtype g_dtype,
                                               int g_aligned, int c_aligned);

#ifdef __cplusplus
}
#endif

#endif /* EMU_BLOCK_OPERATORS_H */
