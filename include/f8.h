/*
 * f8.h -- 8-bit floating point with a scale for each block of 128 in libmxfp4.so:
 * quantisation, products (dense, and each expert's rows with that expert's
 * matrix), their gradient by the rows, and the gradient of a product by its
 * matrices.  Status codes, pointer rules and stream semantics are those of mx4.h
 * (MXFP4_STATUS_*; work enqueued on `stream`, nothing enqueued on a refusal, nothing
 * allocated, no workspace, deterministic results, programmatic dependent launches;
 * a call's outputs overlap neither its inputs nor each other), and so are the
 * experts' row order and offsets (mxfp4_moe_sort) and the element types.
 *
 * Codes are E4M3 bytes (sign, 4 bits of exponent with bias 7, 3 of fraction; largest
 * 448, 0x7F and 0xFF NaN, no infinities), row-major without padding, cols % 16 == 0,
 * 16-byte aligned.  (What is quantised, its rows and the values are read and written fastest where
 * they are 32-byte aligned.)  Scales are FP32 multipliers, of any value (a checkpoint's need be
 * no powers of two):
 *   matrix [rows, cols]      one for each 128x128 block: [ceil(rows/128)][ceil(cols/128)],
 *                            the matrices of a bank one after the other
 *   activations [n, cols]    one for each row's 128 columns: [ceil(cols/128)][n], block
 *                            by block
 * Blocks at the right and lower edge hold what is left.  In products rows, cols and the
 * number of tokens are at most 2^24.
 *
 * A routed layer with its gradients, in this order:
 *   mxfp4_moe_sort, mxfp4_f8_quant (rows gathered into expert order)
 *   mxfp4_f8_moe_mm (the act between two of them is the caller's, as is its gradient),
 *   mxfp4_moe_combine
 *   mxfp4_moe_combine_grad, mxfp4_f8_quant of the gradient's rows
 *   mxfp4_f8_moe_mm_grad (by the rows), mxfp4_moe_mm_grad_w (by the matrices)
 *   mxfp4_moe_dispatch_grad
 */
#ifndef MXFP4_F8_H
#define MXFP4_F8_H

#include "mx4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Quantises [rows, cols] activations.  For each row's 128 columns, with amax their
 * largest magnitude:
 *   scale s = 2^k with the least k >= -126 for which amax <= 448 * 2^k
 *   code = x / s rounded to the nearest E4M3 value, ties to even; the sign of a zero
 *          is kept
 * Both steps are exact but for that one rounding.  A block that holds an infinity or
 * a NaN gets scale NaN and codes 0.
 *   x, type, x_rows, ld, row_of   as mxfp4_quant: `x_rows` rows ld elements apart, output row
 *            i is x row row_of[i] (zeros where out of range) or, with NULL, row i
 *   codes    [rows, cols];  scales [ceil(cols/128)][rows]
 *   values   nullable: what the codes stand for, [rows, cols] of `type`; NaN in a NaN
 *            block.  Exact, except that a value rounded up out of the type's range is
 *            infinite and one below its subnormals is rounded once more. */
int mxfp4_f8_quant(const void* x, int type, int x_rows, int cols, long long ld,
                   const int32_t* row_of, int rows, void* codes, float* scales, void* values,
                   cudaStream_t stream);

/* The same for n_matrices matrices [rows, cols] one after the other (contiguous rows),
 * with blocks of 128x128: codes [n][rows][cols], scales
 * [n][ceil(rows/128)][ceil(cols/128)].  n_matrices <= MXFP4_MOE_MAX_SORTED_EXPERTS. */
int mxfp4_f8_quant_weight(const void* w, int type, int n_matrices, int rows, int cols, void* codes,
                          float* scales, void* values, cudaStream_t stream);

/* Product: Y[t*rows + r] = sum_b (x_scales[b][t] * w_scales[r/128][b]) * sum_{c in b}
 * W[r][c] * X[t][c] over the blocks b of 128 columns; W [rows, cols], X [nb, cols]
 * codes, Y [nb, rows] of y_type (F32 or BF16; the FP32 sum rounded once to nearest
 * even).  Any rows >= 1 and nb >= 1.  On the 8-bit tensor cores; sums within a block
 * and over blocks are FP32, as is the product of the two scales, which must not
 * overflow (the smallest, below 2^-126, lose bits).
 * Error bound (before the rounding to BF16): (ceil(cols/32) + ceil(cols/128) + 8) * 2^-23 *
 * sum_c |W X| with the scales in it.  A NaN code or scale makes the results that take it
 * NaN.  Per token the result does not depend on the other tokens' values, but it may on
 * nb (the order of the sums is chosen by the shape). */
int mxfp4_f8_mm(const void* w, const float* w_scales, int rows, int cols, const void* xq,
                const float* x_scales, int nb, void* Y, int y_type, cudaStream_t stream);

/* Each expert's rows with that expert's matrix: for offsets[e] <= i < offsets[e+1]
 * Y[i*rows + r] as above with W_e.  bank [n_experts][rows][cols] codes, bank_scales
 * [n_experts][ceil(rows/128)][ceil(cols/128)], xq [n_rows, cols] in expert order,
 * x_scales [ceil(cols/128)][n_rows]; offsets as mxfp4_moe_mm_mx (device,
 * int32[n_experts + 1], not decreasing, cut off at n_rows).  Rows of Y that belong to no
 * expert are left untouched. */
int mxfp4_f8_moe_mm(const void* bank, const float* bank_scales, int n_experts, int rows, int cols,
                    const void* xq, const float* x_scales, int n_rows, const int32_t* offsets,
                    void* Y, int y_type, cudaStream_t stream);

/* Gradient of both by the rows: dX[t*cols + c] = sum_b (dy_scales[b][t] *
 * w_scales[b][c/128]) * sum_{r in b} dY[t][r] * W[r][c] over the blocks b of 128 rows of
 * W, with dY quantised as mxfp4_f8_quant does: dyq [nb, rows] codes, dy_scales
 * [ceil(rows/128)][nb], rows % 16 == 0.  The matrix buffers are those of the product.
 * Sums, bound (with rows for cols) and the rest as there. */
int mxfp4_f8_mm_grad(const void* w, const float* w_scales, int rows, int cols, const void* dyq,
                     const float* dy_scales, int nb, void* dX, int dx_type, cudaStream_t stream);
int mxfp4_f8_moe_mm_grad(const void* bank, const float* bank_scales, int n_experts, int rows,
                         int cols, const void* dyq, const float* dy_scales, int n_rows,
                         const int32_t* offsets, void* dX, int dx_type, cudaStream_t stream);

/* Gradient of a product by its matrices: dW_e[r*cols + c] = sum over offsets[e] <= i <
 * offsets[e+1] of dY[i][r] * X[i][c], dY [n_rows, rows] and X [n_rows, cols] both of
 * `type` (BF16 or F16), dW [n_experts][rows][cols] of dw_type (F32 or BF16; the FP32 sum
 * rounded once; written, never added to).  In 16 bits, since the scales of 8-bit codes change
 * along this sum.  An expert without rows gets zeros; rows of dY and X that belong to no expert
 * are not used, whatever they hold.  rows % 8 == 0 and cols % 8 == 0.  Products of two elements
 * are exact; error bound (ceil(m/16) + 8) * 2^-23 * sum_i |dY X| for an expert of m rows, before
 * the rounding to BF16.  mxfp4_mm_grad_w: one matrix, all n_rows rows. */
int mxfp4_mm_grad_w(const void* dy, const void* x, int type, int rows, int cols, int n_rows,
                    void* dW, int dw_type, cudaStream_t stream);
int mxfp4_moe_mm_grad_w(const void* dy, const void* x, int type, int n_experts, int rows, int cols,
                        int n_rows, const int32_t* offsets, void* dW, int dw_type,
                        cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MXFP4_F8_H */
