/*
 * mx4.h -- microscaled 4-bit activations in libmxfp4.so: quantisation to MXFP4,
 * products of two MXFP4 matrices (dense, and each expert's rows with that
 * expert's matrix), and the routing of tokens to experts and back with its
 * gradient.  Status codes, pointer rules and stream semantics are those of
 * mxfp4.h (MXFP4_STATUS_*; work enqueued on `stream`, nothing enqueued on a
 * refusal, nothing allocated, deterministic results).  The kernels are launched
 * as programmatic dependents: their set-up may run while the kernel ahead of
 * them in the stream finishes, but they read and write memory only after it has
 * completed.  The quantisers hold the launch behind them until they are done, so a
 * weight buffer may be written by one and read by mxfp4_mv with launch overlap on.
 * A call's outputs overlap neither its inputs nor each other.
 *
 * An MXFP4 matrix here is a weight buffer of mxfp4.h, whatever it holds: [rows,
 * cols] with cols % 32 == 0, code plane then scale plane, mxfp4_nbytes(rows,
 * cols) bytes, 16-byte aligned.  Activations [tokens, cols] are rows of such a
 * matrix, so what mxfp4_quant writes can be either operand of a product, and
 * mxfp4_dequant reads it back.
 *
 * A routed layer on a prompt, in this order:
 *   mxfp4_moe_sort       expert ids -> the rows' expert order
 *   mxfp4_quant          x rows gathered into that order, as MXFP4
 *   mxfp4_moe_mm_mx      gate and up, each expert's rows with its matrices
 *   mxfp4_swiglu_quant   silu(gate) * up, as MXFP4
 *   mxfp4_moe_mm_mx      down
 *   mxfp4_moe_combine    back to token order with the route weights
 */
#ifndef MX4_H
#define MX4_H

#include "mxfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of dense tensors. */
enum {
    MXFP4_TYPE_F32 = 0,
    MXFP4_TYPE_BF16 = 1,
    MXFP4_TYPE_F16 = 2
};

/* Quantises [rows, cols] values to MXFP4.  Per group of 32 consecutive elements
 * of a row, with amax its largest magnitude:
 *   scale byte k = max(0, floor(log2 amax) - 2 + 127)   (0 for a group of zeros)
 *   code = x * 2^(127-k) rounded to the nearest E2M1 value, ties to even,
 *          magnitudes above 6 to 6; the sign of a zero is kept
 * (2 is the exponent of E2M1's largest binade: the OCP microscaling format's
 * conversion).  Both steps are exact but for that one rounding.  A group that
 * holds an infinity or a NaN gets k = 255 (NaN) and codes 0.
 *   x        x_rows rows of `type`, row i at x + i*ld elements (ld >= cols);
 *            aligned to its element size
 *   row_of   nullable: output row i is x row row_of[i] (device, int32[rows]),
 *            or a row of zeros where row_of[i] is outside [0, x_rows);
 *            NULL: row i, and rows <= x_rows
 *   out      the MXFP4 matrix [rows, cols]
 *   values   nullable: the rounded values, [rows, cols] of `type` (exact in
 *            every type: x's own range holds them), e.g. for a forward pass
 *            through frozen roundings; NaN in a NaN group */
int mxfp4_quant(const void* x, int type, int x_rows, int cols, long long ld,
                const int32_t* row_of, int rows, void* out, void* values, cudaStream_t stream);

/* The same quantisation of act = silu(gate) * up, silu(g) = g / (1 + exp(-g)) in
 * FP32 (the act of mxfp4_moe_gate_up, to within 2^-20 of itself and, where exp(gate)
 * is subnormal, 2^-149 |gate up|): gate and up [rows, cols] of `type`, rows ld
 * elements apart.  swiglu_limit > 0 clamps up to
 * [-limit, limit] and gate to at most limit first (a NaN of either stays one); 0 or
 * less turns the clamp off; NaN is refused.  `values` are exact in F32 and BF16; an
 * act of halves may leave their range although its codes hold it, so F16 values are
 * rounded once more, to the nearest half (infinite from 65520 on, subnormal or zero
 * below 2^-14): a pass through them then differs from one through the codes. */
int mxfp4_swiglu_quant(const void* gate, const void* up, int type, int rows, int cols,
                       long long ld, float swiglu_limit, void* out, void* values,
                       cudaStream_t stream);

/* Product of two MXFP4 matrices: Y[t*rows + r] = sum_c W[r][c] * X[t][c], W
 * [rows, cols], X [nb, cols], Y [nb, rows] of y_type (F32 or BF16; the FP32 sum
 * rounded once to nearest even).  On the block-scaled 4-bit tensor cores, any
 * nb >= 1.  Every product of two elements is exact; sums are FP32, 64 columns
 * added at a time, each addition losing less than 2^-23 of the running sum.
 * Error bound (before the rounding to BF16): (cols / 64 + 8) * 2^-23 * sum_c
 * |W X|, nearly reached where the first 64 columns hold almost all of the sum and
 * each later 64 less than its last bit; sums of one sign that grow evenly come to
 * a sixth of it, and with mixed signs the error is two orders smaller.  A group with scale byte 255 in either operand makes its
 * row (W) or its token (X) NaN.  Per token the result does not depend on the
 * other tokens' values, but it may on nb (the order of the sums is chosen by
 * the shape).  Deterministic. */
int mxfp4_mm_mx(const void* w, int rows, int cols, const void* xq, int nb, void* Y, int y_type,
                cudaStream_t stream);

/* Each expert's rows with that expert's matrix: for offsets[e] <= i < offsets[e+1]
 *   Y[i*rows + r] = sum_c W_e[r][c] * X[i][c].
 * bank: n_experts matrices [rows, cols], expert e at e * mxfp4_nbytes(rows, cols);
 * xq: the MXFP4 matrix [n_rows, cols] in expert order; offsets: device,
 * int32[n_experts + 1], not decreasing, offsets[0] = 0, offsets[n_experts] <=
 * n_rows (as mxfp4_moe_sort writes them; anything past n_rows is cut off there);
 * Y: [n_rows, rows], rows at and past offsets[n_experts] left untouched.
 * n_experts <= MXFP4_MOE_MAX_SORTED_EXPERTS.  Results as mxfp4_mm_mx. */
#define MXFP4_MOE_MAX_SORTED_EXPERTS 1024
int mxfp4_moe_mm_mx(const void* bank, int n_experts, int rows, int cols, const void* xq,
                    int n_rows, const int32_t* offsets, void* Y, int y_type,
                    cudaStream_t stream);

/* Expert order of the pairs p = t*top_k + j (t < n_tokens): a stable counting
 * sort by expert_ids[p] ("rlx-cpu 0.2.17 src/gguf_matmul.rs"
 * grouped_moe_sort_plan).  With P = n_tokens * top_k <= 2^22:
 *   offsets   int32[n_experts + 1]: expert e's rows are offsets[e] .. offsets[e+1]
 *   token_at  int32[P]: the token of row i, -1 for i >= offsets[n_experts]
 *   pos_of    int32[P]: the row of pair p, -1 for a pair whose id is outside
 *             [0, n_experts) (a dropped pair: it has no row)
 * n_experts <= MXFP4_MOE_MAX_SORTED_EXPERTS. */
int mxfp4_moe_sort(const int32_t* expert_ids, int n_tokens, int top_k, int n_experts,
                   int32_t* token_at, int32_t* pos_of, int32_t* offsets, cudaStream_t stream);

/* The tokens' rows in expert order: xs[i] = x[token_at[i]], zeros where token_at[i]
 * is outside [0, n_tokens).  x [n_tokens, width], xs [n_tokens*top_k, width], both of
 * `type`; any width >= 1. */
int mxfp4_moe_dispatch(const void* x, int type, int n_tokens, int top_k, int width,
                       const int32_t* token_at, void* xs, cudaStream_t stream);

/* Its gradient: dx[t] = sum_j dxs[pos_of[t*top_k + j]] over the token's rows, in
 * FP32 in the order of j, rounded once.  A pos_of outside [0, n_tokens*top_k) adds
 * nothing. */
int mxfp4_moe_dispatch_grad(const void* dxs, int type, int n_tokens, int top_k, int width,
                            const int32_t* pos_of, void* dx, cudaStream_t stream);

/* Back to token order with the route weights: y[t] = sum_j route_w[t*top_k + j] *
 * o[pos_of[t*top_k + j]], in FP32 in the order of j, rounded once.  o
 * [n_tokens*top_k, width], y [n_tokens, width] of `type`; route_w
 * [n_tokens*top_k] floats.  Dropped pairs (pos_of outside [0, n_tokens*top_k)) add
 * nothing, whatever their weight. */
int mxfp4_moe_combine(const void* o, int type, int n_tokens, int top_k, int width,
                      const int32_t* pos_of, const float* route_w, void* y, cudaStream_t stream);

/* Its gradient: for every pair p = t*top_k + j with a row i = pos_of[p]
 *   d_o[i] = route_w[p] * dy[t]  (rounded once),  d_route_w[p] = <dy[t], o[i]> (FP32),
 * and d_route_w[p] = 0 for a dropped pair.  Rows of d_o that belong to no pair are
 * left untouched. */
int mxfp4_moe_combine_grad(const void* dy, const void* o, int type, int n_tokens, int top_k,
                           int width, const int32_t* pos_of, const float* route_w, void* d_o,
                           float* d_route_w, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MX4_H */
