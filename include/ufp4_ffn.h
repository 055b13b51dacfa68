/*
 * ufp4_ffn.h -- C ABI of the operators of a feed-forward sublayer, next to the
 * 4-bit GEMMs of ufp4.h and the block operators of ufp4_block.h, in the same
 * library (libufp4.so):
 *   - layer norm with the residual's addition, forward and backward;
 *   - the gated product act(x Wg^T) * (x Wu^T) of two projections on 4-bit
 *     operands in one kernel, dense or grouped by experts, and its backward;
 *   - dropout from a counter-based generator, onto a residual or alone;
 *   - rows in 8-bit integers with one scale each, and the product of two such
 *     operands (scales for each token and channel), dense or grouped, with a
 *     bias or as a gated product: the form that serves a trained layer.
 *
 * The conventions are those of ufp4_block.h: buffer pointers are DEVICE
 * pointers owned by the caller, descriptor structs are HOST memory read during
 * the call, work is enqueued on `stream` as kernel launches only (calls can be
 * captured into a HIP graph), arguments are validated on the host before
 * anything is enqueued, every result is deterministic run to run.  Element
 * types are ufp4_out_dtype codes (UFP4_OUT_F32, UFP4_OUT_BF16).  Floating-point
 * buffers are aligned to their element size and may start at any element.
 * Strides (ld_*) are in elements, at least the row length, and rows times the
 * stride at most 2^60.  Zero rows are accepted: such a call writes what it has
 * to write (zero sums).  Contents of device arrays are not validated by the
 * host; whatever group offsets hold, nothing is read or written out of range.
 */
#ifndef UFP4_FFN_H
#define UFP4_FFN_H

#include "ufp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The activation of a gated product: silu(g) = g / (1 + exp(-g)), gelu(g) =
 * g (1 + erf(g / sqrt 2)) / 2.  NONE: a plain product (int8 calls only). */
typedef enum { UFP4_ACT_NONE = 0, UFP4_ACT_SILU = 1, UFP4_ACT_GELU = 2 } ufp4_act;

/* ------------------------------------------------------------------------
 * Layer norm.   h = round(x + residual)  (an FP32 sum; h = x without one)
 *               mean = mean(h), rstd = 1 / sqrt(mean((h - mean)^2) + eps)
 *               y = (h - mean) * rstd * weight + bias
 * x, residual, h, y are of type `dtype`; weight and bias (NULL: none) of type
 * weight_dtype, either `dtype` or UFP4_OUT_F32.  The statistics are those of
 * the rounded h; the squares are those of the centred values.
 *   residual  NULL: none; h is then ignored, else h is required, dense
 *             [rows, cols]; h may be x or residual itself when that is dense.
 *   y         dense [rows, cols].   mean, rstd  FP32 [rows].
 * ufp4_layernorm_bwd: given dy, the gradient of y, and dh (or NULL), the
 * gradient that reaches h from elsewhere,
 *   xhat = (h - mean) rstd, g = dy weight,
 *   dx = rstd (g - mean(g) - xhat mean(g xhat)) + dh  (of x and the residual)
 *   dw = sum over rows of dy xhat,  db = sum over rows of dy (or NULL)
 * dx is dense and may be dy or dh itself when that is dense.  workspace:
 * device, 16-byte aligned, at least ufp4_layernorm_bwd_workspace_size(rows,
 * cols) bytes, overwritten.  Returns OK, INVALID_ARG (null or misaligned
 * pointer, unknown type, eps negative or NaN), SHAPE, HIP. */
ufp4_status ufp4_layernorm(const void *x, int64_t ld_x, const void *residual, int64_t ld_residual,
                           const void *weight, const void *bias, int32_t dtype,
                           int32_t weight_dtype, int64_t rows, int64_t cols, float eps, void *h,
                           void *y, float *mean, float *rstd, hipStream_t stream);
size_t ufp4_layernorm_bwd_workspace_size(int64_t rows, int64_t cols);
ufp4_status ufp4_layernorm_bwd(const void *dy, int64_t ld_dy, const void *h, int64_t ld_h,
                               const void *weight, const float *mean, const float *rstd,
                               const void *dh, int64_t ld_dh, int32_t dtype, int32_t weight_dtype,
                               int64_t rows, int64_t cols, void *dx, void *dw, void *db,
                               void *workspace, size_t workspace_bytes, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Dropout.   y = residual + (keep ? x / (1 - P) : 0)    (residual NULL: none)
 * The mask is never stored: 16 random bits belong to each element, and keep is
 * bits >= T with T = floor(65536 p + 1/2), P = T / 65536 (so the expectation is
 * exact for the p that is used).  They come from Philox4x32-10 (Salmon,
 * Moraes, Dror and Shaw, SC'11) with `seed` as the key, low word first.  The
 * columns c..c+7 (c a multiple of 8) of row r share one call, whose counter is
 * the 64-bit number r * ceil(cols / 8) + c / 8 in words 0 and 1 and the 64-bit
 * number `offset` + *d_offset (d_offset NULL: 0; sums wrap) in words 2 and 3;
 * column c + 2 i takes the low and c + 2 i + 1 the high half of its word i.
 * The same call with dy for x and no residual is the backward pass.  An
 * element that is dropped is 0 whatever it held.  P = 1 drops everything; P =
 * 0 draws nothing.  x, residual [rows, cols] and y (dense) are of type dtype; y
 * may be x or residual itself when that is dense.  d_offset is read when the
 * kernel runs, so that a captured call draws another mask at each replay if
 * the caller advances it.  Returns OK, INVALID_ARG (also p outside [0, 1]),
 * SHAPE, HIP. */
ufp4_status ufp4_dropout(const void *x, int64_t ld_x, const void *residual, int64_t ld_residual,
                         int32_t dtype, int64_t rows, int64_t cols, double p, uint64_t seed,
                         uint64_t offset, const int64_t *d_offset, void *y, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Gated product on 4-bit operands:  g = x Wg^T, u = x Wu^T, y = act(g) * u.
 * x [T, K] and w are quantized operands as ufp4_gemm_out takes them (same K,
 * grid, RHT and sign mask); w has 2 F rows for each of n_groups experts: Wg's F
 * rows, then Wu's.  y is dense-rowed [T, F] with stride ld_y.  gu, or NULL: g
 * and u [T, 2 F] with stride ld_gu, g in the first F columns, for the backward
 * pass.  Both of type out_dtype, rounded once from FP32 (y from the unrounded
 * g and u).  d_group_offsets NULL: one group of all rows (n_groups 1), else
 * int64 [n_groups + 1] as ufp4_grouped_gemm takes them; rows in no group are
 * left as they are.  g and u are the FP32 sums of ufp4_gemm_out's terms, one per block
 * of 16.  Where there are many tiles of output they are added in its order, one after
 * the other, and g and u are its bits; where there are few, in eight such chains and
 * the chains' sums in order.  T, F and n_groups decide, so a row's last bits may
 * change with the rows beside it; either way a sum is within (K / 16 + 8) 2^-24 of the
 * sum of its terms' sizes, and a call repeated gives the same bits.  Returns OK,
 * INVALID_ARG (also act NONE), SHAPE (also an odd number of rows per group, n_groups
 * outside 1..1024, T = 0 or F = 0), MISMATCH, UNSUPPORTED (K beyond 65536), HIP.
 *
 * ufp4_gated_bwd: from dy [rows, cols] and gu [rows, 2 cols],
 *   dgu = (dy u act'(g) | dy act(g))   dense [rows, 2 cols],
 * all of type dtype; dgu may be gu itself when that is dense.  It is dY of the
 * two projections as one product: quantize it, then DGRAD and WGRAD.
 * act(g) u and its slopes are FP32, rounded once. */
ufp4_status ufp4_gated_gemm(const ufp4_qtensor *x, const ufp4_qtensor *w, int32_t act,
                            int32_t n_groups, const int64_t *d_group_offsets, int32_t out_dtype,
                            void *y, int64_t ld_y, void *gu, int64_t ld_gu, hipStream_t stream);
ufp4_status ufp4_gated_bwd(const void *dy, int64_t ld_dy, const void *gu, int64_t ld_gu,
                           int32_t act, int32_t dtype, int64_t rows, int64_t cols, void *dgu,
                           hipStream_t stream);

/* ------------------------------------------------------------------------
 * Rows in 8-bit integers with one scale each.
 *   scale = max|x| / 127 over the row, q = round(x * (127 * (1 / max|x|))),
 *   to nearest even, each operation rounded to FP32; |q| <= 127.
 * q is dense [rows, kpad] with kpad = cols rounded up to a multiple of 128,
 * zero past the row's end.  A zero row has scale 0 and q 0.  A row that holds
 * an infinity or a NaN has scale NaN and q 0, so that its products are NaN.
 * Returns OK, INVALID_ARG, SHAPE, HIP. */
ufp4_status ufp4_int8_quantize(const void *x, int64_t ld_x, int32_t dtype, int64_t rows,
                               int64_t cols, int8_t *q, float *scale, hipStream_t stream);

/* An operand of the int8 product: rows [rows, kpad] of int8, 16-byte aligned,
 * kpad the multiple of 128 from k on, zeros past k in one of the two operands
 * at least, and an FP32 scale for each row. */
typedef struct {
  const int8_t *q;
  const float *scale;
  int64_t rows, k;
} ufp4_int8_rows;

/* Product of int8 rows:  p[m, n] = scale_a[m] scale_w[n] sum_k qa[m, k] qw[n, k]
 * (+ bias[n], FP32, NULL: none).  act NONE: y = p, [M, N].  act SILU or GELU: w
 * has 2 F rows per group, gate rows first, and y = act(p[:, :F]) * p[:, F:], [M,
 * F].  The sums are exact integers; the scales, the bias and the activation are
 * FP32, rounded once to out_dtype.  d_group_offsets NULL: one group of all
 * rows (n_groups 1); else int64 [n_groups + 1] over a's rows, w has n_groups
 * times the rows of one expert, and a bias as many entries; rows of a in no
 * group leave their rows of y as they are.  Which kernel runs goes by M, N, K and
 * n_groups; results are the same bit for bit.  The FP32 operations are ((sum *
 * scale_a) * scale_w) + bias, each rounded.
 * ufp4_int8_linear: the same with a = ufp4_int8_quantize(x), x [M, k] of type
 * dtype; workspace: device, 16-byte aligned, at least
 * ufp4_int8_linear_workspace_size(M, k, grouped) bytes, overwritten, grouped 0
 * where d_group_offsets is NULL (0 bytes for a few rows, which every workgroup
 * quantizes itself: then it may be NULL; a workspace of the size for grouped 1 makes
 * such a call faster where y has more than 16384 columns).  y may not be x.
 * Returns OK, INVALID_ARG, SHAPE (k of a and w differ, rows not a multiple of
 * the groups, n_groups outside 1..1024), UNSUPPORTED (k beyond 131071: a sum
 * could pass 31 bits), HIP. */
ufp4_status ufp4_int8_gemm(const ufp4_int8_rows *a, const ufp4_int8_rows *w, const float *bias,
                           int32_t act, int32_t n_groups, const int64_t *d_group_offsets,
                           int32_t out_dtype, void *y, int64_t ld_y, hipStream_t stream);
size_t ufp4_int8_linear_workspace_size(int64_t rows, int64_t cols, int32_t grouped);
ufp4_status ufp4_int8_linear(const void *x, int64_t ld_x, int32_t dtype, int64_t rows,
                             int64_t cols, const ufp4_int8_rows *w, const float *bias, int32_t act,
                             int32_t n_groups, const int64_t *d_group_offsets, int32_t out_dtype,
                             void *y, int64_t ld_y, void *workspace, size_t workspace_bytes,
                             hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* UFP4_FFN_H */
