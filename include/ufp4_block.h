/*
 * ufp4_block.h -- C ABI of the operators that stand around the 4-bit GEMMs of
 * ufp4.h in a transformer block, in the same library (libufp4.so):
 *   - RMS norm with the residual's addition, with an output in the input's
 *     type and/or in FP8 E4M3 with one scale per row, forward and backward;
 *   - the MoE router: top-k choices, gates, per-expert counts and the group
 *     offsets of the grouped GEMMs, balance and z loss, and its backward;
 *   - dispatch of tokens to expert order and the gate-weighted combination
 *     back, forward and backward;
 *   - the global gradient norm over many tensors, and clipping by it.
 *
 * The conventions are those of ufp4.h: buffer pointers are DEVICE pointers
 * owned by the caller, descriptor structs are HOST memory read during the
 * call, work is enqueued on `stream` as kernel launches only (calls can be
 * captured into a HIP graph), arguments are validated on the host before
 * anything is enqueued, and every result is deterministic run to run (no
 * floating-point atomics).  Element types are ufp4_out_dtype codes
 * (UFP4_OUT_F32, UFP4_OUT_BF16).  Floating-point buffers are aligned to their
 * element size and may start at any element: the kernels' 16-byte accesses
 * need no more.  Strides (ld_*) are in elements, at least the row length, and
 * rows times the stride at most 2^60.
 * Statistics, sums and gradients are accumulated in FP32 (FP64 where stated)
 * and rounded once to the output's type, to nearest even.  Zero rows or
 * tokens are accepted: such a call writes what it has to write (zero sums).
 *
 * Contents of device arrays are not validated by the host.  A slot outside
 * its array is treated as a choice without a row; nothing is read or written
 * out of range.
 */
#ifndef UFP4_BLOCK_H
#define UFP4_BLOCK_H

#include "ufp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * RMS norm.   h = round(x + residual)  (an FP32 sum; h = x without a residual)
 *             rstd = 1 / sqrt(mean(h^2) + eps),  y = h * rstd * weight
 * x, residual, h, y are of type `dtype`; weight is of type weight_dtype,
 * either `dtype` or UFP4_OUT_F32.  The statistics are those of the rounded h,
 * which is what the backward pass is given.
 * ufp4_rmsnorm:
 *   residual   NULL: none; h is then ignored (h = x), else h is required,
 *              dense [rows, cols].  h may be x or residual itself when that
 *              is dense (the residual stream updated in place).
 *   y          dense [rows, cols], or NULL.
 *   q, scale   dense E4M3 (OCP) bytes [rows, cols] and FP32 [rows], or both
 *              NULL: scale = max|y| / 448 over the row's unrounded y, and
 *              q = round(y / scale), so |q| <= 448, from FP32 values of y and
 *              the quotient (an exact half step may go either way).  A zero
 *              row has scale 0 and q 0; a row that holds an infinity or a
 *              NaN is NaN.
 *   rstd       FP32 [rows].
 * At least one of y and q.  Returns OK, INVALID_ARG (null or misaligned
 * pointer, unknown type, eps negative or NaN), SHAPE, HIP.
 *
 * ufp4_rmsnorm_bwd: given dy, the gradient of y, and dh (or NULL), the
 * gradient that reaches h from elsewhere,
 *   xhat = h rstd, g = dy weight,
 *   dx = rstd (g - xhat mean(g xhat)) + dh     (of x and of the residual)
 *   dw = sum over rows of dy xhat              (of type weight_dtype)
 * dx is dense and may be dy or dh itself when that is dense.  workspace:
 * device, 16-byte aligned, at least ufp4_rmsnorm_bwd_workspace_size(rows,
 * cols) bytes, overwritten. */
ufp4_status ufp4_rmsnorm(const void *x, int64_t ld_x, const void *residual, int64_t ld_residual,
                         const void *weight, int32_t dtype, int32_t weight_dtype, int64_t rows,
                         int64_t cols, float eps, void *h, void *y, uint8_t *q, float *scale,
                         float *rstd, hipStream_t stream);
size_t ufp4_rmsnorm_bwd_workspace_size(int64_t rows, int64_t cols);
ufp4_status ufp4_rmsnorm_bwd(const void *dy, int64_t ld_dy, const void *h, int64_t ld_h,
                             const void *weight, const float *rstd, const void *dh, int64_t ld_dh,
                             int32_t dtype, int32_t weight_dtype, int64_t rows, int64_t cols,
                             void *dx, void *dw, void *workspace, size_t workspace_bytes,
                             hipStream_t stream);

/* ------------------------------------------------------------------------
 * MoE router over logits [tokens, n_experts] (stride ld, type dtype).
 *   lse   = log sum_e exp(l_e),  p_e = exp(l_e - lse)
 *   The token's choices are its k largest logits, the lowest expert first
 *   among equals; an expert whose logit is -inf or NaN is never chosen.
 *   gate  = p of the choice, or with renorm != 0 that over the sum of the
 *   token's chosen p (a softmax over the chosen logits).
 * A token takes no part when valid[token] is 0 (valid NULL: all are valid)
 * or when all its logits are -inf: it has no choices, counts nowhere and its
 * lse is -inf.  A logit of NaN or +inf makes the token's lse, gates and
 * gradients and the losses what IEEE arithmetic makes of them.
 * Outputs (ufp4_routing, all dense):
 *   experts  int32 [tokens, k], by falling logit; -1 where there is none.
 *   gates    FP32  [tokens, k], 0 where there is no choice.
 *   lse      FP32  [tokens].
 *   slots    int32 [tokens, k]: the row of the choice in expert order.  Rows
 *            are ordered by expert, then by token.  Choices that do not exist
 *            share out the rows after those in the same order and are stored
 *            as ~row (negative).
 *   counts   int64 [n_experts], choices per expert.
 *   offsets  int64 [n_experts + 1]: the group offsets that the grouped
 *            calls of ufp4.h take over tokens * k rows: offsets[e] = the sum
 *            of counts before e, and offsets[n_experts] = tokens * k (the
 *            rows without a choice, which dispatch writes as zeros, end the
 *            last group).
 *   n_tokens int64 [1], the number N of tokens that take part.
 *   losses   FP32 [2]: the balance loss
 *              n_experts * sum_e (counts_e / (k N)) (sum_t p_te / N)
 *            and the z loss  sum_t lse_t^2 / N;  both 0 when N is 0.
 * workspace: device, 16-byte aligned, at least
 * ufp4_moe_route_workspace_size(tokens, n_experts) bytes, overwritten (0 for
 * up to 64 tokens: then it may be NULL).
 * 1 <= k <= 16, k <= n_experts <= 1024, tokens * k < 2^31.
 *
 * ufp4_moe_route_bwd: d_logits (dense, type dtype) from d_gates FP32
 * [tokens, k] and d_losses FP32 [2] (device; either may be NULL: zero).  The
 * counts are constants, as usual for this loss; `r` and the logits are those
 * of the forward call.  Returns OK, INVALID_ARG, SHAPE, UNSUPPORTED (k or
 * n_experts beyond the limits, tokens * k >= 2^31), HIP. */
typedef struct {
  int32_t *experts;
  float *gates;
  int32_t *slots;
  float *lse;
  int64_t *counts;
  int64_t *offsets;
  int64_t *n_tokens;
  float *losses;
} ufp4_routing;

size_t ufp4_moe_route_workspace_size(int64_t tokens, int32_t n_experts);
ufp4_status ufp4_moe_route(const void *logits, int64_t ld, int32_t dtype, const uint8_t *valid,
                           int64_t tokens, int32_t n_experts, int32_t k, int32_t renorm,
                           const ufp4_routing *r, void *workspace, size_t workspace_bytes,
                           hipStream_t stream);
ufp4_status ufp4_moe_route_bwd(const void *logits, int64_t ld, int32_t dtype, int64_t tokens,
                               int32_t n_experts, int32_t k, int32_t renorm,
                               const ufp4_routing *r, const float *d_gates,
                               const float *d_losses, void *d_logits, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Token exchange with expert order.  slots int32 [tokens, k] as the router
 * writes them; xs, ys, dxs and dys are dense [tokens * k, cols]; x, dx, y, dy
 * and residual are [tokens, cols] (the outputs dense).  All of type dtype;
 * gates and d_gates FP32 [tokens, k].
 *   dispatch      xs[slot] = x[token], and zeros in the rows without a choice
 *   dispatch_bwd  dx[token] = sum over the token's choices of dxs[slot]
 *   combine       y[token] = residual[token] + sum of gate * ys[slot]
 *                 (residual NULL: none)
 *   combine_bwd   dys[slot] = gate * dy[token] (zeros without a choice),
 *                 d_gate = <ys[slot], dy[token]> (0 without a choice);
 *                 dy itself is the residual's gradient.
 * Rows without a choice are never read.  1 <= k <= 16, tokens * k < 2^31.
 * Returns OK, INVALID_ARG, SHAPE, UNSUPPORTED, HIP. */
ufp4_status ufp4_moe_dispatch(const void *x, int64_t ld_x, const int32_t *slots, int32_t dtype,
                              int64_t tokens, int32_t k, int64_t cols, void *xs,
                              hipStream_t stream);
ufp4_status ufp4_moe_dispatch_bwd(const void *dxs, const int32_t *slots, int32_t dtype,
                                  int64_t tokens, int32_t k, int64_t cols, void *dx,
                                  hipStream_t stream);
ufp4_status ufp4_moe_combine(const void *ys, const int32_t *slots, const float *gates,
                             const void *residual, int64_t ld_residual, int32_t dtype,
                             int64_t tokens, int32_t k, int64_t cols, void *y,
                             hipStream_t stream);
ufp4_status ufp4_moe_combine_bwd(const void *dy, int64_t ld_dy, const void *ys,
                                 const int32_t *slots, const float *gates, int32_t dtype,
                                 int64_t tokens, int32_t k, int64_t cols, void *dys,
                                 float *d_gates, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Global gradient norm and clipping, over n_tensors tensors of any sizes.
 *   norm = sqrt(sum over all tensors and elements of g^2), squares and sums
 *          in FP64, to *norm (FP32, device)
 *   clip: out = g * min(1, max_norm / (norm + eps)) in every tensor, the
 *         coefficient taken from *norm on the device (no synchronisation).
 *         A norm + eps of at most max_norm scales nothing (also where both
 *         are zero or infinite).  A NaN norm gives NaN everywhere, an
 *         infinite one beyond max_norm zeros (NaN where the element is not
 *         finite).  With out == data and a coefficient of 1 nothing is
 *         written.
 * Each tensor is n dense elements of type dtype; out (of type out_dtype) may
 * be data itself when the types agree, and is ignored by ufp4_grad_norm.
 * Tensors must not overlap each other's outputs.  n = 0 is accepted.
 * workspace: device, 16-byte aligned, at least
 * ufp4_grad_norm_workspace_size() bytes, overwritten by ufp4_grad_norm only.
 * Returns OK, INVALID_ARG (also max_norm negative or NaN, eps negative or
 * NaN), SHAPE, HIP. */
typedef struct {
  const void *data;
  void *out;
  int64_t n;
  int32_t dtype;
  int32_t out_dtype;
} ufp4_grad;

size_t ufp4_grad_norm_workspace_size(void);
ufp4_status ufp4_grad_norm(const ufp4_grad *grads, int64_t n_tensors, void *workspace,
                           size_t workspace_bytes, float *norm, hipStream_t stream);
ufp4_status ufp4_grad_clip(const ufp4_grad *grads, int64_t n_tensors, const float *norm,
                           double max_norm, double eps, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* UFP4_BLOCK_H */
