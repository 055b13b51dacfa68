// C ABI of the block operators (include/ufp4_block.h): host-side validation,
// then the launches on the caller's stream.  No allocation of device memory,
// no synchronisation, no state.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/ufp4_block.h"
#include "block_kernels.h"

using namespace ufp4;

namespace {

bool aligned_to(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool known_type(int32_t t) { return t == UFP4_OUT_F32 || t == UFP4_OUT_BF16; }
uintptr_t size_of(int32_t t) { return t == UFP4_OUT_BF16 ? 2 : 4; }
// Not null, and aligned to its element.
bool good(const void *p, uintptr_t size) { return p != nullptr && aligned_to(p, size); }
bool good_or_null(const void *p, uintptr_t size) { return aligned_to(p, size); }

ufp4_status of(hipError_t e) { return e == hipSuccess ? UFP4_OK : UFP4_ERR_HIP; }

// Sizes that keep every element index and byte offset of a tensor in 63 bits.
constexpr int64_t kMaxRows = int64_t(1) << 40;
constexpr int64_t kMaxCols = int64_t(1) << 24;
constexpr int64_t kMaxLd = int64_t(1) << 40;
constexpr int64_t kMaxElems = int64_t(1) << 44;
constexpr int64_t kMaxSpan = int64_t(1) << 60;     // elements from the first row to the last

ufp4_status check_norm_shape(int64_t rows, int64_t cols) {
  if (rows < 0 || cols <= 0 || rows > kMaxRows || cols > kMaxCols || rows > kMaxElems / cols)
    return UFP4_ERR_SHAPE;
  return UFP4_OK;
}
bool bad_ld(int64_t ld, int64_t rows, int64_t cols) {
  return ld < cols || ld > kMaxLd || (rows > 1 && ld > kMaxSpan / rows);
}

ufp4_status check_exchange(int32_t dtype, int64_t tokens, int32_t k, int64_t cols) {
  if (!known_type(dtype)) return UFP4_ERR_INVALID_ARG;
  if (tokens < 0 || k < 1 || cols <= 0 || cols > kMaxCols) return UFP4_ERR_SHAPE;
  if (k > kRouteMaxK || tokens > INT32_MAX / k) return UFP4_ERR_UNSUPPORTED;
  return UFP4_OK;
}

ufp4_status check_route(const void *logits, int64_t ld, int32_t dtype, int64_t tokens,
                        int32_t n_experts, int32_t k, int32_t renorm, const ufp4_routing *r) {
  if (!known_type(dtype) || (renorm != 0 && renorm != 1) || r == nullptr)
    return UFP4_ERR_INVALID_ARG;
  if (tokens < 0 || n_experts < 1 || k < 1 || k > n_experts || bad_ld(ld, tokens, n_experts))
    return UFP4_ERR_SHAPE;
  if (n_experts > kRouteMaxExperts || k > kRouteMaxK || tokens > INT32_MAX / k)
    return UFP4_ERR_UNSUPPORTED;
  if (tokens > 0 && (!good(logits, size_of(dtype)) || !good(r->experts, 4) ||
                     !good(r->gates, 4) || !good(r->lse, 4)))
    return UFP4_ERR_INVALID_ARG;
  if (!good(r->counts, 8) || !good(r->n_tokens, 8)) return UFP4_ERR_INVALID_ARG;
  return UFP4_OK;
}

RouteArgs route_args(const void *logits, int64_t ld, int32_t dtype, int64_t tokens,
                     int32_t n_experts, int32_t k, int32_t renorm, const ufp4_routing *r) {
  RouteArgs a{};
  a.logits = logits;
  a.ld = ld;
  a.bf16 = dtype == UFP4_OUT_BF16;
  a.tokens = tokens;
  a.n_experts = n_experts;
  a.k = k;
  a.renorm = renorm;
  a.experts = r->experts;
  a.gates = r->gates;
  a.slots = r->slots;
  a.lse = r->lse;
  a.counts = r->counts;
  a.offsets = r->offsets;
  a.n_tokens = r->n_tokens;
  a.losses = r->losses;
  return a;
}

ufp4_status check_grads(const ufp4_grad *grads, int64_t n_tensors, bool clip) {
  if (n_tensors < 0 || n_tensors > (int64_t(1) << 32)) return UFP4_ERR_SHAPE;
  if (n_tensors > 0 && grads == nullptr) return UFP4_ERR_INVALID_ARG;
  for (int64_t i = 0; i < n_tensors; ++i) {
    const ufp4_grad &g = grads[i];
    if (!known_type(g.dtype) || (clip && !known_type(g.out_dtype))) return UFP4_ERR_INVALID_ARG;
    if (g.n < 0 || g.n > kMaxElems) return UFP4_ERR_SHAPE;
    if (g.n == 0) continue;
    if (!good(g.data, size_of(g.dtype))) return UFP4_ERR_INVALID_ARG;
    if (clip && (!good(g.out, size_of(g.out_dtype)) ||
                 (g.out == g.data && g.out_dtype != g.dtype)))
      return UFP4_ERR_INVALID_ARG;
  }
  return UFP4_OK;
}

}  // namespace

extern "C" {

ufp4_status ufp4_rmsnorm(const void *x, int64_t ld_x, const void *residual, int64_t ld_residual,
                         const void *weight, int32_t dtype, int32_t weight_dtype, int64_t rows,
                         int64_t cols, float eps, void *h, void *y, uint8_t *q, float *scale,
                         float *rstd, hipStream_t stream) {
  if (!known_type(dtype) || (weight_dtype != dtype && weight_dtype != UFP4_OUT_F32) ||
      !(eps >= 0.0f))
    return UFP4_ERR_INVALID_ARG;
  const ufp4_status s = check_norm_shape(rows, cols);
  if (s != UFP4_OK) return s;
  if (bad_ld(ld_x, rows, cols) || (residual != nullptr && bad_ld(ld_residual, rows, cols)))
    return UFP4_ERR_SHAPE;
  const uintptr_t e = size_of(dtype);
  if (!good(weight, size_of(weight_dtype))) return UFP4_ERR_INVALID_ARG;
  if (rows == 0) return UFP4_OK;
  if ((q == nullptr) != (scale == nullptr) || (y == nullptr && q == nullptr))
    return UFP4_ERR_INVALID_ARG;
  if (!good(x, e) || !good(rstd, 4) || (residual != nullptr && !good(h, e)) ||
      !good_or_null(residual, e) || !good_or_null(y, e) || !good_or_null(scale, 4))
    return UFP4_ERR_INVALID_ARG;
  NormArgs a{};
  a.x = x;
  a.ld_x = ld_x;
  a.res = residual;
  a.ld_res = ld_residual;
  a.w = weight;
  a.bf16 = dtype == UFP4_OUT_BF16;
  a.w_bf16 = weight_dtype == UFP4_OUT_BF16;
  a.rows = rows;
  a.cols = cols;
  a.eps = eps;
  a.h = h;
  a.y = y;
  a.q = q;
  a.scale = scale;
  a.rstd = rstd;
  return of(launch_rmsnorm(a, stream));
}

size_t ufp4_rmsnorm_bwd_workspace_size(int64_t rows, int64_t cols) {
  if (check_norm_shape(rows, cols) != UFP4_OK) return 0;
  return (size_t)norm_bwd_slices(rows, cols) * (size_t)cols * sizeof(float);
}

ufp4_status ufp4_rmsnorm_bwd(const void *dy, int64_t ld_dy, const void *h, int64_t ld_h,
                             const void *weight, const float *rstd, const void *dh, int64_t ld_dh,
                             int32_t dtype, int32_t weight_dtype, int64_t rows, int64_t cols,
                             void *dx, void *dw, void *workspace, size_t workspace_bytes,
                             hipStream_t stream) {
  if (!known_type(dtype) || (weight_dtype != dtype && weight_dtype != UFP4_OUT_F32))
    return UFP4_ERR_INVALID_ARG;
  const ufp4_status s = check_norm_shape(rows, cols);
  if (s != UFP4_OK) return s;
  if (bad_ld(ld_dy, rows, cols) || bad_ld(ld_h, rows, cols) ||
      (dh != nullptr && bad_ld(ld_dh, rows, cols)))
    return UFP4_ERR_SHAPE;
  const uintptr_t e = size_of(dtype), we = size_of(weight_dtype);
  if (!good(weight, we) || !good(dw, we) || !good_or_null(dh, e)) return UFP4_ERR_INVALID_ARG;
  if (!good(workspace, 16) || workspace_bytes < ufp4_rmsnorm_bwd_workspace_size(rows, cols))
    return UFP4_ERR_INVALID_ARG;
  if (rows > 0 && (!good(dy, e) || !good(h, e) || !good(rstd, 4) || !good(dx, e)))
    return UFP4_ERR_INVALID_ARG;
  NormBwdArgs a{};
  a.dy = dy;
  a.ld_dy = ld_dy;
  a.h = h;
  a.ld_h = ld_h;
  a.w = weight;
  a.rstd = rstd;
  a.dh = dh;
  a.ld_dh = ld_dh;
  a.bf16 = dtype == UFP4_OUT_BF16;
  a.w_bf16 = weight_dtype == UFP4_OUT_BF16;
  a.rows = rows;
  a.cols = cols;
  a.dx = dx;
  a.dw = dw;
  a.partial = static_cast<float *>(workspace);
  return of(launch_rmsnorm_bwd(a, stream));
}

size_t ufp4_moe_route_workspace_size(int64_t tokens, int32_t n_experts) {
  if (tokens < 0 || tokens > INT32_MAX || n_experts < 1 || n_experts > kRouteMaxExperts) return 0;
  return route_workspace_bytes(tokens, n_experts);
}

ufp4_status ufp4_moe_route(const void *logits, int64_t ld, int32_t dtype, const uint8_t *valid,
                           int64_t tokens, int32_t n_experts, int32_t k, int32_t renorm,
                           const ufp4_routing *r, void *workspace, size_t workspace_bytes,
                           hipStream_t stream) {
  const ufp4_status s = check_route(logits, ld, dtype, tokens, n_experts, k, renorm, r);
  if (s != UFP4_OK) return s;
  if ((tokens > 0 && !good(r->slots, 4)) || !good(r->offsets, 8) || !good(r->losses, 4))
    return UFP4_ERR_INVALID_ARG;
  const size_t need = ufp4_moe_route_workspace_size(tokens, n_experts);
  if (need > 0 && (!good(workspace, 16) || workspace_bytes < need)) return UFP4_ERR_INVALID_ARG;
  RouteArgs a = route_args(logits, ld, dtype, tokens, n_experts, k, renorm, r);
  a.valid = valid;
  a.workspace = workspace;
  return of(launch_route(a, stream));
}

ufp4_status ufp4_moe_route_bwd(const void *logits, int64_t ld, int32_t dtype, int64_t tokens,
                               int32_t n_experts, int32_t k, int32_t renorm,
                               const ufp4_routing *r, const float *d_gates,
                               const float *d_losses, void *d_logits, hipStream_t stream) {
  const ufp4_status s = check_route(logits, ld, dtype, tokens, n_experts, k, renorm, r);
  if (s != UFP4_OK) return s;
  if (!good_or_null(d_gates, 4) || !good_or_null(d_losses, 4)) return UFP4_ERR_INVALID_ARG;
  if (tokens > 0 && !good(d_logits, size_of(dtype))) return UFP4_ERR_INVALID_ARG;
  RouteArgs a = route_args(logits, ld, dtype, tokens, n_experts, k, renorm, r);
  a.d_gates = d_gates;
  a.d_losses = d_losses;
  a.d_logits = d_logits;
  return of(launch_route_bwd(a, stream));
}

ufp4_status ufp4_moe_dispatch(const void *x, int64_t ld_x, const int32_t *slots, int32_t dtype,
                              int64_t tokens, int32_t k, int64_t cols, void *xs,
                              hipStream_t stream) {
  const ufp4_status s = check_exchange(dtype, tokens, k, cols);
  if (s != UFP4_OK) return s;
  if (bad_ld(ld_x, tokens, cols)) return UFP4_ERR_SHAPE;
  if (tokens == 0) return UFP4_OK;
  const uintptr_t e = size_of(dtype);
  if (!good(x, e) || !good(slots, 4) || !good(xs, e)) return UFP4_ERR_INVALID_ARG;
  ExchangeArgs a{};
  a.in = x;
  a.ld_in = ld_x;
  a.slots = slots;
  a.bf16 = dtype == UFP4_OUT_BF16;
  a.tokens = tokens;
  a.k = k;
  a.cols = cols;
  a.out = xs;
  return of(launch_dispatch(a, stream));
}

ufp4_status ufp4_moe_dispatch_bwd(const void *dxs, const int32_t *slots, int32_t dtype,
                                  int64_t tokens, int32_t k, int64_t cols, void *dx,
                                  hipStream_t stream) {
  const ufp4_status s = check_exchange(dtype, tokens, k, cols);
  if (s != UFP4_OK) return s;
  if (tokens == 0) return UFP4_OK;
  const uintptr_t e = size_of(dtype);
  if (!good(dxs, e) || !good(slots, 4) || !good(dx, e)) return UFP4_ERR_INVALID_ARG;
  ExchangeArgs a{};
  a.in = dxs;
  a.slots = slots;
  a.bf16 = dtype == UFP4_OUT_BF16;
  a.tokens = tokens;
  a.k = k;
  a.cols = cols;
  a.out = dx;
  return of(launch_combine(a, stream));
}

ufp4_status ufp4_moe_combine(const void *ys, const int32_t *slots, const float *gates,
                             const void *residual, int64_t ld_residual, int32_t dtype,
                             int64_t tokens, int32_t k, int64_t cols, void *y,
                             hipStream_t stream) {
  const ufp4_status s = check_exchange(dtype, tokens, k, cols);
  if (s != UFP4_OK) return s;
  if (residual != nullptr && bad_ld(ld_residual, tokens, cols)) return UFP4_ERR_SHAPE;
  if (tokens == 0) return UFP4_OK;
  const uintptr_t e = size_of(dtype);
  if (!good(ys, e) || !good(slots, 4) || !good(gates, 4) || !good_or_null(residual, e) ||
      !good(y, e))
    return UFP4_ERR_INVALID_ARG;
  ExchangeArgs a{};
  a.in = ys;
  a.slots = slots;
  a.gates = gates;
  a.res = residual;
  a.ld_res = ld_residual;
  a.bf16 = dtype == UFP4_OUT_BF16;
  a.tokens = tokens;
  a.k = k;
  a.cols = cols;
  a.out = y;
  return of(launch_combine(a, stream));
}

ufp4_status ufp4_moe_combine_bwd(const void *dy, int64_t ld_dy, const void *ys,
                                 const int32_t *slots, const float *gates, int32_t dtype,
                                 int64_t tokens, int32_t k, int64_t cols, void *dys,
                                 float *d_gates, hipStream_t stream) {
  const ufp4_status s = check_exchange(dtype, tokens, k, cols);
  if (s != UFP4_OK) return s;
  if (bad_ld(ld_dy, tokens, cols)) return UFP4_ERR_SHAPE;
  if (tokens == 0) return UFP4_OK;
  const uintptr_t e = size_of(dtype);
  if (!good(dy, e) || !good(ys, e) || !good(slots, 4) || !good(gates, 4) || !good(dys, e) ||
      !good(d_gates, 4))
    return UFP4_ERR_INVALID_ARG;
  ExchangeArgs a{};
  a.in = ys;
  a.dy = dy;
  a.ld_dy = ld_dy;
  a.slots = slots;
  a.gates = gates;
  a.bf16 = dtype == UFP4_OUT_BF16;
  a.tokens = tokens;
  a.k = k;
  a.cols = cols;
  a.out = dys;
  a.d_gates = d_gates;
  return of(launch_combine_bwd(a, stream));
}

size_t ufp4_grad_norm_workspace_size(void) { return (size_t)kGradMaxBlocks * sizeof(double); }

static_assert(sizeof(ufp4_grad) == 32, "ufp4_grad layout");

ufp4_status ufp4_grad_norm(const ufp4_grad *grads, int64_t n_tensors, void *workspace,
                           size_t workspace_bytes, float *norm, hipStream_t stream) {
  const ufp4_status s = check_grads(grads, n_tensors, false);
  if (s != UFP4_OK) return s;
  if (!good(norm, 4) || !good(workspace, 16) || workspace_bytes < ufp4_grad_norm_workspace_size())
    return UFP4_ERR_INVALID_ARG;
  return of(launch_grad_norm(grads, n_tensors, static_cast<double *>(workspace), norm, stream));
}

ufp4_status ufp4_grad_clip(const ufp4_grad *grads, int64_t n_tensors, const float *norm,
                           double max_norm, double eps, hipStream_t stream) {
  const ufp4_status s = check_grads(grads, n_tensors, true);
  if (s != UFP4_OK) return s;
  if (!good(norm, 4) || !(max_norm >= 0.0) || !(eps >= 0.0)) return UFP4_ERR_INVALID_ARG;
  return of(launch_grad_clip(grads, n_tensors, norm, max_norm, eps, stream));
}

}  // extern "C"
