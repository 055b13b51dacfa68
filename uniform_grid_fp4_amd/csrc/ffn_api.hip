// C ABI of the feed-forward operators (include/ufp4_ffn.h) other than the gated
// product, which stands with the GEMMs it is one of: host-side validation, then
// the launches on the caller's stream.  No allocation of device memory, no
// synchronisation, no state.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ffn_kernels.h"

using namespace ufp4;

namespace {

bool aligned_to(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool known_type(int32_t t) { return t == UFP4_OUT_F32 || t == UFP4_OUT_BF16; }
uintptr_t size_of(int32_t t) { return t == UFP4_OUT_BF16 ? 2 : 4; }
// Not null, and aligned to its element.
bool good(const void *p, uintptr_t size) { return p != nullptr && aligned_to(p, size); }

ufp4_status of(hipError_t e) { return e == hipSuccess ? UFP4_OK : UFP4_ERR_HIP; }

// Sizes that keep every element index and byte offset of a tensor in 63 bits.
constexpr int64_t kMaxRows = int64_t(1) << 40;
constexpr int64_t kMaxCols = int64_t(1) << 24;
constexpr int64_t kMaxLd = int64_t(1) << 40;
constexpr int64_t kMaxElems = int64_t(1) << 44;
constexpr int64_t kMaxSpan = int64_t(1) << 60;     // elements from the first row to the last

bool bad_shape(int64_t rows, int64_t cols) {
  return rows < 0 || cols <= 0 || rows > kMaxRows || cols > kMaxCols || rows > kMaxElems / cols;
}
bool bad_ld(int64_t ld, int64_t rows, int64_t cols) {
  return ld < cols || ld > kMaxLd || (rows > 1 && ld > kMaxSpan / rows);
}
bool bad_act(int32_t act, bool plain) {
  return act != UFP4_ACT_SILU && act != UFP4_ACT_GELU && !(plain && act == UFP4_ACT_NONE);
}

// The right operand, the groups and the output of an int8 product of `rows` rows
// of length k; fills what the kernel takes of them.
ufp4_status int8_product(int64_t rows, int64_t k, const ufp4_int8_rows *w, const float *bias,
                         int32_t act, int32_t n_groups, const int64_t *d_group_offsets,
                         int32_t out_dtype, void *y, int64_t ld_y, Int8GemmArgs &g) {
  if (w == nullptr || bad_act(act, true) || !known_type(out_dtype)) return UFP4_ERR_INVALID_ARG;
  if (!good(w->q, 16) || !good(w->scale, 4) || !aligned_to(bias, 4) ||
      !aligned_to(d_group_offsets, 8))
    return UFP4_ERR_INVALID_ARG;
  if (n_groups < 1 || n_groups > kMaxFfnGroups || (d_group_offsets == nullptr && n_groups != 1))
    return UFP4_ERR_SHAPE;
  if (k < 1 || w->k != k || bad_shape(rows, k) || w->rows < 1 ||
      w->rows % (n_groups * (act == UFP4_ACT_NONE ? 1 : 2)) != 0 ||
      w->rows / n_groups > kMaxCols)
    return UFP4_ERR_SHAPE;
  if (k > kInt8MaxK) return UFP4_ERR_UNSUPPORTED;
  g = Int8GemmArgs{};
  g.w = w->q;
  g.sw = w->scale;
  g.bias = bias;
  g.M = rows;
  g.N = w->rows / n_groups;
  g.kpad = int8_kpad(k);
  g.act = act;
  g.n_groups = n_groups;
  g.goff = d_group_offsets;
  g.out_bf16 = out_dtype == UFP4_OUT_BF16;
  g.y = y;
  g.ld_y = ld_y;
  const int64_t out_n = act == UFP4_ACT_NONE ? g.N : g.N / 2;
  if (bad_ld(ld_y, rows, out_n) || bad_shape(rows, out_n)) return UFP4_ERR_SHAPE;
  if (rows > 0 && !good(y, size_of(out_dtype))) return UFP4_ERR_INVALID_ARG;
  return UFP4_OK;
}

ufp4_status check_quantize(const void *x, int64_t ld_x, int32_t dtype, int64_t rows,
                           int64_t cols) {
  if (!known_type(dtype)) return UFP4_ERR_INVALID_ARG;
  if (bad_shape(rows, cols) || bad_ld(ld_x, rows, cols)) return UFP4_ERR_SHAPE;
  if (rows > 0 && !good(x, size_of(dtype))) return UFP4_ERR_INVALID_ARG;
  return UFP4_OK;
}

Int8QuantArgs quantize_args(const void *x, int64_t ld_x, int32_t dtype, int64_t rows,
                            int64_t cols, int8_t *q, float *scale) {
  Int8QuantArgs a{};
  a.x = x;
  a.ld_x = ld_x;
  a.bf16 = dtype == UFP4_OUT_BF16;
  a.rows = rows;
  a.cols = cols;
  a.kpad = int8_kpad(cols);
  a.q = q;
  a.scale = scale;
  return a;
}

}  // namespace

extern "C" {

ufp4_status ufp4_layernorm(const void *x, int64_t ld_x, const void *residual, int64_t ld_residual,
                           const void *weight, const void *bias, int32_t dtype,
                           int32_t weight_dtype, int64_t rows, int64_t cols, float eps, void *h,
                           void *y, float *mean, float *rstd, hipStream_t stream) {
  if (!known_type(dtype) || (weight_dtype != dtype && weight_dtype != UFP4_OUT_F32) ||
      !(eps >= 0.0f))
    return UFP4_ERR_INVALID_ARG;
  if (bad_shape(rows, cols) || bad_ld(ld_x, rows, cols) ||
      (residual != nullptr && bad_ld(ld_residual, rows, cols)))
    return UFP4_ERR_SHAPE;
  const uintptr_t e = size_of(dtype), we = size_of(weight_dtype);
  if (!good(weight, we) || !aligned_to(bias, we)) return UFP4_ERR_INVALID_ARG;
  if (rows == 0) return UFP4_OK;
  if (!good(x, e) || !good(y, e) || !good(mean, 4) || !good(rstd, 4) ||
      !aligned_to(residual, e) || (residual != nullptr && !good(h, e)))
    return UFP4_ERR_INVALID_ARG;
  LayerNormArgs a{};
  a.x = x;
  a.ld_x = ld_x;
  a.res = residual;
  a.ld_res = ld_residual;
  a.w = weight;
  a.b = bias;
  a.bf16 = dtype == UFP4_OUT_BF16;
  a.w_bf16 = weight_dtype == UFP4_OUT_BF16;
  a.rows = rows;
  a.cols = cols;
  a.eps = eps;
  a.h = h;
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  return of(launch_layernorm(a, stream));
}

size_t ufp4_layernorm_bwd_workspace_size(int64_t rows, int64_t cols) {
  if (bad_shape(rows, cols)) return 0;
  return (size_t)layernorm_bwd_slices(rows, cols) * 2 * (size_t)cols * sizeof(float);
}

ufp4_status ufp4_layernorm_bwd(const void *dy, int64_t ld_dy, const void *h, int64_t ld_h,
                               const void *weight, const float *mean, const float *rstd,
                               const void *dh, int64_t ld_dh, int32_t dtype, int32_t weight_dtype,
                               int64_t rows, int64_t cols, void *dx, void *dw, void *db,
                               void *workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!known_type(dtype) || (weight_dtype != dtype && weight_dtype != UFP4_OUT_F32))
    return UFP4_ERR_INVALID_ARG;
  if (bad_shape(rows, cols) || bad_ld(ld_dy, rows, cols) || bad_ld(ld_h, rows, cols) ||
      (dh != nullptr && bad_ld(ld_dh, rows, cols)))
    return UFP4_ERR_SHAPE;
  const uintptr_t e = size_of(dtype), we = size_of(weight_dtype);
  if (!good(weight, we) || !good(dw, we) || !aligned_to(db, we) || !aligned_to(dh, e))
    return UFP4_ERR_INVALID_ARG;
  if (!good(workspace, 16) || workspace_bytes < ufp4_layernorm_bwd_workspace_size(rows, cols))
    return UFP4_ERR_INVALID_ARG;
  if (rows > 0 &&
      (!good(dy, e) || !good(h, e) || !good(mean, 4) || !good(rstd, 4) || !good(dx, e)))
    return UFP4_ERR_INVALID_ARG;
  LayerNormBwdArgs a{};
  a.dy = dy;
  a.ld_dy = ld_dy;
  a.h = h;
  a.ld_h = ld_h;
  a.w = weight;
  a.mean = mean;
  a.rstd = rstd;
  a.dh = dh;
  a.ld_dh = ld_dh;
  a.bf16 = dtype == UFP4_OUT_BF16;
  a.w_bf16 = weight_dtype == UFP4_OUT_BF16;
  a.rows = rows;
  a.cols = cols;
  a.dx = dx;
  a.dw = dw;
  a.db = db;
  a.partial = static_cast<float *>(workspace);
  return of(launch_layernorm_bwd(a, stream));
}

ufp4_status ufp4_dropout(const void *x, int64_t ld_x, const void *residual, int64_t ld_residual,
                         int32_t dtype, int64_t rows, int64_t cols, double p, uint64_t seed,
                         uint64_t offset, const int64_t *d_offset, void *y, hipStream_t stream) {
  if (!known_type(dtype) || !(p >= 0.0 && p <= 1.0) || !aligned_to(d_offset, 8))
    return UFP4_ERR_INVALID_ARG;
  if (bad_shape(rows, cols) || bad_ld(ld_x, rows, cols) ||
      (residual != nullptr && bad_ld(ld_residual, rows, cols)))
    return UFP4_ERR_SHAPE;
  if (rows == 0) return UFP4_OK;
  const uintptr_t e = size_of(dtype);
  if (!good(x, e) || !good(y, e) || !aligned_to(residual, e)) return UFP4_ERR_INVALID_ARG;
  DropoutArgs a{};
  a.x = x;
  a.ld_x = ld_x;
  a.res = residual;
  a.ld_res = ld_residual;
  a.bf16 = dtype == UFP4_OUT_BF16;
  a.rows = rows;
  a.cols = cols;
  a.limit = (uint32_t)(p * 65536.0 + 0.5);
  a.scale = a.limit < 65536 ? (float)(65536.0 / (65536 - a.limit)) : 0.0f;
  a.seed = seed;
  a.offset = offset;
  a.d_offset = d_offset;
  a.y = y;
  return of(launch_dropout(a, stream));
}

ufp4_status ufp4_gated_bwd(const void *dy, int64_t ld_dy, const void *gu, int64_t ld_gu,
                           int32_t act, int32_t dtype, int64_t rows, int64_t cols, void *dgu,
                           hipStream_t stream) {
  if (!known_type(dtype) || bad_act(act, false)) return UFP4_ERR_INVALID_ARG;
  if (cols > kMaxCols / 2 || bad_shape(rows, 2 * cols) || bad_ld(ld_dy, rows, cols) ||
      bad_ld(ld_gu, rows, 2 * cols))
    return UFP4_ERR_SHAPE;
  if (rows == 0) return UFP4_OK;
  const uintptr_t e = size_of(dtype);
  if (!good(dy, e) || !good(gu, e) || !good(dgu, e)) return UFP4_ERR_INVALID_ARG;
  GatedBwdArgs a{};
  a.dy = dy;
  a.ld_dy = ld_dy;
  a.gu = gu;
  a.ld_gu = ld_gu;
  a.act = act;
  a.bf16 = dtype == UFP4_OUT_BF16;
  a.rows = rows;
  a.cols = cols;
  a.dgu = dgu;
  return of(launch_gated_bwd(a, stream));
}

ufp4_status ufp4_int8_quantize(const void *x, int64_t ld_x, int32_t dtype, int64_t rows,
                               int64_t cols, int8_t *q, float *scale, hipStream_t stream) {
  const ufp4_status s = check_quantize(x, ld_x, dtype, rows, cols);
  if (s != UFP4_OK) return s;
  if (rows == 0) return UFP4_OK;
  if (!good(q, 16) || !good(scale, 4)) return UFP4_ERR_INVALID_ARG;
  return of(launch_int8_quantize(quantize_args(x, ld_x, dtype, rows, cols, q, scale), stream));
}

ufp4_status ufp4_int8_gemm(const ufp4_int8_rows *a, const ufp4_int8_rows *w, const float *bias,
                           int32_t act, int32_t n_groups, const int64_t *d_group_offsets,
                           int32_t out_dtype, void *y, int64_t ld_y, hipStream_t stream) {
  if (a == nullptr) return UFP4_ERR_INVALID_ARG;
  Int8GemmArgs g;
  const ufp4_status s = int8_product(a->rows, a->k, w, bias, act, n_groups, d_group_offsets,
                                     out_dtype, y, ld_y, g);
  if (s != UFP4_OK) return s;
  if (a->rows == 0) return UFP4_OK;
  if (!good(a->q, 16) || !good(a->scale, 4)) return UFP4_ERR_INVALID_ARG;
  g.a = a->q;
  g.sa = a->scale;
  return of(launch_int8_gemm(g, stream));
}

// The codes, then the scales.
size_t ufp4_int8_linear_workspace_size(int64_t rows, int64_t cols, int32_t grouped) {
  if (bad_shape(rows, cols) || (grouped == 0 && int8_fuses(rows, int8_kpad(cols)))) return 0;
  return (size_t)rows * ((size_t)int8_kpad(cols) + sizeof(float));
}

ufp4_status ufp4_int8_linear(const void *x, int64_t ld_x, int32_t dtype, int64_t rows,
                             int64_t cols, const ufp4_int8_rows *w, const float *bias, int32_t act,
                             int32_t n_groups, const int64_t *d_group_offsets, int32_t out_dtype,
                             void *y, int64_t ld_y, void *workspace, size_t workspace_bytes,
                             hipStream_t stream) {
  ufp4_status s = check_quantize(x, ld_x, dtype, rows, cols);
  if (s != UFP4_OK) return s;
  Int8GemmArgs g;
  s = int8_product(rows, cols, w, bias, act, n_groups, d_group_offsets, out_dtype, y, ld_y, g);
  if (s != UFP4_OK) return s;
  if (rows == 0) return UFP4_OK;
  const size_t need =
      ufp4_int8_linear_workspace_size(rows, cols, d_group_offsets != nullptr ? 1 : 0);
  if (need > 0 && (!good(workspace, 16) || workspace_bytes < need)) return UFP4_ERR_INVALID_ARG;
  const int64_t out_n = act == UFP4_ACT_NONE ? g.N : g.N / 2;
  const bool splits = int8_splits(rows, g.kpad, out_n) && good(workspace, 16) &&
                      workspace_bytes >= ufp4_int8_linear_workspace_size(rows, cols, 1);
  int8_t *q = nullptr;
  float *scale = nullptr;
  if (need > 0 || splits) {
    q = static_cast<int8_t *>(workspace);
    scale = reinterpret_cast<float *>(q + rows * g.kpad);
  }
  g.a = q;
  g.sa = scale;
  return of(launch_int8_linear(g, quantize_args(x, ld_x, dtype, rows, cols, q, scale), stream));
}

}  // extern "C"
