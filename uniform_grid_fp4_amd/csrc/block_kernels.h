// Host-side launch interface between the C ABI of the block operators
// (block_api.hip) and their kernels.  Element type codes are ufp4_out_dtype.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/ufp4_block.h"

namespace ufp4 {

struct NormArgs {
  const void *x;
  int64_t ld_x;
  const void *res;          // nullptr: none
  int64_t ld_res;
  const void *w;
  int bf16, w_bf16;         // element types of the rows and of the weight
  int64_t rows, cols;
  float eps;
  void *h;                  // written when there is a residual
  void *y;                  // nullptr: not wanted
  uint8_t *q;               // nullptr: not wanted
  float *scale;
  float *rstd;
  bool stream;              // h and y by streaming stores
};
hipError_t launch_rmsnorm(const NormArgs &a, hipStream_t st);

struct NormBwdArgs {
  const void *dy;
  int64_t ld_dy;
  const void *h;
  int64_t ld_h;
  const void *w;
  const float *rstd;
  const void *dh;           // nullptr: none
  int64_t ld_dh;
  int bf16, w_bf16;
  int64_t rows, cols;
  void *dx;
  bool stream;              // dx by streaming stores
  void *dw;
  float *partial;           // [norm_bwd_slices(rows, cols), cols]
};
int norm_bwd_slices(int64_t rows, int64_t cols);
hipError_t launch_rmsnorm_bwd(const NormBwdArgs &a, hipStream_t st);

constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxK = 16;
constexpr int kRouteTokens = 64;      // tokens per workgroup of the router
struct RouteArgs {
  const void *logits;
  int64_t ld;
  int bf16;
  const uint8_t *valid;     // nullptr: all
  int64_t tokens;
  int n_experts, k, renorm;
  int32_t *experts;
  float *gates;
  int32_t *slots;
  float *lse;
  int64_t *counts, *offsets, *n_tokens;
  float *losses;
  void *workspace;
  // backward only
  const float *d_gates, *d_losses;   // nullptr: zero
  void *d_logits;
};
size_t route_workspace_bytes(int64_t tokens, int n_experts);
hipError_t launch_route(const RouteArgs &a, hipStream_t st);
hipError_t launch_route_bwd(const RouteArgs &a, hipStream_t st);

struct ExchangeArgs {
  const void *in;           // x, dxs, ys
  int64_t ld_in;            // of x (dispatch)
  const void *dy;           // combine_bwd
  int64_t ld_dy;
  const int32_t *slots;
  const float *gates;
  const void *res;          // combine: nullptr: none
  int64_t ld_res;
  int bf16;
  int64_t tokens, cols;
  int k;
  void *out;                // xs, dx, y, dys
  float *d_gates;
  bool stream;              // everything but x, dy and residual by streaming accesses
};
hipError_t launch_dispatch(const ExchangeArgs &a, hipStream_t st);
// The gate-weighted sum with a residual; gates nullptr: plain sum (dispatch's
// backward).
hipError_t launch_combine(const ExchangeArgs &a, hipStream_t st);
hipError_t launch_combine_bwd(const ExchangeArgs &a, hipStream_t st);

constexpr int kGradMaxBlocks = 4096;  // partial sums in the workspace
hipError_t launch_grad_norm(const ufp4_grad *items, int64_t n_items, double *partials, float *norm,
                            hipStream_t st);
hipError_t launch_grad_clip(const ufp4_grad *items, int64_t n_items, const float *norm,
                            double max_norm, double eps, hipStream_t st);

}  // namespace ufp4
