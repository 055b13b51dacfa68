// Host-side launch interface between the C ABI of the feed-forward operators
// (ffn_api.hip) and their kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/ufp4_ffn.h"

namespace ufp4 {

struct LayerNormArgs {
  const void *x;
  int64_t ld_x;
  const void *res;          // nullptr: none
  int64_t ld_res;
  const void *w, *b;        // b nullptr: none
  int bf16, w_bf16;         // element types of the rows and of the weight and bias
  int64_t rows, cols;
  float eps;
  void *h;                  // written when there is a residual
  void *y;
  float *mean, *rstd;
  bool stream;              // h and y by streaming stores
};
hipError_t launch_layernorm(const LayerNormArgs &a, hipStream_t st);

struct LayerNormBwdArgs {
  const void *dy;
  int64_t ld_dy;
  const void *h;
  int64_t ld_h;
  const void *w;
  const float *mean, *rstd;
  const void *dh;           // nullptr: none
  int64_t ld_dh;
  int bf16, w_bf16;
  int64_t rows, cols;
  void *dx;
  bool stream;              // dx by streaming stores
  void *dw, *db;            // db nullptr: not wanted
  float *partial;           // [layernorm_bwd_slices(rows, cols), 2, cols]: dw's and db's sums
};
int layernorm_bwd_slices(int64_t rows, int64_t cols);
hipError_t launch_layernorm_bwd(const LayerNormBwdArgs &a, hipStream_t st);

struct DropoutArgs {
  const void *x;
  int64_t ld_x;
  const void *res;          // nullptr: none
  int64_t ld_res;
  int bf16;
  int64_t rows, cols;
  uint32_t limit;           // an element stays if its 16 bits are at least this; 65536: none does
  float scale;
  uint64_t seed, offset;
  const int64_t *d_offset;  // nullptr: 0
  void *y;
  bool stream;              // y by streaming stores
};
hipError_t launch_dropout(const DropoutArgs &a, hipStream_t st);

struct GatedBwdArgs {
  const void *dy;
  int64_t ld_dy;
  const void *gu;
  int64_t ld_gu;
  int act, bf16;
  int64_t rows, cols;
  void *dgu;
  bool stream;
};
hipError_t launch_gated_bwd(const GatedBwdArgs &a, hipStream_t st);

struct Int8QuantArgs {
  const void *x;
  int64_t ld_x;
  int bf16;
  int64_t rows, cols, kpad;
  int8_t *q;
  float *scale;
};
hipError_t launch_int8_quantize(const Int8QuantArgs &a, hipStream_t st);

struct Int8GemmArgs {
  const int8_t *a, *w;
  const float *sa, *sw;
  const float *bias;        // nullptr: none
  int64_t M, N, kpad;       // N rows of w per group
  int act;                  // gated: the output has N / 2 columns
  int n_groups;
  const int64_t *goff;      // nullptr: one group of all rows
  int out_bf16;
  void *y;
  int64_t ld_y;
};
hipError_t launch_int8_gemm(const Int8GemmArgs &a, hipStream_t st);
// Whether that many rows of one group are quantized by the product's workgroups
// themselves.  It saves a launch, an allocation and, for one row, time on the GPU (us,
// gated, one launch and two: 1 x 2048 to 2 x 8192 10.1 and 10.2, 1 x 32768 to 2 x 1024 36.7 and
// 45.5); more rows take longer than in a kernel of their own, which pays while the
// launch costs more (16 x 1024 to 2 x 2048 6.8 and 5.7, 4 x 2048 to 2 x 8192 11.4 and 10.4, but 16 x
// 2048 to 2 x 8192 17.5 and 11.7, 8 x 4096 to 2 x 2048 12.6 and 9.5).
inline bool int8_fuses(int64_t rows, int64_t kpad) {
  return rows == 1 ? kpad <= 32768 : rows <= 16 && rows * kpad <= 16384;
}
// Whether a workspace that the caller brings all the same is used, for two launches:
// every 16 output columns quantize the rows once more, and beyond so many columns
// that costs more than the launch, but for the fewest elements (us on the GPU, one
// launch and two, to 16384, 32768 and 65536 columns of a plain product: 1 x 2048 10.1 and
// 10.5, 17.1 and 14.8, 30.2 and 25.4; 8 x 2048 15.3 and 11.5, 25.8 and 17.1, 46.6 and 30.2;
// 16 x 1024 13.5 and 8.9, 23.4 and 13.2, 40.9 and 21.7; 16 x 128 8.4 and 4.9, 13.8 and 6.1,
// 23.4 and 8.2.  One eager call after the other the host takes 10 and 13.4: 1 x 512 to
// 32768 10.1 and 13.4, 8 x 512 11.6 and 13.6, 16 x 1024 23.9 and 13.4).
inline bool int8_splits(int64_t rows, int64_t kpad, int64_t out_n) {
  return out_n > 16384 && rows * kpad >= 2048;
}
// Quantizes q.x into q.q and q.scale, which are a.a and a.sa, and multiplies; with
// q.q nullptr (rows that fuse, one group without offsets) in one launch.
hipError_t launch_int8_linear(const Int8GemmArgs &a, const Int8QuantArgs &q, hipStream_t st);

constexpr int kMaxFfnGroups = 1024;
constexpr int64_t kInt8MaxK = 131071;   // 128 * 128 * k stays below 2^31
constexpr int64_t kInt8KAlign = 128;
inline int64_t int8_kpad(int64_t k) { return (k + kInt8KAlign - 1) / kInt8KAlign * kInt8KAlign; }

}  // namespace ufp4
