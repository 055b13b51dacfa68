// Rows in 8-bit integers with one scale each (gfx950):
//   scale = max|x| / 127,  q = round(x * (127 * (1 / max|x|))), nearest even
// One pass: the row stays in registers between its maximum and its codes.  About
// 5 operations per element against 3 bytes (bf16): bound by memory.  30000 x 4096 bf16
// 67 us (369 MB, 5.5 TB/s), FP32 111 us (5.5 TB/s), x 4099 bf16 73 us; 8192 x 2048 11 us.
#include "ffn_kernels.h"
#include "int8_device.h"
#include "row_device.h"

namespace ufp4 {

template <typename T, int TPR, int NV, bool TAIL>
__global__ __launch_bounds__(group_size(TPR)) void int8_quantize_kernel(const Int8QuantArgs a) {
  constexpr int V = Elem<T>::V, ROWS = group_size(TPR) / TPR, STEP = TPR * V;
  __shared__ uint32_t s_max[2][16];
  const int cols = (int)a.cols, kpad = (int)a.kpad;
  const int at = threadIdx.x % TPR, first = at * V;
  const int64_t step = (int64_t)gridDim.x * ROWS;
  int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
  for (int turn = 0; row < a.rows; row += step, turn ^= 1) {
    RowVecs<NV, T, TAIL> v;
    v.load(static_cast<const T *>(a.x) + row * a.ld_x, first, STEP, cols);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float f[V];
      Elem<T>::unpack(v.v[i], f);
#pragma unroll
      for (int j = 0; j < V; ++j) top = max(top, __float_as_uint(fabsf(f[j])));
    }
    const Int8Scale s = int8_scale(span_max<TPR>(top, s_max[turn]));
    if (at == 0) a.scale[row] = s.scale;
    int8_t *q = a.q + row * a.kpad;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c0 = first + i * STEP;
      float f[V];
      Elem<T>::unpack(v.v[i], f);
      uint32_t b[V / 4];
#pragma unroll
      for (int j = 0; j < V / 4; ++j) b[j] = int8x4(f + 4 * j, s);
      if (c0 < cols) __builtin_memcpy(q + vec_start<TAIL, V>(c0, cols), b, V);
    }
    for (int c = cols + at; c < kpad; c += TPR) q[c] = 0;
  }
}

// One workgroup per row at a time, two passes, for rows that the registers do
// not hold and rows of less than a vector.
template <typename T>
__global__ __launch_bounds__(256) void int8_quantize_row_kernel(const Int8QuantArgs a) {
  constexpr int V = Elem<T>::V;
  __shared__ uint32_t s_max[2][4];
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    const T *x = static_cast<const T *>(a.x) + row * a.ld_x;
    uint32_t top = 0;
    for (int64_t c = threadIdx.x * V; c < a.cols; c += 256 * V) {
      float f[V];
      Elem<T>::unpack(load_vec(x + c, a.cols - c), f);
#pragma unroll
      for (int j = 0; j < V; ++j) top = max(top, __float_as_uint(fabsf(f[j])));
    }
    const Int8Scale s = int8_scale(group_max<4>(top, s_max[turn]));
    if (threadIdx.x == 0) a.scale[row] = s.scale;
    int8_t *q = a.q + row * a.kpad;
    // kpad is a multiple of 128: the pad is written with the last vectors
    for (int64_t c = threadIdx.x * V; c < a.kpad; c += 256 * V) {
      float f[V];
#pragma unroll
      for (int j = 0; j < V; ++j) f[j] = 0.0f;
      if (c < a.cols) Elem<T>::unpack(load_vec(x + c, a.cols - c), f);
      uint32_t b[V / 4];
#pragma unroll
      for (int j = 0; j < V / 4; ++j) b[j] = int8x4(f + 4 * j, s);
      __builtin_memcpy(q + c, b, V);
    }
  }
}

template <typename T, bool TAIL>
static hipError_t quantize_rows(const Int8QuantArgs &a, RowShape s, hipStream_t st) {
  const dim3 grid(row_grid(row_groups(a.rows, s.tpr)));
#define UFP4_NORM(TPR, NV)                                                                    \
  if (s.tpr == TPR && s.nv == NV) {                                                           \
    hipLaunchKernelGGL((int8_quantize_kernel<T, TPR, NV, TAIL>), grid, dim3(group_size(TPR)), \
                       0, st, a);                                                             \
    return hipGetLastError();                                                                 \
  }
  UFP4_FWD_SHAPES(UFP4_NORM)
  if constexpr (sizeof(T) == 4) {
    UFP4_NORM(1024, 3)
  }
#undef UFP4_NORM
  return hipErrorInvalidValue;
}

template <typename T>
static hipError_t quantize(const Int8QuantArgs &a, hipStream_t st) {
  if (a.rows == 0) return hipSuccess;
  const RowShape s = row_shape(a.cols, Elem<T>::V);
  if (s.tpr != 0)
    return a.cols % Elem<T>::V ? quantize_rows<T, true>(a, s, st) : quantize_rows<T, false>(a, s, st);
  hipLaunchKernelGGL((int8_quantize_row_kernel<T>), dim3(row_grid(a.rows)), dim3(256), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_int8_quantize(const Int8QuantArgs &a, hipStream_t st) {
  return a.bf16 ? quantize<uint16_t>(a, st) : quantize<float>(a, st);
}

}  // namespace ufp4
