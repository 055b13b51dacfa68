// RMS norm with the residual's addition and an optional E4M3 output with one
// scale per row, and its backward pass (gfx950).
//   h = round(x + r),  rstd = 1 / sqrt(mean(h^2) + eps),  y = h rstd w
//   dx = rstd (g - xhat mean(g xhat)) + dh,  g = dy w,  xhat = h rstd
//   dw = sum over rows of dy xhat
#include "block_device.h"
#include "block_kernels.h"

namespace ufp4 {

constexpr float kE4M3Max = 448.0f;

// What the row's largest |y| gives: the stored scale and the factors that
// take y to q.  1 / scale overflows FP32 below 448 / 2^128, so rows below
// 2^-64 are lifted by 2^64 first (exact).
struct RowScale {
  float scale, lift, inv;
};
__device__ __forceinline__ RowScale row_scale(float top) {
  RowScale s;
  s.scale = top / kE4M3Max;
  s.lift = top < 0x1p-64f ? 0x1p64f : 1.0f;
  s.inv = top > 0.0f ? kE4M3Max / (top * s.lift) : top;   // 0 for a zero row, NaN for NaN
  return s;
}
// Four values to four E4M3 bytes, nearest even.  |y| <= top gives at most
// 448 (1 + 2^-22), which rounds to 448.
__device__ __forceinline__ uint32_t e4m3x4(const float *y, RowScale s) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[0] * s.lift * s.inv, y[1] * s.lift * s.inv, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[2] * s.lift * s.inv, y[3] * s.lift * s.inv, w,
                                                   true);
}

// One workgroup per row at a time, three passes over it; a thread reads back
// only what it wrote itself.
template <typename T, typename W>
__global__ __launch_bounds__(256) void rmsnorm_row_kernel(const NormArgs a) {
  constexpr int V = Elem<T>::V;
  __shared__ float s_sum[4], s_max[4], s_bad[4];
  const W *w = static_cast<const W *>(a.w);
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T *x = static_cast<const T *>(a.x) + row * a.ld_x;
    const T *res = a.res ? static_cast<const T *>(a.res) + row * a.ld_res : nullptr;
    T *h = static_cast<T *>(a.h) + row * a.cols;
    float sum = 0.0f;
    for (int64_t c = threadIdx.x * V; c < a.cols; c += 256 * V) {
      float f[V];
      Elem<T>::unpack(load_vec(x + c, a.cols - c), f);
      if (res != nullptr) {
        float r[V];
        Elem<T>::unpack(load_vec(res + c, a.cols - c), r);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] += r[i];
        const u32x4 packed = Elem<T>::pack(f);
        store_vec(h + c, a.cols - c, packed);
        Elem<T>::unpack(packed, f);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) sum = __builtin_fmaf(f[i], f[i], sum);
    }
    sum = group_sum<4>(sum, s_sum);
    const float rstd = 1.0f / sqrtf(sum / (float)a.cols + a.eps);
    if (threadIdx.x == 0) a.rstd[row] = rstd;
    const T *src = res != nullptr ? h : x;
    float top = 0.0f, bad = 0.0f;
    for (int64_t c = threadIdx.x * V; c < a.cols; c += 256 * V) {
      float f[V];
      Elem<T>::unpack(load_vec(src + c, a.cols - c), f);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        f[i] = f[i] * rstd * (c + i < a.cols ? Elem<W>::get(w[c + i]) : 0.0f);
        top = fmaxf(top, fabsf(f[i]));
        bad += f[i] * 0.0f;                      // NaN once any y is not finite
      }
      if (a.y != nullptr)
        store_vec(static_cast<T *>(a.y) + row * a.cols + c, a.cols - c, Elem<T>::pack(f));
    }
    if (a.q != nullptr) {
      top = group_max<4>(top, s_max);
      top += group_sum<4>(bad, s_bad);
      const RowScale s = row_scale(top);
      if (threadIdx.x == 0) a.scale[row] = s.scale;
      uint8_t *q = a.q + row * a.cols;
      for (int64_t c = threadIdx.x * V; c < a.cols; c += 256 * V) {
        float f[V];
        Elem<T>::unpack(load_vec(src + c, a.cols - c), f);
#pragma unroll
        for (int i = 0; i < V; ++i)
          f[i] = f[i] * rstd * (c + i < a.cols ? Elem<W>::get(w[c + i]) : 0.0f);
#pragma unroll
        for (int i = 0; i < V; i += 4) {
          const uint32_t b = e4m3x4(f + i, s);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (c + i + j < a.cols) q[c + i + j] = (uint8_t)(b >> (8 * j));
        }
      }
    }
    __syncthreads();                             // the next row reuses the LDS words
  }
}

// dx: one workgroup per row at a time, two passes.
template <typename T, typename W>
__global__ __launch_bounds__(256) void rmsnorm_bwd_row_kernel(const NormBwdArgs a) {
  constexpr int V = Elem<T>::V;
  __shared__ float s_sum[4];
  const W *w = static_cast<const W *>(a.w);
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T *dy = static_cast<const T *>(a.dy) + row * a.ld_dy;
    const T *h = static_cast<const T *>(a.h) + row * a.ld_h;
    const T *dh = a.dh ? static_cast<const T *>(a.dh) + row * a.ld_dh : nullptr;
    const float rstd = a.rstd[row];
    float sum = 0.0f;
    for (int64_t c = threadIdx.x * V; c < a.cols; c += 256 * V) {
      float f[V], g[V];
      Elem<T>::unpack(load_vec(h + c, a.cols - c), f);
      Elem<T>::unpack(load_vec(dy + c, a.cols - c), g);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float wv = c + i < a.cols ? Elem<W>::get(w[c + i]) : 0.0f;
        sum = __builtin_fmaf(g[i] * wv, f[i] * rstd, sum);
      }
    }
    const float mean = group_sum<4>(sum, s_sum) / (float)a.cols;
    for (int64_t c = threadIdx.x * V; c < a.cols; c += 256 * V) {
      float f[V], g[V], d[V];
      Elem<T>::unpack(load_vec(h + c, a.cols - c), f);
      Elem<T>::unpack(load_vec(dy + c, a.cols - c), g);
      if (dh != nullptr) Elem<T>::unpack(load_vec(dh + c, a.cols - c), d);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float wv = c + i < a.cols ? Elem<W>::get(w[c + i]) : 0.0f;
        g[i] = rstd * (g[i] * wv - f[i] * rstd * mean);
        if (dh != nullptr) g[i] += d[i];
      }
      store_vec(static_cast<T *>(a.dx) + row * a.cols + c, a.cols - c, Elem<T>::pack(g));
    }
    __syncthreads();                             // the next row reuses the LDS words
  }
}

// dw, first half: workgroup (chunk of 256 columns, slice of rows) sums its
// rows in order.  Runs before the dx kernel, which may write over dy.
template <typename T>
__global__ __launch_bounds__(256) void rmsnorm_dw_kernel(const NormBwdArgs a, int64_t per_slice) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= a.cols) return;
  const int64_t r0 = (int64_t)blockIdx.y * per_slice;
  const int64_t r1 = min(r0 + per_slice, a.rows);
  const T *dy = static_cast<const T *>(a.dy) + c;
  const T *h = static_cast<const T *>(a.h) + c;
  float sum = 0.0f;
  for (int64_t r = r0; r < r1; ++r)
    sum = __builtin_fmaf(Elem<T>::get(dy[r * a.ld_dy]), Elem<T>::get(h[r * a.ld_h]) * a.rstd[r],
                         sum);
  a.partial[(int64_t)blockIdx.y * a.cols + c] = sum;
}

// dw, second half: the slices' sums in slice order.
template <typename W>
__global__ __launch_bounds__(256) void rmsnorm_dw_final_kernel(const NormBwdArgs a, int slices) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= a.cols) return;
  float sum = 0.0f;
  for (int s = 0; s < slices; ++s) sum += a.partial[(int64_t)s * a.cols + c];
  static_cast<W *>(a.dw)[c] = Elem<W>::put(sum);
}

// A launch holds fewer than 2^32 threads; rows beyond the grid are looped over.
static unsigned row_grid(int64_t rows) { return (unsigned)(rows < (1 << 20) ? rows : (1 << 20)); }

template <typename T, typename W>
static hipError_t norm_fwd(const NormArgs &a, hipStream_t st) {
  if (a.rows == 0) return hipSuccess;
  hipLaunchKernelGGL((rmsnorm_row_kernel<T, W>), dim3(row_grid(a.rows)), dim3(256), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_rmsnorm(const NormArgs &a, hipStream_t st) {
  if (!a.bf16) return norm_fwd<float, float>(a, st);
  return a.w_bf16 ? norm_fwd<uint16_t, uint16_t>(a, st) : norm_fwd<uint16_t, float>(a, st);
}

int norm_bwd_slices(int64_t rows, int64_t cols) {
  (void)cols;
  const int64_t s = (rows + 63) / 64;
  return s < 1 ? 1 : (s > 256 ? 256 : (int)s);
}

template <typename T, typename W>
static hipError_t norm_bwd(const NormBwdArgs &a, hipStream_t st) {
  const int slices = norm_bwd_slices(a.rows, a.cols);
  const int64_t per = (a.rows + slices - 1) / slices;
  const unsigned chunks = (unsigned)((a.cols + 255) / 256);
  hipLaunchKernelGGL((rmsnorm_dw_kernel<T>), dim3(chunks, slices), dim3(256), 0, st, a, per);
  hipLaunchKernelGGL((rmsnorm_dw_final_kernel<W>), dim3(chunks), dim3(256), 0, st, a, slices);
  if (a.rows > 0)
    hipLaunchKernelGGL((rmsnorm_bwd_row_kernel<T, W>), dim3(row_grid(a.rows)), dim3(256), 0,
                       st, a);
  return hipGetLastError();
}

hipError_t launch_rmsnorm_bwd(const NormBwdArgs &a, hipStream_t st) {
  if (!a.bf16) return norm_bwd<float, float>(a, st);
  return a.w_bf16 ? norm_bwd<uint16_t, uint16_t>(a, st) : norm_bwd<uint16_t, float>(a, st);
}

}  // namespace ufp4
