// Token exchange with expert order (gfx950): dispatch, combine and their
// backward passes.  A token's k choices hold the rows given by its slots
// (negative: ~row is a row without a choice).  All four move whole rows and
// compute next to nothing: they are bound by memory.
#include "block_device.h"
#include "block_kernels.h"

namespace ufp4 {

// The row of a slot, or -1 for one outside the array.
__device__ __forceinline__ int64_t slot_row(int32_t slot, int64_t rows) {
  const int32_t r = slot < 0 ? ~slot : slot;
  return r < rows ? r : -1;
}

// Thread = one vector of one token's row, written to its k rows.
template <typename T>
__global__ __launch_bounds__(256) void dispatch_kernel(const ExchangeArgs a, int64_t chunks) {
  constexpr int V = Elem<T>::V;
  const int64_t rows = a.tokens * a.k;
  for (int64_t b = blockIdx.x; b < a.tokens * chunks; b += gridDim.x) {
    const int64_t t = b / chunks;
    const int64_t c = ((b - t * chunks) * 256 + threadIdx.x) * V;
    if (c >= a.cols) continue;
    const u32x4 v = load_vec(static_cast<const T *>(a.in) + t * a.ld_in + c, a.cols - c);
    for (int j = 0; j < a.k; ++j) {
      const int32_t slot = a.slots[t * a.k + j];
      const int64_t r = slot_row(slot, rows);
      if (r >= 0)
        store_vec(static_cast<T *>(a.out) + r * a.cols + c, a.cols - c, slot < 0 ? u32x4(0) : v);
    }
  }
}

// Thread = one vector of one token's row: the (weighted) sum of its k rows.
template <typename T, bool GATED>
__global__ __launch_bounds__(256) void combine_kernel(const ExchangeArgs a, int64_t chunks) {
  constexpr int V = Elem<T>::V;
  const int64_t rows = a.tokens * a.k;
  for (int64_t b = blockIdx.x; b < a.tokens * chunks; b += gridDim.x) {
    const int64_t t = b / chunks;
    const int64_t c = ((b - t * chunks) * 256 + threadIdx.x) * V;
    if (c >= a.cols) continue;
    float sum[V];
#pragma unroll
    for (int i = 0; i < V; ++i) sum[i] = 0.0f;
    for (int j = 0; j < a.k; ++j) {
      const int32_t slot = a.slots[t * a.k + j];
      if (slot < 0 || slot >= rows) continue;
      const float g = GATED ? a.gates[t * a.k + j] : 1.0f;
      float f[V];
      Elem<T>::unpack(load_vec(static_cast<const T *>(a.in) + (int64_t)slot * a.cols + c,
                               a.cols - c), f);
#pragma unroll
      for (int i = 0; i < V; ++i) sum[i] = GATED ? __builtin_fmaf(g, f[i], sum[i]) : sum[i] + f[i];
    }
    if (GATED && a.res != nullptr) {
      float f[V];
      Elem<T>::unpack(load_vec(static_cast<const T *>(a.res) + t * a.ld_res + c, a.cols - c), f);
#pragma unroll
      for (int i = 0; i < V; ++i) sum[i] += f[i];
    }
    store_vec(static_cast<T *>(a.out) + t * a.cols + c, a.cols - c, Elem<T>::pack(sum));
  }
}

// One workgroup per token at a time: for each choice, dys = g dy and the dot
// product of ys and dy.
template <typename T>
__global__ __launch_bounds__(256) void combine_bwd_kernel(const ExchangeArgs a) {
  constexpr int V = Elem<T>::V;
  __shared__ float s_dot[4];
  const int64_t rows = a.tokens * a.k;
  for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
    const T *dy = static_cast<const T *>(a.dy) + t * a.ld_dy;
    for (int j = 0; j < a.k; ++j) {
      const int32_t slot = a.slots[t * a.k + j];
      const int64_t r = slot_row(slot, rows);
      const bool chosen = slot >= 0 && r >= 0;
      const float g = chosen ? a.gates[t * a.k + j] : 0.0f;
      float dot = 0.0f;
      for (int64_t c = threadIdx.x * V; c < a.cols; c += 256 * V) {
        float f[V], d[V];
        Elem<T>::unpack(load_vec(dy + c, a.cols - c), d);
        if (chosen) {
          Elem<T>::unpack(load_vec(static_cast<const T *>(a.in) + r * a.cols + c, a.cols - c), f);
#pragma unroll
          for (int i = 0; i < V; ++i) dot = __builtin_fmaf(f[i], d[i], dot);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] = chosen ? d[i] * g : 0.0f;
        if (r >= 0)
          store_vec(static_cast<T *>(a.out) + r * a.cols + c, a.cols - c, Elem<T>::pack(d));
      }
      dot = group_sum<4>(dot, s_dot);
      if (threadIdx.x == 0) a.d_gates[t * a.k + j] = dot;
      __syncthreads();
    }
  }
}

// A launch holds fewer than 2^32 threads; work beyond the grid is looped over.
static unsigned grid_of(int64_t blocks) {
  return (unsigned)(blocks < (1 << 23) ? blocks : (1 << 23));
}

template <typename T>
static hipError_t exchange(const ExchangeArgs &a, int what, hipStream_t st) {
  if (a.tokens == 0) return hipSuccess;
  const int64_t per = 256 * Elem<T>::V, chunks = (a.cols + per - 1) / per;
  const dim3 grid(grid_of(a.tokens * chunks)), block(256);
  if (what == 0)
    hipLaunchKernelGGL((dispatch_kernel<T>), grid, block, 0, st, a, chunks);
  else if (what == 1)
    hipLaunchKernelGGL((combine_kernel<T, false>), grid, block, 0, st, a, chunks);
  else if (what == 2)
    hipLaunchKernelGGL((combine_kernel<T, true>), grid, block, 0, st, a, chunks);
  else
    hipLaunchKernelGGL((combine_bwd_kernel<T>), dim3(grid_of(a.tokens)), block, 0, st, a);
  return hipGetLastError();
}

hipError_t launch_dispatch(const ExchangeArgs &a, hipStream_t st) {
  return a.bf16 ? exchange<uint16_t>(a, 0, st) : exchange<float>(a, 0, st);
}
hipError_t launch_combine(const ExchangeArgs &a, hipStream_t st) {
  const int what = a.gates != nullptr ? 2 : 1;
  return a.bf16 ? exchange<uint16_t>(a, what, st) : exchange<float>(a, what, st);
}
hipError_t launch_combine_bwd(const ExchangeArgs &a, hipStream_t st) {
  return a.bf16 ? exchange<uint16_t>(a, 3, st) : exchange<float>(a, 3, st);
}

}  // namespace ufp4
