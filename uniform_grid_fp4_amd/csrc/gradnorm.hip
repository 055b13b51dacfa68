// Global gradient norm over many tensors, and clipping by it (gfx950).
//   norm = sqrt(sum g^2),  out = g min(1, max_norm / (norm + eps))
// The list of tensors travels in the kernel arguments, kGradPerLaunch at a
// time, so a call needs no table in device memory and can be captured.  A
// tensor is cut into pieces of kPiece elements; workgroup b takes pieces b,
// b + grid, ...  Squares and sums are FP64: an FP32 square overflows at
// 1.8e19 and a sum over 10^9 elements needs more than 24 bits.  The FP64
// multiply-adds run at half the memory's pace or better, so both passes are
// bound by memory: 201M bf16 elements (403 MB) are summed in 70-73 us (5.6 TB/s)
// and scaled into another buffer in 133 us (805 MB, 6.1 TB/s, part of the input
// still cached).  Hundreds of small tensors are bound by the host, which lists
// them: 432 tensors take 9 launches and 50 us of GPU time in a call of 250 us.
#include "block_device.h"
#include "block_kernels.h"

namespace ufp4 {

constexpr int kGradPerLaunch = 128;
constexpr int kPiece = 16384;                    // elements

struct GradTable {
  const void *data[kGradPerLaunch];
  void *out[kGradPerLaunch];
  int64_t n[kGradPerLaunch];
  int32_t first[kGradPerLaunch + 1];             // number of pieces before each tensor
  uint8_t bf16[kGradPerLaunch];                  // bit 0: data, bit 1: out
  int32_t items;
};
static_assert(sizeof(GradTable) <= 3800, "kernel arguments");

// The tensor that holds piece p: the last one with first <= p.
__device__ __forceinline__ int item_of(const GradTable &g, int32_t p) {
  int lo = 0, hi = g.items;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (g.first[mid] <= p) lo = mid; else hi = mid;
  }
  return lo;
}

// Eight elements of a tensor as FP32.
template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += Elem<T>::V) {
    float v[Elem<T>::V];
    Elem<T>::unpack(*reinterpret_cast<const u32x4_any *>(p + i), v);
#pragma unroll
    for (int j = 0; j < Elem<T>::V; ++j) f[i + j] = v[j];
  }
}
template <typename O>
__device__ __forceinline__ void store8(O *p, const float (&f)[8], bool stream) {
#pragma unroll
  for (int i = 0; i < 8; i += Elem<O>::V) {
    float v[Elem<O>::V];
#pragma unroll
    for (int j = 0; j < Elem<O>::V; ++j) v[j] = f[i + j];
    store_as(p + i, Elem<O>::V, Elem<O>::pack(v), stream);
  }
}

// A piece: runs of 8 elements per thread, kRuns of them in flight, then what
// is left by single elements.
constexpr int kRuns = 4;
template <typename T>
__device__ __forceinline__ double piece_squares(const T *p, int n) {
  double sum = 0.0;
  int c = threadIdx.x * 8;
  for (; c + (kRuns - 1) * 2048 + 8 <= n; c += kRuns * 2048) {
    float f[kRuns][8];
#pragma unroll
    for (int r = 0; r < kRuns; ++r) load8(p + c + r * 2048, f[r]);
#pragma unroll
    for (int r = 0; r < kRuns; ++r)
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = __builtin_fma((double)f[r][i], (double)f[r][i], sum);
  }
  for (; c < n; c += 2048) {
    if (c + 8 <= n) {
      float f[8];
      load8(p + c, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = __builtin_fma((double)f[i], (double)f[i], sum);
    } else {
      for (int i = c; i < n; ++i) {
        const double f = (double)Elem<T>::get(p[i]);
        sum = __builtin_fma(f, f, sum);
      }
    }
  }
  return sum;
}

__global__ __launch_bounds__(256) void grad_squares_kernel(const GradTable g, double *partials) {
  __shared__ double s_sum[4];
  double sum = 0.0;
  const int32_t pieces = g.first[g.items];
  for (int32_t p = blockIdx.x; p < pieces; p += gridDim.x) {
    const int i = item_of(g, p);
    const int64_t at = (int64_t)(p - g.first[i]) * kPiece;
    const int n = (int)min(g.n[i] - at, (int64_t)kPiece);
    sum += (g.bf16[i] & 1) ? piece_squares(static_cast<const uint16_t *>(g.data[i]) + at, n)
                           : piece_squares(static_cast<const float *>(g.data[i]) + at, n);
  }
  sum = lanes_sum(sum);
  if ((threadIdx.x & 63) == 0) s_sum[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) partials[blockIdx.x] = ((s_sum[0] + s_sum[1]) + s_sum[2]) + s_sum[3];
}

// The partial sums in a fixed order: to the root of their sum (norm given), or
// folded into partials[0].
__global__ __launch_bounds__(256) void grad_norm_kernel(double *partials, int n, float *norm) {
  __shared__ double s_sum[4];
  double sum = 0.0;
  for (int i = threadIdx.x; i < n; i += 256) sum += partials[i];
  sum = lanes_sum(sum);
  if ((threadIdx.x & 63) == 0) s_sum[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    sum = ((s_sum[0] + s_sum[1]) + s_sum[2]) + s_sum[3];
    if (norm != nullptr) *norm = (float)sqrt(sum); else partials[0] = sum;
  }
}

template <typename T, typename O>
__device__ __forceinline__ void piece_scale(const T *p, O *out, int n, float coef, bool stream) {
  int c = threadIdx.x * 8;
  for (; c + (kRuns - 1) * 2048 + 8 <= n; c += kRuns * 2048) {
    float f[kRuns][8];
#pragma unroll
    for (int r = 0; r < kRuns; ++r) load8(p + c + r * 2048, f[r]);
#pragma unroll
    for (int r = 0; r < kRuns; ++r) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[r][i] *= coef;
      store8(out + c + r * 2048, f[r], stream);
    }
  }
  for (; c < n; c += 2048) {
    if (c + 8 <= n) {
      float f[8];
      load8(p + c, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] *= coef;
      store8(out + c, f, stream);
    } else {
      for (int i = c; i < n; ++i) out[i] = Elem<O>::put(Elem<T>::get(p[i]) * coef);
    }
  }
}

__global__ __launch_bounds__(256) void grad_scale_kernel(const GradTable g, const float *norm,
                                                         double max_norm, double eps, bool stream) {
  // a norm within the limit first: 0 / 0 and inf / inf are within it; a NaN stays
  const double size = (double)*norm + eps;
  const float coef = size <= max_norm ? 1.0f : (float)(max_norm / size);
  const int32_t pieces = g.first[g.items];
  // from the last piece to the first: what the norm read last is still cached
  for (int32_t p = pieces - 1 - (int32_t)blockIdx.x; p >= 0; p -= gridDim.x) {
    const int i = item_of(g, p);
    if (coef == 1.0f && g.data[i] == g.out[i]) continue;
    const int64_t at = (int64_t)(p - g.first[i]) * kPiece;
    const int n = (int)min(g.n[i] - at, (int64_t)kPiece);
    const uint16_t *hs = static_cast<const uint16_t *>(g.data[i]) + at;
    const float *fs = static_cast<const float *>(g.data[i]) + at;
    uint16_t *hd = static_cast<uint16_t *>(g.out[i]) + at;
    float *fd = static_cast<float *>(g.out[i]) + at;
    switch (g.bf16[i]) {
      case 0: piece_scale(fs, fd, n, coef, stream); break;
      case 1: piece_scale(hs, fd, n, coef, stream); break;
      case 2: piece_scale(fs, hd, n, coef, stream); break;
      default: piece_scale(hs, hd, n, coef, stream); break;
    }
  }
}

// Pieces of one launch: the largest tensor accepted has 2^30, and a piece index
// plus the grid stays within 32 bits.
constexpr int64_t kMaxPieces = int64_t(1) << 30;

// Calls launch(table, pieces) for each table that the list fills.
template <typename F>
static hipError_t each_table(const ufp4_grad *items, int64_t n_items, F launch) {
  GradTable g{};
  int64_t pieces = 0;
  for (int64_t i = 0; i <= n_items; ++i) {
    const int64_t mine = i < n_items ? (items[i].n + kPiece - 1) / kPiece : 0;
    if (g.items > 0 &&
        (i == n_items || g.items == kGradPerLaunch || pieces + mine > kMaxPieces)) {
      g.first[g.items] = (int32_t)pieces;
      const hipError_t e = launch(g, (int32_t)pieces);
      if (e != hipSuccess) return e;
      g.items = 0;
      pieces = 0;
    }
    if (mine == 0) continue;
    g.data[g.items] = items[i].data;
    g.out[g.items] = items[i].out;
    g.n[g.items] = items[i].n;
    g.first[g.items] = (int32_t)pieces;
    g.bf16[g.items] = (uint8_t)((items[i].dtype == UFP4_OUT_BF16) | (items[i].out_dtype == UFP4_OUT_BF16) << 1);
    ++g.items;
    pieces += mine;
  }
  return hipSuccess;
}

constexpr int kGradGrid = 2048;

hipError_t launch_grad_norm(const ufp4_grad *items, int64_t n_items, double *partials, float *norm,
                            hipStream_t st) {
  int used = 0;
  const hipError_t e = each_table(items, n_items, [&](const GradTable &g, int32_t pieces) {
    const int grid = pieces < kGradGrid ? pieces : kGradGrid;
    if (used + grid > kGradMaxBlocks) {          // fold what is there into one partial sum
      hipLaunchKernelGGL(grad_norm_kernel, dim3(1), dim3(256), 0, st, partials, used,
                         static_cast<float *>(nullptr));
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      used = 1;
    }
    hipLaunchKernelGGL(grad_squares_kernel, dim3(grid), dim3(256), 0, st, g, partials + used);
    used += grid;
    return hipGetLastError();
  });
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(grad_norm_kernel, dim3(1), dim3(256), 0, st, partials, used, norm);
  return hipGetLastError();
}

hipError_t launch_grad_clip(const ufp4_grad *items, int64_t n_items, const float *norm,
                            double max_norm, double eps, hipStream_t st) {
  int64_t bytes = 0;
  for (int64_t i = 0; i < n_items; ++i)
    bytes += items[i].n * (items[i].out_dtype == UFP4_OUT_BF16 ? 2 : 4);
  const bool stream = bytes >= kStreamBytes;
  return each_table(items, n_items, [&](const GradTable &g, int32_t pieces) {
    const int grid = pieces < kGradGrid ? pieces : kGradGrid;
    hipLaunchKernelGGL(grad_scale_kernel, dim3(grid), dim3(256), 0, st, g, norm, max_norm, eps,
                       stream);
    return hipGetLastError();
  });
}

}  // namespace ufp4
