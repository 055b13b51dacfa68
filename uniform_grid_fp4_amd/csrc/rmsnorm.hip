// RMS norm with the residual's addition and an optional E4M3 output with one
// scale per row, and its backward pass (gfx950).
//   h = round(x + r),  rstd = 1 / sqrt(mean(h^2) + eps),  y = h rstd w
//   dx = rstd (g - xhat mean(g xhat)) + dh,  g = dy w,  xhat = h rstd
//   dw = sum over rows of dy xhat
// About 12 operations per element forward and 16 backward against 6 to 10
// bytes: bound by memory.  Sums are FP32 along a row (a lane's chain is a 64th
// of it or less, and one vector in rows of up to 16 vectors) and over the rows
// of dw; h is rounded once to the stream's type, and the statistics are those of
// the rounded h that the backward sees; y, q and the gradients are rounded once
// from FP32.
#include "block_kernels.h"
#include "row_device.h"

namespace ufp4 {

constexpr float kE4M3Max = 448.0f;

// What the row's largest |y| gives: the stored scale and the factors that
// take y to q.  1 / scale overflows FP32 below 448 / 2^128, so rows below
// 2^-64 are lifted by 2^64 first (exact).  The maximum is taken over the bits
// of |y| as unsigned numbers, where infinities and NaN are the largest: either
// makes the whole row NaN.
struct RowScale {
  float scale, lift, inv;
};
__device__ __forceinline__ RowScale row_scale(uint32_t top_bits) {
  const float top = top_bits >= 0x7F800000u ? __uint_as_float(0x7FC00000u)
                                            : __uint_as_float(top_bits);
  RowScale s;
  s.scale = top / kE4M3Max;
  s.lift = top < 0x1p-64f ? 0x1p64f : 1.0f;
  s.inv = top > 0.0f ? kE4M3Max / (top * s.lift) : top;   // 0 for a zero row, NaN for NaN
  return s;
}
// Four values to four E4M3 bytes, nearest even.  |y| <= top gives at most
// 448 (1 + 2^-22), which rounds to 448.  y and its product with 448 / top are
// rounded to FP32 first, so a quotient that is half a step exactly, as one in some
// 2000 of bf16 rows is, may go to either neighbour.
__device__ __forceinline__ uint32_t e4m3x4(const float *y, RowScale s) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[0] * s.lift * s.inv, y[1] * s.lift * s.inv, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[2] * s.lift * s.inv, y[3] * s.lift * s.inv, w,
                                                   true);
}

// Rows held in registers: TPR threads (16 lanes, a wave, or a workgroup) hold a
// row as NV vectors each, so x and the residual are read once and everything
// else happens in registers.  TAIL: the row length is not a multiple of the
// vector.  A row per workgroup at a time, with the hardware starting the next
// workgroup as one ends: a grid that fills the GPU once and walks over rows with
// the next row's loads in flight took 350 us where this takes 317 us (32768 x
// 6144 bf16 with residual and E4M3), 302 us with streaming stores: 1.81 GB at
// 6.0 TB/s, the rate that the fastest of these kernels reach; a plain copy of 2 GB
// reaches 4.9 TB/s here.  8192 x 2048 takes 23-28 us (134 MB, 4.8-5.8 TB/s,
// partly from the 256 MB cache), 4096 x 12288 FP32 135 us (805 MB, 6.0 TB/s), one
// row 3.2 us.
template <typename T, typename W, int TPR, int NV, bool TAIL>
__global__ __launch_bounds__(group_size(TPR)) void rmsnorm_kernel(const NormArgs a) {
  constexpr int V = Elem<T>::V, ROWS = group_size(TPR) / TPR, STEP = TPR * V;
  __shared__ float s_sum[2][16];
  __shared__ uint32_t s_max[2][16];
  const int cols = (int)a.cols;
  const int first = (threadIdx.x % TPR) * V;
  WeightVec<T, W, TAIL> w[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) w[i].load(static_cast<const W *>(a.w), first + i * STEP, cols);
  const int64_t step = (int64_t)gridDim.x * ROWS;
  int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
  const T *x = static_cast<const T *>(a.x), *res = static_cast<const T *>(a.res);
  // 16 lanes or a wave leave the loop on their own; a workgroup has one row
  for (int turn = 0; row < a.rows; row += step, turn ^= 1) {
    RowVecs<NV, T, TAIL> h, r0;
    h.load(x + row * a.ld_x, first, STEP, cols);
    if (res != nullptr) r0.load(res + row * a.ld_res, first, STEP, cols);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float f[V];
      Elem<T>::unpack(h.v[i], f);
      if (res != nullptr) {
        float r[V];
        Elem<T>::unpack(r0.v[i], r);
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] += r[j];
        h.v[i] = Elem<T>::pack(f);
        Elem<T>::unpack(h.v[i], f);
      }
#pragma unroll
      for (int j = 0; j < V; ++j)
        sum = elsewhere<TAIL, V>(first + i * STEP, cols, j) ? sum
                                                            : __builtin_fmaf(f[j], f[j], sum);
    }
    sum = span_sum<TPR>(sum, s_sum[turn]);
    const float rstd = 1.0f / sqrtf(sum / (float)cols + a.eps);
    if (first == 0) a.rstd[row] = rstd;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float f[V], g[V];
      // only now, when every lane of the row has read its own: h may be x or the
      // residual, and two lanes may share elements
      if (res != nullptr)
        row_store<T, TAIL>(static_cast<T *>(a.h) + row * a.cols, first + i * STEP, cols, h.v[i],
                           a.stream);
      Elem<T>::unpack(h.v[i], f);
      w[i].get(g);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        f[j] = f[j] * rstd * g[j];
        top = max(top, __float_as_uint(fabsf(f[j])));
      }
      if (a.y != nullptr)
        row_store<T, TAIL>(static_cast<T *>(a.y) + row * a.cols, first + i * STEP, cols,
                           Elem<T>::pack(f), a.stream);
    }
    if (a.q == nullptr) continue;
    top = span_max<TPR>(top, s_max[turn]);
    const RowScale s = row_scale(top);
    if (first == 0) a.scale[row] = s.scale;
    uint8_t *q = a.q + row * a.cols;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float f[V], g[V];
      Elem<T>::unpack(h.v[i], f);
      w[i].get(g);
#pragma unroll
      for (int j = 0; j < V; ++j) f[j] = f[j] * rstd * g[j];
      const int c0 = first + i * STEP;
      uint32_t b[V / 4];
#pragma unroll
      for (int j = 0; j < V / 4; ++j) b[j] = e4m3x4(f + 4 * j, s);
      if (c0 < cols) __builtin_memcpy(q + vec_start<TAIL, V>(c0, cols), b, V);
    }
  }
}

// One workgroup per row at a time, three passes over it; a thread reads back
// only what it wrote itself.  4096 x 16384 FP32 with residual 254 us (1.07 GB,
// 4.2 TB/s; the second pass hits the caches), 4096 x 32768 bf16 342 us.
template <typename T, typename W>
__global__ __launch_bounds__(256) void rmsnorm_row_kernel(const NormArgs a) {
  constexpr int V = Elem<T>::V;
  __shared__ float s_sum[4];
  __shared__ uint32_t s_max[4];
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
    uint32_t top = 0;
    for (int64_t c = threadIdx.x * V; c < a.cols; c += 256 * V) {
      float f[V];
      Elem<T>::unpack(load_vec(src + c, a.cols - c), f);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        f[i] = f[i] * rstd * (c + i < a.cols ? Elem<W>::get(w[c + i]) : 0.0f);
        top = max(top, __float_as_uint(fabsf(f[i])));
      }
      if (a.y != nullptr)
        store_vec(static_cast<T *>(a.y) + row * a.cols + c, a.cols - c, Elem<T>::pack(f));
    }
    if (a.q != nullptr) {
      top = group_max<4>(top, s_max);
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

// Backward with rows held in registers as above: dx, and the workgroup's share
// of dw, which stays in registers over all its rows (in the order of the
// rows) and goes to partial[workgroup][cols] at the end, the four waves of a
// wave-per-row workgroup added in wave order.  Reads dy, h and dh once: 8192 x
// 2048 bf16 26 us and 4 us for dw's second half (134 MB, 4.5 TB/s); 16384 x
// 6144 163 and 6 us (805 MB, 4.8 TB/s), bound by memory.  Loading the next row ahead
// changed nothing (the other workgroup of the CU covers the wait).
template <typename T, typename W, int TPR, int NV, bool TAIL>
__global__ __launch_bounds__(group_size(TPR)) void rmsnorm_bwd_kernel(const NormBwdArgs a) {
  constexpr int V = Elem<T>::V, ROWS = group_size(TPR) / TPR, STEP = TPR * V;
  __shared__ float s_sum[2][16];
  const int cols = (int)a.cols;
  const int first = (threadIdx.x % TPR) * V;
  WeightVec<T, W, TAIL> w[NV];
  float acc[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    w[i].load(static_cast<const W *>(a.w), first + i * STEP, cols);
#pragma unroll
    for (int j = 0; j < V; ++j) acc[i][j] = 0.0f;
  }
  const int64_t step = (int64_t)gridDim.x * ROWS;
  int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
  const T *dy = static_cast<const T *>(a.dy), *h = static_cast<const T *>(a.h);
  const T *dh = static_cast<const T *>(a.dh);
  for (int turn = 0; row < a.rows; row += step, turn ^= 1) {
    RowVecs<NV, T, TAIL> vd, vy, vh;
    vy.load(dy + row * a.ld_dy, first, STEP, cols);
    vh.load(h + row * a.ld_h, first, STEP, cols);
    const float rstd = a.rstd[row];
    if (dh != nullptr) vd.load(dh + row * a.ld_dh, first, STEP, cols);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float f[V], g[V], wf[V];
      Elem<T>::unpack(vh.v[i], f);
      Elem<T>::unpack(vy.v[i], g);
      w[i].get(wf);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        f[j] *= rstd;
        if (elsewhere<TAIL, V>(first + i * STEP, cols, j)) g[j] = f[j] = 0.0f;
        acc[i][j] = __builtin_fmaf(g[j], f[j], acc[i][j]);
        sum = __builtin_fmaf(g[j] * wf[j], f[j], sum);
      }
    }
    // dx may be dy or dh: with shared elements every lane's dh has to be here
    // before another's dx is stored
    if (TAIL && dh != nullptr) {
#pragma unroll
      for (int i = 0; i < NV; ++i) asm volatile("" ::"v"(vd.v[i]));
    }
    const float mean = span_sum<TPR>(sum, s_sum[turn]) / (float)cols;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float f[V], g[V], wf[V];
      Elem<T>::unpack(vh.v[i], f);
      Elem<T>::unpack(vy.v[i], g);
      w[i].get(wf);
#pragma unroll
      for (int j = 0; j < V; ++j) f[j] = rstd * __builtin_fmaf(-f[j] * rstd, mean, g[j] * wf[j]);
      if (dh != nullptr) {
        Elem<T>::unpack(vd.v[i], g);
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] += g[j];
      }
      row_store<T, TAIL>(static_cast<T *>(a.dx) + row * a.cols, first + i * STEP, cols,
                         Elem<T>::pack(f), a.stream);
    }
  }
  float *partial = a.partial + (int64_t)blockIdx.x * a.cols;
  if (ROWS == 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c0 = first + i * STEP;
        if (c0 < cols && !elsewhere<TAIL, V>(c0, cols, j))
          partial[vec_start<TAIL, V>(c0, cols) + j] = acc[i][j];
      }
    return;
  }
  __shared__ float s_acc[ROWS][STEP + 1];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c0 = first + i * STEP;
      if (c0 < cols && !elsewhere<TAIL, V>(c0, cols, j))
        s_acc[threadIdx.x / TPR][vec_start<TAIL, V>(c0, cols) + j - i * STEP] = acc[i][j];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < STEP && i * STEP + c < cols; c += 256) {
      float t = s_acc[0][c];
#pragma unroll
      for (int r = 1; r < ROWS; ++r) t += s_acc[r][c];
      partial[i * STEP + c] = t;
    }
  }
}

// dx: one workgroup per row at a time, two passes.  With dw's own pass over dy
// and h before it, the backward of 4096 x 16384 FP32 takes 138 + 265 + 5 us (1.07
// GB, 2.6 TB/s), of 4096 x 32768 bf16 163 + 376 + 9 us.
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

// dw, second half: the slices' sums in a fixed order, 64 runs of slices side
// by side for 16 columns per workgroup.
template <typename W>
__global__ __launch_bounds__(1024) void rmsnorm_dw_final_kernel(const NormBwdArgs a, int slices) {
  __shared__ float s_sum[64][17];
  const int col = threadIdx.x & 15, run = threadIdx.x >> 4;
  const int64_t c = (int64_t)blockIdx.x * 16 + col;
  float sum = 0.0f;
  if (c < a.cols) {
#pragma unroll 4
    for (int s = run; s < slices; s += 64) sum += a.partial[(int64_t)s * a.cols + c];
  }
  s_sum[run][col] = sum;
  __syncthreads();
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    if (run < o) s_sum[run][col] += s_sum[run + o][col];
    __syncthreads();
  }
  if (run == 0 && c < a.cols) static_cast<W *>(a.dw)[c] = Elem<W>::put(s_sum[0][col]);
}

// The backward pass also keeps dw's sums, and a wave with four vectors per lane
// has few registers left for its loads: 193 to 256 vectors take a workgroup
// with one each (8192 x 2048 bf16 26.7 us, a wave per row 27.8; 3000 x 2047 17
// and 22 us).  With fewer too many of its threads would idle (30000 x 1280: 77
// us, a wave per row 57 us).
static RowShape bwd_shape(int64_t cols, int v) {
  const int64_t n = (cols + v - 1) / v;
  return n > 192 && n <= 256 ? RowShape{256, 1} : row_shape(cols, v);
}
// Workgroups of the backward pass.  Each writes a row of partial sums, so more
// of them cost traffic and a longer second half; fewer leave the memory idle
// (16384 x 6144 bf16: 256 workgroups 168 us, 512 160 us, 1024 175 us; 8192 x
// 2048: 34, 28 and 30 us).
constexpr int kNormBwdGrid = 512;
#define UFP4_BWD_SHAPES(F) F(16, 1) F(64, 1) F(64, 2) F(64, 3) F(256, 1) UFP4_LONG_SHAPES(F)

template <typename T, typename W, bool TAIL>
static hipError_t norm_fwd_rows(const NormArgs &a, RowShape s, hipStream_t st) {
  const int64_t groups = row_groups(a.rows, s.tpr);
  const dim3 grid(row_grid(groups));
#define UFP4_NORM(TPR, NV)                                                                   \
  if (s.tpr == TPR && s.nv == NV) {                                                          \
    hipLaunchKernelGGL((rmsnorm_kernel<T, W, TPR, NV, TAIL>), grid, dim3(group_size(TPR)),   \
                       0, st, a);                                                            \
    return hipGetLastError();                                                                \
  }
  UFP4_FWD_SHAPES(UFP4_NORM)
  if constexpr (sizeof(T) == 4) {
    UFP4_NORM(1024, 3)
  }
#undef UFP4_NORM
  return hipErrorInvalidValue;
}

template <typename T, typename W>
static hipError_t norm_fwd(NormArgs a, hipStream_t st) {
  if (a.rows == 0) return hipSuccess;
  a.stream = a.rows * a.cols * (int64_t)sizeof(T) >= kStreamBytes;
  const RowShape s = row_shape(a.cols, Elem<T>::V);
  if (s.tpr != 0)
    return a.cols % Elem<T>::V ? norm_fwd_rows<T, W, true>(a, s, st)
                               : norm_fwd_rows<T, W, false>(a, s, st);
  hipLaunchKernelGGL((rmsnorm_row_kernel<T, W>), dim3(row_grid(a.rows)), dim3(256), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_rmsnorm(const NormArgs &a, hipStream_t st) {
  if (!a.bf16) return norm_fwd<float, float>(a, st);
  return a.w_bf16 ? norm_fwd<uint16_t, uint16_t>(a, st) : norm_fwd<uint16_t, float>(a, st);
}

// Rows of partial sums that dw goes through: the workgroups of the register
// kernel, or the looping kernel's slices of rows.  The element type is not
// known here, so this is the larger of the two types' needs.
static int bwd_slices(int64_t rows, int64_t cols, int v) {
  const RowShape s = bwd_shape(cols, v);
  int64_t n = s.tpr != 0 ? row_groups(rows, s.tpr) : (rows + 63) / 64;
  const int64_t most = s.tpr != 0 ? kNormBwdGrid : 256;
  if (n > most) n = most;
  return n < 1 ? 1 : (int)n;
}
int norm_bwd_slices(int64_t rows, int64_t cols) {
  const int a = bwd_slices(rows, cols, Elem<uint16_t>::V), b = bwd_slices(rows, cols, Elem<float>::V);
  return a > b ? a : b;
}

template <typename T, typename W, bool TAIL>
static hipError_t norm_bwd_rows(const NormBwdArgs &a, RowShape s, int slices, hipStream_t st) {
#define UFP4_NORM(TPR, NV)                                                                   \
  if (s.tpr == TPR && s.nv == NV) {                                                          \
    hipLaunchKernelGGL((rmsnorm_bwd_kernel<T, W, TPR, NV, TAIL>), dim3(slices),              \
                       dim3(group_size(TPR)), 0, st, a);                                     \
    return hipGetLastError();                                                                \
  }
  UFP4_BWD_SHAPES(UFP4_NORM)
  if constexpr (sizeof(T) == 4) {
    UFP4_NORM(1024, 3)
  }
#undef UFP4_NORM
  return hipErrorInvalidValue;
}

template <typename T, typename W>
static hipError_t norm_bwd(NormBwdArgs a, hipStream_t st) {
  a.stream = a.rows * a.cols * (int64_t)sizeof(T) >= kStreamBytes;
  const int slices = bwd_slices(a.rows, a.cols, Elem<T>::V);
  const RowShape s = bwd_shape(a.cols, Elem<T>::V);
  if (s.tpr != 0) {
    const hipError_t e = a.cols % Elem<T>::V ? norm_bwd_rows<T, W, true>(a, s, slices, st)
                                             : norm_bwd_rows<T, W, false>(a, s, slices, st);
    if (e != hipSuccess) return e;
  } else {
    const int64_t per = (a.rows + slices - 1) / slices;
    const unsigned chunks = (unsigned)((a.cols + 255) / 256);
    hipLaunchKernelGGL((rmsnorm_dw_kernel<T>), dim3(chunks, slices), dim3(256), 0, st, a, per);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && a.rows > 0) {
      hipLaunchKernelGGL((rmsnorm_bwd_row_kernel<T, W>), dim3(row_grid(a.rows)), dim3(256), 0,
                         st, a);
      e = hipGetLastError();
    }
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((rmsnorm_dw_final_kernel<W>), dim3((unsigned)((a.cols + 15) / 16)),
                     dim3(1024), 0, st, a, slices);
  return hipGetLastError();
}

hipError_t launch_rmsnorm_bwd(const NormBwdArgs &a, hipStream_t st) {
  if (!a.bf16) return norm_bwd<float, float>(a, st);
  return a.w_bf16 ? norm_bwd<uint16_t, uint16_t>(a, st) : norm_bwd<uint16_t, float>(a, st);
}

}  // namespace ufp4
