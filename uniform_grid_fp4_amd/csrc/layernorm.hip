// Layer norm with the residual's addition, and its backward pass (gfx950).
//   h = round(x + r),  mean = mean(h),  rstd = 1 / sqrt(mean((h - mean)^2) + eps)
//   y = (h - mean) rstd w + b
//   dx = rstd (g - mean(g) - xhat mean(g xhat)) + dh,  g = dy w,
//   dw = sum over rows of dy xhat,  db = sum over rows of dy
// The variance is that of the centred values, which are at hand in registers:
// mean(h^2) - mean^2 would lose what they have in common.  About 12 operations
// per element forward and 18 backward against 6 to 10 bytes: bound by memory.
// Sums are FP32 along a row and over the rows of dw and db; h is rounded once to
// the stream's type, and the statistics are those of the rounded h that the
// backward sees; y and the gradients are rounded once from FP32.
#include "ffn_kernels.h"
#include "row_device.h"

namespace ufp4 {

// Whether element j of the vector of column c0 counts in this lane's sums.
template <bool TAIL, int V>
__device__ __forceinline__ bool counts(int c0, int cols, int j) {
  return c0 < cols && !elsewhere<TAIL, V>(c0, cols, j);
}

// Two sums over the TPR threads that hold a row, through one exchange; s is of
// another turn than the last exchange's.
template <int TPR>
__device__ __forceinline__ void span_sums(float &a, float &b, float (*s)[16]) {
  if constexpr (TPR == 16) {
    a = row_sum(a);
    b = row_sum(b);
  } else {
    a = lanes_sum(a);
    b = lanes_sum(b);
    if constexpr (TPR > 64) {
      constexpr int WAVES = TPR / 64;
      if ((threadIdx.x & 63) == 0) {
        s[0][threadIdx.x % TPR >> 6] = a;
        s[1][threadIdx.x % TPR >> 6] = b;
      }
      __syncthreads();
      a = s[0][0];
      b = s[1][0];
#pragma unroll
      for (int i = 1; i < WAVES; ++i) {
        a += s[0][i];
        b += s[1][i];
      }
    }
  }
}

// A row per TPR threads at a time, as NV vectors each.  Two sums per row go
// through LDS words of their own: between two uses of either lies the other's
// barrier.  8192 x 2048 bf16 with residual 24 us (134 MB, 5.6 TB/s, partly from the
// 256 MB cache), 16384 x 6144 139 us (805 MB, 5.8 TB/s), 4096 x 8192 FP32 100 us (537
// MB, 5.4 TB/s), one row 3.2 us: bound by memory.
template <typename T, typename W, int TPR, int NV, bool TAIL>
__global__ __launch_bounds__(group_size(TPR)) void layernorm_kernel(const LayerNormArgs a) {
  constexpr int V = Elem<T>::V, ROWS = group_size(TPR) / TPR, STEP = TPR * V;
  __shared__ float s_mean[16], s_var[16];
  const int cols = (int)a.cols;
  const int first = (threadIdx.x % TPR) * V;
  WeightVec<T, W, TAIL> w[NV], b[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    w[i].load(static_cast<const W *>(a.w), first + i * STEP, cols);
    if (a.b != nullptr) b[i].load(static_cast<const W *>(a.b), first + i * STEP, cols);
  }
  const int64_t step = (int64_t)gridDim.x * ROWS;
  int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
  const T *x = static_cast<const T *>(a.x), *res = static_cast<const T *>(a.res);
  // 16 lanes or a wave leave the loop on their own; a workgroup has one row
  for (; row < a.rows; row += step) {
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
        sum = elsewhere<TAIL, V>(first + i * STEP, cols, j) ? sum : sum + f[j];
    }
    const float mean = span_sum<TPR>(sum, s_mean) / (float)cols;
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float f[V];
      Elem<T>::unpack(h.v[i], f);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float d = f[j] - mean;
        sum = counts<TAIL, V>(first + i * STEP, cols, j) ? __builtin_fmaf(d, d, sum) : sum;
      }
    }
    const float var = span_sum<TPR>(sum, s_var) / (float)cols;
    const float rstd = 1.0f / sqrtf(var + a.eps);
    if (first == 0) {
      a.mean[row] = mean;
      a.rstd[row] = rstd;
    }
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
      for (int j = 0; j < V; ++j) f[j] = (f[j] - mean) * rstd * g[j];
      if (a.b != nullptr) {
        b[i].get(g);
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] += g[j];
      }
      row_store<T, TAIL>(static_cast<T *>(a.y) + row * a.cols, first + i * STEP, cols,
                         Elem<T>::pack(f), a.stream);
    }
  }
}

// One workgroup per row at a time, three passes over it (the later two find it
// in the caches); a thread reads back only what it wrote itself.
template <typename T, typename W>
__global__ __launch_bounds__(256) void layernorm_row_kernel(const LayerNormArgs a) {
  constexpr int V = Elem<T>::V;
  __shared__ float s_mean[4], s_var[4];
  const W *w = static_cast<const W *>(a.w), *b = static_cast<const W *>(a.b);
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
      for (int i = 0; i < V; ++i) sum += f[i];
    }
    const float mean = group_sum<4>(sum, s_mean) / (float)a.cols;
    const T *src = res != nullptr ? h : x;
    sum = 0.0f;
    for (int64_t c = threadIdx.x * V; c < a.cols; c += 256 * V) {
      float f[V];
      Elem<T>::unpack(load_vec(src + c, a.cols - c), f);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float d = c + i < a.cols ? f[i] - mean : 0.0f;
        sum = __builtin_fmaf(d, d, sum);
      }
    }
    const float rstd = 1.0f / sqrtf(group_sum<4>(sum, s_var) / (float)a.cols + a.eps);
    if (threadIdx.x == 0) {
      a.mean[row] = mean;
      a.rstd[row] = rstd;
    }
    for (int64_t c = threadIdx.x * V; c < a.cols; c += 256 * V) {
      float f[V];
      Elem<T>::unpack(load_vec(src + c, a.cols - c), f);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (c + i >= a.cols) continue;
        f[i] = (f[i] - mean) * rstd * Elem<W>::get(w[c + i]);
        if (b != nullptr) f[i] += Elem<W>::get(b[c + i]);
      }
      store_vec(static_cast<T *>(a.y) + row * a.cols + c, a.cols - c, Elem<T>::pack(f));
    }
  }
}

// Threads of a workgroup of the backward pass: it holds 512 / TPR rows at once,
// whose sums of dw and db it joins, so that fewer partial rows are written.
constexpr int bwd_threads(int tpr) { return tpr < 512 ? 512 : tpr; }

// Backward with rows held in registers: dx, and the workgroup's share of dw and
// db, which stay in registers over all its rows (in the order of the rows) and
// go to partial[workgroup][0 and 1][cols] at the end, the rows of a workgroup
// that holds several added in their order.  8192 x 2048 bf16 29 us and 4 us for the
// second half of dw and db (134 MB and 17 MB of partial sums; with one row of 256
// threads per workgroup 33 and 4); 16384 x 6144 156 us together (805 MB, 5.2 TB/s).
// Loading the next row ahead cost registers and gained nothing.
template <typename T, typename W, int TPR, int NV, bool TAIL>
__global__ __launch_bounds__(bwd_threads(TPR)) void layernorm_bwd_kernel(const LayerNormBwdArgs a) {
  constexpr int THREADS = bwd_threads(TPR);
  constexpr int V = Elem<T>::V, ROWS = THREADS / TPR, STEP = TPR * V;
  __shared__ float s_sums[2][ROWS][2][16];
  const int cols = (int)a.cols;
  const int first = (threadIdx.x % TPR) * V;
  WeightVec<T, W, TAIL> w[NV];
  float acc[NV][V], acb[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    w[i].load(static_cast<const W *>(a.w), first + i * STEP, cols);
#pragma unroll
    for (int j = 0; j < V; ++j) acc[i][j] = acb[i][j] = 0.0f;
  }
  const int64_t step = (int64_t)gridDim.x * ROWS;
  int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
  const T *dy = static_cast<const T *>(a.dy), *h = static_cast<const T *>(a.h);
  const T *dh = static_cast<const T *>(a.dh);
  // 16 lanes or a wave leave the loop on their own.  The rows of a workgroup with
  // barriers leave it together: one past the end repeats the last one and counts
  // nowhere.
  constexpr bool TOGETHER = TPR > 64 && ROWS > 1;
  for (int turn = 0; TOGETHER ? row - threadIdx.x / TPR < a.rows : row < a.rows;
       row += step, turn ^= 1) {
    const int64_t mine = row;
    const bool live = !TOGETHER || row < a.rows;
    if (TOGETHER && !live) row = a.rows - 1;
    RowVecs<NV, T, TAIL> vd, vy, vh;
    vy.load(dy + row * a.ld_dy, first, STEP, cols);
    vh.load(h + row * a.ld_h, first, STEP, cols);
    const float mean = a.mean[row], rstd = a.rstd[row];
    if (dh != nullptr) vd.load(dh + row * a.ld_dh, first, STEP, cols);
    float sg = 0.0f, sgx = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float f[V], g[V], wf[V];
      Elem<T>::unpack(vh.v[i], f);
      Elem<T>::unpack(vy.v[i], g);
      w[i].get(wf);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        // what is not of the row, or another lane's, counts nowhere
        f[j] = (f[j] - mean) * rstd;
        if (!live || !counts<TAIL, V>(first + i * STEP, cols, j)) g[j] = f[j] = 0.0f;
        acc[i][j] = __builtin_fmaf(g[j], f[j], acc[i][j]);
        acb[i][j] += g[j];
        g[j] *= wf[j];
        sg += g[j];
        sgx = __builtin_fmaf(g[j], f[j], sgx);
      }
    }
    // dx may be dy or dh: with shared elements every lane's dh has to be here
    // before another's dx is stored
    if (TAIL && dh != nullptr) {
#pragma unroll
      for (int i = 0; i < NV; ++i) asm volatile("" ::"v"(vd.v[i]));
    }
    span_sums<TPR>(sg, sgx, s_sums[turn][threadIdx.x / TPR]);
    const float mg = sg / (float)cols, mgx = sgx / (float)cols;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float f[V], g[V], wf[V];
      Elem<T>::unpack(vh.v[i], f);
      Elem<T>::unpack(vy.v[i], g);
      w[i].get(wf);
#pragma unroll
      for (int j = 0; j < V; ++j)
        f[j] = rstd * __builtin_fmaf(-(f[j] - mean) * rstd, mgx,
                                     __builtin_fmaf(g[j], wf[j], -mg));
      if (dh != nullptr) {
        Elem<T>::unpack(vd.v[i], g);
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] += g[j];
      }
      if (live)
        row_store<T, TAIL>(static_cast<T *>(a.dx) + row * a.cols, first + i * STEP, cols,
                           Elem<T>::pack(f), a.stream);
    }
    if (TOGETHER) row = mine;
  }
  float *partial = a.partial + (int64_t)blockIdx.x * 2 * a.cols;
  if (ROWS == 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c0 = first + i * STEP;
        if (counts<TAIL, V>(c0, cols, j)) {
          float *p = partial + vec_start<TAIL, V>(c0, cols) + j;
          p[0] = acc[i][j];
          if (a.db != nullptr) p[a.cols] = acb[i][j];
        }
      }
    return;
  }
  __shared__ float s_acc[ROWS][STEP + 1];
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if (which == 1 && a.db == nullptr) break;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c0 = first + i * STEP;
        if (counts<TAIL, V>(c0, cols, j))
          s_acc[threadIdx.x / TPR][vec_start<TAIL, V>(c0, cols) + j - i * STEP] =
              which ? acb[i][j] : acc[i][j];
      }
      __syncthreads();
      for (int c = threadIdx.x; c < STEP && i * STEP + c < cols; c += THREADS) {
        float t = s_acc[0][c];
#pragma unroll
        for (int r = 1; r < ROWS; ++r) t += s_acc[r][c];
        partial[which * a.cols + i * STEP + c] = t;
      }
    }
  }
}

// dx: one workgroup per row at a time, two passes.
template <typename T, typename W>
__global__ __launch_bounds__(256) void layernorm_bwd_row_kernel(const LayerNormBwdArgs a) {
  constexpr int V = Elem<T>::V;
  __shared__ float s_g[4], s_gx[4];
  const W *w = static_cast<const W *>(a.w);
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T *dy = static_cast<const T *>(a.dy) + row * a.ld_dy;
    const T *h = static_cast<const T *>(a.h) + row * a.ld_h;
    const T *dh = a.dh ? static_cast<const T *>(a.dh) + row * a.ld_dh : nullptr;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float sg = 0.0f, sgx = 0.0f;
    for (int64_t c = threadIdx.x * V; c < a.cols; c += 256 * V) {
      float f[V], g[V];
      Elem<T>::unpack(load_vec(h + c, a.cols - c), f);
      Elem<T>::unpack(load_vec(dy + c, a.cols - c), g);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (c + i >= a.cols) continue;
        g[i] *= Elem<W>::get(w[c + i]);
        sg += g[i];
        sgx = __builtin_fmaf(g[i], (f[i] - mean) * rstd, sgx);
      }
    }
    const float mg = group_sum<4>(sg, s_g) / (float)a.cols;
    const float mgx = group_sum<4>(sgx, s_gx) / (float)a.cols;
    for (int64_t c = threadIdx.x * V; c < a.cols; c += 256 * V) {
      float f[V], g[V], d[V];
      Elem<T>::unpack(load_vec(h + c, a.cols - c), f);
      Elem<T>::unpack(load_vec(dy + c, a.cols - c), g);
      if (dh != nullptr) Elem<T>::unpack(load_vec(dh + c, a.cols - c), d);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float wv = c + i < a.cols ? Elem<W>::get(w[c + i]) : 0.0f;
        g[i] = rstd * __builtin_fmaf(-(f[i] - mean) * rstd, mgx,
                                     __builtin_fmaf(g[i], wv, -mg));
        if (dh != nullptr) g[i] += d[i];
      }
      store_vec(static_cast<T *>(a.dx) + row * a.cols + c, a.cols - c, Elem<T>::pack(g));
    }
  }
}

// dw and db, first half: workgroup (chunk of 256 columns, slice of rows) sums
// its rows in order.  Runs before the dx kernel, which may write over dy.
template <typename T>
__global__ __launch_bounds__(256) void layernorm_dw_kernel(const LayerNormBwdArgs a,
                                                           int64_t per_slice) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= a.cols) return;
  const int64_t r0 = (int64_t)blockIdx.y * per_slice;
  const int64_t r1 = min(r0 + per_slice, a.rows);
  const T *dy = static_cast<const T *>(a.dy) + c;
  const T *h = static_cast<const T *>(a.h) + c;
  float sum = 0.0f, sb = 0.0f;
  for (int64_t r = r0; r < r1; ++r) {
    const float g = Elem<T>::get(dy[r * a.ld_dy]);
    sum = __builtin_fmaf(g, (Elem<T>::get(h[r * a.ld_h]) - a.mean[r]) * a.rstd[r], sum);
    sb += g;
  }
  float *p = a.partial + (int64_t)blockIdx.y * 2 * a.cols + c;
  p[0] = sum;
  if (a.db != nullptr) p[a.cols] = sb;
}

// dw and db (blockIdx.y), second half: the slices' sums in a fixed order, 64
// runs of slices side by side for 16 columns per workgroup.
template <typename W>
__global__ __launch_bounds__(1024) void layernorm_dw_final_kernel(const LayerNormBwdArgs a,
                                                                  int slices) {
  __shared__ float s_sum[64][17];
  const int col = threadIdx.x & 15, run = threadIdx.x >> 4;
  const int64_t c = (int64_t)blockIdx.x * 16 + col;
  const float *partial = a.partial + (int64_t)blockIdx.y * a.cols;
  float sum = 0.0f;
  if (c < a.cols) {
#pragma unroll 4
    for (int s = run; s < slices; s += 64) sum += partial[(int64_t)s * 2 * a.cols + c];
  }
  s_sum[run][col] = sum;
  __syncthreads();
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    if (run < o) s_sum[run][col] += s_sum[run + o][col];
    __syncthreads();
  }
  if (run == 0 && c < a.cols)
    static_cast<W *>(blockIdx.y ? a.db : a.dw)[c] = Elem<W>::put(s_sum[0][col]);
}

// The backward pass keeps the sums of dw and db next to three rows: with four
// vectors per lane of a wave it would spill, so 193 to 256 vectors take 256 threads
// with one each.  With fewer, too many of them would idle (30000 x 1280 bf16: 71 us,
// a wave per row 63).  In the same way twice the threads take two vectors each where
// half would take four, and in FP32, whose partial rows of that length are few beside
// the rows, 512 threads one each where 256 would take two (16000 x 1536: 80 and 77 us, 4099 x
// 1411: 24 and 23; bf16 8192 x 4096: 59 and 62).
static RowShape bwd_shape(int64_t cols, int v) {
  const int64_t n = (cols + v - 1) / v;
  const RowShape s = row_shape(cols, v);
  if (v == Elem<float>::V && n > 256 && n <= 512) return {512, 1};
  if (s.nv != 4) return s;
  return n <= 256 ? RowShape{256, 1} : RowShape{s.tpr * 2, 2};
}
// Workgroups of the backward pass, each of which writes its partial sums: two per
// CU where a thread holds one vector and two fit (8192 x 2048 bf16: 33 us, one per
// CU 38; 60000 x 256: 33 and 41), else one (30000 x 1280: 68 and 63 us, 2000 x 12000: 86
// and 65; 16384 x 6144: 168 and 156).
static int bwd_grid(RowShape s) { return s.nv == 1 ? 512 : 256; }

#define UFP4_BWD_SHAPES(F)                                                                   \
  F(16, 1) F(64, 1) F(64, 2) F(64, 3) F(256, 1) F(256, 2) F(256, 3) F(512, 2) F(512, 3) F(1024, 2)

template <typename T, typename W, bool TAIL>
static hipError_t fwd_rows(const LayerNormArgs &a, RowShape s, hipStream_t st) {
  const dim3 grid(row_grid(row_groups(a.rows, s.tpr)));
#define UFP4_NORM(TPR, NV)                                                                   \
  if (s.tpr == TPR && s.nv == NV) {                                                          \
    hipLaunchKernelGGL((layernorm_kernel<T, W, TPR, NV, TAIL>), grid, dim3(group_size(TPR)), \
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
static hipError_t layernorm_fwd(LayerNormArgs a, hipStream_t st) {
  if (a.rows == 0) return hipSuccess;
  a.stream = a.rows * a.cols * (int64_t)sizeof(T) >= kStreamBytes;
  const RowShape s = row_shape(a.cols, Elem<T>::V);
  if (s.tpr != 0)
    return a.cols % Elem<T>::V ? fwd_rows<T, W, true>(a, s, st) : fwd_rows<T, W, false>(a, s, st);
  hipLaunchKernelGGL((layernorm_row_kernel<T, W>), dim3(row_grid(a.rows)), dim3(256), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_layernorm(const LayerNormArgs &a, hipStream_t st) {
  if (!a.bf16) return layernorm_fwd<float, float>(a, st);
  return a.w_bf16 ? layernorm_fwd<uint16_t, uint16_t>(a, st) : layernorm_fwd<uint16_t, float>(a, st);
}

// Rows of partial sums that dw and db go through: the workgroups of the
// register kernel, or the looping kernel's slices of rows.  The element type is
// not known to the caller, so this is the larger of the two types' needs.
static int bwd_slices(int64_t rows, int64_t cols, int v) {
  const RowShape s = bwd_shape(cols, v);
  const int per = s.tpr != 0 ? bwd_threads(s.tpr) / s.tpr : 64;
  int64_t n = (rows + per - 1) / per;
  const int64_t most = s.tpr != 0 ? bwd_grid(s) : 256;
  if (n > most) n = most;
  return n < 1 ? 1 : (int)n;
}
int layernorm_bwd_slices(int64_t rows, int64_t cols) {
  const int a = bwd_slices(rows, cols, Elem<uint16_t>::V), b = bwd_slices(rows, cols, Elem<float>::V);
  return a > b ? a : b;
}

template <typename T, typename W, bool TAIL>
static hipError_t bwd_rows(const LayerNormBwdArgs &a, RowShape s, int slices, hipStream_t st) {
#define UFP4_NORM(TPR, NV)                                                                   \
  if (s.tpr == TPR && s.nv == NV) {                                                          \
    hipLaunchKernelGGL((layernorm_bwd_kernel<T, W, TPR, NV, TAIL>), dim3(slices),            \
                       dim3(bwd_threads(TPR)), 0, st, a);                                    \
    return hipGetLastError();                                                                \
  }
  UFP4_BWD_SHAPES(UFP4_NORM)
  if constexpr (sizeof(T) == 4) {
    UFP4_NORM(512, 1)
    UFP4_NORM(1024, 3)
  }
#undef UFP4_NORM
  return hipErrorInvalidValue;
}

template <typename T, typename W>
static hipError_t layernorm_bwd(LayerNormBwdArgs a, hipStream_t st) {
  a.stream = a.rows * a.cols * (int64_t)sizeof(T) >= kStreamBytes;
  const int slices = bwd_slices(a.rows, a.cols, Elem<T>::V);
  const RowShape s = bwd_shape(a.cols, Elem<T>::V);
  hipError_t e;
  if (s.tpr != 0) {
    e = a.cols % Elem<T>::V ? bwd_rows<T, W, true>(a, s, slices, st)
                            : bwd_rows<T, W, false>(a, s, slices, st);
  } else {
    const int64_t per = (a.rows + slices - 1) / slices;
    const unsigned chunks = (unsigned)((a.cols + 255) / 256);
    hipLaunchKernelGGL((layernorm_dw_kernel<T>), dim3(chunks, slices), dim3(256), 0, st, a, per);
    e = hipGetLastError();
    if (e == hipSuccess && a.rows > 0) {
      hipLaunchKernelGGL((layernorm_bwd_row_kernel<T, W>), dim3(row_grid(a.rows)), dim3(256), 0,
                         st, a);
      e = hipGetLastError();
    }
  }
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((layernorm_dw_final_kernel<W>),
                     dim3((unsigned)((a.cols + 15) / 16), a.db != nullptr ? 2 : 1), dim3(1024), 0,
                     st, a, slices);
  return hipGetLastError();
}

hipError_t launch_layernorm_bwd(const LayerNormBwdArgs &a, hipStream_t st) {
  if (!a.bf16) return layernorm_bwd<float, float>(a, st);
  return a.w_bf16 ? layernorm_bwd<uint16_t, uint16_t>(a, st) : layernorm_bwd<uint16_t, float>(a, st);
}

}  // namespace ufp4
