// Product of int8 rows with a scale each (gfx950):
//   p[m, n] = sa[m] sw[n] sum_k qa[m, k] qw[n, k] (+ bias[n]);  gated: act(p_gate) * p_up
// on v_mfma_i32_*_i8, whose sums are exact: any order and split of K gives the
// same bits.
#include "act_device.h"
#include "block_device.h"
#include "ffn_kernels.h"

namespace ufp4 {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

constexpr int kXcd = 8;
constexpr int kStageK = 128;                     // bytes of K per LDS stage, one row's line

__device__ __forceinline__ int64_t clamped(int64_t v, int64_t n) {
  return v < 0 ? 0 : (v > n ? n : v);
}

// The group and the tile in it of tile t, where group e has ceil(rows of e / bm)
// * per_row tiles.  Offsets are clamped to [0, M], a decreasing pair is an empty
// group.  Every wave finds it by itself: a lane sums a run of groups, a scan over
// the lanes finds the run, and the run is walked.
struct GroupTile {
  int e;                                         // -1: past the last tile
  int64_t row0, rows, local, tiles_m;
};
__device__ __forceinline__ GroupTile group_tile(const Int8GemmArgs &a, int bm, int64_t per_row,
                                                int64_t t) {
  GroupTile g{0, 0, a.M, t, (a.M + bm - 1) / bm};
  if (a.goff == nullptr) {
    if (t >= g.tiles_m * per_row) g.e = -1;
    return g;
  }
  const int lane = threadIdx.x & 63;
  const int per = (a.n_groups + 63) / 64;
  auto tiles_of = [&](int e) -> int64_t {
    if (e >= a.n_groups) return 0;
    const int64_t n = clamped(a.goff[e + 1], a.M) - clamped(a.goff[e], a.M);
    return n > 0 ? (n + bm - 1) / bm : 0;
  };
  int64_t mine = 0;
  for (int i = 0; i < per; ++i) mine += tiles_of(lane * per + i);
  mine *= per_row;
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int64_t v = __shfl_up(incl, o, 64);
    if (lane >= o) incl += v;
  }
  const uint64_t over = __ballot(incl > t);
  if (over == 0) {
    g.e = -1;
    return g;
  }
  const int src = __builtin_ctzll(over);
  int64_t base = __shfl(incl - mine, src, 64);
  for (int e = src * per;; ++e) {
    const int64_t n = tiles_of(e);
    if (t < base + n * per_row) {
      g.e = e;
      g.row0 = clamped(a.goff[e], a.M);
      g.rows = clamped(a.goff[e + 1], a.M) - g.row0;
      g.local = t - base;
      g.tiles_m = n;
      return g;
    }
    base += n * per_row;
  }
}

__device__ __forceinline__ void put(const Int8GemmArgs &a, int64_t row, int64_t col, float v) {
  if (a.out_bf16) static_cast<uint16_t *>(a.y)[row * a.ld_y + col] = to_bf16_bits(v);
  else static_cast<float *>(a.y)[row * a.ld_y + col] = v;
}
__device__ __forceinline__ float gated(int act, float gate, float up) {
  return up * (act == UFP4_ACT_SILU ? act_value<UFP4_ACT_SILU>(gate)
                                    : act_value<UFP4_ACT_GELU>(gate));
}

// ---------------------------------------------------------------------------
// Few rows of x per group: w is read once, straight into the matrix
// instruction's registers, by workgroups of 16 columns (gated: 16 of either
// projection) whose four waves take every fourth 64 bytes of K; their sums meet
// in LDS.  MT tiles of 16 rows of x at a time, in a loop over the group's rows.
// ---------------------------------------------------------------------------
template <int MT, bool GATED>
__global__ __launch_bounds__(256) void int8_rows_kernel(const Int8GemmArgs a) {
  constexpr int P = GATED ? 2 : 1, WAVES = 4, U = 4;
  __shared__ int s_acc[WAVES][P * MT][256];
  const int64_t out_n = a.N / P;                  // output columns
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l16 = lane & 15, chunk = (lane >> 4) * 16;
  int64_t row0 = 0, rows = a.M;
  const int e = blockIdx.y;
  if (a.goff != nullptr) {
    row0 = clamped(a.goff[e], a.M);
    rows = clamped(a.goff[e + 1], a.M) - row0;
  }
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int64_t units = a.kpad / 64;
  const int8_t *pw[P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int64_t n = min(n0 + l16, out_n - 1);
    pw[p] = a.w + ((int64_t)e * a.N + p * out_n + n) * a.kpad + chunk;
  }
  for (int64_t m0 = 0; m0 < rows; m0 += 16 * MT) {
    const int8_t *pa[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t)
      pa[t] = a.a + (row0 + min(m0 + 16 * t + l16, rows - 1)) * a.kpad + chunk;
    i32x4 acc[P][MT];
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int t = 0; t < MT; ++t) acc[p][t] = i32x4(0);
    int64_t k = wave;
    for (; k + (U - 1) * WAVES < units; k += U * WAVES) {
      i32x4 w[U][P], x[U][MT];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t at = (k + u * WAVES) * 64;
#pragma unroll
        for (int p = 0; p < P; ++p) w[u][p] = *reinterpret_cast<const i32x4 *>(pw[p] + at);
#pragma unroll
        for (int t = 0; t < MT; ++t) x[u][t] = *reinterpret_cast<const i32x4 *>(pa[t] + at);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int t = 0; t < MT; ++t)
            acc[p][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(x[u][t], w[u][p], acc[p][t], 0, 0, 0);
    }
    for (; k < units; k += WAVES) {
      i32x4 w[P];
#pragma unroll
      for (int p = 0; p < P; ++p) w[p] = *reinterpret_cast<const i32x4 *>(pw[p] + k * 64);
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const i32x4 x = *reinterpret_cast<const i32x4 *>(pa[t] + k * 64);
#pragma unroll
        for (int p = 0; p < P; ++p)
          acc[p][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(x, w[p], acc[p][t], 0, 0, 0);
      }
    }
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          s_acc[wave][p * MT + t][(4 * (lane >> 4) + r) * 16 + l16] = acc[p][t][r];
    __syncthreads();
    const int64_t col = n0 + (threadIdx.x & 15);
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const int64_t m = m0 + 16 * t + (threadIdx.x >> 4);
      if (m >= rows || col >= out_n) continue;
      const float sa = a.sa[row0 + m];
      float v[P];
#pragma unroll
      for (int p = 0; p < P; ++p) {
        int sum = 0;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) sum += s_acc[w][p * MT + t][threadIdx.x];
        const int64_t n = (int64_t)e * a.N + p * out_n + col;
        v[p] = (float)sum * sa * a.sw[n];
        if (a.bias != nullptr) v[p] += a.bias[n];
      }
      put(a, row0 + m, col, GATED ? gated(a.act, v[0], v[P - 1]) : v[0]);
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Many rows: BM x BN tiles of p, staged through LDS.
// ---------------------------------------------------------------------------
template <int WM, int WN, int MT, bool GATED>
__global__ __launch_bounds__(64 * WM * WN) void int8_tile_kernel(const Int8GemmArgs a,
                                                                 int64_t tiles_n,
                                                                 int64_t first) {
  constexpr int NT = 2, THREADS = 64 * WM * WN;
  constexpr int BM = 32 * MT * WM, BN = 32 * NT * WN;
  constexpr int OUT = GATED ? BN / 2 : BN;        // output columns of a tile
  constexpr int AL = BM * kStageK / (16 * THREADS), BL = BN * kStageK / (16 * THREADS);
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  constexpr int kStage = (BM + BN) * kStageK;
  const int64_t out_n = a.N / (GATED ? 2 : 1);

  // The workgroups of an XCD (every eighth) walk a contiguous range of tiles, so
  // that a panel stays in one L2.
  const unsigned per = gridDim.x / kXcd;          // the grid is a multiple of the XCDs
  const int64_t t = first + blockIdx.x % kXcd * per + blockIdx.x / kXcd;
  const GroupTile g = group_tile(a, BM, tiles_n, t);
  if (g.e < 0) return;
  const int64_t tm = g.local / tiles_n, tn = g.local - tm * tiles_n;
  const int64_t row0 = g.row0 + tm * BM;
  const int rows = (int)min((int64_t)BM, g.rows - tm * BM);
  const int64_t col0 = tn * OUT;
  const int cols = (int)min((int64_t)OUT, out_n - col0);

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave % WM, wn = wave / WM;
  const int8_t *pa[AL], *pb[BL];
#pragma unroll
  for (int i = 0; i < AL; ++i) {
    const int item = i * THREADS + threadIdx.x;
    const int r = item >> 3, c = (item & 7) ^ (r & 7);
    pa[i] = a.a + (row0 + min(r, rows - 1)) * a.kpad + c * 16;
  }
#pragma unroll
  for (int i = 0; i < BL; ++i) {
    const int item = i * THREADS + threadIdx.x;
    const int r = item >> 3, c = (item & 7) ^ (r & 7);
    int64_t n;
    if (GATED) n = (int64_t)((r >> 5) & 1) * out_n + col0 + min((r >> 6) * 32 + (r & 31), cols - 1);
    else n = col0 + min(r, cols - 1);
    pb[i] = a.w + ((int64_t)g.e * a.N + n) * a.kpad + c * 16;
  }
  i32x16 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
  const int64_t stages = a.kpad / kStageK;
  i32x4 ra[AL], rb[BL];
  auto load = [&](int64_t s) {
#pragma unroll
    for (int i = 0; i < AL; ++i) ra[i] = *reinterpret_cast<const i32x4 *>(pa[i] + s * kStageK);
#pragma unroll
    for (int i = 0; i < BL; ++i) rb[i] = *reinterpret_cast<const i32x4 *>(pb[i] + s * kStageK);
  };
  auto store = [&](uint8_t *st) {
#pragma unroll
    for (int i = 0; i < AL; ++i)
      *reinterpret_cast<i32x4 *>(st + (i * THREADS + threadIdx.x) * 16) = ra[i];
#pragma unroll
    for (int i = 0; i < BL; ++i)
      *reinterpret_cast<i32x4 *>(st + BM * kStageK + (i * THREADS + threadIdx.x) * 16) = rb[i];
  };
  const int l32 = lane & 31, half = lane >> 5;
  load(0);
  store(lds);
  __syncthreads();
  for (int64_t s = 0; s < stages; ++s) {
    const uint8_t *st = lds + (s & 1) * kStage;
    if (s + 1 < stages) load(s + 1);
#pragma unroll
    for (int kk = 0; kk < kStageK / 32; ++kk) {
      const int slot = ((2 * kk + half) ^ (l32 & 7)) * 16;
      i32x4 fa[MT], fb[NT];
#pragma unroll
      for (int i = 0; i < MT; ++i)
        fa[i] = *reinterpret_cast<const i32x4 *>(st + ((wm * MT + i) * 32 + l32) * kStageK + slot);
#pragma unroll
      for (int j = 0; j < NT; ++j)
        fb[j] = *reinterpret_cast<const i32x4 *>(st + (BM + (wn * NT + j) * 32 + l32) * kStageK +
                                                 slot);
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fa[i], fb[j], acc[i][j], 0, 0, 0);
    }
    if (s + 1 < stages) store(lds + ((s + 1) & 1) * kStage);
    __syncthreads();
  }
#pragma unroll
  for (int j = 0; j < (GATED ? 1 : NT); ++j) {
    const int col = GATED ? wn * 32 + l32 : (wn * NT + j) * 32 + l32;
    if (col >= cols) continue;
    const int64_t n = (int64_t)g.e * a.N + col0 + col;
    const float sw = a.sw[n], su = GATED ? a.sw[n + out_n] : 0.0f;
    const float bw = a.bias ? a.bias[n] : 0.0f, bu = GATED && a.bias ? a.bias[n + out_n] : 0.0f;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int m = (wm * MT + i) * 32 + 8 * (r >> 2) + 4 * half + (r & 3);
        if (m >= rows) continue;
        const float sa = a.sa[row0 + m];
        float v = (float)acc[i][j][r] * sa * sw;
        if (a.bias) v += bw;
        if (GATED) {
          float u = (float)acc[i][1][r] * sa * su;
          if (a.bias) u += bu;
          v = gated(a.act, v, u);
        }
        put(a, row0 + m, col0 + col, v);
      }
  }
}

// ---------------------------------------------------------------------------
template <int MT, bool GATED>
static hipError_t launch_rows(const Int8GemmArgs &a, hipStream_t st) {
  const int64_t out_n = a.N / (GATED ? 2 : 1);
  hipLaunchKernelGGL((int8_rows_kernel<MT, GATED>),
                     dim3((unsigned)((out_n + 15) / 16), (unsigned)a.n_groups), dim3(256), 0, st, a);
  return hipGetLastError();
}

template <int WM, int WN, int MT, bool GATED>
static hipError_t launch_tiles(const Int8GemmArgs &a, hipStream_t st) {
  constexpr int BM = 32 * MT * WM, BN = 64 * WN;
  constexpr size_t kLds = 2 * (BM + BN) * kStageK;
  const int64_t out_n = a.N / (GATED ? 2 : 1);
  const int64_t tiles_n = (out_n + (GATED ? BN / 2 : BN) - 1) / (GATED ? BN / 2 : BN);
  const int64_t tiles_m = (a.M + BM - 1) / BM + (a.goff ? a.n_groups : 0);
  const int64_t total = (tiles_m * tiles_n + kXcd - 1) / kXcd * kXcd;
  constexpr int64_t kMost = 1 << 22;              // tiles of a launch: below 2^32 threads
  auto *kernel = int8_tile_kernel<WM, WN, MT, GATED>;
  const hipError_t e = hipFuncSetAttribute((const void *)kernel,
                                           hipFuncAttributeMaxDynamicSharedMemorySize, (int)kLds);
  if (e != hipSuccess) return e;
  for (int64_t first = 0; first < total; first += kMost) {
    const unsigned n = (unsigned)(total - first < kMost ? total - first : kMost);
    hipLaunchKernelGGL(kernel, dim3(n), dim3(64 * WM * WN), kLds, st, a, tiles_n, first);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

template <bool GATED>
static hipError_t int8_gemm(const Int8GemmArgs &a, hipStream_t st) {
  const int64_t rows = (a.M + a.n_groups - 1) / a.n_groups;
  if (rows <= 16) return launch_rows<1, GATED>(a, st);
  if (rows <= 64) return launch_rows<4, GATED>(a, st);
  const int64_t big = ((a.M + 255) / 256) * ((a.N + 255) / 256);
  if (big >= 256) return launch_tiles<2, 4, 4, GATED>(a, st);
  return launch_tiles<2, 2, 2, GATED>(a, st);
}

hipError_t launch_int8_gemm(const Int8GemmArgs &a, hipStream_t st) {
  if (a.M == 0) return hipSuccess;
  return a.act == UFP4_ACT_NONE ? int8_gemm<false>(a, st) : int8_gemm<true>(a, st);
}

}  // namespace ufp4
