// Product of int8 rows with a scale each (gfx950):
//   p[m, n] = sa[m] sw[n] sum_k qa[m, k] qw[n, k] (+ bias[n]);  gated: act(p_gate) * p_up
// on v_mfma_i32_*_i8, whose sums are exact: any order and split of K gives the
// same bits.
#include <atomic>
#include <cmath>

#include "act_device.h"
#include "block_device.h"
#include "ffn_kernels.h"
#include "group_device.h"
#include "int8_device.h"

namespace ufp4 {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef float floatx4 __attribute__((ext_vector_type(4)));

constexpr int kXcd = 8, kCus = 256;
constexpr int kStageK = 128;                     // bytes of K per LDS stage: a row's piece is a line

// One value of the result from its exact sums: the same operations in every
// kernel, so that which one runs shows in no bit.
// No bias is one of -0, which changes no sum, and costs less than the choice.
template <int ACT>
__device__ __forceinline__ float finish(int gate, int up, float sa, float sg, float su, float bg,
                                        float bu) {
  const float v = (float)gate * sa * sg + bg;
  if constexpr (ACT != UFP4_ACT_NONE) return ((float)up * sa * su + bu) * act_value<ACT>(v);
  return v;
}
constexpr float kNoBias = -0.0f;
__device__ __forceinline__ void put(const Int8GemmArgs &a, int64_t row, int64_t col, float v) {
  if (a.out_bf16) static_cast<uint16_t *>(a.y)[row * a.ld_y + col] = to_bf16_bits(v);
  else static_cast<float *>(a.y)[row * a.ld_y + col] = v;
}

// ---------------------------------------------------------------------------
// Few rows of x per group: bound by reading w, which goes once, straight into
// the matrix instruction's registers.  A workgroup has 16 columns (gated: of
// either projection); its eight waves take every eighth line of 128 bytes of its
// rows, and their sums meet in LDS.  MT tiles of 16 rows of x at a time, in a loop
// over the group's rows.  The two loads of a line follow each other, and all
// loads of a turn go before its products: 128 rows over 32 experts of 6144 to 2 x
// 2048 columns take 131 us (805 MB, 6.1 TB/s), in the order of the products 155 us, with
// streaming loads 150-200 us; one row to 2 x 8192 columns 7.6 us.
// ---------------------------------------------------------------------------
constexpr int kRowWaves = 8;
template <int MT, int ACT>
__global__ __launch_bounds__(64 * kRowWaves) void int8_rows_kernel(const Int8GemmArgs a) {
  constexpr bool GATED = ACT != UFP4_ACT_NONE;
  constexpr int P = GATED ? 2 : 1;
  __shared__ int s_acc[kRowWaves][P * MT][256];
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
  const int kpad = (int)a.kpad;
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
    for (int k = wave * kStageK; k < kpad; k += kRowWaves * kStageK) {
      i32x4 w[P][2], x[MT][2];
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int u = 0; u < 2; ++u)
          w[p][u] = *reinterpret_cast<const i32x4 *>(pw[p] + k + u * 64);
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int u = 0; u < 2; ++u)
          x[t][u] = *reinterpret_cast<const i32x4 *>(pa[t] + k + u * 64);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int t = 0; t < MT; ++t)
            acc[p][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(x[t][u], w[p][u], acc[p][t], 0, 0, 0);
    }
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          s_acc[wave][p * MT + t][(4 * (lane >> 4) + r) * 16 + l16] = acc[p][t][r];
    __syncthreads();
    for (int i = threadIdx.x; i < MT * 256; i += 64 * kRowWaves) {
      const int tile = i >> 8, at = i & 255;
      const int64_t m = m0 + 16 * tile + (at >> 4), col = n0 + (at & 15);
      if (m >= rows || col >= out_n) continue;
      int sum[2] = {0, 0};
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int w = 0; w < kRowWaves; ++w) sum[p] += s_acc[w][p * MT + tile][at];
      const int64_t n = (int64_t)e * a.N + col, up = GATED ? n + out_n : n;
      const bool bias = a.bias != nullptr;
      put(a, row0 + m, col,
          finish<ACT>(sum[0], sum[1], a.sa[row0 + m], a.sw[n], a.sw[up],
                      bias ? a.bias[n] : kNoBias, bias ? a.bias[up] : kNoBias));
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// The same for so few rows of x, in one group, that every workgroup quantizes them
// by itself: one launch instead of two, and no workspace.  The waves share out the
// rows (or parts of one), their largest elements meet in LDS, the codes go to LDS,
// and the products read them there.  The first loads of w are on their way
// meanwhile.  1 x 2048 to 2 x 8192 columns, bf16: 10 us (34 MB, 3.4 TB/s; 9 us with one
// set of weights that stays in the caches): bound by latency, of the row, of two
// exchanges and of w.
// ---------------------------------------------------------------------------
template <typename T, int ACT>
__global__ __launch_bounds__(64 * kRowWaves) void int8_fused_kernel(const Int8GemmArgs a,
                                                                    const Int8QuantArgs q) {
  constexpr bool GATED = ACT != UFP4_ACT_NONE;
  constexpr int P = GATED ? 2 : 1, V = Elem<T>::V;
  __shared__ int s_acc[kRowWaves][P][256];
  __shared__ uint32_t s_top[16][kRowWaves];
  extern __shared__ __attribute__((aligned(16))) uint8_t s_x[];
  const int64_t out_n = a.N / P;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l16 = lane & 15, chunk = (lane >> 4) * 16;
  const int rows = (int)a.M, kpad = (int)a.kpad, cols = (int)q.cols;
  const int line = kpad + 16;                     // 16 more to spread the rows over the banks
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int8_t *pw[P];
  i32x4 w[P][2];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    pw[p] = a.w + (p * out_n + min(n0 + l16, out_n - 1)) * a.kpad + chunk;
    // a wave beyond K loads the first line and does not use it
    const int k = wave * kStageK < kpad ? wave * kStageK : 0;
#pragma unroll
    for (int u = 0; u < 2; ++u) w[p][u] = *reinterpret_cast<const i32x4 *>(pw[p] + k + u * 64);
  }

  // waves per row: 8 for one row, down to 1; beyond 8 rows a wave has two
  const int parts = rows == 1 ? 8 : rows == 2 ? 4 : rows <= 4 ? 2 : 1;
  const int part = wave % parts, row_step = kRowWaves / parts;
  const int step = parts * 64 * V, c_first = (part * 64 + lane) * V;
  const T *x = static_cast<const T *>(q.x);
  for (int r = wave / parts; r < rows; r += row_step) {
    uint32_t top = 0;
    for (int c = c_first; c < cols; c += step) {
      float f[V];
      Elem<T>::unpack(load_vec(x + r * q.ld_x + c, cols - c), f);
#pragma unroll
      for (int j = 0; j < V; ++j) top = max(top, __float_as_uint(fabsf(f[j])));
    }
    top = lanes_max(top);
    if (lane == 0) s_top[r][part] = top;
  }
  __syncthreads();
  for (int r = wave / parts; r < rows; r += row_step) {
    uint32_t top = s_top[r][0];
    for (int i = 1; i < parts; ++i) top = max(top, s_top[r][i]);
    const Int8Scale s = int8_scale(top);
    for (int c = c_first; c < kpad; c += step) {
      float f[V];
#pragma unroll
      for (int j = 0; j < V; ++j) f[j] = 0.0f;
      if (c < cols) Elem<T>::unpack(load_vec(x + r * q.ld_x + c, cols - c), f);
#pragma unroll
      for (int j = 0; j < V / 4; ++j)
        *reinterpret_cast<uint32_t *>(s_x + r * line + c + 4 * j) = int8x4(f + 4 * j, s);
    }
  }
  __syncthreads();

  i32x4 acc[P];
#pragma unroll
  for (int p = 0; p < P; ++p) acc[p] = i32x4(0);
  const uint8_t *px = s_x + min(l16, rows - 1) * line + chunk;
  for (int k = wave * kStageK; k < kpad; k += kRowWaves * kStageK) {
    i32x4 f[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) f[u] = *reinterpret_cast<const i32x4 *>(px + k + u * 64);
    i32x4 next[P][2];
    const int k1 = k + kRowWaves * kStageK < kpad ? k + kRowWaves * kStageK : k;
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int u = 0; u < 2; ++u)
        next[p][u] = *reinterpret_cast<const i32x4 *>(pw[p] + k1 + u * 64);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int p = 0; p < P; ++p)
        acc[p] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f[u], w[p][u], acc[p], 0, 0, 0);
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int u = 0; u < 2; ++u) w[p][u] = next[p][u];
  }
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int r = 0; r < 4; ++r) s_acc[wave][p][(4 * (lane >> 4) + r) * 16 + l16] = acc[p][r];
  __syncthreads();
  if (threadIdx.x >= 256) return;
  const int m = threadIdx.x >> 4;
  const int64_t n = n0 + l16, up = GATED ? n + out_n : n;
  if (m >= rows || n >= out_n) return;
  int sum[2] = {0, 0};
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int i = 0; i < kRowWaves; ++i) sum[p] += s_acc[i][p][threadIdx.x];
  uint32_t top = s_top[m][0];
  for (int i = 1; i < parts; ++i) top = max(top, s_top[m][i]);
  const bool bias = a.bias != nullptr;
  put(a, m, n,
      finish<ACT>(sum[0], sum[1], int8_scale(top).scale, a.sw[n], a.sw[up],
                  bias ? a.bias[n] : kNoBias, bias ? a.bias[up] : kNoBias));
}

// ---------------------------------------------------------------------------
// Many rows: BM x BN tiles of p (BM = 32 MT WM, BN = 64 WN), one per workgroup of
// WM x WN waves, a wave owning 32 MT x 64 of it in 32x32 tiles; gated: its two
// tiles of a row are the gate's and the up projection's of the same 32 columns.
// Where the tiles are fewer than the CUs, a workgroup has KS such sets of waves,
// each with its own stages of K (every KS-th) and its own LDS, so that one set's
// products cover another's waits; their integer sums meet in LDS.
//
// K goes through LDS in stages of 128 bytes per row, double-buffered, brought
// there by buffer loads that write LDS directly (16 bytes a lane, no registers).
// The loads of a stage are in flight while the one before is multiplied.  A
// fragment is read from LDS one step of 32 bytes before its products, across the
// stages too: the last step of a stage waits for the next stage's loads and the
// other waves' reads, reads the next stage's first fragments, sends the loads of
// the stage after it into the buffer that is now free, and only then issues its
// own products.  Rows are 128 bytes, so a fragment's 32 rows fall on the same
// banks: the 16-byte pieces of a row are kept in an order of its own (piece c at
// place c ^ swizzle(row)), which the loads make by the address each lane asks for.
//
// w is the matrix instruction's first operand and x its second, so a lane ends
// with four neighbouring columns of one row: the epilogue packs them, passes them
// through LDS and writes 16 bytes a lane.  The largest tiles have a CU to
// themselves, with nothing beside them to hide their start: their workgroups go
// on to other tiles, whose first two stages are under way during the epilogue.
// 8192 x 2048 to 2 x 8192 columns, silu, bf16: 280 us (1.96 POP/s; a workgroup per tile
// 296; a library product of the same size 287 with its int32 output); 8192 x 8192 to
// 8192: 474 us (2.32 POP/s; 500).  Earlier steps of the first: fragments read in their
// own step 300-320 us instead of 273 on that day's card, stages of 64 bytes 290-297,
// 128 x 128 tiles 298, 128 x 128 per wave (4 waves) 300-315.  What bounds it: reads of LDS
// (24 KB per 8.4 MOP of a wave) and the products take about the same time, under
// them the clock falls to 1.9 GHz (zeros in place of the data: 225 us), and the
// epilogue's vector work, 4 to 5 us a tile, runs beside neither.
// ---------------------------------------------------------------------------
__device__ __forceinline__ int swizzle(int row) {
  return ((row >> 1) & 3) | ((((row >> 3) ^ (row >> 4)) & 1) << 2);
}
// Waits for all of this wave's loads into LDS, and for its LDS accesses.
__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
// Writes to LDS that do not wait for the loads into it (elsewhere), as the compiler's
// own would; wait_lds() before they are read.
__device__ __forceinline__ uint32_t lds_address(uint8_t *p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)p;
}
__device__ __forceinline__ void write_lds(uint8_t *p, uint2 v) {
  asm volatile("ds_write_b64 %0, %1" ::"v"(lds_address(p)), "v"(v) : "memory");
}
__device__ __forceinline__ void write_lds(uint8_t *p, floatx4 v) {
  asm volatile("ds_write_b128 %0, %1" ::"v"(lds_address(p)), "v"(v) : "memory");
}
// Between the waves of a workgroup; memory accesses stay on their side.
__device__ __forceinline__ void meet() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}
// 16 bytes per lane from base + voffset + soffset to dst + 16 * lane.
__device__ __forceinline__ void load_lds(const int8_t *base, int voffset, int soffset,
                                         uint8_t *dst) {
  const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<int8_t *>(base), (short)0, 0x7FFFFFF0, 0x00020000);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(
      r, (__attribute__((address_space(3))) void *)dst, 16, voffset, soffset, 0, 0);
}

// The first n columns of a vector (none for n <= 0).
template <typename T>
__device__ __forceinline__ void store_cols(T *p, int n, u32x4 v) {
  if (n > 0) store_vec(p, n, v);
}

constexpr int kBandRows = 8;       // tile rows that neighbouring workgroups share w's panels over
constexpr int kLine = 64 + 16;     // bytes of a row's piece in the epilogue; 16 more spread the banks
template <int WM, int WN, int MT, int KS>
struct TileShape {
  static constexpr int kThreads = 64 * WM * WN * KS, kBM = 32 * MT * WM, kBN = 64 * WN;
  static constexpr int kStage = (kBM + kBN) * kStageK;
  // the workgroup goes on to other tiles: it has the CU to itself
  static constexpr bool kStays = 2 * kStage > 80 * 1024 && KS == 1;
  static constexpr int kLines = WM * WN * 32 * kLine;
  // the stages; the rows' scales; the columns' scales and biases; the epilogue's lines,
  // where the next tile's stages come in under it
  static constexpr size_t kLds =
      KS * 2 * kStage + (kBM + 2 * kBN) * sizeof(float) + (kStays ? kLines : 0);
};

// a / b; both are small where it counts.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((uint64_t)(a | b) >> 31) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

template <int WM, int WN, int MT, int KS, int ACT>
__global__ __attribute__((amdgpu_flat_work_group_size(64 * WM * WN * KS, 64 * WM * WN * KS),
                          amdgpu_waves_per_eu(2, 2))) void
int8_tile_kernel(const Int8GemmArgs a, int64_t tiles_n, int64_t first) {
  using S = TileShape<WM, WN, MT, KS>;
  constexpr bool GATED = ACT != UFP4_ACT_NONE;
  constexpr int NT = 2, WAVES = WM * WN, BM = S::kBM, BN = S::kBN;
  constexpr int OUT = GATED ? BN / 2 : BN;        // output columns of a tile
  constexpr int AL = BM / (8 * WAVES), BL = BN / (8 * WAVES);   // loads per lane and stage
  static_assert(AL * 8 * WAVES == BM && BL * 8 * WAVES == BN, "rows per load");
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  float *s_sa = reinterpret_cast<float *>(lds + KS * 2 * S::kStage);
  float *s_sw = s_sa + BM, *s_bias = s_sw + BN;
  uint8_t *lines = S::kStays ? reinterpret_cast<uint8_t *>(s_bias + BN) : lds;
  const int64_t out_n = a.N / (GATED ? 2 : 1);

  const int lane = threadIdx.x & 63;
  const int id = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = id / WAVES, wave = id % WAVES; // of K, of the part
  const int wm = wave % WM, wn = wave / WM;
  const int l32 = lane & 31, half = lane >> 5;
  const int kpad = (int)a.kpad;
  const int total = kpad / kStageK;
  const int stages = (total - part + KS - 1) / KS, turns = (total + KS - 1) / KS;
  uint8_t *const mine = lds + part * 2 * S::kStage;

  // A tile: its place, its loads and its scales.  The scales wait in registers for
  // the epilogue: a write to LDS would wait for all loads into it.
  int64_t row0 = 0, col0 = 0;
  int rows = 0, cols = 0;
  const int8_t *base_a = nullptr, *base_w = nullptr, *base_u = nullptr;
  int va[AL], vw[BL];
  float scale_a[(BM + S::kThreads - 1) / S::kThreads];
  float scale_w[(BN + S::kThreads - 1) / S::kThreads], bias[(BN + S::kThreads - 1) / S::kThreads];
  // The workgroups of an XCD (every eighth) walk a contiguous eighth of the tiles, in
  // bands of kBandRows tile rows, column by column: their panels meet in one L2.  Of
  // the tiles that there are: eighths of the grid, which is cut for the most tiles that
  // the groups can have, would leave the last XCDs idle.
  auto place = [&](int64_t at) __attribute__((always_inline)) -> bool {
    const GroupTile g = group_tile(a.goff, a.n_groups, a.M, BM, tiles_n, [=](int64_t tiles) {
      const int64_t per = (tiles + kXcd - 1) / kXcd;
      return at / kXcd < per ? at % kXcd * per + at / kXcd : tiles;
    });
    if (g.e < 0) return false;
    const int64_t band = quotient(g.local, kBandRows * tiles_n);
    const int64_t in_band = g.local - band * kBandRows * tiles_n;
    const int64_t deep = min((int64_t)kBandRows, g.tiles_m - band * kBandRows);
    const int64_t tn = quotient(in_band, deep), tm = band * kBandRows + in_band - tn * deep;
    row0 = g.row0 + tm * BM;
    rows = (int)min((int64_t)BM, g.rows - tm * BM);
    col0 = tn * OUT;
    cols = (int)min((int64_t)OUT, out_n - col0);
    const int64_t w_row = (int64_t)g.e * a.N + col0;
    // A load takes eight rows; rows past the tile's repeat its last one (their
    // products are not stored).  Offsets stay below 256 rows of 2^17 bytes.
    base_a = a.a + row0 * a.kpad;
    base_w = a.w + w_row * a.kpad;
    base_u = base_w + (GATED ? out_n * a.kpad : 0);
#pragma unroll
    for (int i = 0; i < AL; ++i) {
      const int r = (i * WAVES + wave) * 8 + (lane >> 3);
      va[i] = min(r, rows - 1) * kpad + ((lane & 7) ^ swizzle(r)) * 16;
    }
#pragma unroll
    for (int i = 0; i < BL; ++i) {
      const int r = (i * WAVES + wave) * 8 + (lane >> 3);
      const int n = GATED ? (r >> 6) * 32 + (r & 31) : r;
      vw[i] = min(n, cols - 1) * kpad + ((lane & 7) ^ swizzle(r)) * 16;
    }
#pragma unroll
    for (int i = 0; i * S::kThreads < BM; ++i)
      scale_a[i] = a.sa[row0 + min((int)threadIdx.x + i * S::kThreads, rows - 1)];
#pragma unroll
    for (int i = 0; i * S::kThreads < BN; ++i) {
      const int r = min((int)threadIdx.x + i * S::kThreads, BN - 1);
      const int n = min(GATED ? (r >> 6) * 32 + (r & 31) : r, cols - 1);
      const int64_t w = w_row + n + (GATED && (r >> 5) & 1 ? out_n : 0);
      scale_w[i] = a.sw[w];
      bias[i] = a.bias != nullptr ? a.bias[w] : kNoBias;
    }
    return true;
  };
  auto issue = [&](int stage) __attribute__((always_inline)) {
    uint8_t *st = mine + (stage & 1) * S::kStage + wave * 1024;
    const int k0 = (stage * KS + part) * kStageK;
#pragma unroll
    for (int i = 0; i < AL; ++i) load_lds(base_a, va[i], k0, st + i * WAVES * 1024);
#pragma unroll
    for (int i = 0; i < BL; ++i) {
      // runs of 32 rows of either projection; a load's eight are of one
      const bool up = GATED && (((i * WAVES + wave) >> 2) & 1) != 0;
      load_lds(up ? base_u : base_w, vw[i], k0, st + BM * kStageK + i * WAVES * 1024);
    }
  };

  int64_t at = first + blockIdx.x;
  if (!place(at)) return;
  if (stages > 0) issue(0);
  if (stages > 1) issue(1);
  for (;;) {
    i32x16 acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
    constexpr int KK = kStageK / 32;
    i32x4 fa[2][MT], fw[2][NT];
    const uint8_t *pa = mine + (wm * MT * 32 + l32) * kStageK;
    const uint8_t *pw = mine + (BM + wn * NT * 32 + l32) * kStageK;
    const int sw32 = swizzle(l32);
    auto read = [&](int into, int stage, int kk) __attribute__((always_inline)) {
      const int from = (stage & 1) * S::kStage + ((2 * kk + half) ^ sw32) * 16;
#pragma unroll
      for (int i = 0; i < MT; ++i)
        fa[into][i] = *reinterpret_cast<const i32x4 *>(pa + from + i * 32 * kStageK);
#pragma unroll
      for (int j = 0; j < NT; ++j)
        fw[into][j] = *reinterpret_cast<const i32x4 *>(pw + from + j * 32 * kStageK);
    };
    wait_loads();
    wait_lds();
    meet();
    read(0, 0, 0);
    for (int s = 0; s < turns; ++s) {
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) {
        if (kk + 1 < KK) {
          read((kk + 1) & 1, s, kk + 1);
        } else if (s + 1 < turns) {
          wait_loads();                           // of stage s + 1
          wait_lds();                             // this wave's last fragments of stage s
          meet();
          read((kk + 1) & 1, s + 1, 0);
          if (s + 2 < stages) issue(s + 2);
        }
        // the reads and loads above go out before the products below
        __builtin_amdgcn_sched_barrier(0);
        if (KS == 1 || s < stages) {              // a part may have one stage less
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[kk & 1][j], fa[kk & 1][i],
                                                                acc[i][j], 0, 0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
#pragma unroll
    for (int i = 0; i * S::kThreads < BM; ++i)
      if (const int r = threadIdx.x + i * S::kThreads; r < BM) s_sa[r] = scale_a[i];
#pragma unroll
    for (int i = 0; i * S::kThreads < BN; ++i)
      if (const int r = threadIdx.x + i * S::kThreads; r < BN) {
        s_sw[r] = scale_w[i];
        s_bias[r] = bias[i];
      }
    wait_lds();
    meet();                                       // the scales are there, the stages' LDS is free
    const int64_t e_row0 = row0, e_col0 = col0;
    const int e_rows = rows, e_cols = cols;
    bool more = false;
    if (S::kStays) {
      at += gridDim.x;
      more = place(at);
      if (more) {
        issue(0);
        if (stages > 1) issue(1);
      }
    }
    if (KS > 1) {
      // the parts' sums meet in the first one's waves
      i32x4 *sums = reinterpret_cast<i32x4 *>(lds) + wave * (MT * NT * 4 * 64) + lane;
      constexpr int PART = WAVES * MT * NT * 4 * 64;
      static_assert((KS - 1) * PART * 16 <= KS * 2 * S::kStage, "sums in LDS");
      if (part > 0) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const i32x4 v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                               acc[i][j][4 * q + 3]};
              sums[(part - 1) * PART + ((i * NT + j) * 4 + q) * 64] = v;
            }
      }
      wait_lds();
      meet();
      if (part == 0) {
#pragma unroll
        for (int from = 0; from < KS - 1; ++from)
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const i32x4 v = sums[from * PART + ((i * NT + j) * 4 + q) * 64];
#pragma unroll
                for (int z = 0; z < 4; ++z) acc[i][j][4 * q + z] += v[z];
              }
      }
      wait_lds();
      meet();                                     // a wave's lines lie over others' sums
      if (part > 0) return;
    }

    // Epilogue, 64 bytes of 32 rows of the wave at a time through its own piece of
    // LDS: a lane has columns 8 q + 4 half + 0..3 of row l32.
    static_assert(S::kStays || S::kLines <= KS * 2 * S::kStage, "epilogue LDS");
    uint8_t *line = lines + wave * 32 * kLine;
    constexpr int W = GATED ? 32 : 64;            // output columns of the wave
    const int wcol = wn * W, left = e_cols - wcol;   // columns of the wave that exist
    auto value = [&](int i, int j, int q, float sa, float (&v)[4]) __attribute__((always_inline)) {
      const int n0 = wn * 64 + j * 32 + 8 * q + 4 * half, n1 = GATED ? n0 + 32 : n0;
      const floatx4 sg = *reinterpret_cast<const floatx4 *>(s_sw + n0);
      const floatx4 su = *reinterpret_cast<const floatx4 *>(s_sw + n1);
      const floatx4 bg = *reinterpret_cast<const floatx4 *>(s_bias + n0);
      const floatx4 bu = *reinterpret_cast<const floatx4 *>(s_bias + n1);
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        const int r = q * 4 + z;
        v[z] = finish<ACT>(acc[i][j][r], acc[i][1][r], sa, sg[z], su[z], bg[z], bu[z]);
      }
    };
    // the 32 rows' pieces of columns c.. from LDS, 16 bytes a lane: four lanes a row
    auto flush = [&](int m0, int c, auto *y) __attribute__((always_inline)) {
      constexpr int V = 16 / (int)sizeof(*y);
      wait_lds();                                 // the wave's own lines; its lanes run together
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = x * 16 + (lane >> 2), p = lane & 3, m = m0 + r;
        const u32x4 v = *reinterpret_cast<const u32x4 *>(line + r * kLine + p * 16);
        if (m < e_rows)
          store_cols(y + (e_row0 + m) * a.ld_y + e_col0 + wcol + c + p * V, left - c - p * V, v);
      }
      wait_lds();
    };
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int m0 = (wm * MT + i) * 32;
      const float sa = s_sa[m0 + l32];
#pragma unroll
      for (int j = 0; j < W / 32; ++j) {
        if (a.out_bf16) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float v[4];
            value(i, j, q, sa, v);
            uint2 w;
            w.x = (uint32_t)to_bf16_bits(v[0]) | (uint32_t)to_bf16_bits(v[1]) << 16;
            w.y = (uint32_t)to_bf16_bits(v[2]) | (uint32_t)to_bf16_bits(v[3]) << 16;
            write_lds(line + l32 * kLine + (8 * q + 4 * half) * 2, w);
          }
          flush(m0, j * 32, static_cast<uint16_t *>(a.y));
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              float v[4];
              value(i, j, 2 * h + q, sa, v);
              write_lds(line + l32 * kLine + (8 * q + 4 * half) * 4,
                        floatx4{v[0], v[1], v[2], v[3]});
            }
            flush(m0, j * 32 + h * 16, static_cast<float *>(a.y));
          }
        }
      }
    }
    if (!more) return;
  }
}

// ---------------------------------------------------------------------------
template <int MT, int ACT>
static hipError_t launch_rows(const Int8GemmArgs &a, hipStream_t st) {
  const int64_t out_n = a.N / (ACT != UFP4_ACT_NONE ? 2 : 1);
  hipLaunchKernelGGL((int8_rows_kernel<MT, ACT>),
                     dim3((unsigned)((out_n + 15) / 16), (unsigned)a.n_groups),
                     dim3(64 * kRowWaves), 0, st, a);
  return hipGetLastError();
}

// The dynamic-LDS limit is a per-device function attribute: set once on each
// device the kernel runs on (a bit per device id; concurrent first calls at worst
// both set it, which is harmless).
template <int WM, int WN, int MT, int KS, int ACT>
static hipError_t allow_lds(const void *kernel, size_t bytes) {
  static std::atomic<uint64_t> configured{0};
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
  if (bit != 0 && (configured.load(std::memory_order_acquire) & bit) != 0) return hipSuccess;
  e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == hipSuccess) configured.fetch_or(bit, std::memory_order_release);
  return e;
}

template <int WM, int WN, int MT, int KS, int ACT>
static hipError_t launch_tiles(const Int8GemmArgs &a, hipStream_t st) {
  using S = TileShape<WM, WN, MT, KS>;
  const int64_t out_n = a.N / (ACT != UFP4_ACT_NONE ? 2 : 1);
  const int64_t out = ACT != UFP4_ACT_NONE ? S::kBN / 2 : S::kBN;
  const int64_t tiles_n = (out_n + out - 1) / out;
  const int64_t tiles_m = (a.M + S::kBM - 1) / S::kBM + (a.goff ? a.n_groups : 0);
  const int64_t total = (tiles_m * tiles_n + kXcd - 1) / kXcd * kXcd;
  constexpr int64_t kMost = 1 << 22;              // tiles of a launch: below 2^32 threads
  auto *kernel = int8_tile_kernel<WM, WN, MT, KS, ACT>;
  hipError_t e = allow_lds<WM, WN, MT, KS, ACT>((const void *)kernel, S::kLds);
  if (e != hipSuccess) return e;
  const int64_t most = S::kStays ? kCus : kMost;
  for (int64_t first = 0; first < total; first += kMost) {
    const unsigned n = (unsigned)(total - first < most ? total - first : most);
    hipLaunchKernelGGL(kernel, dim3(n), dim3(S::kThreads), S::kLds, st, a, tiles_n, first);
    e = hipGetLastError();
    if (e != hipSuccess || S::kStays) return e;
  }
  return hipSuccess;
}

// Which tiles: those whose time, estimated from their number per CU at even groups,
// is least.  A CU holds one workgroup of 256 x 256, two of 128 x 128, three of 64 x
// 128, or one of those that split K; the last one to start costs as much as a full
// set.  A workgroup's start and end cost as much as the added stages of K.  Measured,
// us:
//                                  256x256 128x128 64x128 64x128/2 64x64/4
//   8192 x 2048 to 2 x 8192, gated     290     324    466      571     826
//   10000 x 2048 to 2 x 1408, gated,
//     32 groups                        115     116    137      187     258
//   24000 x 64 to 2 x 3648, gated,
//     32 groups                        120     130    186      373     775
//   3808 x 6065 to 2172, 8 groups       82      98    118      142     168
//   4000 x 4096 to 4096                 68      83     94      131     169
//   2000 x 4096 to 4096                 55      41     48       65      86
//   1500 x 4096 to 4096                 54      39     45       50      66
//   1000 x 4096 to 4096                 49      27     25       34      43
//   905 x 2560 to 2 x 768, gated        34      17     15       13      17
//   500 x 2048 to 2048                  28      13     10        9       8
//   200 x 4096 to 4096                  47      24     20       16      13
//   1000 x 6080 to 128                  65      28     20       18      14
template <int ACT>
static hipError_t launch_best_tiles(const Int8GemmArgs &a, hipStream_t st) {
  const int64_t per = (a.M + a.n_groups - 1) / a.n_groups;      // rows of an even group
  const double stages = (double)(a.kpad / kStageK);
  auto per_cu = [&](int64_t bm, int64_t bn) {
    return (double)((per + bm - 1) / bm * ((a.N + bn - 1) / bn) * a.n_groups) / kCus;
  };
  const double middle = per_cu(128, 128), small = per_cu(64, 128);
  const double pairs = std::floor(middle / 2.0), left = middle - 2.0 * pairs;
  const double whole = std::floor(small);
  const double t[5] = {
      std::ceil(per_cu(256, 256)) * 1.74 * (stages + 4.5) + 4.0,
      (pairs * 1.15 + (left <= 0.0 ? 0.0 : left <= 1.0 ? 0.95 : 1.1)) * (stages + 3.5),
      (small <= 1.0   ? 0.63
       : small <= 2.0 ? 0.81
                      : whole * 0.4 + (small > whole ? 0.85 : 0.0)) * (stages + 3.5),
      std::ceil(small) * 0.42 * (stages + 9.0),
      std::ceil(per_cu(64, 64)) * 0.29 * (stages + 12.5)};
  int best = 0;
  for (int i = 1; i < 5; ++i)
    if (t[i] < t[best]) best = i;
  switch (best) {
    case 0: return launch_tiles<2, 4, 4, 1, ACT>(a, st);
    case 1: return launch_tiles<2, 2, 2, 1, ACT>(a, st);
    case 2: return launch_tiles<2, 2, 1, 1, ACT>(a, st);
    case 3: return launch_tiles<2, 2, 1, 2, ACT>(a, st);
    default: return launch_tiles<2, 1, 1, 4, ACT>(a, st);
  }
}

template <int ACT>
static hipError_t int8_gemm(const Int8GemmArgs &a, hipStream_t st) {
  const int64_t rows = (a.M + a.n_groups - 1) / a.n_groups;
  const int64_t out_n = a.N / (ACT != UFP4_ACT_NONE ? 2 : 1);
  const int64_t groups16 = (out_n + 15) / 16 * a.n_groups;      // workgroups of the rows kernel
  // Up to 16 rows the rows kernel reads w at the memory's rate.  With more rows it
  // reads them in every workgroup, which pays while there are few (32 rows, 8192 to
  // 2048 columns: 13 us, tiles 22; 48 rows, 1024 to 2 x 2048: 5.0 and 6.0; 32 rows, 2048
  // to 2 x 8192: 10.1 and 10.1; 64 rows, 2048 to 2 x 4096: 8.6 and 8.1; 300 rows over 8
  // experts, 2048 to 2 x 1024: 14.5 and 12.3).  Where the rows of each group lie is known
  // on the GPU only, so both this rule and that of the tiles take the groups to be even.
  // An expert with more rows than that has its weights read again for every 16 of them, 3
  // us each at this size (2048 to 2 x 2048; even, half the rows with one expert, all: 512
  // rows over 32 experts 46, 72 and 100 us; 1024 over 64 113, 154 and 203; with tiles 1024
  // over 32 45, 53 and 18; 4096 over 8 42, 67 and 41).
  if (rows <= 16) return launch_rows<1, ACT>(a, st);
  if (rows <= 32 && groups16 <= 512) return launch_rows<2, ACT>(a, st);
  if (rows <= 64 && groups16 <= 256) return launch_rows<4, ACT>(a, st);
  return launch_best_tiles<ACT>(a, st);
}

template <typename T, int ACT>
static hipError_t launch_fused(const Int8GemmArgs &a, const Int8QuantArgs &q, hipStream_t st) {
  const int64_t out_n = a.N / (ACT != UFP4_ACT_NONE ? 2 : 1);
  hipLaunchKernelGGL((int8_fused_kernel<T, ACT>), dim3((unsigned)((out_n + 15) / 16)),
                     dim3(64 * kRowWaves), (size_t)(a.M * (a.kpad + 16)), st, a, q);
  return hipGetLastError();
}
template <typename T>
static hipError_t fused(const Int8GemmArgs &a, const Int8QuantArgs &q, hipStream_t st) {
  if (a.act == UFP4_ACT_NONE) return launch_fused<T, UFP4_ACT_NONE>(a, q, st);
  return a.act == UFP4_ACT_SILU ? launch_fused<T, UFP4_ACT_SILU>(a, q, st)
                                : launch_fused<T, UFP4_ACT_GELU>(a, q, st);
}
hipError_t launch_int8_linear(const Int8GemmArgs &a, const Int8QuantArgs &q, hipStream_t st) {
  if (a.M == 0) return hipSuccess;
  if (q.q == nullptr)
    return q.bf16 ? fused<uint16_t>(a, q, st) : fused<float>(a, q, st);
  const hipError_t e = launch_int8_quantize(q, st);
  return e == hipSuccess ? launch_int8_gemm(a, st) : e;
}

hipError_t launch_int8_gemm(const Int8GemmArgs &a, hipStream_t st) {
  if (a.M == 0) return hipSuccess;
  if (a.act == UFP4_ACT_NONE) return int8_gemm<UFP4_ACT_NONE>(a, st);
  return a.act == UFP4_ACT_SILU ? int8_gemm<UFP4_ACT_SILU>(a, st) : int8_gemm<UFP4_ACT_GELU>(a, st);
}

}  // namespace ufp4
