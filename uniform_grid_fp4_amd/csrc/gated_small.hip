// The gated product act(x Wg^T) * (x Wu^T) on 4-bit operands for few output
// tiles (gfx950): what gemm.hip's gated kernel computes, for problems whose 128 x
// 64 tiles would leave most of the GPU idle and run along K one stage after the
// other.
//   g = (1/L^2) sum_kb sa sb P_kb,  P_kb = sum over the 16 elements of block kb
//
// A workgroup has 32 rows and 32 columns of either projection, and its eight
// waves split K: each takes every eighth run of four blocks, straight from
// memory into registers, and expands its own nibbles.  Per block the arithmetic is
// gemm.hip's: two FP8 products, one FP32 outer product of the scales, one FMA per
// output.  The eight partial sums meet in LDS and are added in the order of the
// waves.  Nothing is shared between waves before that, so there are no barriers
// along K, for 4 to 8 times the reads of the L2.  Bound by the cache lines that its
// loads touch (192 per wave and run, every row another line): reading each row's
// run once per wave and exchanging words between the halves of the wave, instead of
// in both halves, took 512 x 2048 columns, K = 2048, from 42 to 35 us.  Two workgroups
// fit a CU, with at most 128 registers: 29 us; 8 rows over 32 experts of 5120 columns, K
// = 64, 27 -> 16; 1266 x 1143, K = 384, 21 -> 14.5; 14 rows over 8 experts of 2355 columns, K
// = 5793, 53 us either way (164 MB, 3.1 TB/s).  Loading a run ahead would spill.
#include "act_device.h"
#include "block_device.h"
#include "group_device.h"
#include "ufp4_device.h"
#include "ufp4_kernels.h"

namespace ufp4 {

typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef float floatx32 __attribute__((ext_vector_type(32)));
typedef uint32_t u32x4_dword __attribute__((ext_vector_type(4), aligned(4)));

constexpr int kSmallWaves = 8;
constexpr int kSmallRows = 32, kSmallCols = 32;

// The products of one block: this lane's half of the block's nibbles of its row
// of x, of the gate's and of the up projection's, its row's scale, and the scale
// of its column (lanes 0-31 the gate's, 32-63 the up projection's).
template <int GRID>
__device__ __forceinline__ void block_product(uint32_t x, uint32_t g, uint32_t u, float sx, float sw,
                                              floatx16 (&acc)[2]) {
  floatx16 zero;
#pragma unroll
  for (int r = 0; r < 16; ++r) zero[r] = 0.0f;
  floatx32 zero32;
#pragma unroll
  for (int r = 0; r < 32; ++r) zero32[r] = 0.0f;
  const long fx = __builtin_bit_cast(long, nib8_to_fp8<GRID>(x));
  const long fg = __builtin_bit_cast(long, nib8_to_fp8<GRID>(g));
  const long fu = __builtin_bit_cast(long, nib8_to_fp8<GRID>(u));
  const floatx32 S = __builtin_amdgcn_mfma_f32_32x32x1f32(sx, sw, zero32, 1, 0, 0);
  const floatx16 p0 = __builtin_amdgcn_mfma_f32_32x32x16_fp8_fp8(fx, fg, zero, 0, 0, 0);
#pragma unroll
  for (int r = 0; r < 16; ++r) acc[0][r] = fmaf(S[r], p0[r], acc[0][r]);
  const floatx16 p1 = __builtin_amdgcn_mfma_f32_32x32x16_fp8_fp8(fx, fu, zero, 0, 0, 0);
#pragma unroll
  for (int r = 0; r < 16; ++r) acc[1][r] = fmaf(S[16 + r], p1[r], acc[1][r]);
}

// Four blocks of a row.  A lane of the wave's lower half loads the first two, its
// counterpart in the upper half the other two: 32 rows and 32 bytes of each, in
// one access.  Exchanging the upper half of a block's first word with the lower half
// of its second gives both halves their own four bytes of the first pair's block
// and of the second's.
struct FourBlocks {
  uint32_t w[4];
  __device__ __forceinline__ explicit FourBlocks(u32x4_dword v) {
    const auto a = __builtin_amdgcn_permlane32_swap(v[0], v[1], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(v[2], v[3], false, false);
    w[0] = a[0];
    w[1] = b[0];
    w[2] = a[1];
    w[3] = b[1];
  }
};

template <int GRID>
__global__ __launch_bounds__(64 * kSmallWaves) __attribute__((amdgpu_waves_per_eu(4, 4))) void
gated_small_kernel(const GemmArgs a, int64_t tiles_n) {
  __shared__ float s_acc[kSmallWaves][2][kSmallRows * kSmallCols];
  const GroupTile t = group_tile(a.goff, a.n_groups, a.M, kSmallRows, tiles_n,
                                 [](int64_t) { return (int64_t)blockIdx.x; });
  if (t.e < 0) return;
  // row tiles next to each other share w's rows
  const int64_t tn = t.local / t.tiles_m, tm = t.local - tn * t.tiles_m;
  const int64_t row0 = t.row0 + tm * kSmallRows, col0 = tn * kSmallCols;
  const int rows = (int)min((int64_t)kSmallRows, t.rows - tm * kSmallRows);
  const int cols = (int)min((int64_t)kSmallCols, a.N - col0);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l32 = lane & 31, half = lane >> 5;
  const int nkb = (int)(a.kpad / 16);
  // Rows and columns past the end repeat the last one; they are not stored.  Lanes
  // differ by 32-bit offsets from bases in scalar registers, but for the scales of w:
  // a half has the gate's and a half the up projection's.
  const int64_t w_row = (int64_t)t.e * 2 * a.N + col0;
  const uint8_t *qx = a.a_codes + row0 * (nkb * 8), *qg = a.b_codes + w_row * (nkb * 8);
  const uint8_t *qu = qg + a.N * (nkb * 8);
  const uint32_t rx = min(l32, rows - 1) * nkb, rw = min(l32, cols - 1) * nkb;
  const float *sx = a.a_scales + row0 * nkb;
  const float *sw = a.b_scales + (w_row + half * a.N) * nkb + rw;

  floatx16 acc[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[i][r] = 0.0f;
  const int runs = nkb / 4;                       // of four blocks
  for (int i = wave; i < runs; i += kSmallWaves) {
    const u32x4_dword vx = *reinterpret_cast<const u32x4_dword *>(qx + i * 32 + (rx * 8 + half * 16));
    const u32x4_dword vg = *reinterpret_cast<const u32x4_dword *>(qg + i * 32 + (rw * 8 + half * 16));
    const u32x4_dword vu = *reinterpret_cast<const u32x4_dword *>(qu + i * 32 + (rw * 8 + half * 16));
    const u32x4_dword fx = *reinterpret_cast<const u32x4_dword *>(sx + i * 4 + rx);
    const u32x4_dword fw = *reinterpret_cast<const u32x4_dword *>(sw + i * 4);
    __builtin_amdgcn_sched_barrier(0);            // all loads go out before the products
    const FourBlocks x(vx), g(vg), u(vu);
#pragma unroll
    for (int b = 0; b < 4; ++b)
      block_product<GRID>(x.w[b], g.w[b], u.w[b], __uint_as_float(fx[b]), __uint_as_float(fw[b]),
                          acc);
  }
  // the last blocks, one to a wave
  if (const int k = runs * 4 + wave; k < nkb)
    block_product<GRID>(*reinterpret_cast<const uint32_t *>(qx + k * 8 + (rx * 8 + half * 4)),
                        *reinterpret_cast<const uint32_t *>(qg + k * 8 + (rw * 8 + half * 4)),
                        *reinterpret_cast<const uint32_t *>(qu + k * 8 + (rw * 8 + half * 4)),
                        sx[k + rx], sw[k], acc);
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r)
      s_acc[wave][i][(8 * (r >> 2) + 4 * half + (r & 3)) * kSmallCols + l32] = acc[i][r];
  __syncthreads();
  constexpr float l2 = (GRID == kGridUniform) ? 49.0f : (GRID == kGridE2M1) ? 144.0f : 16.0f;
  for (int i = threadIdx.x; i < kSmallRows * kSmallCols; i += 64 * kSmallWaves) {
    const int m = i / kSmallCols, n = i % kSmallCols;
    if (m >= rows || n >= cols) continue;
    float v[2];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      float sum = s_acc[0][p][i];
#pragma unroll
      for (int w = 1; w < kSmallWaves; ++w) sum += s_acc[w][p][i];
      v[p] = sum * (1.0f / l2);
    }
    const float y = v[1] * (a.act == UFP4_ACT_SILU ? act_value<UFP4_ACT_SILU>(v[0])
                                                   : act_value<UFP4_ACT_GELU>(v[0]));
    const int64_t row = row0 + m, col = col0 + n;
    if (a.out_bf16) {
      static_cast<uint16_t *>(a.c)[row * a.ldc + col] = to_bf16_bits(y);
      if (a.gu == nullptr) continue;
      uint16_t *p = static_cast<uint16_t *>(a.gu) + row * a.ld_gu + col;
      p[0] = to_bf16_bits(v[0]);
      p[a.N] = to_bf16_bits(v[1]);
    } else {
      static_cast<float *>(a.c)[row * a.ldc + col] = y;
      if (a.gu == nullptr) continue;
      float *p = static_cast<float *>(a.gu) + row * a.ld_gu + col;
      p[0] = v[0];
      p[a.N] = v[1];
    }
  }
}

template <int GRID>
static hipError_t small_t(const GemmArgs &g, unsigned blocks, int64_t tiles_n, hipStream_t st) {
  hipLaunchKernelGGL((gated_small_kernel<GRID>), dim3(blocks), dim3(64 * kSmallWaves), 0, st, g,
                     tiles_n);
  return hipGetLastError();
}
hipError_t launch_gated_small(const GemmArgs &g, hipStream_t st) {
  const int64_t tiles_n = (g.N + kSmallCols - 1) / kSmallCols;
  const int64_t tiles_m = (g.M + kSmallRows - 1) / kSmallRows + (g.goff != nullptr ? g.n_groups : 0);
  // the caller's rule keeps this below 2^21 workgroups
  const unsigned blocks = (unsigned)(tiles_m * tiles_n);
  if (g.grid == kGridUniform) return small_t<kGridUniform>(g, blocks, tiles_n, st);
  if (g.grid == kGridE2M1) return small_t<kGridE2M1>(g, blocks, tiles_n, st);
  return small_t<kGridE2M1Max2>(g, blocks, tiles_n, st);
}

}  // namespace ufp4
