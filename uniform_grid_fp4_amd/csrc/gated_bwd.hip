// Backward pass of a gated product y = act(g) * u (gfx950):
//   dg = dy u act'(g),  du = dy act(g)
// from dy [rows, cols] and gu = (g | u) [rows, 2 cols] into dgu = (dg | du), dY
// of the two projections as one product.  About 25 operations and 10 bytes per
// element in bf16: bound by memory.  8192 x 8192 silu 106 us (671 MB, 6.3 TB/s, partly from
// the 256 MB cache), 98304 x 1408 237 us (1384 MB, 5.8 TB/s).
#include "act_device.h"
#include "block_device.h"
#include "ffn_kernels.h"

namespace ufp4 {

// The vectors of all rows in one sequence, `vecs` to a row, 256 to a workgroup and
// turn: with workgroups of one row's vectors 24338 x 528, gelu, took 35 us instead of 24,
// 24338 x 529 39 instead of 31 (23 us at the memory's rate; rows of odd length
// cost unaligned stores).  A vector is read whole before it is written: dgu may be gu.
template <typename T, int ACT>
__global__ __launch_bounds__(256) void gated_bwd_kernel(const GatedBwdArgs a, int vecs) {
  constexpr int V = Elem<T>::V;
  const int64_t total = a.rows * vecs;
  for (int64_t at = (int64_t)blockIdx.x * 256; at < total; at += (int64_t)gridDim.x * 256) {
    const int64_t row0 = at / vecs;               // wave-uniform; what is left fits 32 bits
    const unsigned in = (unsigned)(at - row0 * vecs) + threadIdx.x;
    const int64_t row = row0 + in / (unsigned)vecs;
    if (row >= a.rows) return;
    const int64_t c = (int64_t)(in % (unsigned)vecs) * V, left = a.cols - c;
    const T *gu = static_cast<const T *>(a.gu) + row * a.ld_gu + c;
    T *out = static_cast<T *>(a.dgu) + row * 2 * a.cols + c;
    float g[V], u[V], d[V];
    const u32x4 vg = load_vec(gu, left), vu = load_vec(gu + a.cols, left);
    const u32x4 vd = load_vec(static_cast<const T *>(a.dy) + row * a.ld_dy + c, left);
    Elem<T>::unpack(vg, g);
    Elem<T>::unpack(vu, u);
    Elem<T>::unpack(vd, d);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const ActPair p = act_pair<ACT>(g[j]);
      g[j] = d[j] * u[j] * p.slope;
      u[j] = d[j] * p.value;
    }
    store_as(out, left, Elem<T>::pack(g), a.stream);
    store_as(out + a.cols, left, Elem<T>::pack(u), a.stream);
  }
}

template <typename T>
static hipError_t gated_bwd(GatedBwdArgs a, hipStream_t st) {
  if (a.rows == 0) return hipSuccess;
  a.stream = 2 * a.rows * a.cols * (int64_t)sizeof(T) >= kStreamBytes;
  constexpr int V = Elem<T>::V;
  const int vecs = (int)((a.cols + V - 1) / V);
  const int64_t turns = (a.rows * vecs + 255) / 256;
  constexpr int64_t kMost = 1 << 20;
  const dim3 grid((unsigned)(turns < kMost ? turns : kMost));
  if (a.act == UFP4_ACT_SILU)
    hipLaunchKernelGGL((gated_bwd_kernel<T, UFP4_ACT_SILU>), grid, dim3(256), 0, st, a, vecs);
  else
    hipLaunchKernelGGL((gated_bwd_kernel<T, UFP4_ACT_GELU>), grid, dim3(256), 0, st, a, vecs);
  return hipGetLastError();
}

hipError_t launch_gated_bwd(const GatedBwdArgs &a, hipStream_t st) {
  return a.bf16 ? gated_bwd<uint16_t>(a, st) : gated_bwd<float>(a, st);
}

}  // namespace ufp4
