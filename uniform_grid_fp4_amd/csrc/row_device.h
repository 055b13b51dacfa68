// Rows held in registers, for the kernels that work row by row (gfx950): TPR
// threads (16 lanes, a wave, or a workgroup) hold a row as NV 16-byte vectors
// each.  TAIL: the row length is not a multiple of the vector.
#pragma once

#include "block_device.h"

namespace ufp4 {

// Sum / maximum over the TPR threads that hold a row: a DPP row, a wave, or the
// workgroup.
template <int TPR>
__device__ __forceinline__ float span_sum(float v, float *s) {
  if constexpr (TPR == 16) return row_sum(v);
  else return group_sum<TPR / 64>(v, s);
}
template <int TPR>
__device__ __forceinline__ uint32_t span_max(uint32_t v, uint32_t *s) {
  if constexpr (TPR == 16) return row_max(v);
  else return group_max<TPR / 64>(v, s);
}

constexpr int group_size(int tpr) { return tpr < 256 ? 256 : tpr; }
// Where the vector that begins at column c0 lies: with TAIL, one that passes the
// end of the row is taken back to end with it.  Its first c0 - start elements
// belong to another lane; they count in no sum, and both lanes store the same
// values there.  (Masked accesses, element by element in one lane, made the
// whole row wait: 16384 x 2047 bf16 backward 139 us, this way 55 us.)
template <bool TAIL, int V>
__device__ __forceinline__ int vec_start(int c0, int cols) {
  return TAIL ? min(c0, cols - V) : c0;
}
// Whether element j of the vector of c0 is another lane's.
template <bool TAIL, int V>
__device__ __forceinline__ bool elsewhere(int c0, int cols, int j) {
  return TAIL && vec_start<TAIL, V>(c0, cols) + j < c0;
}

template <int NV, typename T, bool TAIL>
struct RowVecs {
  static constexpr int V = Elem<T>::V;
  u32x4 v[NV];
  __device__ __forceinline__ void load(const T *p, int first, int step, int cols) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c0 = first + i * step;
      v[i] = c0 < cols
                 ? (u32x4)*reinterpret_cast<const u32x4_any *>(p + vec_start<TAIL, V>(c0, cols))
                 : u32x4(0);
    }
  }
};
template <typename T, bool TAIL>
__device__ __forceinline__ void row_store(T *p, int c0, int cols, u32x4 v, bool stream) {
  constexpr int V = Elem<T>::V;
  if (c0 < cols) store_as(p + vec_start<TAIL, V>(c0, cols), V, v, stream);
}

// The weights of one vector's columns: packed as the rows are when the types
// agree, FP32 otherwise.
template <typename T, typename W, bool TAIL>
struct WeightVec {
  static constexpr int V = Elem<T>::V;
  float f[V];
  __device__ __forceinline__ void load(const W *w, int c0, int cols) {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = 0.0f;
    if (c0 >= cols) return;
    constexpr int VW = Elem<W>::V;
    w += vec_start<TAIL, V>(c0, cols);
#pragma unroll
    for (int i = 0; i < V; i += VW) {
      float g[VW];
      Elem<W>::unpack(*reinterpret_cast<const u32x4_any *>(w + i), g);
#pragma unroll
      for (int j = 0; j < VW; ++j) f[i + j] = g[j];
    }
  }
  __device__ __forceinline__ void get(float (&g)[V]) const {
#pragma unroll
    for (int i = 0; i < V; ++i) g[i] = f[i];
  }
};
template <bool TAIL>
struct WeightVec<uint16_t, uint16_t, TAIL> {
  u32x4 v;
  __device__ __forceinline__ void load(const uint16_t *w, int c0, int cols) {
    v = c0 < cols
            ? (u32x4)*reinterpret_cast<const u32x4_any *>(w + vec_start<TAIL, 8>(c0, cols))
            : u32x4(0);
  }
  __device__ __forceinline__ void get(float (&g)[8]) const { Elem<uint16_t>::unpack(v, g); }
};

// A launch holds fewer than 2^32 threads; rows beyond the grid are looped over.
inline unsigned row_grid(int64_t rows) { return (unsigned)(rows < (1 << 20) ? rows : (1 << 20)); }

// Threads per row and vectors per thread for a row of so many 16-byte vectors
// of v elements: 16 lanes take up to 16, a wave up to 4 per lane, longer rows a workgroup
// of 256 to 1024 threads with up to 4 each; (0, 0) beyond, and for less than a vector (the looping
// kernels).
// 1024 threads leave 128 registers each, too few for bf16's backward.
struct RowShape {
  int tpr, nv;
};
inline RowShape row_shape(int64_t cols, int v) {
  constexpr RowShape kShapes[] = {{16, 1},  {64, 1},  {64, 2},  {64, 3},  {64, 4},  {256, 2},
                                  {256, 3}, {256, 4}, {512, 3}, {512, 4}, {1024, 3}};
  if (cols < v) return {0, 0};
  const int64_t n = (cols + v - 1) / v;
  for (const RowShape &s : kShapes)
    if (n <= s.tpr * s.nv && (s.tpr < 1024 || v == Elem<float>::V)) return s;
  return {0, 0};
}
inline int64_t row_groups(int64_t rows, int tpr) {
  const int per = group_size(tpr) / tpr;
  return (rows + per - 1) / per;
}

#define UFP4_LONG_SHAPES(F) F(256, 2) F(256, 3) F(256, 4) F(512, 3) F(512, 4)
#define UFP4_FWD_SHAPES(F) F(16, 1) F(64, 1) F(64, 2) F(64, 3) F(64, 4) UFP4_LONG_SHAPES(F)

}  // namespace ufp4
