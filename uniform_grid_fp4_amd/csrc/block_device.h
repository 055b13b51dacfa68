// Device helpers of the block operators (gfx950): 16-byte vectors of bf16 or
// FP32 elements at any element alignment, and fixed-order reductions.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ufp4 {

// gfx950 global memory takes 16-byte accesses at any address (the HSA ABI
// runs with unaligned access enabled), so a row may start at any element.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

__device__ __forceinline__ uint16_t to_bf16_bits(float f) {
  return __builtin_bit_cast(uint16_t, (__bf16)f);       // nearest even, NaN kept
}

// A type's vector: V elements in 16 bytes, unpacked to FP32 and packed again.
template <typename T>
struct Elem;
template <>
struct Elem<uint16_t> {       // bf16 bit patterns
  static constexpr int V = 8;
  __device__ static __forceinline__ float get(uint16_t b) {
    return __uint_as_float((uint32_t)b << 16);
  }
  __device__ static __forceinline__ uint16_t put(float f) { return to_bf16_bits(f); }
  __device__ static __forceinline__ void unpack(u32x4 w, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ static __forceinline__ u32x4 pack(const float (&f)[8]) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = (uint32_t)to_bf16_bits(f[2 * i]) | (uint32_t)to_bf16_bits(f[2 * i + 1]) << 16;
    return w;
  }
};
template <>
struct Elem<float> {
  static constexpr int V = 4;
  __device__ static __forceinline__ float get(float f) { return f; }
  __device__ static __forceinline__ float put(float f) { return f; }
  __device__ static __forceinline__ void unpack(u32x4 w, float (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(w[i]);
  }
  __device__ static __forceinline__ u32x4 pack(const float (&f)[4]) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(f[i]);
    return w;
  }
};

// V elements from p, of which the first n exist (the others read as zero).
template <typename T>
__device__ __forceinline__ u32x4 load_vec(const T *p, int64_t n) {
  constexpr int V = Elem<T>::V;
  if (n >= V) return *reinterpret_cast<const u32x4_any *>(p);
  float f[V];
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = i < n ? Elem<T>::get(p[i]) : 0.0f;
  return Elem<T>::pack(f);
}
template <typename T>
__device__ __forceinline__ void store_vec(T *p, int64_t n, u32x4 w) {
  constexpr int V = Elem<T>::V;
  if (n >= V) {
    *reinterpret_cast<u32x4_any *>(p) = w;
    return;
  }
  float f[V];
  Elem<T>::unpack(w, f);
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (i < n) p[i] = Elem<T>::put(f[i]);
}

// Streaming accesses, for tensors that the 256 MB memory-side cache cannot
// hold until their next reader anyway: the caches stay with what is used again
// (6144 columns, 16384 x 8 rows: dispatch 354 -> 309 us).  A smaller output is
// left to the caches for that reader (a norm of 32768 x 2048 and a reader of
// its output: 143 us, with streaming stores 147 us).
constexpr int64_t kStreamBytes = int64_t(256) << 20;
template <typename T>
__device__ __forceinline__ u32x4 load_as(const T *p, int64_t n, bool stream) {
  if (stream && n >= Elem<T>::V) {
    // The empty statements keep the compiler from making one access, without
    // the hint, of the two branches' (here and below).
    asm volatile("");
    const u32x4 w = __builtin_nontemporal_load(reinterpret_cast<const u32x4_any *>(p));
    asm volatile("");
    return w;
  }
  return load_vec(p, n);
}
template <typename T>
__device__ __forceinline__ void store_as(T *p, int64_t n, u32x4 w, bool stream) {
  if (stream && n >= Elem<T>::V) {
    asm volatile("");
    __builtin_nontemporal_store((u32x4_any)w, reinterpret_cast<u32x4_any *>(p));
    asm volatile("");
  } else {
    store_vec(p, n, w);
  }
}

// Sum / maximum over the 16 lanes of a DPP row, in every lane, by rotations of
// 8, 4, 2 and 1: each step adds two values that both lanes of a pair hold, so
// all lanes get the same bits.
template <int ROT>
__device__ __forceinline__ float row_rotate(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp(
      (int)__float_as_uint(v), 0x120 + ROT, 0xF, 0xF, true));
}
__device__ __forceinline__ float row_sum(float v) {
  v += row_rotate<8>(v);
  v += row_rotate<4>(v);
  v += row_rotate<2>(v);
  v += row_rotate<1>(v);
  return v;
}
template <int ROT>
__device__ __forceinline__ uint32_t row_rotate(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x120 + ROT, 0xF, 0xF, true);
}
// fmaxf drops a NaN operand; callers that must keep NaN test for it apart.
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, row_rotate<8>(v));
  v = fmaxf(v, row_rotate<4>(v));
  v = fmaxf(v, row_rotate<2>(v));
  v = fmaxf(v, row_rotate<1>(v));
  return v;
}
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  v = max(v, row_rotate<8>(v));
  v = max(v, row_rotate<4>(v));
  v = max(v, row_rotate<2>(v));
  return max(v, row_rotate<1>(v));
}
// The four rows of a wave: v_permlane16_swap_b32 of a value with itself gives
// every pair of rows the first's and the second's value, v_permlane32_swap_b32
// every pair of halves.
struct Pair {
  uint32_t a, b;
};
__device__ __forceinline__ Pair row_pairs(uint32_t v) {
  const auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  return {p[0], p[1]};
}
__device__ __forceinline__ Pair half_pairs(uint32_t v) {
  const auto p = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return {p[0], p[1]};
}
__device__ __forceinline__ float rows_sum(float v) {
  Pair p = row_pairs(__float_as_uint(v));
  v = __uint_as_float(p.a) + __uint_as_float(p.b);
  p = half_pairs(__float_as_uint(v));
  return __uint_as_float(p.a) + __uint_as_float(p.b);
}
__device__ __forceinline__ float lanes_sum(float v) { return rows_sum(row_sum(v)); }
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  Pair p = row_pairs(row_max(v));
  p = half_pairs(max(p.a, p.b));
  return max(p.a, p.b);
}
__device__ __forceinline__ double lanes_sum(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// Sum / maximum over a workgroup of WAVES waves, in every thread: the waves'
// results go through s[0..WAVES) and are taken in wave order.  The caller
// separates two uses of the same s with a barrier.
template <int WAVES>
__device__ __forceinline__ float group_sum(float v, float *s) {
  v = lanes_sum(v);
  if (WAVES == 1) return v;
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  float t = s[0];
#pragma unroll
  for (int i = 1; i < WAVES; ++i) t += s[i];
  return t;
}
template <int WAVES>
__device__ __forceinline__ uint32_t group_max(uint32_t v, uint32_t *s) {
  v = lanes_max(v);
  if (WAVES == 1) return v;
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  uint32_t t = s[0];
#pragma unroll
  for (int i = 1; i < WAVES; ++i) t = max(t, s[i]);
  return t;
}

}  // namespace ufp4
