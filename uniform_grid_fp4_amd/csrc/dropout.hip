// Dropout from a counter-based generator (gfx950):
//   y = residual + (keep ? x * scale : 0)
// The mask is never stored: both passes draw it from Philox4x32-10, keyed by
// the seed and counted by (row, eight columns, offset), one call for eight
// elements of 16 bits each.  Per element a call's 20 wide multiplies and 20
// three-input xors come to 5 instructions, next to some 6 for the element
// itself and 4 to 12 bytes: bound by memory, with the vector unit about half
// busy at bf16.  32768 x 6144 bf16: onto a residual 187 us (1208 MB, 6.5 TB/s), alone (as
// in the backward pass) 138 us (805 MB, 5.8 TB/s); 257 x 1411 FP32 3.4 us.
#include "block_device.h"
#include "ffn_kernels.h"
#include "ufp4_device.h"

namespace ufp4 {

constexpr int kGroup = 8;                        // columns that share a call

// n / d for n below 2^31 by a multiplication: m = floor(2^(31 + s) / d) + 1
// with 2^s >= d, so that n m / 2^(31 + s) lies in [n / d, n / d + 1 / d).
struct Divisor {
  uint32_t m, s, d;
};
static Divisor divisor(uint32_t d) {
  uint32_t s = 0;
  while (((uint64_t)1 << s) < d) ++s;
  return {(uint32_t)((((uint64_t)1 << (31 + s)) / d) + 1), s, d};
}
__device__ __forceinline__ uint32_t divided(uint32_t n, Divisor v) {
  return (uint32_t)(((uint64_t)n * v.m) >> 31 >> v.s);
}

// The first n of the eight elements at p, in pieces of 4, 2 and 1 (one lane in a
// row has fewer than eight, and its wave waits for it).
template <typename T>
struct Group;
template <>
struct Group<uint16_t> {
  u32x4 v;
  __device__ __forceinline__ void load(const uint16_t *p, int n, bool stream) {
    if (n >= 8) {
      v = load_as(p, 8, stream);
      return;
    }
    typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
    typedef uint32_t u32_any __attribute__((aligned(2)));
    uint32_t w[4] = {0, 0, 0, 0};
    int at = 0;
    if (n & 4) {
      const u32x2_any t = *reinterpret_cast<const u32x2_any *>(p);
      w[0] = t[0];
      w[1] = t[1];
      at = 4;
    }
    if (n & 2) {
      const uint32_t t = *reinterpret_cast<const u32_any *>(p + at);
      if (at) w[2] = t; else w[0] = t;
      at += 2;
    }
    if (n & 1) {
      const uint32_t t = p[at];
      if (at == 6) w[3] = t; else if (at == 4) w[2] = t; else if (at == 2) w[1] = t; else w[0] = t;
    }
    v = u32x4{w[0], w[1], w[2], w[3]};
  }
  __device__ __forceinline__ void get(float (&f)[8]) const { Elem<uint16_t>::unpack(v, f); }
  __device__ __forceinline__ static void store(uint16_t *p, int n, const float (&f)[8],
                                               bool stream) {
    const u32x4 v = Elem<uint16_t>::pack(f);
    if (n >= 8) {
      store_as(p, 8, v, stream);
      return;
    }
    typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
    typedef uint32_t u32_any __attribute__((aligned(2)));
    int at = 0;
    if (n & 4) {
      *reinterpret_cast<u32x2_any *>(p) = u32x2_any{v[0], v[1]};
      at = 4;
    }
    if (n & 2) {
      *reinterpret_cast<u32_any *>(p + at) = at ? v[2] : v[0];
      at += 2;
    }
    if (n & 1) p[at] = (uint16_t)(at == 6 ? v[3] : at == 4 ? v[2] : at == 2 ? v[1] : v[0]);
  }
};
template <>
struct Group<float> {
  float v[8];
  __device__ __forceinline__ void load(const float *p, int n, bool stream) {
    if (n >= 8) {
      float lo[4], hi[4];
      Elem<float>::unpack(load_as(p, 4, stream), lo);
      Elem<float>::unpack(load_as(p + 4, 4, stream), hi);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = lo[i];
        v[4 + i] = hi[i];
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : 0.0f;
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = v[i];
  }
  __device__ __forceinline__ static void store(float *p, int n, const float (&f)[8],
                                               bool stream) {
    if (n >= 8) {
      const float lo[4] = {f[0], f[1], f[2], f[3]}, hi[4] = {f[4], f[5], f[6], f[7]};
      store_as(p, 4, Elem<float>::pack(lo), stream);
      store_as(p + 4, 4, Elem<float>::pack(hi), stream);
      return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = f[i];
  }
};

// Groups [0, n) of the rows from row0 on, one per thread and turn; n < 2^31.
template <typename T>
__global__ __launch_bounds__(256) void dropout_kernel(const DropoutArgs a, int64_t row0,
                                                      uint32_t n, Divisor per_row) {
  const uint64_t offset = a.offset + (a.d_offset != nullptr ? (uint64_t)*a.d_offset : 0);
  const T *x = static_cast<const T *>(a.x), *res = static_cast<const T *>(a.res);
  T *y = static_cast<T *>(a.y);
  for (uint32_t i = blockIdx.x * 256u + threadIdx.x; i < n; i += gridDim.x * 256u) {
    const uint32_t r = divided(i, per_row);
    const int64_t row = row0 + r;
    const int64_t c = (int64_t)(i - r * per_row.d) * kGroup;
    const int left = (int)min((int64_t)kGroup, a.cols - c);
    Group<T> gx, gr;
    gx.load(x + row * a.ld_x + c, left, a.stream);
    if (res != nullptr) gr.load(res + row * a.ld_res + c, left, a.stream);
    float f[8], g[8];
    gx.get(f);
    if (a.limit != 0) {
      const uint64_t at = (uint64_t)row0 * per_row.d + i;
      const U32x4 bits = philox4x32_10((uint32_t)at, (uint32_t)(at >> 32), (uint32_t)offset,
                                       (uint32_t)(offset >> 32), (uint32_t)a.seed,
                                       (uint32_t)(a.seed >> 32));
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t u = j & 1 ? bits.w[j / 2] >> 16 : bits.w[j / 2] & 0xFFFFu;
        f[j] = u >= a.limit ? f[j] * a.scale : 0.0f;
      }
    }
    if (res != nullptr) {
      gr.get(g);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] += g[j];
    }
    Group<T>::store(y + row * a.cols + c, left, f, a.stream);
  }
}

template <typename T>
static hipError_t dropout(DropoutArgs a, hipStream_t st) {
  a.stream = a.rows * a.cols * (int64_t)sizeof(T) >= kStreamBytes;
  const int64_t groups = (a.cols + kGroup - 1) / kGroup;
  const Divisor d = divisor((uint32_t)groups);
  // so many rows a launch that their groups, and a step beyond, stay below 2^31
  const int64_t per = ((int64_t(1) << 30) + groups - 1) / groups;
  for (int64_t row0 = 0; row0 < a.rows; row0 += per) {
    const int64_t rows = a.rows - row0 < per ? a.rows - row0 : per;
    const int64_t n = rows * groups;
    const int64_t blocks = (n + 255) / 256;
    const unsigned grid = (unsigned)(blocks < 65536 ? blocks : 65536);
    hipLaunchKernelGGL((dropout_kernel<T>), dim3(grid), dim3(256), 0, st, a, row0, (uint32_t)n, d);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_dropout(const DropoutArgs &a, hipStream_t st) {
  return a.bf16 ? dropout<uint16_t>(a, st) : dropout<float>(a, st);
}

}  // namespace ufp4
