// A row's scale and codes in int8 (gfx950), for the quantizer and for the product
// that quantizes its few rows itself.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ufp4 {

// What the row's largest |x| gives.  The maximum is taken over the bits of |x|
// as unsigned numbers, where infinities and NaN are the largest: either makes
// the scale NaN and the codes zero.  The reciprocal leaves the normal numbers at
// either end, so rows beyond 2^64 or below 2^-64 are moved by 2^64 first (exact,
// but for elements that are nothing next to the largest).
struct Int8Scale {
  float scale, lift, inv;
};
__device__ __forceinline__ Int8Scale int8_scale(uint32_t top_bits) {
  const float top = __uint_as_float(top_bits);
  if (top_bits >= 0x7F800000u) return {__uint_as_float(0x7FC00000u), 1.0f, 0.0f};
  Int8Scale s;
  s.scale = top / 127.0f;
  s.lift = top < 0x1p-64f ? 0x1p64f : top > 0x1p64f ? 0x1p-64f : 1.0f;
  s.inv = top > 0.0f ? 127.0f * (1.0f / (top * s.lift)) : 0.0f;
  return s;
}
// Four codes of a row in one word; |x| <= top gives at most 127 (1 + 2^-23),
// which rounds to 127.  Where the scale is NaN, 0 for every element: the product
// with zero may be NaN and is not converted.
__device__ __forceinline__ uint32_t int8x4(const float *x, Int8Scale s) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float t = x[i] * s.lift * s.inv;
    w |= ((uint32_t)(int)rintf(t == t ? t : 0.0f) & 0xFFu) << (8 * i);
  }
  return w;
}

}  // namespace ufp4
