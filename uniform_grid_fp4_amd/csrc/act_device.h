// The activations of gated products and their slopes, in FP32 (gfx950).
//   silu(g) = g p,  silu'(g) = p (1 + g (1 - p)),  p = 1 / (1 + exp(-g))
//   gelu(g) = g c,  gelu'(g) = c + g exp(-g^2 / 2) / sqrt(2 pi),
//   c = erfc(-g / sqrt 2) / 2   (no cancellation where 1 + erf would lose c)
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/ufp4_ffn.h"

namespace ufp4 {

struct ActPair {
  float value, slope;
};

// 1 / x to nearest but for a last bit: the hardware's reciprocal (within one
// step) and one Newton step.  x in [1, inf].
__device__ __forceinline__ float recip(float x) {
  const float r = __builtin_amdgcn_rcpf(x);
  const float e = __builtin_fmaf(-x, r, 1.0f);
  return x < 0x1p126f ? __builtin_fmaf(e, r, r) : r;
}

template <int ACT>
__device__ __forceinline__ float act_value(float g) {
  if (ACT == UFP4_ACT_SILU) return g * recip(1.0f + expf(-g));
  return g * (0.5f * erfcf(-0.70710678118654752f * g));
}

template <int ACT>
__device__ __forceinline__ ActPair act_pair(float g) {
  if (ACT == UFP4_ACT_SILU) {
    const float p = recip(1.0f + expf(-g));
    return {g * p, p * (1.0f + g * (1.0f - p))};
  }
  const float c = 0.5f * erfcf(-0.70710678118654752f * g);
  return {g * c, c + g * (0.39894228040143268f * expf(-0.5f * g * g))};
}

}  // namespace ufp4
