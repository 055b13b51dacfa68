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

// p = 1 / (1 + exp(-g)) within 4 steps.  exp(-g) = 2^n 2^f with -g log2(e) = n +
// f, f taken from the product's two halves (log2(e) as two floats), so that no
// digit is lost in a large g; the exponential and the reciprocal are the
// hardware's, within a step.  Beyond 104 either way p is 1 or 0 (or NaN).
__device__ __forceinline__ float sigmoid(float g) {
  const float c = __builtin_amdgcn_fmed3f(g, -104.0f, 104.0f);
  const float n = __builtin_rintf(c * -1.4426950216293335f);
  float f = __builtin_fmaf(c, -1.4426950216293335f, -n);
  f = __builtin_fmaf(c, -1.925963e-8f, f);
  const float e = __builtin_ldexpf(__builtin_amdgcn_exp2f(f), (int)n);
  return __builtin_amdgcn_rcpf(1.0f + e);
}

template <int ACT>
__device__ __forceinline__ float act_value(float g) {
  if (ACT == UFP4_ACT_SILU) return g * sigmoid(g);
  return g * (0.5f * erfcf(-0.70710678118654752f * g));
}

template <int ACT>
__device__ __forceinline__ ActPair act_pair(float g) {
  if (ACT == UFP4_ACT_SILU) {
    const float p = sigmoid(g);
    return {g * p, p * (1.0f + g * (1.0f - p))};
  }
  const float c = 0.5f * erfcf(-0.70710678118654752f * g);
  return {g * c, c + g * (0.39894228040143268f * expf(-0.5f * g * g))};
}

}  // namespace ufp4
