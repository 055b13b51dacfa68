// The activations of gated products and their slopes, in FP32 (gfx950).
//   silu(g) = g p,  silu'(g) = p (1 + g (1 - p)),  p = 1 / (1 + exp(-g))
//   gelu(g) = g c,  gelu'(g) = c + g exp(-g^2 / 2) / sqrt(2 pi),
//   c = erfc(-g / sqrt 2) / 2   (relative accuracy kept where 1 + erf would lose c)
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/ufp4_ffn.h"

namespace ufp4 {

struct ActPair {
  float value, slope;
};

// p = 1 / (1 + exp(-g)) by the hardware's exponential and reciprocal, within a step
// each.  The rounding of -g log2(e) moves exp(-g) by 1.3 |g| half steps of itself and
// so p: by less than one where g >= 0 (exp(-g) is small beside the 1), by 1.3 |g| half
// steps of a p that is itself exp(g) where g < 0.  Taking the exponent apart to spare
// a p of 1e-9 those 26 half steps cost 5 more instructions of an epilogue that has 20.
__device__ __forceinline__ float sigmoid(float g) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.4426950408889634f));
}

// c = erfc(-g / sqrt 2) / 2.  For z = |g| / sqrt 2 in the form erfc(z) = t exp(P(t)
// - z^2), t = 1 / (1 + z / 2) (Press et al., Numerical Recipes), P of degree 9 fitted
// by least squares at Chebyshev nodes; with its coefficients in FP32, as they stand
// here, it is within 1.01e-7 of log(erfc(z) exp(z^2) / t) over t in [0.155, 1], where
// erfc is above the smallest number.  In FP32 erfc(z) is within 6 (1 + z^2) half steps;
// the rounding of the exponent is what grows.  The device library's erfcf, with its
// branches, took the gated int8 product of 1387 x 180 to 2 x 5568 from 20 to 49 us.
__device__ __forceinline__ float normal_share(float g) {
  const float z = fabsf(g) * 0.70710678118654752f;
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.5f, z, 1.0f));
  float p = 0.15155121684074402f;
  p = __builtin_fmaf(p, t, -0.7168052792549133f);
  p = __builtin_fmaf(p, t, 1.241164207458496f);
  p = __builtin_fmaf(p, t, -0.8082337975502014f);
  p = __builtin_fmaf(p, t, 0.011933238245546818f);
  p = __builtin_fmaf(p, t, -0.0474550798535347f);
  p = __builtin_fmaf(p, t, 0.051060404628515244f);
  p = __builtin_fmaf(p, t, 0.38322609663009644f);
  p = __builtin_fmaf(p, t, 0.9990261793136597f);
  p = __builtin_fmaf(p, t, -1.2654671669006348f);
  const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(-z, z, p) * 1.4426950408889634f);
  const float h = 0.5f * t * e;
  return g <= 0.0f ? h : 1.0f - h;
}

template <int ACT>
__device__ __forceinline__ float act_value(float g) {
  if (ACT == UFP4_ACT_SILU) return g * sigmoid(g);
  return g * normal_share(g);
}

template <int ACT>
__device__ __forceinline__ ActPair act_pair(float g) {
  if (ACT == UFP4_ACT_SILU) {
    const float p = sigmoid(g);
    return {g * p, p * (1.0f + g * (1.0f - p))};
  }
  const float c = normal_share(g);
  const float phi = 0.39894228040143268f * __builtin_amdgcn_exp2f(g * g * -0.72134752044448170f);
  return {g * c, c + g * phi};
}

}  // namespace ufp4
