// glu.cuh -- the gate functions of gated experts, h = f(g) * u, and their derivatives.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace moe {

// f(g) in 32 bits.  FAST (bf16 results): the hardware exponential and erff, whose errors
// (a few units of 2^-22 relative, 2^-23 absolute) vanish in the rounding to 8 bits; else
// expf and erfcf, which keep relative accuracy where f(g) is tiny.
template <int FN, bool FAST>
__device__ __forceinline__ float glu_f(float g) {
  if (FN == kGluSilu) return FAST ? __fdividef(g, 1.f + __expf(-g)) : g / (1.f + expf(-g));
  if (FN == kGluGelu) {
    const float z = g * 0.70710678118654752f;
    return FAST ? 0.5f * g * (1.f + erff(z)) : 0.5f * g * erfcf(-z);
  }
  return fmaxf(g, 0.f);
}

// f(g) and f'(g): silu s(1 + g(1 - s)), s = 1/(1 + e^-g); gelu F(g) + g e^(-g^2/2)/sqrt(2 pi)
// with F the normal distribution; relu 1 for g > 0.
template <int FN, bool FAST>
__device__ __forceinline__ void glu_f_df(float g, float& f, float& df) {
  if (FN == kGluSilu) {
    const float s = FAST ? __fdividef(1.f, 1.f + __expf(-g)) : 1.f / (1.f + expf(-g));
    f = g * s;
    df = s * (1.f + g * (1.f - s));
  } else if (FN == kGluGelu) {
    const float z = g * 0.70710678118654752f;
    const float c = FAST ? 0.5f * (1.f + erff(z)) : 0.5f * erfcf(-z);
    f = g * c;
    df = c + g * 0.39894228040143268f * (FAST ? __expf(-0.5f * g * g) : expf(-0.5f * g * g));
  } else {
    f = fmaxf(g, 0.f);
    df = g > 0.f ? 1.f : 0.f;
  }
}

}  // namespace moe
