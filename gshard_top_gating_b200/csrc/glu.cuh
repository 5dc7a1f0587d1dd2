// glu.cuh -- the gate functions of gated experts, h = f(g) * u, and their derivatives.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace moe {

// The normal distribution F(g) and its density e^(-g^2/2) / sqrt(2 pi), both from one
// exponential: F(-|g|) = erfc(z) / 2 with z = |g| / sqrt 2 and Hastings' approximation
// erfc(z) = (a1 t + ... + a5 t^5) e^(-z^2), t = 1 / (1 + p z) (Abramowitz and Stegun,
// "Handbook of Mathematical Functions", 7.1.26), off by at most 1.5e-7.
__device__ __forceinline__ void normal_fast(float g, float& cdf, float& pdf) {
  const float e = __expf(-0.5f * g * g);
  const float t = __fdividef(1.f, fmaf(fabsf(g), 0.3275911f * 0.70710678f, 1.f));
  float s = fmaf(t, 1.061405429f, -1.453152027f);
  s = fmaf(t, s, 1.421413741f);
  s = fmaf(t, s, -0.284496736f);
  s = fmaf(t, s, 0.254829592f);
  const float q = 0.5f * s * t * e;
  cdf = g > 0.f ? 1.f - q : q;
  pdf = 0.39894228040143268f * e;
}

// f(g) in 32 bits.  FAST (bf16 results): the hardware exponential and reciprocal and the
// approximation above, whose errors (about 2^-21) vanish in the rounding to 8 bits -- with
// erff, dh on 8 x 2048 x 2048 x 8192 took 616 us, the product alone 350 --; else expf and
// erfcf.
template <int FN, bool FAST>
__device__ __forceinline__ float glu_f(float g) {
  if (FN == kGluSilu) return FAST ? __fdividef(g, 1.f + __expf(-g)) : g / (1.f + expf(-g));
  if (FN == kGluGelu) {
    if (!FAST) return 0.5f * g * erfcf(-g * 0.70710678118654752f);
    float c, d;
    normal_fast(g, c, d);
    return g * c;
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
    float c, d;
    if (FAST) {
      normal_fast(g, c, d);
    } else {
      c = 0.5f * erfcf(-g * 0.70710678118654752f);
      d = 0.39894228040143268f * expf(-0.5f * g * g);
    }
    f = g * c;
    df = fmaf(g, d, c);
  } else {
    f = fmaxf(g, 0.f);
    df = g > 0.f ? 1.f : 0.f;
  }
}

}  // namespace moe
