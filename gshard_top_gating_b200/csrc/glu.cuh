// glu.cuh -- the gate functions of gated experts, h = f(g) * u, and their derivatives.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace moe {

// The normal distribution F(g) and its density e^(-g^2/2) / sqrt(2 pi), both from one
// exponential: F(-|g|) = erfc(z) / 2 with z = |g| / sqrt 2, and erfc(z) e^(z^2) as a polynomial
// t P(t) in t = 1 / (1 + 0.434 z), P of degree 5.  Its coefficients are a fit of the relative
// error over 0 <= z <= 9.5, where e^(-z^2) leaves the range of 32 bits (iterated reweighted least
// squares against the exact function): F(-|g|) is off by at most 3.9e-6 of itself, in the far
// tail as near 0, before the exponential's own error (1e-5 of itself at g = -9).
__device__ __forceinline__ void normal_fast(float g, float& cdf, float& pdf) {
  const float e = __expf(-0.5f * g * g);
  const float t = __fdividef(1.f, fmaf(fabsf(g), 0.434f * 0.70710678f, 1.f));
  float s = fmaf(t, -0.15204786f, 0.38831508f);
  s = fmaf(t, s, 0.0061460095f);
  s = fmaf(t, s, 0.27604872f);
  s = fmaf(t, s, 0.23612294f);
  s = fmaf(t, s, 0.24541432f);
  const float q = 0.5f * s * t * e;
  cdf = g > 0.f ? 1.f - q : q;
  pdf = 0.39894228040143268f * e;
}

// f(g) in 32 bits.  FAST (bf16 and 8-bit results): the hardware exponential and reciprocal and the
// approximation above, off by 2^-15 of f at most where that rounds to 2^-8 -- with erff, dh on
// 8 x 2048 x 2048 x 8192 took 616 us, the product alone 350 --; else expf and erfcf.
template <int FN, bool FAST>
__device__ __forceinline__ float glu_f(float g) {
  if (FN == kGluSilu) return FAST ? __fdividef(g, 1.f + __expf(-g)) : g / (1.f + expf(-g));
  if (FN == kGluGelu) {
    if (!FAST) return 0.5f * g * erfcf(-g * 0.70710678118654752f);
    float c, d;
    normal_fast(g, c, d);
    return g * c;
  }
  return g <= 0.f ? 0.f : g;      // a NaN stays one
}

// f(g) and f'(g): silu s(1 + g(1 - s)), s = 1/(1 + e^-g); gelu F(g) + g e^(-g^2/2)/sqrt(2 pi)
// with F the normal distribution; relu 1 for g > 0.  Where g is NaN both are, for every f.
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
    f = g <= 0.f ? 0.f : g;
    df = g > 0.f ? 1.f : f;       // 0, or NaN
  }
}

// g and u as a bf16 forward keeps them for its backward, in 16 bits, 32 columns of a row alike:
// fp16 where all their magnitudes are in [2^-17, 65504), which is never less exact than bf16 and
// from 2^-14 on eight times more so, else bf16.  The lowest bit of the first of the 32 says which
// (1: fp16).  That one becomes the nearest code with this lowest bit, either way, so it is off by
// at most a step where the others are by half of one: 2^-10 of itself in fp16 (2^-24 in all
// below 2^-14, where fp16 is subnormal), 2^-7 in bf16.  dx and dW13 are then
// off by 2.4e-3 of their norm, the roundings of dg, du and the results; with g and u in bf16
// alone by 3.0e-3, for 1 to 3% less time (15 experts of 1365 rows, M = 256, H = 3008: 325 us
// against 348, as the epilogues of `up` and `dh` bound small M).
__device__ __forceinline__ bool gu_fine(float least, float most) { return least >= 0x1p-17f && most < 65504.f; }
__device__ __forceinline__ bool gu_is_fine(uint32_t first) { return first & 1u; }
// The first of 32 in bf16, rounded to the nearest even code.
__device__ __forceinline__ uint32_t gu_first_wide(float v) {
  const uint32_t x = __float_as_uint(v);
  return (min((x & 0x7fffffffu) + 0x10000u, 0x7fffffffu) >> 16 & 0x7ffeu) | (x >> 16 & 0x8000u);
}
// In fp16, to an odd code: towards zero, which leaves 2k or 2k + 1, then 2k + 1.
__device__ __forceinline__ uint32_t gu_first_fine(float v) { return __half_as_ushort(__float2half_rz(v)) | 1u; }
__device__ __forceinline__ void pack_gu(const uint32_t (&v)[32], bool live, uint32_t (&pk)[16]) {
  float least = fabsf(__uint_as_float(v[0])), most = least;
#pragma unroll
  for (int j = 1; j < 32; ++j) {
    const float m = fabsf(__uint_as_float(v[j]));
    least = fminf(least, m);
    most = fmaxf(most, m);
  }
  const bool fine = gu_fine(least, most);
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float a = __uint_as_float(v[2 * j]), b = __uint_as_float(v[2 * j + 1]);
    pk[j] = !live ? 0u : fine ? pack_f16x2(a, b) : pack_bf16x2(a, b);
  }
  if (live) {
    const float first = __uint_as_float(v[0]);
    pk[0] = (pk[0] & 0xffff0000u) | (fine ? gu_first_fine(first) : gu_first_wide(first));
  }
}
// One of them, where the warp holds the 32 columns (and the row is live for all of it or none).
__device__ __forceinline__ uint16_t pack_gu_lane(float v, bool live) {
  const float m = fabsf(v);
  const bool fine = __all_sync(0xffffffffu, gu_fine(m, m) || isnan(v));
  uint32_t c = (fine ? pack_f16x2(v, 0.f) : pack_bf16x2(v, 0.f)) & 0xffffu;
  if ((threadIdx.x & 31) == 0) c = fine ? gu_first_fine(v) : gu_first_wide(v);
  return live ? (uint16_t)c : 0;
}
// Both of a word: FINE, all lanes hold fp16; else each lane as `fine` says.
template <bool FINE>
__device__ __forceinline__ void unpack_gu(uint32_t w, bool fine, float& a, float& b) {
  a = bf16lo(w);
  b = bf16hi(w);
  if (FINE || fine) unpack_f16x2(w, a, b);
}

}  // namespace moe
