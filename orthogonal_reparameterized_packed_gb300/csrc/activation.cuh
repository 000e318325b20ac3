// The activations of poetx_linear_* and their derivatives in fp32.
// FAST (bf16 results): exp and the quotient by the approximate intrinsics: the
// quotient within 2 ulp, exp(x) within 2 + 1.2 |x| (2^-16 relative at x = -87, where
// bf16's range ends), far below bf16's 2^-8; otherwise full fp32 accuracy.
#pragma once

#include <cuda_bf16.h>

#include "poetx.h"

namespace poetx {

template <bool FAST>
__device__ __forceinline__ float sigmoid_f(float z) {
  return FAST ? __fdividef(1.f, 1.f + __expf(-z)) : 1.f / (1.f + expf(-z));
}

// Phi(z), the standard normal distribution, with `e` = exp(-z^2 / 2).  FAST: for
// z <= 0, Phi(z) / e as a polynomial in t = 1 / (1 + c |z|), without a term of order
// 0 (as 7.1.26 of Abramowitz and Stegun, Handbook of Mathematical Functions, has
// it), c and the coefficients fitted here: the largest of the error over 2^-21 and
// the relative error over 2^-13 is least over 0 >= z >= -14 (linear programming).  In fp32
// it is within 3e-7, and relatively within 2^-14 besides e's error, so that the tail
// z Phi(z) keeps bf16's accuracy (7.1.26 itself is off by 1 % at z = -8).
// (erfcf's branches made the epilogue of a 2048 x 5632 x 2048 product take 47 us
// instead of 34.)
template <bool FAST>
__device__ __forceinline__ float normal_cdf(float z, float e) {
  if (!FAST) return 0.5f * erfcf(-0.7071067811865476f * z);
  const float t = __fdividef(1.f, fmaf(0.29521707f, fabsf(z), 1.f));
  float q = fmaf(-0.16737619f, t, 0.50032765f);
  q = fmaf(q, t, -0.10591569f);
  q = fmaf(q, t, 0.31997606f);
  q = fmaf(q, t, 0.21603106f);
  q = fmaf(q, t, 0.23695697f);
  q *= 0.5f * t * e;
  return z > 0.f ? 1.f - q : q;
}

// u of gelu_tanh: tanh(u) = 2 sigmoid(2u) - 1
__device__ __forceinline__ float gelu_u(float z) {
  return 0.7978845608028654f * fmaf(0.044715f * z * z, z, z);
}

template <int ACT, bool FAST>
__device__ __forceinline__ float act_f(float z) {
  if (ACT == POETX_ACT_RELU) return z <= 0.f ? 0.f : z;  // NaN stays NaN
  if (ACT == POETX_ACT_SILU) return z * sigmoid_f<FAST>(z);
  if (ACT == POETX_ACT_GELU) return z * normal_cdf<FAST>(z, FAST ? __expf(-0.5f * z * z) : 0.f);
  if (ACT == POETX_ACT_GELU_TANH) return z * sigmoid_f<FAST>(2.f * gelu_u(z));
  return z;
}

// d act / dz, but for relu (act_grad)
template <int ACT, bool FAST>
__device__ __forceinline__ float act_df(float z) {
  if (ACT == POETX_ACT_SILU) {
    const float s = sigmoid_f<FAST>(z);
    return s * (1.f + z * (1.f - s));
  }
  if (ACT == POETX_ACT_GELU) {
    const float e = FAST ? __expf(-0.5f * z * z) : expf(-0.5f * z * z);
    return fmaf(z * 0.3989422804014327f, e, normal_cdf<FAST>(z, e));
  }
  if (ACT == POETX_ACT_GELU_TANH) {
    // s (1 - s) is 0 from |z| = 11 on and comes first; z^2 must not leave the range
    const float s = sigmoid_f<FAST>(2.f * gelu_u(z)), zz = fminf(z * z, 1e30f);
    return s + s * (1.f - s) * z * (2.f * 0.7978845608028654f * fmaf(0.134145f, zz, 1.f));
  }
  return 1.f;
}

// dy act'(z).  relu selects: where z is not above 0 (0 and NaN among them) the
// gradient is 0, an infinite or NaN dy too, which a product with 0 would keep.
template <int ACT, bool FAST>
__device__ __forceinline__ float act_grad(float dy, float z) {
  if (ACT == POETX_ACT_NONE) return dy;
  if (ACT == POETX_ACT_RELU) return z > 0.f ? dy : 0.f;
  return dy * act_df<ACT, FAST>(z);
}

}  // namespace poetx
