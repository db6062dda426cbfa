// Activations of the linear layers and their derivatives, in fp32.
//
// kFast forms serve bf16 operands, whose results are rounded to bf16 (2^-8) in most calls: the
// hardware exponential, the approximate division and, for the normal distribution function, a
// polynomial whose exponential the derivative shares.  Their values are good to 2e-5 of their
// size down to about 2e-37, where the exponential or its reciprocal leaves the normal numbers.
#pragma once

#include <type_traits>

#include "../../include/moe.h"
#include "common.cuh"

namespace moe {

// The hardware's reciprocal (1 ulp) and power of two (2 ulp), results under 2^-126 as 0.
__device__ __forceinline__ float rcp_ftz(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float exp2_ftz(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Phi(z) for kFast; *e = exp(-z^2 / 2).  With x = |z| / sqrt 2, Phi(-|z|) = e^(-x^2) f(x) / 2,
// and f, which falls from 1 like 1 / x, is t P(t) with t = 1 / (1 + 0.49 x).  P (degree 6) is
// fitted to f on 0 <= x <= 9.6 for the least of the larger of its relative error over 1e-5 and
// its share of Phi's absolute error over 7e-8, in a third of both; float arithmetic brings that
// to 9e-6 of Phi's size over the whole tail and 1.7e-7 absolute.
__device__ __forceinline__ float normal_cdf_fast(float z, float* e) {
  const float t = rcp_ftz(fmaf(0.49f * 0.70710678f, fabsf(z), 1.0f));
  float poly = fmaf(t, 0.08903342f, -0.37844392f);
  poly = fmaf(t, poly, 0.45524510f);
  poly = fmaf(t, poly, -0.0054650893f);
  poly = fmaf(t, poly, 0.29349263f);
  poly = fmaf(t, poly, 0.26927288f);
  poly = fmaf(t, poly, 0.27686502f);
  *e = exp2_ftz(-0.72134752f * z * z);
  const float tail = (0.5f * t) * (poly * *e);  // Phi(-|z|)
  return z < 0.f ? tail : 1.0f - tail;
}

// y = act(z).
template <bool kFast>
__device__ __forceinline__ float act_value(int act, float z) {
  switch (act) {
    case MOE_ACT_RELU:
      return z > 0.f ? z : (z != z ? z : 0.f);
    case MOE_ACT_GELU: {
      if (kFast) {
        float e;
        return z * normal_cdf_fast(z, &e);
      }
      return 0.5f * z * erfcf(-0.70710678118654752f * z);
    }
    case MOE_ACT_GELU_TANH: {
      // (1 + tanh u) / 2 is the logistic function of 2u
      const float u2 = 1.5957691216057308f * fmaf(0.044715f * z * z, z, z);
      return kFast ? __fdividef(z, 1.0f + __expf(-u2)) : z / (1.0f + expf(-u2));
    }
    case MOE_ACT_SILU:
      return kFast ? silu_bf16out(z) : silu_f(z);
    default:
      return z;
  }
}

// Several values at once: one switch for all of them.
template <bool kFast, int N>
__device__ __forceinline__ void act_values(int act, float (&v)[N]) {
  auto each = [&](auto a) {
#pragma unroll
    for (int q = 0; q < N; ++q) v[q] = act_value<kFast>(decltype(a)::value, v[q]);
  };
  switch (act) {
    case MOE_ACT_RELU: each(std::integral_constant<int, MOE_ACT_RELU>{}); break;
    case MOE_ACT_GELU: each(std::integral_constant<int, MOE_ACT_GELU>{}); break;
    case MOE_ACT_GELU_TANH: each(std::integral_constant<int, MOE_ACT_GELU_TANH>{}); break;
    case MOE_ACT_SILU: each(std::integral_constant<int, MOE_ACT_SILU>{}); break;
    default: break;
  }
}

// d act / d z (ReLU: 0 at 0).
template <bool kFast>
__device__ __forceinline__ float act_slope(int act, float z) {
  switch (act) {
    case MOE_ACT_RELU:
      return z > 0.f ? 1.f : 0.f;
    case MOE_ACT_GELU: {
      if (kFast) {
        float e;
        const float cdf = normal_cdf_fast(z, &e);
        return fmaf(z * 0.39894228f, e, cdf);
      }
      return 0.5f * erfcf(-0.70710678118654752f * z) +
             z * 0.3989422804014327f * expf(-0.5f * z * z);
    }
    case MOE_ACT_GELU_TANH: {
      constexpr float c = 1.5957691216057308f;
      const float z2 = z * z;
      const float u2 = c * fmaf(0.044715f * z2, z, z);
      const float p = kFast ? rcp_ftz(1.0f + __expf(-u2)) : 1.0f / (1.0f + expf(-u2));
      const float q = p * (1.0f - p);
      return q > 0.f ? fmaf(z * q, c * fmaf(0.134145f, z2, 1.0f), p) : p;
    }
    case MOE_ACT_SILU: {
      // p (1 + z q) with q = 1 - p; for z < 0 the bracket is q (1 + z + e^z), which vanishes at
      // z0 and is there d + e^z0 (e^d - 1) with d = z - z0, whose terms have one sign: nothing
      // cancels
      const float d = (z + 1.2784645557403564f) - 1.2979282759673083e-08f;
      const float t = kFast ? __expf(-fabsf(z)) : expf(-fabsf(z));
      const float r = kFast ? rcp_ftz(1.0f + t) : 1.0f / (1.0f + t);
      const float p = z > 0.f ? r : t * r, q = z > 0.f ? t * r : r;
      float bracket = fmaf(z, q, 1.0f);
      if (kFast) {  // a column's sum is float32, so near z0 the slope keeps its accuracy too
        const float series =  // e^d - 1 to 2e-6 of itself for |d| < 1/4
            d * fmaf(d, fmaf(d, fmaf(d, fmaf(d, 1.0f / 120.f, 1.0f / 24.f), 1.0f / 6.f), 0.5f), 1.0f);
        bracket = fabsf(d) < 0.25f ? q * fmaf(0.27846454f, series, d) : bracket;
      } else if (z < 0.f) {
        bracket = q * fmaf(0.2784645427610737f, expm1f(d), d);
      }
      return p * bracket;
    }
    default:
      return 1.f;
  }
}

}  // namespace moe
