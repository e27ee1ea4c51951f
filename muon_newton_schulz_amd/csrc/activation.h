// The activations of a layer and their slopes, on float32 values in registers.
#pragma once
#include <hip/hip_runtime.h>

namespace mns {

enum Act { ACT_NONE = 0, ACT_RELU = 1, ACT_RELU2 = 2, ACT_GELU = 3, ACT_SILU = 4 };

// Phi(z), the normal distribution's mass below z, and, with SLOPE, phi(z), its density.
//
// EXACT (float32 storage): erfc to float32. Else (bfloat16 storage, whose rounding is up to 2^-8 of a value):
// erfc(x) e^(x^2) on x >= 0 as a polynomial of degree 5 in t = 1 / (1 + 0.53 x), fitted here to the least
// largest relative error up to x = 9.5 (2.9e-5 of Phi in either tail, where e^(-x^2) leaves float32's
// normal numbers): one reciprocal, one exponential and ten multiply-adds, where float32's erfc takes
// several times that. An epilogue has 256 x 256 values a block and nothing to hide them behind.
template <bool EXACT, bool SLOPE>
__device__ __forceinline__ float normal_cdf(float z, float& density) {
  const float e = __builtin_amdgcn_exp2f(z * z * -0.72134752044f);      // e^(-z^2 / 2)
  density = SLOPE ? e * 0.39894228040f : 0.f;
  if constexpr (EXACT) {
    if (SLOPE) density = expf(-0.5f * z * z) * 0.39894228040f;
    return 0.5f * erfcf(z * -0.70710678119f);
  } else {
    const float t = __builtin_amdgcn_rcpf(1.f + fabsf(z) * (0.53f * 0.70710678119f));
    float q = -0.18196194364f;
    q = fmaf(q, t, 0.40301403400f);
    q = fmaf(q, t, 0.16524518902f);
    q = fmaf(q, t, 0.31580967563f);
    q = fmaf(q, t, 0.29788199973f);
    q *= 0.5f * t * e;
    return z >= 0.f ? 1.f - q : q;
  }
}

// 1 / (1 + e^-z).
template <bool EXACT>
__device__ __forceinline__ float sigmoid(float z) {
  if constexpr (EXACT) {
    const float e = expf(-fabsf(z));                  // no overflow on either side
    return (z >= 0.f ? 1.f : e) / (1.f + e);
  } else {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(z * -1.44269504089f));
  }
}

// v <- act(v). A NaN stays one: the tests are for <= 0, which a NaN fails.
template <bool EXACT, int N>
__device__ __forceinline__ void activate(int act, float (&v)[N]) {
  float unused;
  switch (act) {
    case ACT_RELU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = v[i] <= 0.f ? 0.f : v[i];
      break;
    case ACT_RELU2:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = v[i] <= 0.f ? 0.f : v[i] * v[i];
      break;
    case ACT_GELU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] *= normal_cdf<EXACT, false>(v[i], unused);
      break;
    case ACT_SILU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] *= sigmoid<EXACT>(v[i]);
      break;
    default:
      break;
  }
}

// v <- v act'(z).
template <bool EXACT, int N>
__device__ __forceinline__ void times_slope(int act, float (&v)[N], const float (&z)[N]) {
  switch (act) {
    case ACT_RELU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = z[i] <= 0.f ? 0.f : v[i];
      break;
    case ACT_RELU2:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = z[i] <= 0.f ? 0.f : v[i] * (2.f * z[i]);
      break;
    case ACT_GELU:
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float density;
        const float cdf = normal_cdf<EXACT, true>(z[i], density);
        v[i] *= fmaf(z[i], density, cdf);
      }
      break;
    case ACT_SILU:
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float s = sigmoid<EXACT>(z[i]);
        // EXACT: 1 - s from the other side, which keeps its last bits where s is near 1
        const float other = EXACT ? sigmoid<EXACT>(-z[i]) : 1.f - s;
        v[i] *= s * fmaf(z[i], other, 1.f);
      }
      break;
    default:
      break;
  }
}

}  // namespace mns
