// The activations of a layer and their slopes, on float32 values in registers.
#pragma once
#include <hip/hip_runtime.h>

namespace mns {

enum Act { ACT_NONE = 0, ACT_RELU = 1, ACT_RELU2 = 2, ACT_GELU = 3, ACT_SILU = 4 };

// gelu and its slope, z Phi(z) and Phi(z) + z phi(z), Phi the normal distribution's mass below z and phi
// its density. EXACT (float32 storage): by float32's erfc. Else (bfloat16 storage) by two approximations of
// Q(a) = Phi(-a), a = |z|, fitted here to the least largest relative error, in about 15 and 24 instructions'
// time where float32's erfc takes several times that (an epilogue has 256 x 256 values a block and little to
// hide them behind):
//   log2 Q as a polynomial of degree 8 in a: 1.5e-5 of Q up to a = 5, 2.1e-4 up to 8 and 2.8e-3, below half a
//   bfloat16 step, up to 13.2, where Q leaves float32's normal numbers; gelu = max(z, 0) - a Q;
//   Q e^(a^2 / 2) as one of degree 7 in t = 1 / (1 + 0.5 a / sqrt 2): 1.3e-6 of Q, and z^2 2^-24 for the
//   exponential's rounded argument; the slope is 1 - S or S with S = e^(-a^2 / 2) (that - a / sqrt(2 pi)), so
//   both terms share the exponential.
// They are this close because what is rounded to bfloat16 from a value that is off by r falls on the other
// side for about r 2^8 of the elements: with 2e-4 and 2.9e-5 of Q (one and two terms fewer) 1.5 and 0.9 % of
// normally distributed elements did, now 0.1 % and less. A NaN stays one.
template <bool EXACT>
__device__ __forceinline__ float gelu(float z) {
  if constexpr (EXACT) {
    return 0.5f * z * erfcf(z * -0.70710678119f);
  } else {
    // Q is 0 from a = 15 on (2^-167), where the polynomial turns; a NaN passes through this minimum
    const float a = __builtin_elementwise_minimum(fabsf(z), 15.f);
    float p = 5.07311775e-08f;
    p = fmaf(p, a, -2.83297572e-06f);
    p = fmaf(p, a, 6.81215533e-05f);
    p = fmaf(p, a, -9.40051919e-04f);
    p = fmaf(p, a, 8.43972154e-03f);
    p = fmaf(p, a, -5.36463074e-02f);
    p = fmaf(p, a, -4.58936363e-01f);
    p = fmaf(p, a, -1.15100300e+00f);
    p = fmaf(p, a, -1.00002003e+00f);
    return fmaf(-a, __builtin_amdgcn_exp2f(p), fmaxf(z, 0.f));
  }
}

template <bool EXACT>
__device__ __forceinline__ float gelu_slope(float z) {
  if constexpr (EXACT) {
    const float density = expf(-0.5f * z * z) * 0.39894228040f;
    return fmaf(z, density, 0.5f * erfcf(z * -0.70710678119f));
  } else {
    const float a = fabsf(z), e = __builtin_amdgcn_exp2f(z * z * -0.72134752044f);
    const float t = __builtin_amdgcn_rcpf(fmaf(a, 0.5f * 0.70710678119f, 1.f));
    float q = 4.4651631266e-02f;
    q = fmaf(q, t, -1.8030735850e-01f);
    q = fmaf(q, t, 1.9733217359e-01f);
    q = fmaf(q, t, 1.7013832927e-02f);
    q = fmaf(q, t, 1.4147923887e-01f);
    q = fmaf(q, t, 1.3865421712e-01f);
    q = fmaf(q, t, 1.4117570221e-01f);
    const float s = e * fmaf(q, t, a * -0.39894228040f);
    return z >= 0.f ? 1.f - s : s;
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
      for (int i = 0; i < N; ++i) v[i] = gelu<EXACT>(v[i]);
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
      for (int i = 0; i < N; ++i) v[i] *= gelu_slope<EXACT>(z[i]);
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
