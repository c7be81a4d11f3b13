// The activations of the matrix product's epilogue and their slopes (internal header).
// gelu(z) = z Phi(z) with Phi the normal distribution function, exact (erf) GELU;
// gelu'(z) = Phi(z) + z exp(-z^2 / 2) / sqrt(2 pi).
#pragma once

#include "pe_common.cuh"

namespace pe {

// Results rounded to bf16: Phi(-|z|) = erfc(x) / 2 with x = |z| / sqrt 2, and erfc(x) =
// exp(-x^2) t P(t) with t = 1 / (1 + x / 2) and a polynomial P of degree 6 fitted here (equal
// ripples of the relative error, x from 0 to 9.5). Relative error 1.2e-6 plus that of the
// exponential, 2e-7 z^2, on both tails: far below bf16's 2^-9. `bell` receives
// exp(-z^2 / 2), which the slope needs too.
__device__ __forceinline__ float normal_fast(float z, float& bell) {
  const float x = fabsf(z);
  const float t = __fdividef(1.f, fmaf(0.5f * 0.70710678f, x, 1.f));
  bell = ex2(z * z * (-0.5f * kLog2e));
  float p = 0.08912372f;
  p = fmaf(p, t, -0.35997975f);
  p = fmaf(p, t, 0.39377043f);
  p = fmaf(p, t, 0.0346651f);
  p = fmaf(p, t, 0.28271717f);
  p = fmaf(p, t, 0.27735412f);
  p = fmaf(p, t, 0.28234804f);
  const float tail = 0.5f * p * t * bell;
  return z < 0.f ? tail : 1.f - tail;
}

// T: the type the result is rounded to. fp32 takes CUDA's own functions. Infinite z give the
// limits, 0 and infinity, a slope of 0 and 1.
template <typename T>
__device__ __forceinline__ float normal(float z, float& bell) {
  if constexpr (sizeof(T) == 4) {
    bell = expf(-0.5f * z * z);
    return normcdff(z);
  } else {
    return normal_fast(z, bell);
  }
}
__device__ __forceinline__ float times_normal(float z, float phi) {
  return fmaxf(z, -3.402823466e38f) * phi;     // phi carries a NaN
}

template <typename T>
__device__ __forceinline__ float gelu(float z) {
  if constexpr (sizeof(T) == 4) {
    return times_normal(z, normcdff(z));
  } else {
    float bell;
    return times_normal(z, normal_fast(z, bell));
  }
}

// gelu and its slope together.
template <typename T>
__device__ __forceinline__ float gelu_slope(float z, float& value) {
  constexpr float kDensity = 0.3989422804014327f;     // 1 / sqrt(2 pi)
  float bell;
  const float phi = normal<T>(z, bell);
  value = times_normal(z, phi);
  return fmaf(fminf(fmaxf(z, -64.f), 64.f) * kDensity, bell, phi);
}

inline bool activation_ok(int act) { return act >= PE_ACT_NONE && act <= PE_ACT_GEGLU; }

}  // namespace pe
