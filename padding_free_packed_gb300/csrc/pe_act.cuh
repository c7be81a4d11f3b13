// The activations of the matrix product's epilogue and their slopes (internal header).
// gelu(z) = z Phi(z) with Phi the normal distribution function, exact (erf) GELU;
// gelu'(z) = Phi(z) + z exp(-z^2 / 2) / sqrt(2 pi).
#pragma once

#include "pe_sm103.cuh"

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

// The same for results rounded to bf16, two numbers at a time in paired arithmetic. With a =
// |z| and q = Phi(-a),
//   gelu = max(z, 0) - a q,    gelu' = m for z < 0, 1 - m otherwise, m = q - a bell / sqrt(2 pi),
// which keeps both tails as exact as normal_fast without computing two. a is cut off at 64,
// where q is long zero: infinities give the limits, and a NaN stays one.
struct GeluPair {
  uint64_t a, q, bell;

  __device__ __forceinline__ GeluPair(float z0, float z1) {
    using namespace sm103;
    auto cut = [](float z) {
      float r;
      asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(z)), "f"(64.f));
      return r;
    };
    a = f2(cut(z0), cut(z1));
    float d0, d1, e0, e1, t0, t1;
    f2_split(ffma2(a, both(0.5f * 0.70710678f), both(1.f)), d0, d1);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t0) : "f"(d0));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t1) : "f"(d1));
    f2_split(fmul2(fmul2(a, a), both(-0.5f * kLog2e)), e0, e1);
    bell = f2(ex2(e0), ex2(e1));
    const uint64_t t = f2(t0, t1);
    uint64_t p = ffma2(both(0.5f * 0.08912372f), t, both(0.5f * -0.35997975f));
    p = ffma2(p, t, both(0.5f * 0.39377043f));
    p = ffma2(p, t, both(0.5f * 0.0346651f));
    p = ffma2(p, t, both(0.5f * 0.28271717f));
    p = ffma2(p, t, both(0.5f * 0.27735412f));
    p = ffma2(p, t, both(0.5f * 0.28234804f));
    q = fmul2(fmul2(p, t), bell);
  }
  static __device__ __forceinline__ uint64_t both(float x) { return sm103::f2(x, x); }
  static __device__ __forceinline__ uint64_t minus(uint64_t x) {
    return x ^ 0x8000000080000000ull;
  }
  __device__ __forceinline__ uint64_t value(float z0, float z1) const {
    return sm103::ffma2(minus(a), q, sm103::f2(fmaxf(z0, 0.f), fmaxf(z1, 0.f)));
  }
  __device__ __forceinline__ uint64_t slope(float z0, float z1) const {
    using namespace sm103;
    const uint64_t m = ffma2(fmul2(minus(a), both(0.3989422804014327f)), bell, q);
    float m0, m1, n0, n1;
    f2_split(m, m0, m1);
    f2_split(fadd2(both(1.f), minus(m)), n0, n1);
    return f2(z0 < 0.f ? m0 : n0, z1 < 0.f ? m1 : n1);
  }
};

inline bool activation_ok(int act) { return act >= PE_ACT_NONE && act <= PE_ACT_GEGLU; }

}  // namespace pe
