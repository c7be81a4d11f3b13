// 8-bit floating-point helpers of the 8-bit layer kernels (internal header).
#pragma once

#include "pe_common.cuh"

namespace pe {

constexpr int kFp8Block = 128;             // elements along a row that share a scale

// Largest finite value of each 8-bit type.
__host__ __device__ constexpr float fp8_largest(bool e5m2) { return e5m2 ? 57344.f : 448.f; }

// Smallest block magnitude that quantisation works with, a power of two: the
// scale it gives, and that scale's reciprocal, are still normal fp32 numbers.
__host__ __device__ constexpr float fp8_smallest_amax(bool e5m2) {
  return e5m2 ? 7.703719777548943e-34f : 6.018531076210112e-36f;   // 2^-110, 2^-117
}

// max that returns NaN when either operand is NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Two fp32 values rounded to 8 bits (nearest, ties to even), lo in the low byte.
template <bool kE5M2>
__device__ __forceinline__ uint32_t fp8x2(float lo, float hi) {
  uint16_t r;
  if constexpr (kE5M2)
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

template <bool kE5M2>
__device__ __forceinline__ uint32_t fp8x4(float a, float b, float c, float d) {
  return fp8x2<kE5M2>(a, b) | (fp8x2<kE5M2>(c, d) << 16);
}

// A block with largest magnitude amax: the magnitude it is quantised with, the factor
// that takes its elements to the 8-bit range, and its scale. Both quotients are the
// nearest fp32 numbers: the rounded 1 / F alone would put the same bias of up to 0.75
// of a rounding on every scale, an approximate reciprocal two roundings more on every
// factor. Measured: 32299 x 768 normalised 28.7 us against 28.5 with both of these, 90487
// x 500 fp32 41.6 against 41.1, 32299 x 2304 quantised both ways 53.1 against 52.6.
template <bool kE5M2>
__device__ __forceinline__ float fp8_block(float amax) {
  return max_nan(amax, fp8_smallest_amax(kE5M2));
}
// F / block from a reciprocal improved once and the exact remainder of its product
// (Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990). A call of the division took registers that rows of odd width do
// not have (90487 x 501 bf16 114 us, 85 without). Equal to the division for all 2^23
// significands in 14 binades, the first and the last among them. The power of two keeps
// the reciprocal normal; an infinite block gives 0.
template <bool kE5M2>
__device__ __forceinline__ float fp8_factor(float block) {
  constexpr float kDown = 0x1p-9f, kLargest = fp8_largest(kE5M2) * kDown;
  const float a = block * kDown;
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(a));
  y = fmaf(y, fmaf(-a, y, 1.f), y);
  const float q = kLargest * y;
  return isinf(block) ? 0.f : fmaf(fmaf(-a, q, kLargest), y, q);
}
// A known divisor: the product with its rounded reciprocal, corrected once by the exact
// remainder, is the rounded quotient (Brisebarre, Muller and Raina, "Accelerating
// correctly rounded floating-point division when the divisor is known in advance",
// 2004; compared with division for all 2^23 significands). An infinity stays one.
template <bool kE5M2>
__device__ __forceinline__ float fp8_scale(float block) {
  constexpr float kLargest = fp8_largest(kE5M2), kInverse = 1.f / kLargest;
  const float q = block * kInverse;
  const float rest = fmaf(-kLargest, q, block);
  return isinf(block) ? block : fmaf(rest, kInverse, q);
}

inline bool fp8_type_ok(pe_fp8_type t) { return t == PE_E4M3 || t == PE_E5M2; }

// The layout every 8-bit matrix has: 16-byte aligned rows.
inline bool fp8_layout_ok(const void* p, int64_t ld, int64_t cols) {
  return aligned(p, 16) && ld % 16 == 0 && ld >= cols;
}

}  // namespace pe
