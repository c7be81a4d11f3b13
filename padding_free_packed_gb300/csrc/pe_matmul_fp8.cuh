// Internal interface of the 8-bit matrix product's kernels.
#pragma once

#include "pe_fp8.cuh"
#include "pe_sm103.cuh"

namespace pe {

struct MatmulFp8 {
  const uint8_t* a;
  const uint8_t* b;
  int64_t a_ld, b_ld;
  const float* a_scales;   // [ceil(k / 128)][m]
  const float* b_scales;   // [ceil(k / 128)][ceil(n / 128)]
  int32_t m, n, k;
  bool a_e5m2, b_e5m2, out_fp32;
  void* out;
};

// How a product runs. The choice depends on the sizes alone (the workspace size
// follows it); it counts the 152 SMs of the device these kernels are built for.
struct MatmulPlan {
  int32_t rows;      // of a per CTA of the narrow kernel: 16, 32 or 64; 0: the pair kernel
  int32_t split;     // narrow: CTAs of a cluster that share a tile's sum
  bool runs;         // pair: equal runs of blocks of k, parts summed by a second kernel
};
MatmulPlan matmul_plan(int64_t m, int64_t n, int64_t k);

// Pairs of CTAs on 256 x 256 tiles, for products with many rows.
size_t matmul_pair_workspace();
pe_status matmul_pair(const MatmulFp8& p, bool runs, void* workspace, DeviceStatus* status,
                      cudaStream_t stream);

// Few rows: 128 rows of b by 16, 32 or 64 rows of a per CTA, the sum over k split
// over a cluster.
pe_status matmul_rows(const MatmulFp8& p, int32_t rows, int32_t split, DeviceStatus* status,
                      cudaStream_t stream);

// Tensor map of row-major [rows, cols] of `type` (elements of `size` bytes), rows
// `pitch` bytes apart, boxes of box_rows rows of 128 bytes, 128-byte swizzle.
pe_status matmul_map(CUtensorMap* map, CUtensorMapDataType type, int size, const void* base,
                     int64_t rows, int64_t cols, int64_t pitch, uint32_t box_rows);
// The same for `planes` such matrices, one after the other (0: without that dimension).
pe_status matmul_map_planes(CUtensorMap* map, CUtensorMapDataType type, int size,
                            const void* base, int64_t rows, int64_t cols, int64_t pitch,
                            uint32_t box_rows, int32_t planes);

// The address, on the current device, of the status word that every product's waits share.
pe_status matmul_status_word(DeviceStatus** out);

namespace sm103 {

// mbar_wait for the waits of every block of k: a few attempts (each suspends the
// thread for a while) before the clock and the abort flag are looked at. Not with a
// short limit, which is kept by polling.
__device__ __forceinline__ bool eager_wait(uint32_t bar, uint32_t parity,
                                           volatile WaitGuard* guard, DeviceStatus* status,
                                           int where) {
  if (mbar_test_wait(bar, parity)) return true;
  if (guard->limit_ns >= kPollBelowNs) {
    for (int i = 0; i < 16; ++i)
      if (mbar_try_wait(bar, parity)) return true;
  }
  return mbar_wait(bar, parity, guard, status, where);
}
// The same for a whole warp: true only if true in every lane.
__device__ __forceinline__ bool eager_warp_wait(uint32_t bar, uint32_t parity,
                                                volatile WaitGuard* guard, DeviceStatus* status,
                                                int where) {
  return __all_sync(0xffffffffu, eager_wait(bar, parity, guard, status, where));
}

// Four bytes to shared memory without a register on the way (zero unless `in`).
__device__ __forceinline__ void copy_async4(void* dst, const float* src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(in ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int kPending>
__device__ __forceinline__ void copy_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

// The product of a block's two scales may leave the range of normal fp32 numbers although
// the block's part of the result does not (quantisation makes scales from 2^-126 up); it
// is then added in two steps. Whether a scale is one of which that can happen: neither
// zero nor from 2^-62 to 2^63.
__device__ __forceinline__ bool scale_is_far(float x) {
  const uint32_t twice = __float_as_uint(x) << 1;       // without the sign
  return twice != 0 && twice - ((127u - 62u) << 24) >= (126u << 24);
}
// Factors x and y so that sum + (d x) y, the second step a fused multiply-add, is the sum
// with d a b: 1 and a b where a b is a normal number (the same bits as sum + d (a b)), or
// zero, infinite or NaN because a or b is; else y is a power of two that keeps d x in
// range. d, the block's sum of products, is zero or from 2^-32 to 2^39: with a b below
// 2^-126, x y = a b 2^64 2^-64; with a b above 2^128, a b 2^-96 2^96, where x is cut off
// at the largest number, beyond which only d = 0 has a finite result.
__device__ __forceinline__ float2 far_factors(float a, float b) {
  constexpr float kLargest = 3.402823466e38f, kSmallest = 0x1p-126f;
  const float s = fabsf(a * b);
  if ((s >= kSmallest && s <= kLargest) || a == 0.f || b == 0.f || !(fabsf(a) <= kLargest) ||
      !(fabsf(b) <= kLargest))
    return make_float2(1.f, a * b);
  if (s < 1.f) return make_float2(a * 0x1p64f * b, 0x1p-64f);
  const float x = (a * 0x1p-48f) * (b * 0x1p-48f);
  return make_float2(fminf(fmaxf(x, -kLargest), kLargest), 0x1p96f);
}

// Instruction descriptor of kind::f8f6f4: fp32 accumulator, both operands K-major.
constexpr uint32_t idesc_fp8(int M, int N, bool a_e5m2, bool b_e5m2) {
  return (1u << 4) | ((a_e5m2 ? 1u : 0u) << 7) | ((b_e5m2 ? 1u : 0u) << 10) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

}  // namespace sm103
}  // namespace pe
