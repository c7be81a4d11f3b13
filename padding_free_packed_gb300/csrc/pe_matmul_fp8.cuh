// Internal interface of the 8-bit matrix product's kernels.
#pragma once

#include "pe_fp8.cuh"

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

// Pairs of CTAs on 256 x 256 tiles, for products with many rows.
size_t matmul_pair_workspace(int64_t m, int64_t n, int64_t k);
pe_status matmul_pair(const MatmulFp8& p, void* workspace, DeviceStatus* status,
                      cudaStream_t stream);

}  // namespace pe
