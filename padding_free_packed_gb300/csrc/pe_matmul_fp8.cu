// Matrix product of 8-bit operands with a scale for each block of 128.
#include "pe_fp8.cuh"

namespace pe {

namespace {

constexpr int kTileM = 64, kTileN = 64, kTileK = 32;

__device__ DeviceStatus g_matmul_status;

template <bool kE5M2>
__device__ __forceinline__ float from_fp8(uint8_t v) {
  uint32_t h2;
  const uint16_t pair = v;
  if constexpr (kE5M2)
    asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h2) : "h"(pair));
  else
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(pair));
  float f;
  asm("{.reg .f16 l, h; mov.b32 {l, h}, %1; cvt.f32.f16 %0, l;}" : "=f"(f) : "r"(h2));
  return f;
}

struct Args {
  const uint8_t *a, *b;
  int64_t a_ld, b_ld, m, n, k;
  const float *a_scales, *b_scales;
  void* out;
};

template <bool kA5, bool kB5, typename TOut>
__global__ void __launch_bounds__(256) matmul_simple_kernel(const Args p) {
  __shared__ float as[kTileK][kTileM + 1], bs[kTileK][kTileN + 1];
  const int64_t i0 = (int64_t)blockIdx.x * kTileM, j0 = (int64_t)blockIdx.y * kTileN;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t nb = (p.n + 127) / 128;
  float acc[4][4] = {}, blk[4][4] = {};
  for (int64_t l0 = 0; l0 < p.k; l0 += kTileK) {
    for (int e = threadIdx.x; e < kTileK * kTileM; e += 256) {
      const int l = e % kTileK, r = e / kTileK;
      const bool in = l0 + l < p.k;
      as[l][r] = in && i0 + r < p.m ? from_fp8<kA5>(p.a[(i0 + r) * p.a_ld + l0 + l]) : 0.f;
      bs[l][r] = in && j0 + r < p.n ? from_fp8<kB5>(p.b[(j0 + r) * p.b_ld + l0 + l]) : 0.f;
    }
    __syncthreads();
    for (int l = 0; l < kTileK; ++l)
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          blk[u][v] = fmaf(as[l][ty * 4 + u], bs[l][tx * 4 + v], blk[u][v]);
    __syncthreads();
    if ((l0 + kTileK) % kFp8Block == 0 || l0 + kTileK >= p.k) {
      const int64_t c = l0 / kFp8Block;
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int64_t i = i0 + ty * 4 + u, j = j0 + tx * 4 + v;
          if (i < p.m && j < p.n)
            acc[u][v] = fmaf(p.a_scales[c * p.m + i] * p.b_scales[c * nb + j / 128], blk[u][v],
                             acc[u][v]);
          blk[u][v] = 0.f;
        }
    }
  }
#pragma unroll
  for (int u = 0; u < 4; ++u)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int64_t i = i0 + ty * 4 + u, j = j0 + tx * 4 + v;
      if (i < p.m && j < p.n) static_cast<TOut*>(p.out)[i * p.n + j] = from_f32<TOut>(acc[u][v]);
    }
}

template <bool kA5, bool kB5>
pe_status launch(const Args& p, pe_dtype out_dtype, cudaStream_t stream) {
  const dim3 grid((unsigned)ceil_div(p.m, kTileM), (unsigned)ceil_div(p.n, kTileN));
  if (out_dtype == PE_FP32)
    matmul_simple_kernel<kA5, kB5, float><<<grid, 256, 0, stream>>>(p);
  else
    matmul_simple_kernel<kA5, kB5, __nv_bfloat16><<<grid, 256, 0, stream>>>(p);
  PE_CUDA_TRY(cudaGetLastError());
  return PE_OK;
}

}  // namespace

}  // namespace pe

using namespace pe;

extern "C" size_t pe_matmul_fp8_workspace_size(int64_t m, int64_t n, int64_t k) {
  (void)m;
  (void)n;
  (void)k;
  return 0;
}

extern "C" pe_status pe_matmul_fp8(pe_fp8_type a_type, const void* a, int64_t a_ld,
                                   const float* a_scales, pe_fp8_type b_type, const void* b,
                                   int64_t b_ld, const float* b_scales, int64_t m, int64_t n,
                                   int64_t k, pe_dtype out_dtype, void* out, void* workspace,
                                   size_t workspace_bytes, pe_stream_t stream_) {
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (!fp8_type_ok(a_type) || !fp8_type_ok(b_type) ||
      (out_dtype != PE_BF16 && out_dtype != PE_FP32))
    return PE_ERR_UNSUPPORTED;
  if (m < 0 || n < 0 || k < 0) return PE_ERR_INVALID_ARG;
  if (m >= (1LL << 31) || n >= (1LL << 31) || k >= (1LL << 31)) return PE_ERR_OVERFLOW;
  if (ceil_div(n, kTileN) > 65535) return PE_ERR_OVERFLOW;
  if (m == 0 || n == 0) return PE_OK;
  if (!out || (k > 0 && (!a || !b || !a_scales || !b_scales))) return PE_ERR_INVALID_ARG;
  if (k > 0 && (!fp8_layout_ok(a, a_ld, k) || !fp8_layout_ok(b, b_ld, k)))
    return PE_ERR_UNSUPPORTED;
  if (!device_is_sm103()) return PE_ERR_UNSUPPORTED;
  if (k == 0) {
    PE_CUDA_TRY(cudaMemsetAsync(out, 0, (size_t)m * (size_t)n * (out_dtype == PE_FP32 ? 4 : 2),
                                stream));
    return PE_OK;
  }
  (void)workspace;
  (void)workspace_bytes;
  const Args p = {static_cast<const uint8_t*>(a), static_cast<const uint8_t*>(b), a_ld, b_ld, m,
                  n, k, a_scales, b_scales, out};
  if (a_type == PE_E5M2)
    return b_type == PE_E5M2 ? launch<true, true>(p, out_dtype, stream)
                             : launch<true, false>(p, out_dtype, stream);
  return b_type == PE_E5M2 ? launch<false, true>(p, out_dtype, stream)
                           : launch<false, false>(p, out_dtype, stream);
}

extern "C" pe_status pe_read_matmul_status(pe_stream_t stream_) {
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  void* word = nullptr;
  if (cudaGetSymbolAddress(&word, g_matmul_status) != cudaSuccess) return PE_ERR_CUDA;
  DeviceStatus st = {};
  PE_CUDA_TRY(cudaMemcpyAsync(&st, word, sizeof(st), cudaMemcpyDeviceToHost, stream));
  PE_CUDA_TRY(cudaMemsetAsync(word, 0, sizeof(st), stream));
  PE_CUDA_TRY(cudaStreamSynchronize(stream));
  return static_cast<pe_status>(st.code);
}
