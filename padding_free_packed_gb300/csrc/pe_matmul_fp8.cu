// Matrix product of 8-bit operands with a scale for each block of 128.
#include <atomic>

#include "pe_matmul_fp8.cuh"

namespace pe {

namespace {

// The kernels hold row, column and k coordinates of whole tiles in int32.
constexpr int64_t kMaxSize = (1LL << 31) - 1024;

__device__ DeviceStatus g_matmul_status;

constexpr int kMaxDevices = 64;
std::atomic<DeviceStatus*> g_status_address[kMaxDevices];

// The status word's address on the current device.
pe_status status_word(DeviceStatus** out) {
  int dev = 0;
  PE_CUDA_TRY(cudaGetDevice(&dev));
  if (dev < 0 || dev >= kMaxDevices) return PE_ERR_CUDA;
  DeviceStatus* word = g_status_address[dev].load();
  if (!word) {
    void* p = nullptr;
    PE_CUDA_TRY(cudaGetSymbolAddress(&p, g_matmul_status));
    word = static_cast<DeviceStatus*>(p);
    g_status_address[dev].store(word);
  }
  *out = word;
  return PE_OK;
}

}  // namespace

}  // namespace pe

using namespace pe;

extern "C" size_t pe_matmul_fp8_workspace_size(int64_t m, int64_t n, int64_t k) {
  if (m <= 0 || n <= 0 || k <= 0) return 0;
  return matmul_pair_workspace(m, n, k);
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
  if (m >= kMaxSize || n >= kMaxSize || k >= kMaxSize) return PE_ERR_OVERFLOW;
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
  const size_t need = pe_matmul_fp8_workspace_size(m, n, k);
  if (need && (!workspace || !aligned(workspace, 16) || workspace_bytes < need))
    return PE_ERR_WORKSPACE;
  DeviceStatus* status = nullptr;
  PE_TRY(status_word(&status));
  const MatmulFp8 p = {static_cast<const uint8_t*>(a),
                       static_cast<const uint8_t*>(b),
                       a_ld,
                       b_ld,
                       a_scales,
                       b_scales,
                       (int32_t)m,
                       (int32_t)n,
                       (int32_t)k,
                       a_type == PE_E5M2,
                       b_type == PE_E5M2,
                       out_dtype == PE_FP32,
                       out};
  return matmul_pair(p, workspace, status, stream);
}

extern "C" pe_status pe_read_matmul_status(pe_stream_t stream_) {
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  DeviceStatus* word = nullptr;
  PE_TRY(status_word(&word));
  DeviceStatus st = {};
  PE_CUDA_TRY(cudaMemcpyAsync(&st, word, sizeof(st), cudaMemcpyDeviceToHost, stream));
  PE_CUDA_TRY(cudaMemsetAsync(word, 0, sizeof(st), stream));
  PE_CUDA_TRY(cudaStreamSynchronize(stream));
  return static_cast<pe_status>(st.code);
}
