// Matrix product of 8-bit operands with a scale for each block of 128: the C entry,
// the choice among the kernels, and the status word of their waits.
#include <cudaTypedefs.h>

#include <atomic>

#include "pe_matmul_fp8.cuh"

namespace pe {

namespace {

// The kernels hold row, column and k coordinates of whole tiles in int32.
constexpr int64_t kMaxSize = (1LL << 31) - 1024;
// They count blocks of 256 x 256 x 128 in int32 too. Sizes up to kMaxSize give up to
// 2^70 of them, hence the quotient.
bool sizes_ok(int64_t m, int64_t n, int64_t k) {
  constexpr int64_t kMaxBlocks = 1LL << 30;
  if (m >= kMaxSize || n >= kMaxSize || k >= kMaxSize) return false;
  if (m == 0 || n == 0 || k == 0) return true;
  return ceil_div(m, 256) * ceil_div(n, 256) <= (kMaxBlocks - 1) / ceil_div(k, kFp8Block);
}

__device__ DeviceStatus g_matmul_status;

constexpr int kMaxDevices = 64;
std::atomic<DeviceStatus*> g_status_address[kMaxDevices];

std::atomic<PFN_cuTensorMapEncodeTiled_v12000> g_encode{nullptr};

}  // namespace

// The status word's address on the current device.
pe_status matmul_status_word(DeviceStatus** out) {
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

// Estimated microseconds of every way, from times measured on a GB300 (m x n x k,
// bf16 out; T: rows of a per CTA, S: split; pair: whole tiles of the pair kernel, runs:
// equal runs of blocks):
//   1 x 2304 x 768     T16 4.4   T32 4.9   T64 5.9   pair 8.9
//   320 x 2304 x 768   T16 8.9   T32 6.6   T64 6.7   pair 8.8
//   640 x 2304 x 768   T16 13.0  T32 9.9   T64 8.5   pair 8.8
//   2500 x 2304 x 768                      T64 20.1  pair 12.6, runs 22.6
//   768 x 768 x 9001             T64,S2 21.0         pair 34.9, runs 18.7
//   200 x 200 x 20000  T16,S8 11.8  T32,S8 11.0  T64,S8 13.4
// A narrow CTA takes kFixed and kBlock for each block of k; CTAs that share an SM slow
// each other, and the join of a split costs kJoin. Splitting pays from a sum of 7 blocks
// on, with two blocks or more a CTA (S1 and the best split):
//   6 blocks  1 x 2304 x 768 4.4, 4.5    64 x 768 x 768 4.8, 5.05   200 x 768 x 768 4.9, 5.2
//   7 blocks  1 x 1024 x 896 4.9, S3 4.85, S7 4.5
//   8 blocks  1 x 2304 x 1024 5.2, S4 4.7, S8 5.3    1 x 1024 x 1024 5.2, S4 4.7, S8 4.8
// Whole tiles take 0.41 for each block of a wave of pairs; runs have no last wave, but
// parts, a second kernel and worse sharing of the operands in L2:
//   2304 x 768, 27 tiles   k 4097: whole 20.1, runs 21.7   5000: 22.9, 23.4   6000: 26.0, 24.8
//                          k 9000: 36, 28.5                32299: 109, 62
//   2304 x 1152, 45 tiles  k 4096: whole 19.8, runs 26.2   9000: 36.4, 37.5   32299: 118, 102
//   2304 x 2304, 81 tiles  k 4096: whole 34.5, runs 36.1   6000: 47.5, 44.2   8192: 60.6, 52.1
//   128 tiles, 64 blocks: whole 61.3, runs 71.5            160, 16: 28.8, 38.2
//   256 tiles, 128 blocks: 229, 231    400, 40: 112, 123   1024, 64: 404, 449
// Beyond two tiles a pair runs are never better, and are not asked for.
MatmulPlan matmul_plan(int64_t m, int64_t n, int64_t k) {
  constexpr int64_t kSms = 152, kPairs = kSms / 2;
  const int64_t blocks = ceil_div(k, kFp8Block);
  const int64_t tiles = ceil_div(m, 256) * ceil_div(n, 256);
  const double whole = 6 + (double)ceil_div(tiles, kPairs) * (0.41 * (double)blocks + 1);
  const double runs = 15 + 0.045 * (double)tiles + 0.48 * (double)(tiles * blocks) / kPairs;
  MatmulPlan plan = {0, 1, tiles <= 2 * kPairs && runs < whole};
  double best = plan.runs ? runs : whole;
  constexpr int32_t kRows[3] = {16, 32, 64};
  constexpr double kFixed[3] = {3.0, 3.4, 3.6}, kBlock[3] = {0.285, 0.30, 0.43},
                   kJoin[3] = {0.8, 0.8, 1.5};
  for (int i = 0; i < 3; ++i) {
    const int64_t ctas = ceil_div(m, kRows[i]) * ceil_div(n, 128);
    if (ctas > 8 * kSms || ceil_div(m, kRows[i]) > 65535) continue;
    int64_t split = kSms / ctas < blocks / 2 ? kSms / ctas : blocks / 2;
    split = blocks < 7 || split < 1 ? 1 : split > 8 ? 8 : split;
    const double shared = (double)ceil_div(ctas * split, kSms) - 1;
    const double t = kFixed[i] + kBlock[i] * (double)ceil_div(blocks, split) * (1 + 0.6 * shared) +
                     1.2 * shared + (split > 1 ? kJoin[i] : 0);
    if (t < best) {
      best = t;
      plan = {kRows[i], (int32_t)split, false};
    }
  }
  return plan;
}

pe_status matmul_map(CUtensorMap* map, CUtensorMapDataType type, int size, const void* base,
                     int64_t rows, int64_t cols, int64_t pitch, uint32_t box_rows) {
  return matmul_map_planes(map, type, size, base, rows, cols, pitch, box_rows, 0);
}

pe_status matmul_map_planes(CUtensorMap* map, CUtensorMapDataType type, int size,
                            const void* base, int64_t rows, int64_t cols, int64_t pitch,
                            uint32_t box_rows, int32_t planes) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = g_encode.load();
  if (!encode) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult qres;
    PE_CUDA_TRY(cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000,
                                                 cudaEnableDefault, &qres));
    if (qres != cudaDriverEntryPointSuccess || !fn) return PE_ERR_CUDA;
    encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    g_encode.store(encode);
  }
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                        static_cast<cuuint64_t>(planes)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(pitch),
                           static_cast<cuuint64_t>(pitch) * static_cast<cuuint64_t>(rows)};
  cuuint32_t box[3] = {128u / size, box_rows, 1};
  cuuint32_t elem_strides[3] = {1, 1, 1};
  CUresult r = encode(map, type, planes ? 3 : 2, const_cast<void*>(base), dims, strides, box,
                      elem_strides, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                      CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? PE_OK : PE_ERR_CUDA;
}

}  // namespace pe

using namespace pe;

extern "C" size_t pe_matmul_fp8_workspace_size(int64_t m, int64_t n, int64_t k) {
  if (m <= 0 || n <= 0 || k <= 0 || !sizes_ok(m, n, k)) return 0;
  return matmul_plan(m, n, k).runs ? matmul_pair_workspace() : 0;
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
  if (!sizes_ok(m, n, k)) return PE_ERR_OVERFLOW;
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
  const MatmulPlan plan = matmul_plan(m, n, k);
  const size_t need = plan.runs ? matmul_pair_workspace() : 0;
  if (need && (!workspace || !aligned(workspace, 16) || workspace_bytes < need))
    return PE_ERR_WORKSPACE;
  DeviceStatus* status = nullptr;
  PE_TRY(matmul_status_word(&status));
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
  if (plan.rows) return matmul_rows(p, plan.rows, plan.split, status, stream);
  return matmul_pair(p, plan.runs, workspace, status, stream);
}

extern "C" pe_status pe_read_matmul_status(pe_stream_t stream_) {
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  DeviceStatus* word = nullptr;
  PE_TRY(matmul_status_word(&word));
  DeviceStatus st = {};
  PE_CUDA_TRY(cudaMemcpyAsync(&st, word, sizeof(st), cudaMemcpyDeviceToHost, stream));
  PE_CUDA_TRY(cudaMemsetAsync(word, 0, sizeof(st), stream));
  PE_CUDA_TRY(cudaStreamSynchronize(stream));
  return static_cast<pe_status>(st.code);
}
