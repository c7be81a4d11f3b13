// Backward of the matrix product's activation and bias: dz = dy act'(z), and the sums of dz
// over the rows, dbias. With geglu, z = (gate, up), y = gelu(gate) up:
//   dgate = dy up gelu'(gate), dup = dy gelu(gate).
// A bandwidth kernel: dy and z are read once and dz written once; a thread keeps the sums of
// its own columns in fp32 registers over all of its rows, the warps of a block add theirs in
// shared memory, and a second kernel adds the blocks' lines in a fixed order.
// Measured (GB300, device time): 32299 x 1152 bf16 geglu in 60 us (6.2 TB/s, 0.91 of the
// measured copy rate), gelu 41 us (0.80), relu 37 us (0.89), column sums alone 169151 x 1024
// 53.6 us (0.95), 20000 x 1152 fp32 geglu 80 us (0.85). A grid that the device holds at a time
// took 64 us to 60, paired arithmetic 68 to 64. bf16 rows of odd width move two bytes at a time
// (20000 x 1001 gelu 50 us, 0.36).
#include <math.h>

#include "pe_act.cuh"
#include "pe_vec.cuh"

namespace pe {

namespace {

constexpr int kThreads = 256;
constexpr int kLanes = 16;                     // threads across a block's columns
constexpr int kRowLanes = kThreads / kLanes;
constexpr int kMaxBlocks = 304;                // along the rows

template <typename T>
struct Args {
  const T* dy;           // dy and z may be dz: not read through the read-only path
  const T* z;
  int64_t rows;
  int32_t features;
  T* dz;
  float* part;           // [gridDim.y][columns of z], or null
  float* dbias;          // few rows: written by the strip's cluster of gridDim.y blocks
};

// Rows that a cluster of eight blocks takes for each strip of columns, 16 for each of a
// block's threads (1001 x 333 gelu fp32: one launch 5.5 us, two 8.3).
constexpr int64_t kFewRows = 16 * kClusterLines * kRowLanes;


// V neighbouring columns per access, kRows rows of a thread in flight.
template <typename T, int V, int kAct, int kRows>
__global__ void __launch_bounds__(kThreads)
activation_bwd_kernel(const Args<T> a) {
  constexpr int kParts = kAct == PE_ACT_GEGLU ? 2 : 1;
  constexpr bool kPaired = kAct >= PE_ACT_GELU && sizeof(T) == 2 && V > 1;
  __shared__ float sums[kRowLanes][kParts][kLanes * V];
  const int x = threadIdx.x % kLanes, y = threadIdx.x / kLanes;
  const int32_t F = a.features, c = (blockIdx.x * kLanes + x) * V;
  const int64_t ld = (int64_t)kParts * F;
  float sum[kParts][V];
#pragma unroll
  for (int p = 0; p < kParts; ++p)
#pragma unroll
    for (int v = 0; v < V; ++v) sum[p][v] = 0.f;
  if (c < F) {
    const int64_t step = (int64_t)gridDim.y * kRowLanes;
    for (int64_t r0 = (int64_t)blockIdx.y * kRowLanes + y; r0 < a.rows; r0 += kRows * step) {
      Vec<T, V> dy[kRows], z[kRows][kParts];
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        const int64_t r = r0 + u * step;
        if (r < a.rows) {
          dy[u] = load_vec<T, V>(a.dy + r * F + c);
          if constexpr (kAct != PE_ACT_NONE) {
#pragma unroll
            for (int p = 0; p < kParts; ++p) z[u][p] = load_vec<T, V>(a.z + r * ld + p * F + c);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        const int64_t r = r0 + u * step;
        if (r < a.rows) {
          float d[kParts][V];
          if constexpr (kPaired) {
            using namespace sm103;
#pragma unroll
            for (int j = 0; j < V / 2; ++j) {
              const float z0 = z[u][0].get(2 * j), z1 = z[u][0].get(2 * j + 1);
              const GeluPair at(z0, z1);
              const uint64_t g = dy[u].pair(j), slope = at.slope(z0, z1);
              if constexpr (kAct == PE_ACT_GEGLU) {
                f2_split(fmul2(fmul2(g, z[u][1].pair(j)), slope), d[0][2 * j], d[0][2 * j + 1]);
                f2_split(fmul2(g, at.value(z0, z1)), d[1][2 * j], d[1][2 * j + 1]);
              } else {
                f2_split(fmul2(g, slope), d[0][2 * j], d[0][2 * j + 1]);
              }
            }
          }
#pragma unroll
          for (int v = 0; v < (kPaired ? 0 : V); ++v) {
            const float g = dy[u].get(v);
            if constexpr (kAct == PE_ACT_GEGLU) {
              float value;
              const float slope = gelu_slope<T>(z[u][0].get(v), value);
              d[0][v] = g * z[u][1].get(v) * slope;
              d[1][v] = g * value;
            } else if constexpr (kAct == PE_ACT_GELU) {
              float value;
              d[0][v] = g * gelu_slope<T>(z[u][0].get(v), value);
            } else if constexpr (kAct == PE_ACT_RELU) {
              d[0][v] = z[u][0].get(v) > 0.f ? g : 0.f;
            } else {
              d[0][v] = g;
            }
          }
#pragma unroll
          for (int p = 0; p < kParts; ++p) {
#pragma unroll
            for (int v = 0; v < V; ++v) sum[p][v] += d[p][v];
            if constexpr (kAct != PE_ACT_NONE) {
              Vec<T, V> o;
              o.put(d[p]);
              store_vec<T, V>(a.dz + r * ld + p * F + c, o);
            }
          }
        }
      }
    }
  }
  if (!a.part && !a.dbias) return;
  griddep_launch_dependents();                 // the second kernel may come to wait for this one
#pragma unroll
  for (int p = 0; p < kParts; ++p)
#pragma unroll
    for (int v = 0; v < V; ++v) sums[y][p][x * V + v] = sum[p][v];
  __syncthreads();
  __shared__ float line[kParts * kLanes * V];  // this block's sums of the strip's columns
  for (int e = threadIdx.x; e < kParts * kLanes * V; e += kThreads) {
    const int p = e / (kLanes * V), at = e % (kLanes * V);
    const int32_t col = blockIdx.x * kLanes * V + at;
    float total = 0.f;
#pragma unroll
    for (int i = 0; i < kRowLanes; ++i) total += sums[i][p][at];
    if (!a.part)
      line[e] = total;
    else if (col < F)
      a.part[(int64_t)blockIdx.y * ld + (int64_t)p * F + col] = total;
  }
  if (a.part) return;
  // The strip's gate columns, then its up columns.
  const int32_t first = blockIdx.x * kLanes * V;
  const int32_t wide = F - first < kLanes * V ? F - first : kLanes * V;
  sm103::cluster_sync();                       // every block's line is complete
  const uint32_t here = sm103::smem_u32(line), blocks = gridDim.y;
  for (int e = (int)(blockIdx.y * kThreads + threadIdx.x); e < kParts * kLanes * V;
       e += (int)blocks * kThreads) {
    const int p = e / (kLanes * V), at = e % (kLanes * V);
    float total = 0.f;
    for (uint32_t b = 0; b < blocks; ++b)
      total += sm103::load_cluster_f32(sm103::peer_address(here + 4 * e, b));
    if (at < wide) a.dbias[(int64_t)p * F + first + at] = total;
  }
  sm103::cluster_sync();                       // the lines have been read
}

template <typename T, int V, int kAct>
pe_status launch(const Args<T>& a, cudaStream_t stream) {
  // 6 to 8 loads of a thread in flight, with narrow ones more.
  constexpr int kRows = (kAct == PE_ACT_NONE ? 8 : kAct == PE_ACT_GEGLU ? 2 : 4) *
                        (kAct != PE_ACT_NONE && V * sizeof(T) < 16 ? 2 : 1);
  constexpr int kParts = kAct == PE_ACT_GEGLU ? 2 : 1;
  const int64_t strips = ceil_div(a.features, kLanes * V);
  int64_t lines = ceil_div(a.rows, kRowLanes);
  if (a.dbias && a.rows <= kFewRows) {
    if (lines > kClusterLines) lines = kClusterLines;
    Args<T> few = a;
    few.part = nullptr;
    return launch_clusters(activation_bwd_kernel<T, V, kAct, kRows>,
                           dim3((unsigned)strips, (unsigned)lines), dim3(1, (unsigned)lines),
                           kThreads, 0, stream, few);
  }
  static DeviceNumber known;
  const int resident =
      resident_blocks(activation_bwd_kernel<T, V, kAct, kRows>, kThreads, 0, known);
  if (resident < 1) return PE_ERR_CUDA;
  int64_t most = (int64_t)device_sm_count() * resident / strips;
  if (most < 1) most = 1;
  if (lines > most) lines = most;
  if (lines > kMaxBlocks) lines = kMaxBlocks;
  activation_bwd_kernel<T, V, kAct, kRows>
      <<<dim3((unsigned)strips, (unsigned)lines), kThreads, 0, stream>>>(a);
  PE_CUDA_TRY(cudaGetLastError());
  if (!a.part) return PE_OK;
  return launch_sum_parts(a.part, (int32_t)lines, kParts * a.features, a.dbias, 0, nullptr, stream);
}

template <typename T, int V>
pe_status launch_act(int act, const Args<T>& a, cudaStream_t stream) {
  switch (act) {
    case PE_ACT_GEGLU: return launch<T, V, PE_ACT_GEGLU>(a, stream);
    case PE_ACT_GELU: return launch<T, V, PE_ACT_GELU>(a, stream);
    case PE_ACT_RELU: return launch<T, V, PE_ACT_RELU>(a, stream);
    default: return launch<T, V, PE_ACT_NONE>(a, stream);
  }
}

template <typename T>
pe_status run(int act, const void* dy, const void* z, int64_t rows, int32_t features, void* dz,
              float* dbias, void* workspace, cudaStream_t stream) {
  const Args<T> a = {static_cast<const T*>(dy),
                     static_cast<const T*>(z),
                     rows,
                     features,
                     static_cast<T*>(dz),
                     dbias ? static_cast<float*>(workspace) : nullptr,
                     dbias};
  constexpr int V = 16 / sizeof(T);
  if (vectors<V>(features, a.dy, a.z, a.dz)) return launch_act<T, V>(act, a, stream);
  if (V > 4 && vectors<4>(features, a.dy, a.z, a.dz))
    return launch_act<T, 4>(act, a, stream);
  if (vectors<2>(features, a.dy, a.z, a.dz)) return launch_act<T, 2>(act, a, stream);
  return launch_act<T, 1>(act, a, stream);
}

// Columns of z are counted in int32, up to a block's past the last one.
constexpr int32_t kMaxFeatures = (1 << 30) - 1024;

}  // namespace

}  // namespace pe

using namespace pe;

extern "C" size_t pe_activation_bwd_workspace_size(pe_activation activation, int64_t rows,
                                                   int32_t features) {
  if (!activation_ok(activation) || rows <= kFewRows || features < 1 || features > kMaxFeatures)
    return 0;
  return (size_t)kMaxBlocks * (size_t)features * (activation == PE_ACT_GEGLU ? 2 : 1) *
         sizeof(float);
}

extern "C" pe_status pe_activation_bwd(pe_dtype dtype, pe_activation activation, const void* dy,
                                       const void* pre, int64_t rows, int32_t features, void* dz,
                                       float* dbias, void* workspace, size_t workspace_bytes,
                                       pe_stream_t stream_) {
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (dtype != PE_BF16 && dtype != PE_FP32) return PE_ERR_UNSUPPORTED;
  if (!activation_ok(activation) || rows < 0 || features < 1) return PE_ERR_INVALID_ARG;
  if (features > kMaxFeatures) return PE_ERR_OVERFLOW;
  if (activation == PE_ACT_NONE && (pre || dz || !dbias)) return PE_ERR_INVALID_ARG;
  if (!by_elements(PE_FP32, dbias)) return PE_ERR_UNSUPPORTED;
  if (rows > 0) {
    if (!dy || (activation != PE_ACT_NONE && (!pre || !dz))) return PE_ERR_INVALID_ARG;
    if (activation == PE_ACT_GEGLU && dz == dy) return PE_ERR_INVALID_ARG;
    if (!by_elements(dtype, dy, pre, dz)) return PE_ERR_UNSUPPORTED;
    const size_t need =
        dbias ? pe_activation_bwd_workspace_size(activation, rows, features) : 0;
    if (need && (!workspace || !aligned(workspace, 16) || workspace_bytes < need))
      return PE_ERR_WORKSPACE;
  }
  if (!device_is_sm103()) return PE_ERR_UNSUPPORTED;
  if (rows == 0) {
    if (dbias)
      PE_CUDA_TRY(cudaMemsetAsync(
          dbias, 0, (size_t)features * (activation == PE_ACT_GEGLU ? 8 : 4), stream));
    return PE_OK;
  }
  if (dtype == PE_FP32)
    return run<float>(activation, dy, pre, rows, features, dz, dbias, workspace, stream);
  return run<__nv_bfloat16>(activation, dy, pre, rows, features, dz, dbias, workspace, stream);
}
