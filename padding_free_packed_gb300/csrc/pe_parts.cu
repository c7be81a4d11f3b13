// Sums over rows that a backward's blocks left one line each.
#include "pe_vec.cuh"

namespace pe {

namespace {

// 32 columns per block, 32 rows of threads, each adding every 32nd line. `part` is not
// __restrict__: the kernel before may still write it at this one's start, so its loads must
// not pass for loads of constant memory, which could be moved before the wait.
__global__ void __launch_bounds__(1024)
sum_parts_kernel(const float* part, int32_t blocks, int32_t c0, float* out0, int32_t c1,
                 float* out1) {
  __shared__ float sum[32][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int32_t cols = c0 + c1, c = blockIdx.x * 32 + x;
  griddep_wait();
  float s = 0.f;
  if (c < cols) {
    for (int32_t b = y; b < blocks; b += 320) {                       // ten lines in flight
      float v[10];
#pragma unroll
      for (int j = 0; j < 10; ++j)
        v[j] = b + 32 * j < blocks ? part[(int64_t)(b + 32 * j) * cols + c] : 0.f;
#pragma unroll
      for (int j = 0; j < 10; ++j) s += v[j];
    }
  }
  sum[y][x] = s;
  __syncthreads();
  s = warp_sum(sum[x][y]);
  const int32_t to = blockIdx.x * 32 + y;
  if (x == 0 && to < cols) {
    if (to < c0)
      out0[to] = s;
    else if (out1)
      out1[to - c0] = s;
  }
}

}  // namespace

pe_status launch_sum_parts(const float* part, int32_t blocks, int32_t c0, float* out0, int32_t c1,
                           float* out1, cudaStream_t stream) {
  return launch_after_previous(sum_parts_kernel, dim3((unsigned)ceil_div(c0 + c1, 32)),
                               dim3(1024), 0, stream, part, blocks, c0, out0, c1, out1);
}

}  // namespace pe
