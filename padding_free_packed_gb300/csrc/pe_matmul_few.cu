// Matrix product with bias, activation and residual, fp32 operands and few products, such as a
// token's: out = act(a b^T + bias) + residual.
//
// A single token's product reads b once and little else. In parts of bf16 b is read and
// written twice over in another kernel first; here it is multiplied as it lies, by fp32
// multiply-adds, since four rows of them for each number of b are less than its way from HBM.
// A warp takes a column of out (a row of b; with geglu the gate's and the up part's) in
// pieces of 512 bytes, up to eight warps of a block share the column's sum over k where there
// are few columns, and join in the order of k. An infinity or a NaN of an operand makes its
// sums NaN, as in the products by parts: x - x, 0 or NaN, is added up beside the products.
// Measured (GB300, device time; by parts on the tensor cores): 1 x 2304 x 768 3.7 us (11.7), 1 x
// 768 x 768 2.7 (9.5), 1 x 64 x 30000 6.0 (60), 1 x 8192 x 8192 53 us (212; 5.0 TB/s, 0.74 of
// the measured copy rate), 4 x 2304 x 768 5.4 (11.9), 16 x 768 x 768 6.6 (9.8). What bounds it is
// bytes in flight, with four rows the loads of a from the caches. Loads of b eight steps ahead
// and a's in turn took 1 x 8192 x 8192 from 69 us (four ahead) to 53; masked steps instead of
// shorter batches at the end took it to 76.
#include <type_traits>

#include "pe_matmul.cuh"

namespace pe {

namespace {

using namespace sm103;

constexpr int kThreads = 256, kWarps = kThreads / 32;

struct Params {
  MatmulEpilogue e;
  const float* a;
  const float* b;
  int64_t a_ld, b_ld;
  int32_t k;
  int32_t split;             // warps of a column: 1, 2, 4 or 8
  int32_t groups;            // of rows of a
};

// Products of V neighbouring elements of k, and their x - x.
template <int M, int kCols, int V>
struct Sums {
  float s[M][kCols][V], bad_a[M], bad_b[kCols];

  __device__ Sums() {
#pragma unroll
    for (int m = 0; m < M; ++m) {
      bad_a[m] = 0.f;
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        bad_b[c] = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) s[m][c][v] = 0.f;
      }
    }
  }
  __device__ __forceinline__ void add(const float (&x)[M][V], const float (&y)[kCols][V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int m = 0; m < M; ++m) bad_a[m] += x[m][v] - x[m][v];
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        bad_b[c] += y[c][v] - y[c][v];
#pragma unroll
        for (int m = 0; m < M; ++m) s[m][c][v] = fmaf(x[m][v], y[c][v], s[m][c][v]);
      }
    }
  }
  __device__ float of(int m, int c) const {
    float t = bad_a[m] + bad_b[c];
#pragma unroll
    for (int v = 0; v < V; ++v) t += s[m][c][v];
    return t;
  }
};

template <int V>
__device__ __forceinline__ void load_v(const float* p, float (&x)[V]) {
  if constexpr (V == 4) {
    const float4 q = *reinterpret_cast<const float4*>(p);
    x[0] = q.x, x[1] = q.y, x[2] = q.z, x[3] = q.w;
  } else {
    x[0] = *p;
  }
}

// V: 4 where rows start at multiples of 16 bytes. Pointers are not __restrict__: the kernel
// before may still write what they show at this one's start.
template <int M, int V, int kAct>
__global__ void __launch_bounds__(kThreads)
matmul_few_kernel(const __grid_constant__ Params p) {
  constexpr int kCols = kAct == PE_ACT_GEGLU ? 2 : 1;
  __shared__ float joined[kWarps][M][kCols];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t columns = kWarps / p.split;                // of this block
  const int32_t own = warp / p.split, slice = warp - own * p.split;
  // Blocks of the same columns are neighbours, so that they find b in L2.
  const int32_t block = blockIdx.x / p.groups, row0 = (blockIdx.x - block * p.groups) * M;
  const int32_t col = block * columns + own;
  griddep_wait();                          // what the kernel before this one wrote is read below
  griddep_launch_dependents();             // the next one waits for this one's end in turn
  if (col < p.e.n) {
    const float* b[kCols];
#pragma unroll
    for (int c = 0; c < kCols; ++c) b[c] = p.b + ((int64_t)c * p.e.n + col) * p.b_ld;
    const float* a[M];
#pragma unroll
    for (int m = 0; m < M; ++m)                            // past the last row: the first
      a[m] = p.a + (row0 + m < p.e.m ? row0 + m : row0) * p.a_ld;
    Sums<M, kCols, V> sums;
    const int32_t whole = p.k / V, step = 32 * p.split;
    auto load_b = [&](int32_t i, float (&y)[kCols][V]) {
#pragma unroll
      for (int c = 0; c < kCols; ++c) load_v<V>(b[c] + (int64_t)i * V, y[c]);
    };
    auto add = [&](int32_t i, const float (&y)[kCols][V]) {
      float x[M][V];
#pragma unroll
      for (int m = 0; m < M; ++m) load_v<V>(a[m] + (int64_t)i * V, x[m]);
      sums.add(x, y);
    };
    // b, from HBM, several steps ahead; a, from the caches, when it is its turn.
    int32_t i = slice * 32 + lane;
    auto steps = [&](auto flight) {
      constexpr int kF = decltype(flight)::value;
      for (; i < whole - (kF - 1) * step; i += kF * step) {
        float y[kF][kCols][V];
#pragma unroll
        for (int f = 0; f < kF; ++f) load_b(i + f * step, y[f]);
#pragma unroll
        for (int f = 0; f < kF; ++f) add(i + f * step, y[f]);
      }
    };
    steps(std::integral_constant<int, 8 / kCols>());
    steps(std::integral_constant<int, 3>());
    steps(std::integral_constant<int, 1>());
    if (V > 1 && slice == 0 && lane < p.k - whole * V) {   // the last elements of k
      float x[M][V] = {}, y[kCols][V] = {};
#pragma unroll
      for (int c = 0; c < kCols; ++c) y[c][0] = b[c][whole * V + lane];
#pragma unroll
      for (int m = 0; m < M; ++m)
        x[m][0] = a[m][whole * V + lane];
      sums.add(x, y);
    }
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        float t = sums.of(m, c);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
        if (lane == 0) joined[warp][m][c] = t;
      }
  }
  __syncthreads();
  // A thread for each column and row.
  const int32_t at = threadIdx.x / M, of_group = threadIdx.x % M, row = row0 + of_group;
  const int32_t out_col = block * columns + at;
  if (at >= columns || out_col >= p.e.n || row >= p.e.m) return;
  float z[kCols];
#pragma unroll
  for (int c = 0; c < kCols; ++c) {
    z[c] = 0.f;
    for (int s = 0; s < p.split; ++s) z[c] += joined[at * p.split + s][of_group][c];
    if (p.e.bias) z[c] += io_get(p.e.bias, (int64_t)c * p.e.n + out_col, p.e.out_fp32);
  }
  float y = z[0];
  if constexpr (kAct == PE_ACT_RELU) y = y < 0.f ? 0.f : y;
  if constexpr (kAct >= PE_ACT_GELU) y = gelu_fp32(y);
  if constexpr (kAct == PE_ACT_GEGLU) y *= z[1];
  if (p.e.residual) y += io_get(p.e.residual, row * p.e.residual_ld + out_col, p.e.out_fp32);
  if (p.e.pre) {
#pragma unroll
    for (int c = 0; c < kCols; ++c)
      io_put(p.e.pre, row * p.e.pre_ld + (int64_t)c * p.e.n + out_col, p.e.out_fp32, z[c]);
  }
  io_put(p.e.out, row * p.e.out_ld + out_col, p.e.out_fp32, y);
}

template <int M, int V>
pe_status launch(Params p, cudaStream_t stream) {
  const auto kernel = p.e.act == PE_ACT_GEGLU  ? matmul_few_kernel<M, V, PE_ACT_GEGLU>
                      : p.e.act == PE_ACT_GELU ? matmul_few_kernel<M, V, PE_ACT_GELU>
                      : p.e.act == PE_ACT_RELU ? matmul_few_kernel<M, V, PE_ACT_RELU>
                                               : matmul_few_kernel<M, V, PE_ACT_NONE>;
  p.groups = (int32_t)ceil_div(p.e.m, M);
  const int64_t blocks = ceil_div(p.e.n, kWarps / p.split) * p.groups;
  return launch_after_previous(kernel, dim3((unsigned)blocks), dim3(kThreads), 0, stream, p);
}

}  // namespace

pe_status matmul_few(const Matmul& q, cudaStream_t stream) {
  Params p = {q.e,    static_cast<const float*>(q.a.base), static_cast<const float*>(q.b.base),
              q.a.ld, q.b.ld,                              q.k,
              1,      1};
  // Sixteen warps an SM where there are columns and elements of k enough for them.
  while (p.split < kWarps && (int64_t)p.e.n * p.split * ceil_div(p.e.m, 4) < 16 * 152 && q.k >= 512 * p.split)
    p.split *= 2;
  const bool vector = aligned(p.a, 16) && aligned(p.b, 16) && p.b_ld % 4 == 0 &&
                      (p.a_ld % 4 == 0 || p.e.m == 1);
  if (p.e.m == 1) return vector ? launch<1, 4>(p, stream) : launch<1, 1>(p, stream);
  if (p.e.m == 2) return vector ? launch<2, 4>(p, stream) : launch<2, 1>(p, stream);
  return vector ? launch<4, 4>(p, stream) : launch<4, 1>(p, stream);
}

}  // namespace pe
