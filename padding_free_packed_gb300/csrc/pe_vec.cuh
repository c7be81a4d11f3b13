// Rows of bf16 or fp32 moved in vectors, and sums over a warp and over the threads that
// share a row (internal header).
#pragma once

#include "pe_common.cuh"
#include "pe_sm103.cuh"

namespace pe {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kClusterLines = 8;               // blocks of a cluster that add their sums

// V consecutive elements of a row, kept as loaded: bf16 pairs stay in one register
// until they are used.
template <typename T, int V>
struct Vec;
template <int V>
struct alignas(4 * V) Vec<float, V> {
  float w[V];
  __device__ float get(int v) const { return w[v]; }
  __device__ uint64_t pair(int j) const { return sm103::f2(w[2 * j], w[2 * j + 1]); }
  __device__ void put_pair(int j, uint64_t x) { sm103::f2_split(x, w[2 * j], w[2 * j + 1]); }
  __device__ void zero() {
#pragma unroll
    for (int v = 0; v < V; ++v) w[v] = 0.f;
  }
  __device__ void put(const float* x) {
#pragma unroll
    for (int v = 0; v < V; ++v) w[v] = x[v];
  }
  __device__ void add(const Vec& o) {
#pragma unroll
    for (int v = 0; v < V; ++v) w[v] += o.w[v];
  }
};
template <int V>
struct alignas(2 * V) Vec<__nv_bfloat16, V> {
  uint32_t w[V / 2];
  __device__ float get(int v) const {
    return __uint_as_float(v & 1 ? w[v >> 1] & 0xffff0000u : w[v >> 1] << 16);
  }
  // Elements 2 j and 2 j + 1 for paired fp32 arithmetic, and back, rounded.
  __device__ uint64_t pair(int j) const { return sm103::f2(get(2 * j), get(2 * j + 1)); }
  __device__ void put_pair(int j, uint64_t x) {
    float lo, hi;
    sm103::f2_split(x, lo, hi);
    w[j] = sm103::pack_bf16x2(lo, hi);
  }
  __device__ void zero() {
#pragma unroll
    for (int v = 0; v < V / 2; ++v) w[v] = 0u;
  }
  __device__ void put(const float* x) {
#pragma unroll
    for (int v = 0; v < V / 2; ++v) {
      const __nv_bfloat162 pair = __floats2bfloat162_rn(x[2 * v], x[2 * v + 1]);
      w[v] = *reinterpret_cast<const uint32_t*>(&pair);
    }
  }
  // The rounded fp32 sum, two at a time: an fp32 sum of bf16 numbers is exact
  // unless one is below 2^-16 of the other, when rounding it first changes nothing.
  __device__ void add(const Vec& o) {
#pragma unroll
    for (int v = 0; v < V / 2; ++v) {
      const __nv_bfloat162 sum = __hadd2_rn(*reinterpret_cast<const __nv_bfloat162*>(&w[v]),
                                            *reinterpret_cast<const __nv_bfloat162*>(&o.w[v]));
      w[v] = *reinterpret_cast<const uint32_t*>(&sum);
    }
  }
};
template <>
struct Vec<__nv_bfloat16, 1> {
  __nv_bfloat16 w[1];
  __device__ float get(int) const { return __bfloat162float(w[0]); }
  __device__ void zero() { w[0] = __float2bfloat16_rn(0.f); }
  __device__ void put(const float* x) { w[0] = __float2bfloat16_rn(x[0]); }
  __device__ void add(const Vec& o) { w[0] = __float2bfloat16_rn(get(0) + o.get(0)); }
};

// One access of a vector's bytes.
template <int kBytes>
struct Bits;
template <>
struct Bits<2> { using type = uint16_t; };
template <>
struct Bits<4> { using type = uint32_t; };
template <>
struct Bits<8> { using type = uint2; };
template <>
struct Bits<16> { using type = uint4; };

template <typename T, int V>
__device__ __forceinline__ Vec<T, V> load_vec(const T* p) {
  using B = typename Bits<(int)sizeof(T) * V>::type;
  Vec<T, V> v;
  *reinterpret_cast<B*>(v.w) = *reinterpret_cast<const B*>(p);
  return v;
}
template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const Vec<T, V>& v) {
  using B = typename Bits<(int)sizeof(T) * V>::type;
  *reinterpret_cast<B*>(p) = *reinterpret_cast<const B*>(v.w);
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(kFull, x, off);
  return x;
}

// A barrier of the kGroup threads that share a row.
template <int kGroup>
__device__ __forceinline__ void group_sync(int group) {
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(kGroup) : "memory");
}

// The columns' sums that a backward's blocks leave, part[b][c] for c < c0 + c1, added in a
// fixed order: columns below c0 into out0, the others into out1 (unless that is null). Runs
// after the kernel before it in the stream.
pe_status launch_sum_parts(const float* part, int32_t blocks, int32_t c0, float* out0, int32_t c1,
                           float* out1, cudaStream_t stream);

// Few rows need no second kernel: the blocks form a cluster and add their lines in shared
// memory. `line` is this block's, at the same place in every block; the blocks deal the
// columns among them and add them in the order of the blocks.
__device__ __forceinline__ void sum_lines_of_cluster(const float* line, int32_t blocks, int32_t c0,
                                                     float* out0, int32_t c1, float* out1) {
  using namespace sm103;
  cluster_sync();                              // every block's line is complete
  const uint32_t here = smem_u32(line);
  const int32_t step = blocks * (int32_t)blockDim.x;
  for (int32_t c = (int32_t)(cluster_rank() * blockDim.x + threadIdx.x); c < c0 + c1; c += step) {
    float v[kClusterLines], s = 0.f;
#pragma unroll
    for (int b = 0; b < kClusterLines; ++b)
      v[b] = b < blocks ? load_cluster_f32(peer_address(here + 4 * c, b)) : 0.f;
#pragma unroll
    for (int b = 0; b < kClusterLines; ++b) s += v[b];
    if (c < c0)
      out0[c] = s;
    else if (out1)
      out1[c - c0] = s;
  }
  cluster_sync();                              // the lines have been read
}

// Whether rows of C channels and their tensors allow accesses of V channels.
template <int V, typename T, typename... P>
bool vectors(int32_t C, const T* p, P... rest) {
  bool ok = C % V == 0 && aligned(p, V * sizeof(T));
  ((ok = ok && aligned(rest, V * sizeof(T))), ...);
  return ok;
}

}  // namespace pe
