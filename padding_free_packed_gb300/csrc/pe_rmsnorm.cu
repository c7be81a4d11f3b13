// RMSNorm of packed token rows, with the residual's addition and an 8-bit
// output, and its backward.
//   forward:  h = x, or x + residual rounded to the I/O type (stored, and
//             normalised as stored); y = h rstd w, rstd = 1 / sqrt(mean(h^2) + eps);
//             in 8 bits: one scale for each 128 channels of a row.
//   backward: with n = h rstd, dx = rstd (w dy - n mean(w dy n)) (+ dresidual);
//             dw = sum over rows of dy n.
// All are bandwidth kernels: a row is read once, held in the registers of 1 to 8
// warps, and every output written once. Statistics, products and sums are fp32. Very
// wide rows take two passes of which the second finds the row in the caches.
// Measured (GB300, device time): forward with residual and 8-bit output 32299 x 768
// bf16 in 28.7 us (6.1 TB/s, 0.90 of the measured copy rate), 90487 x 500 fp32 in
// 42 us (0.81), one row of 768 in 1.7; backward with the residual's gradient 32299 x
// 768 bf16 in 39.3 us (5.05 TB/s, 0.74; 2 to 3 us of it the second kernel). The
// backward waits for memory: 64 threads a row with 16 weight sums each, three blocks of
// 256 threads an SM; rows through a shared-memory ring did not help (46.5 us). bf16 rows
// of odd width move two bytes at a time, 0.4 to 0.55 of the copy rate (32299 x 777 in 71
// us, backward 58); reading them by aligned 8-byte words shifted together, with the sum
// written two bytes at a time, took 81.
#include <math.h>

#include "pe_fp8.cuh"
#include "pe_vec.cuh"

namespace pe {

namespace {

constexpr int kThreads = 256;

// 8-bit output of a forward: none, e4m3 or e5m2.
enum Mode { kNoFp8 = 0, kE4M3 = 1, kE5M2 = 2 };

template <typename T>
struct FwdArgs {
  const T* x;          // may be res_out or y: not read through the read-only path
  const T* res;
  const T* w;
  int64_t N;
  int32_t C;
  float inv_c;         // 1 / C
  float eps;
  T* y;
  T* res_out;
  uint8_t* y8;
  int64_t y8_ld;
  float* scales;
};

// Channels of one step of a warp: U vectors of V per lane, lane-major inside a
// vector group, so a step covers 32 V U channels and always whole blocks of
// 128: one block for V U = 4 (32 lanes share it), two for V = 8 (16 lanes each).
template <int V, int U>
__device__ __forceinline__ int32_t channel(int32_t step, int u, int lane) {
  return (step * U + u) * 32 * V + lane * V;
}

// V neighbouring 8-bit values.
template <int V, bool e5>
__device__ __forceinline__ void store_fp8(uint8_t* p, const float* q, float f) {
  if constexpr (V == 8) {
    uint2 o;
    o.x = fp8x4<e5>(q[0] * f, q[1] * f, q[2] * f, q[3] * f);
    o.y = fp8x4<e5>(q[4] * f, q[5] * f, q[6] * f, q[7] * f);
    *reinterpret_cast<uint2*>(p) = o;
  } else if constexpr (V == 4) {
    *reinterpret_cast<uint32_t*>(p) = fp8x4<e5>(q[0] * f, q[1] * f, q[2] * f, q[3] * f);
  } else if constexpr (V == 2) {
    *reinterpret_cast<uint16_t*>(p) = (uint16_t)fp8x2<e5>(q[0] * f, q[1] * f);
  } else {
    *p = (uint8_t)fp8x2<e5>(q[0] * f, 0.f);
  }
}

// Output of one step from its h: y in T when wanted, and the 8-bit block.
template <typename T, int V, int U, int kMode>
__device__ __forceinline__ void emit(const FwdArgs<T>& a, int64_t t, int32_t step, int lane,
                                     const float (&h)[U * V], const Vec<T, V> (&w)[U],
                                     float rstd) {
  float y[U * V];
  float amax = 0.f;
#pragma unroll
  for (int u = 0; u < U; ++u) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      y[u * V + v] = h[u * V + v] * rstd * w[u].get(v);
      amax = max_nan(amax, fabsf(y[u * V + v]));
    }
  }
  if (a.y) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int32_t c = channel<V, U>(step, u, lane);
      if (c < a.C) {
        Vec<T, V> o;
        o.put(y + u * V);
        store_vec<T, V>(a.y + t * a.C + c, o);
      }
    }
  }
  if constexpr (kMode != kNoFp8) {
    constexpr bool e5 = kMode == kE5M2;
    constexpr int lanes = kFp8Block / (U * V);   // lanes that share a block
#pragma unroll
    for (int off = lanes / 2; off > 0; off >>= 1)
      amax = max_nan(amax, __shfl_xor_sync(kFull, amax, off));
    const float block = fp8_block<e5>(amax);
    const float factor = fp8_factor<e5>(block);
    const int32_t c0 = channel<V, U>(step, 0, lane);
    if (lane % lanes == 0 && c0 < a.C)
      a.scales[(int64_t)(c0 / kFp8Block) * a.N + t] = fp8_scale<e5>(block);
    uint8_t* row = a.y8 + t * a.y8_ld;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int32_t c = channel<V, U>(step, u, lane);
      if (c < a.C) {
        store_fp8<V, e5>(row + c, y + u * V, factor);
      }
    }
  }
}

// Block maxima of kIter steps at once, a block of each step in kLanes neighbouring
// lanes: every exchange halves the steps a lane carries, so three steps take five
// shuffles instead of twelve, and each lane ends with one step's maximum.
__host__ __device__ constexpr int pow2_at_least(int n) {
  int p = 1;
  while (p < n) p *= 2;
  return p;
}
// The lane (within its block's lanes) that ends with step `it`.
template <int kIter, int kLanes>
__host__ __device__ constexpr int holder(int it) {
  int lane = 0;
  for (int half = pow2_at_least(kIter) / 2, off = kLanes / 2; half > 0; half /= 2, off /= 2)
    if (it & half) lane += off;
  return lane;
}
template <int kIter, int kLanes>
__device__ __forceinline__ float max_of_blocks(const float (&amax)[kIter], int lane) {
  constexpr int P = pow2_at_least(kIter);
  static_assert(P <= kLanes, "one lane at least for every step");
  float m[P];
#pragma unroll
  for (int i = 0; i < P; ++i) m[i] = i < kIter ? amax[i < kIter ? i : 0] : 0.f;
  int off = kLanes / 2;
#pragma unroll
  for (int half = P / 2; half > 0; half /= 2, off /= 2) {
    const bool upper = lane & off;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float give = upper ? m[i] : m[i + half], keep = upper ? m[i + half] : m[i];
      m[i] = max_nan(keep, __shfl_xor_sync(kFull, give, off));
    }
  }
#pragma unroll
  for (; off > 0; off /= 2) m[0] = max_nan(m[0], __shfl_xor_sync(kFull, m[0], off));
  return m[0];
}

// x[0] .. x[N - 1], N a power of two: the second half is added to the first, and again.
template <int N>
__device__ __forceinline__ float sum_of_halves(float (&x)[N]) {
#pragma unroll
  for (int half = N / 2; half > 0; half /= 2)
#pragma unroll
    for (int i = 0; i < half; ++i) x[i] += x[i + half];
  return x[0];
}

// Vectors of a warp that make up a whole block of 128 channels.
template <int V>
constexpr int kUnit = V < 4 ? 4 / V : 1;

// kWarps warps per row of up to 32 V kUnit kIter kWarps channels, held in registers:
// all loads of a row are issued before any arithmetic. A warp has every kWarps-th
// step of the row, so whole blocks. A row's sum of squares does not depend on kWarps,
// nor its bits on the rows beside it: a lane's steps j, j + 8, .. make up its sum j,
// the sums are added as ((0 4) (2 6)) ((1 5) (3 7)), a pair of halves at a time in
// whichever warp holds both, and the lanes' totals last.
template <typename T, int V, int kIter, int kWarps, int kBlocks, int kMode>
__global__ void __launch_bounds__(kThreads, kBlocks) rmsnorm_row_kernel(const FwdArgs<T> a) {
  constexpr int U = kUnit<V>, kVecs = kIter * U, kRows = kThreads / (32 * kWarps);
  constexpr int kSums = 8 / kWarps;          // sums of a lane in each warp
  __shared__ float red[2][kThreads];
  const int lane = threadIdx.x & 31, group = (threadIdx.x >> 5) / kWarps;
  const int warp = (threadIdx.x >> 5) % kWarps;
  int phase = 0;
  for (int64_t t = (int64_t)blockIdx.x * kRows + group; t < a.N;
       t += (int64_t)gridDim.x * kRows) {
    Vec<T, V> hv[kVecs], rv[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int32_t c = channel<V, U>(i / U * kWarps + warp, i % U, lane);
      hv[i].zero();
      if (c < a.C) hv[i] = load_vec<T, V>(a.x + t * a.C + c);
    }
    if (a.res) {
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {
        const int32_t c = channel<V, U>(i / U * kWarps + warp, i % U, lane);
        if (c < a.C) rv[i] = load_vec<T, V>(a.res + t * a.C + c);
      }
    }
    float sums[kSums];
#pragma unroll
    for (int i = 0; i < kSums; ++i) sums[i] = 0.f;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int32_t c = channel<V, U>(i / U * kWarps + warp, i % U, lane);
      if (a.res && c < a.C) {
        hv[i].add(rv[i]);
        if (a.res_out) store_vec<T, V>(a.res_out + t * a.C + c, hv[i]);
      }
      float& sq = sums[i / U % kSums];
#pragma unroll
      for (int v = 0; v < V; ++v) sq = fmaf(hv[i].get(v), hv[i].get(v), sq);
    }
    float sq = sum_of_halves<kSums>(sums);
    if constexpr (kWarps > 1) {              // two sets of sums: one barrier a row
      red[phase][threadIdx.x] = sq;
      group_sync<32 * kWarps>(group);
      float all[kWarps];
#pragma unroll
      for (int i = 0; i < kWarps; ++i) all[i] = red[phase][(group * kWarps + i) * 32 + lane];
      sq = sum_of_halves<kWarps>(all);
      phase ^= 1;
    }
    sq = warp_sum(sq);
    const float rstd = rsqrtf(fmaf(sq, a.inv_c, a.eps));
    float y[kVecs][V], amax[kIter];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int32_t c = channel<V, U>(i / U * kWarps + warp, i % U, lane);
      Vec<T, V> w;
      w.zero();
      if (c < a.C) w = load_vec<T, V>(a.w + c);
      if (i % U == 0) amax[i / U] = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        y[i][v] = hv[i].get(v) * rstd * w.get(v);
        amax[i / U] = max_nan(amax[i / U], fabsf(y[i][v]));
      }
      if (a.y && c < a.C) {
        Vec<T, V> o;
        o.put(y[i]);
        store_vec<T, V>(a.y + t * a.C + c, o);
      }
    }
    if constexpr (kMode != kNoFp8) {
      // One lane computes one block's scale; the factors go back by shuffles.
      constexpr bool e5 = kMode == kE5M2;
      constexpr int lanes = kFp8Block / (V * U);
      const float mine = fp8_block<e5>(max_of_blocks<kIter, lanes>(amax, lane));
      const float factor = fp8_factor<e5>(mine), scale = fp8_scale<e5>(mine);
      uint8_t* row = a.y8 + t * a.y8_ld;
#pragma unroll
      for (int it = 0; it < kIter; ++it) {
        const int from = (lane & ~(lanes - 1)) + holder<kIter, lanes>(it);
        const float f = __shfl_sync(kFull, factor, from);
        const int32_t block = channel<V, U>(it * kWarps + warp, 0, lane) / kFp8Block;
        if (lane == from && block * kFp8Block < a.C) a.scales[(int64_t)block * a.N + t] = scale;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int32_t c = channel<V, U>(it * kWarps + warp, u, lane);
          if (c < a.C) store_fp8<V, e5>(row + c, y[it * U + u], f);
        }
      }
    }
  }
}

// One warp per row of any width: the sum of squares, then the output, in two
// passes over the row of which the second finds it in the caches. A lane
// touches the same channels in both passes, so x, residual, residual_out and y
// may share buffers (h is read back from residual_out when it is stored).
template <typename T, int V, int kMode>
__global__ void __launch_bounds__(kThreads)
rmsnorm_any_kernel(const FwdArgs<T> a) {
  constexpr int U = kUnit<V>;
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
  const int32_t steps = (a.C + 32 * V * U - 1) / (32 * V * U);
  for (int64_t t = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); t < a.N;
       t += warps) {
    const T* xr = a.x + t * a.C;
    const T* rr = a.res ? a.res + t * a.C : nullptr;
    T* hr = a.res_out ? a.res_out + t * a.C : nullptr;
    float sq = 0.f;
    for (int32_t step = 0; step < steps; ++step) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int32_t c = channel<V, U>(step, u, lane);
        if (c < a.C) {
          Vec<T, V> hv = load_vec<T, V>(xr + c);
          if (rr) {
            hv.add(load_vec<T, V>(rr + c));
            if (hr) store_vec<T, V>(hr + c, hv);
          }
#pragma unroll
          for (int v = 0; v < V; ++v) sq = fmaf(hv.get(v), hv.get(v), sq);
        }
      }
    }
    const float rstd = rsqrtf(fmaf(warp_sum(sq), a.inv_c, a.eps));
    for (int32_t step = 0; step < steps; ++step) {
      float h[U * V];
      Vec<T, V> w[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int32_t c = channel<V, U>(step, u, lane);
#pragma unroll
        for (int v = 0; v < V; ++v) h[u * V + v] = 0.f;
        w[u].zero();
        if (c < a.C) {
          w[u] = load_vec<T, V>(a.w + c);
          Vec<T, V> hv = load_vec<T, V>((hr ? hr : xr) + c);
          if (rr && !hr) hv.add(load_vec<T, V>(rr + c));
#pragma unroll
          for (int v = 0; v < V; ++v) h[u * V + v] = hv.get(v);
        }
      }
      emit<T, V, U, kMode>(a, t, step, lane, h, w, rstd);
    }
  }
}

unsigned row_grid(int64_t rows, int rows_per_block, int blocks_per_sm) {
  const int64_t blocks = ceil_div(rows, rows_per_block);
  const int64_t cap = (int64_t)device_sm_count() * blocks_per_sm;
  return (unsigned)(blocks < cap ? blocks : cap);
}

template <typename T, int V, int kIter, int kWarps, int kBlocks, int kMode>
void launch_row(const FwdArgs<T>& a, cudaStream_t stream) {
  rmsnorm_row_kernel<T, V, kIter, kWarps, kBlocks, kMode>
      <<<row_grid(a.N, kThreads / (32 * kWarps), 16), kThreads, 0, stream>>>(a);
}

// The form for V neighbouring channels per access: warps a row, vectors a lane and
// blocks an SM, by the row's width. Few rows (up to four an SM) take a block each, in us
// (otherwise): bf16 76 x 768 2.0 (2.8), 608 x 768 2.6 (2.8), 1216 x 768 3.8 (2.9), 304 x
// 333 2.8 (4.7), 608 x 1501 4.4 (5.1), 1216 x 1501 7.5 (5.6); fp32 608 x 2304 3.6 (4.3).
// Many rows keep 16 to 20 channels a lane: with more the registers leave too few
// rows in flight, with fewer the barrier shows. bf16, residual, 8-bit output:
//   90487 x 500  V 4: 1 warp 53 us, 2 warps 65;      V 1: 1 warp 86, 2 warps 100
//   32299 x 768  V 8: 1 warp 29 us, 2 warps 32 (fp32 40000 rows: 62 both)
//   32299 x 1024 V 8: 1 warp 38 us, 2 warps 38, 4 warps 47
//   32299 x 2304 V 4: 4 warps 83 us, 8 warps 99;     V 8: 2 warps 84, 1 warp 97
//   32299 x 2001 V 1: 8 warps 141 us, 4 warps 252, two passes 212
template <typename T, int V, int kMode>
void launch_rows(const FwdArgs<T>& a, cudaStream_t stream) {
  const int32_t C = a.C;
  const bool few = a.N <= 4 * (int64_t)device_sm_count() && C > 256;
  if constexpr (V == 8) {
    if (C > 2048 && C <= 2560) return launch_rows<T, 4, kMode>(a, stream);
    if (few && C <= 2048) return launch_row<T, V, 1, 8, 6, kMode>(a, stream);
    if (C <= 256) return launch_row<T, V, 1, 1, 6, kMode>(a, stream);
    if (C <= 512) return launch_row<T, V, 2, 1, 4, kMode>(a, stream);
    if (C <= 768) return launch_row<T, V, 3, 1, 3, kMode>(a, stream);
    if (C <= 1024) return launch_row<T, V, 2, 2, 4, kMode>(a, stream);
    if (C <= 1536) return launch_row<T, V, 3, 2, 3, kMode>(a, stream);
    if (C <= 2048) return launch_row<T, V, 2, 4, 4, kMode>(a, stream);
    if (C <= 4096) return launch_row<T, V, 2, 8, 4, kMode>(a, stream);
  } else {
    if (!few) {
      if (C <= 256) return launch_row<T, V, 2, 1, V == 1 ? 4 : 6, kMode>(a, stream);
      if (C <= 512) return launch_row<T, V, 4, 1, 4, kMode>(a, stream);
      if (C <= 768) return launch_row<T, V, 3, 2, 4, kMode>(a, stream);
      if constexpr (V > 1) {
        if (C <= 1024) return launch_row<T, V, 4, 2, 4, kMode>(a, stream);
      }
      if (C > 1024 && C <= 1536) return launch_row<T, V, 3, 4, 4, kMode>(a, stream);
      if constexpr (V > 1) {
        if (C > 1024 && C <= 2560)
          return launch_row<T, V, 5, 4, V == 4 ? 4 : 3, kMode>(a, stream);
      }
    }
    if (C <= 1 * 1024) return launch_row<T, V, 1, 8, 6, kMode>(a, stream);
    if (C <= 2 * 1024) return launch_row<T, V, 2, 8, 4, kMode>(a, stream);
    if (C <= 3 * 1024) return launch_row<T, V, 3, 8, 4, kMode>(a, stream);
  }
  rmsnorm_any_kernel<T, V, kMode><<<row_grid(a.N, kThreads / 32, 16), kThreads, 0, stream>>>(a);
}

template <typename T, int kMode>
pe_status launch_fwd(const FwdArgs<T>& a, cudaStream_t stream) {
  constexpr int V = 16 / sizeof(T);
  if (vectors<V>(a.C, a.x, a.w, a.y, a.res, a.res_out))
    launch_rows<T, V, kMode>(a, stream);
  else if (vectors<4>(a.C, a.x, a.w, a.y, a.res, a.res_out))
    launch_rows<T, 4, kMode>(a, stream);
  else if (vectors<2>(a.C, a.x, a.w, a.y, a.res, a.res_out))
    launch_rows<T, 2, kMode>(a, stream);
  else
    launch_rows<T, 1, kMode>(a, stream);
  PE_CUDA_TRY(cudaGetLastError());
  return PE_OK;
}

template <typename T>
pe_status run_fwd(int mode, const void* x, const void* res, const void* w, int64_t N, int32_t C,
                  float eps, void* y8, int64_t y8_ld, float* scales, void* y, void* res_out,
                  cudaStream_t stream) {
  const FwdArgs<T> a = {static_cast<const T*>(x),
                        static_cast<const T*>(res),
                        static_cast<const T*>(w),
                        N,
                        C,
                        1.f / (float)C,
                        eps,
                        static_cast<T*>(y),
                        static_cast<T*>(res_out),
                        static_cast<uint8_t*>(y8),
                        y8_ld,
                        scales};
  if (mode == kE4M3) return launch_fwd<T, kE4M3>(a, stream);
  if (mode == kE5M2) return launch_fwd<T, kE5M2>(a, stream);
  return launch_fwd<T, kNoFp8>(a, stream);
}

// ---------------------------------------------------------------- backward
constexpr int32_t kBwdMaxChannels = 16384;
constexpr int kBwdMaxBlocks = 640;

template <typename T>
struct BwdArgs {
  const T* dy;         // may be dx: not read through the read-only path
  const T* h;
  const T* w;
  const T* dres;
  int64_t N;
  int32_t C;
  float inv_c;         // 1 / C
  float eps;
  T* dx;
  float* part;         // [gridDim.x][C] sums of this block's rows
};

// kGroup threads per row (a warp, or the whole block), each with kIter vectors
// of V channels, the same for all of its rows: the weight's gradient stays in
// fp32 registers until the block's last row. Blocks of warps add their warps'
// sums in warp order.
template <typename T, int V, int kIter, int kGroup, int kBlocks>
__global__ void __launch_bounds__(kGroup > kThreads ? kGroup : kThreads, kBlocks)
rmsnorm_bwd_kernel(const BwdArgs<T> a) {
  constexpr int kBlock = kGroup > kThreads ? kGroup : kThreads;
  constexpr int kGroups = kBlock / kGroup;
  extern __shared__ float sums[];            // kGroup == 32: every warp's
  __shared__ float2 red[2][kBlock / 32];
  const int g = threadIdx.x % kGroup, group = threadIdx.x / kGroup;
  float dw[kIter * V];
#pragma unroll
  for (int i = 0; i < kIter * V; ++i) dw[i] = 0.f;
  int phase = 0;
  for (int64_t t = (int64_t)blockIdx.x * kGroups + group; t < a.N;
       t += (int64_t)gridDim.x * kGroups) {
    Vec<T, V> dyv[kIter], hv[kIter], rv[kIter];
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
      const int32_t c = (it * kGroup + g) * V;
      dyv[it].zero();
      hv[it].zero();
      if (c < a.C) {
        dyv[it] = load_vec<T, V>(a.dy + t * a.C + c);
        hv[it] = load_vec<T, V>(a.h + t * a.C + c);
        if (a.dres) rv[it] = load_vec<T, V>(a.dres + t * a.C + c);
      }
    }
    float sq = 0.f, dot = 0.f;
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
      const int32_t c = (it * kGroup + g) * V;
      Vec<T, V> wv;                          // from the caches, here and below
      if (c < a.C) wv = load_vec<T, V>(a.w + c);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float h = hv[it].get(v);
        sq = fmaf(h, h, sq);
        if (c < a.C) dot = fmaf(dyv[it].get(v) * wv.get(v), h, dot);
      }
    }
    sq = warp_sum(sq);
    dot = warp_sum(dot);
    if constexpr (kGroup > 32) {
      if ((threadIdx.x & 31) == 0) red[phase][threadIdx.x >> 5] = make_float2(sq, dot);
      group_sync<kGroup>(group);
      sq = dot = 0.f;
#pragma unroll
      for (int i = 0; i < kGroup / 32; ++i) {
        const float2 r = red[phase][group * (kGroup / 32) + i];
        sq += r.x;
        dot += r.y;
      }
      phase ^= 1;
    }
    const float rstd = rsqrtf(fmaf(sq, a.inv_c, a.eps));
    const float along = rstd * (dot * a.inv_c) * rstd;   // mean(w dy n) rstd
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
      const int32_t c = (it * kGroup + g) * V;
      if (c < a.C) {
        const Vec<T, V> wv = load_vec<T, V>(a.w + c);
        float dx[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float dy = dyv[it].get(v), n = hv[it].get(v) * rstd;
          dx[v] = rstd * (dy * wv.get(v)) - n * along;
          if (a.dres) dx[v] += rv[it].get(v);
          dw[it * V + v] = fmaf(dy, n, dw[it * V + v]);
        }
        Vec<T, V> o;
        o.put(dx);
        store_vec<T, V>(a.dx + t * a.C + c, o);
      }
    }
  }
  float* part = a.part + (int64_t)blockIdx.x * a.C;
  if constexpr (kGroups == 1) {
#pragma unroll
    for (int it = 0; it < kIter; ++it)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int32_t c = (it * kGroup + g) * V + v;
        if (c < a.C) part[c] = dw[it * V + v];
      }
  } else {
    // [group][vector element][thread], a row padded so that neither access conflicts.
    constexpr int kLine = kGroup + 1;
    float* mine = sums + group * (kIter * V * kLine);
#pragma unroll
    for (int i = 0; i < kIter * V; ++i) mine[i * kLine + g] = dw[i];
    __syncthreads();
    for (int32_t c = threadIdx.x; c < a.C; c += kBlock) {
      const int vec = c / V, i = vec / kGroup * V + c % V;
      float total = 0.f;
#pragma unroll
      for (int w = 0; w < kGroups; ++w)
        total += sums[(w * kIter * V + i) * kLine + vec % kGroup];
      part[c] = total;
    }
  }
}

// dweight[c] = the blocks' sums, added in a fixed order: 32 columns per block,
// 32 rows of threads, each adding every 32nd block's sum. `part` is not __restrict__:
// the kernel before may still write it at this one's start, so its loads must not pass
// for loads of constant memory, which could be moved before the wait.
__global__ void __launch_bounds__(1024)
rmsnorm_dweight_kernel(const float* part, int32_t blocks, int32_t C, float* dweight) {
  __shared__ float sum[32][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int32_t c = blockIdx.x * 32 + x;
  griddep_wait();
  float s = 0.f;
  if (c < C)
    for (int32_t b = y; b < blocks; b += 32) s += part[(int64_t)b * C + c];
  sum[y][x] = s;
  __syncthreads();
  s = warp_sum(sum[x][y]);
  if (x == 0 && blockIdx.x * 32 + y < C) dweight[blockIdx.x * 32 + y] = s;
}

template <typename T, int V, int kIter, int kGroup, int kBlocks>
pe_status launch_bwd_kernel(const BwdArgs<T>& a, float* dweight, cudaStream_t stream) {
  constexpr int kBlock = kGroup > kThreads ? kGroup : kThreads;
  unsigned grid = row_grid(a.N, kBlock / kGroup, kBlocks);
  if (grid > kBwdMaxBlocks) grid = kBwdMaxBlocks;
  constexpr size_t smem =
      kGroup < kBlock ? (size_t)(kBlock / kGroup) * kIter * V * (kGroup + 1) * sizeof(float) : 0;
  static_assert(smem <= 47 << 10, "the sums fit without an opt-in");
  rmsnorm_bwd_kernel<T, V, kIter, kGroup, kBlocks><<<grid, kBlock, smem, stream>>>(a);
  PE_CUDA_TRY(cudaGetLastError());
  return launch_after_previous(rmsnorm_dweight_kernel, dim3((unsigned)ceil_div(a.C, 32)),
                               dim3(1024), 0, stream, (const float*)a.part, (int32_t)grid, a.C,
                               dweight);
}

// The form for V neighbouring channels per access: vectors a thread, threads a row and
// blocks an SM, by the row's width; 8 to 20 weight sums a thread. With the residual's
// gradient:
//   bf16 32299 x 768   V 8: 64 threads 40.1 us, 32 40.5, 128 43.7, 256 (two blocks) 108
//   bf16 32299 x 2304  V 4: 128 threads 106 us;      V 8: 64 112, 128 116, 256 118
//   fp32 40000 x 1024  V 4: 128 threads 99 us, 64 104, 256 112, 32 118
//   fp32 20000 x 2304  V 4: 256 threads 113 us, 128 120, 64 175
//   bf16 90487 x 501   V 1: 64 threads 91 us, 32 105, 128 110, 256 170
template <typename T, int V>
pe_status launch_bwd(const BwdArgs<T>& a, float* dweight, cudaStream_t stream) {
  constexpr bool bf16 = sizeof(T) == 2;
  const int32_t C = a.C;
  if constexpr (V == 8) {
    if (C <= 256) return launch_bwd_kernel<T, V, 1, 32, 3>(a, dweight, stream);
    if (C <= 512) return launch_bwd_kernel<T, V, 2, 32, 3>(a, dweight, stream);
    if (C <= 1024) return launch_bwd_kernel<T, V, 2, 64, 3>(a, dweight, stream);
    if (C <= 2048) return launch_bwd_kernel<T, V, 2, 128, 3>(a, dweight, stream);
    if (C <= 2560) return launch_bwd<T, 4>(a, dweight, stream);
    if (C <= 4096) return launch_bwd_kernel<T, V, 2, 256, 4>(a, dweight, stream);
    return launch_bwd_kernel<T, V, 2, 1024, 1>(a, dweight, stream);
  } else if constexpr (V == 4) {
    if (C <= 256) return launch_bwd_kernel<T, V, 2, 32, 3>(a, dweight, stream);
    if constexpr (bf16) {
      if (C <= 512) return launch_bwd_kernel<T, V, 4, 32, 3>(a, dweight, stream);
      if (C <= 1024) return launch_bwd_kernel<T, V, 4, 64, 3>(a, dweight, stream);
      if (C <= 2560) return launch_bwd_kernel<T, V, 5, 128, 3>(a, dweight, stream);
    } else {
      if (C <= 768) return launch_bwd_kernel<T, V, 3, 64, 3>(a, dweight, stream);
      if (C <= 1024) return launch_bwd_kernel<T, V, 2, 128, 4>(a, dweight, stream);
    }
    if (C <= 3 * 1024) return launch_bwd_kernel<T, V, 3, 256, 4>(a, dweight, stream);
    return launch_bwd_kernel<T, V, 4, 1024, 1>(a, dweight, stream);
  } else {
    if constexpr (V == 2) {
      if constexpr (bf16) {
        if (C <= 512) return launch_bwd_kernel<T, V, 8, 32, 3>(a, dweight, stream);
        if (C <= 1024) return launch_bwd_kernel<T, V, 8, 64, 3>(a, dweight, stream);
      } else {
        if (C <= 256) return launch_bwd_kernel<T, V, 4, 32, 3>(a, dweight, stream);
        if (C <= 1024) return launch_bwd_kernel<T, V, 4, 128, 4>(a, dweight, stream);
      }
      if (C <= 2304) return launch_bwd_kernel<T, V, 9, 128, bf16 ? 3 : 2>(a, dweight, stream);
    } else {
      if (C <= 256) return launch_bwd_kernel<T, V, 8, 32, 4>(a, dweight, stream);
      if (C <= 512) return launch_bwd_kernel<T, V, 8, 64, 3>(a, dweight, stream);
      if (C <= 1024) return launch_bwd_kernel<T, V, 8, 128, bf16 ? 4 : 3>(a, dweight, stream);
      if (C <= 2304) return launch_bwd_kernel<T, V, 9, 256, 3>(a, dweight, stream);
    }
    return launch_bwd_kernel<T, V, 16 / V, 1024, 1>(a, dweight, stream);
  }
}

template <typename T>
pe_status run_bwd(const void* dy, const void* h, const void* w, const void* dres, int64_t N,
                  int32_t C, float eps, void* dx, float* dweight, void* ws,
                  cudaStream_t stream) {
  const BwdArgs<T> a = {static_cast<const T*>(dy),
                        static_cast<const T*>(h),
                        static_cast<const T*>(w),
                        static_cast<const T*>(dres),
                        N,
                        C,
                        1.f / (float)C,
                        eps,
                        static_cast<T*>(dx),
                        static_cast<float*>(ws)};
  if (sizeof(T) == 2 && vectors<8>(C, a.dy, a.w, a.h, a.dx, a.dres))
    return launch_bwd<T, 16 / sizeof(T)>(a, dweight, stream);
  if (vectors<4>(C, a.dy, a.w, a.h, a.dx, a.dres)) return launch_bwd<T, 4>(a, dweight, stream);
  if (vectors<2>(C, a.dy, a.w, a.h, a.dx, a.dres)) return launch_bwd<T, 2>(a, dweight, stream);
  return launch_bwd<T, 1>(a, dweight, stream);
}

// Channels are counted in int32, up to a whole step of a warp (256) past the last one.
constexpr int32_t kMaxChannels = 0x7fffffff - 1024;

bool dtype_ok(pe_dtype d) { return d == PE_BF16 || d == PE_FP32; }

pe_status check_fwd(pe_dtype dtype, const void* x, const void* residual, const void* weight,
                    int64_t N, int32_t C, float eps, const void* y, const void* residual_out) {
  if (!dtype_ok(dtype)) return PE_ERR_UNSUPPORTED;
  if (N < 0 || C < 1 || !(eps > 0.f) || !isfinite(eps)) return PE_ERR_INVALID_ARG;
  if (C > kMaxChannels) return PE_ERR_OVERFLOW;
  if (N > 0 && (!x || !weight || (residual_out && (!residual || residual_out == y))))
    return PE_ERR_INVALID_ARG;
  return PE_OK;
}

}  // namespace

}  // namespace pe

using namespace pe;

extern "C" pe_status pe_rmsnorm(pe_dtype dtype, const void* x, const void* residual,
                                const void* weight, int64_t N, int32_t C, float eps, void* y,
                                void* residual_out, pe_stream_t stream_) {
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  PE_TRY(check_fwd(dtype, x, residual, weight, N, C, eps, y, residual_out));
  if (N == 0) return PE_OK;
  if (!y) return PE_ERR_INVALID_ARG;
  if (!device_is_sm103()) return PE_ERR_UNSUPPORTED;
  if (dtype == PE_FP32)
    return run_fwd<float>(kNoFp8, x, residual, weight, N, C, eps, nullptr, 0, nullptr, y,
                          residual_out, stream);
  return run_fwd<__nv_bfloat16>(kNoFp8, x, residual, weight, N, C, eps, nullptr, 0, nullptr, y,
                                residual_out, stream);
}

extern "C" pe_status pe_rmsnorm_fp8(pe_dtype dtype, pe_fp8_type fp8_type, const void* x,
                                    const void* residual, const void* weight, int64_t N,
                                    int32_t C, float eps, void* y8, int64_t y8_ld,
                                    float* y8_scales, void* y, void* residual_out,
                                    pe_stream_t stream_) {
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (!fp8_type_ok(fp8_type)) return PE_ERR_UNSUPPORTED;
  PE_TRY(check_fwd(dtype, x, residual, weight, N, C, eps, y, residual_out));
  if (N == 0) return PE_OK;
  if (!y8 || !y8_scales) return PE_ERR_INVALID_ARG;
  if (!fp8_layout_ok(y8, y8_ld, C)) return PE_ERR_UNSUPPORTED;
  if (!device_is_sm103()) return PE_ERR_UNSUPPORTED;
  const int mode = fp8_type == PE_E5M2 ? kE5M2 : kE4M3;
  if (dtype == PE_FP32)
    return run_fwd<float>(mode, x, residual, weight, N, C, eps, y8, y8_ld, y8_scales, y,
                          residual_out, stream);
  return run_fwd<__nv_bfloat16>(mode, x, residual, weight, N, C, eps, y8, y8_ld, y8_scales, y,
                                residual_out, stream);
}

extern "C" size_t pe_rmsnorm_bwd_workspace_size(int32_t C) {
  return C < 1 ? 0 : (size_t)kBwdMaxBlocks * (size_t)C * sizeof(float);
}

extern "C" pe_status pe_rmsnorm_bwd(pe_dtype dtype, const void* dy, const void* h,
                                    const void* weight, const void* dresidual, int64_t N,
                                    int32_t C, float eps, void* dx, float* dweight,
                                    void* workspace, size_t workspace_bytes,
                                    pe_stream_t stream_) {
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (!dtype_ok(dtype)) return PE_ERR_UNSUPPORTED;
  if (N < 0 || C < 1 || !(eps > 0.f) || !isfinite(eps) || !dweight) return PE_ERR_INVALID_ARG;
  if (C > kBwdMaxChannels) return PE_ERR_UNSUPPORTED;
  if (N > 0) {
    if (!dy || !h || !weight || !dx) return PE_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 16) ||
        workspace_bytes < pe_rmsnorm_bwd_workspace_size(C))
      return PE_ERR_WORKSPACE;
  }
  if (!device_is_sm103()) return PE_ERR_UNSUPPORTED;
  if (N == 0) {
    PE_CUDA_TRY(cudaMemsetAsync(dweight, 0, (size_t)C * sizeof(float), stream));
    return PE_OK;
  }
  if (dtype == PE_FP32)
    return run_bwd<float>(dy, h, weight, dresidual, N, C, eps, dx, dweight, workspace, stream);
  return run_bwd<__nv_bfloat16>(dy, h, weight, dresidual, N, C, eps, dx, dweight, workspace,
                                stream);
}
