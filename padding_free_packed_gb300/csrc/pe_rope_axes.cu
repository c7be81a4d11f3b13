// Rotary positions with several axes (time, height, width): pair i of a head's channels
// (i, i + D / 2) belongs to one axis and turns by that axis's position times the pair's
// frequency, theta^(-2 i / D), or theta^(-j / s) for the j-th of the s pairs of an axis with
// frequencies of its own. The inverse turns back, which is the backward.
//
// A bandwidth kernel: a warp takes a token, forms the cosine and sine of each pair once for
// all heads of q and k, and reads and writes every channel once, in 16-byte vectors from both
// halves of a head. Angles are counted in turns modulo one, in 64-bit fixed point: a position
// times the frequency as a fraction of 2^64, which wraps as turns do, so far positions lose
// nothing and no double-precision arithmetic runs on the GPU.
// Measured (GB300, device time): q and k of 169151 tokens, 16 heads x 64 bf16, out of one
// buffer of q, k and v, in 203 us (6.8 TB/s, the measured copy rate).
#include <math.h>

#include "pe_vec.cuh"

namespace pe {

namespace {

constexpr int kThreads = 256;
constexpr int kBlocksPerSm = 32;               // 16: 208 us in the case above, 3: 246
constexpr int kMaxHalf = 128;                  // head_dim <= 256
constexpr int kMaxAxes = 4;

struct Tensor {
  const void* in;        // in may be out: not read through the read-only path
  void* out;
  int64_t in_stride, out_stride;               // elements from a token to the next
  int32_t heads;
};

struct Plan {
  uint64_t turns[kMaxHalf];                    // of each pair, a position, times 2^64
  int32_t ends[kMaxAxes];                      // one past the last pair of each axis
};

template <typename T, int V, int kFlight>
__global__ void __launch_bounds__(kThreads)
rope_axes_kernel(const Tensor q, const Tensor k, const int32_t* __restrict__ pos, int64_t N,
                 int32_t D, const __grid_constant__ Plan plan, float sign) {
  __shared__ float table[kThreads / 32][2][kMaxHalf];   // per warp: cos, sin
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t half = D / 2, chunks = half / V, items = (q.heads + k.heads) * chunks;
  const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
  float* cs = table[warp][0];
  float* sn = table[warp][1];
  for (int64_t t = (int64_t)blockIdx.x * (kThreads / 32) + warp; t < N; t += warps) {
    auto locate = [&](int32_t item, const T*& in, T*& out, int32_t& i0) {
      const int32_t h = item / chunks;
      i0 = (item - h * chunks) * V;
      if (h < q.heads) {
        in = static_cast<const T*>(q.in) + t * q.in_stride + h * D + i0;
        out = static_cast<T*>(q.out) + t * q.out_stride + h * D + i0;
      } else {
        in = static_cast<const T*>(k.in) + t * k.in_stride + (h - q.heads) * D + i0;
        out = static_cast<T*>(k.out) + t * k.out_stride + (h - q.heads) * D + i0;
      }
    };
    Vec<T, V> x1[kFlight], x2[kFlight];
    auto load = [&](int32_t first) {
#pragma unroll
      for (int u = 0; u < kFlight; ++u) {
        const int32_t item = first + 32 * u + lane;
        if (item < items) {
          const T* in;
          T* out;
          int32_t i0;
          locate(item, in, out, i0);
          x1[u] = load_vec<T, V>(in);
          x2[u] = load_vec<T, V>(in + half);
        }
      }
    };
    load(0);                                   // in flight while the angles are formed
    for (int32_t i = lane; i < half; i += 32) {
      int axis = 0;
#pragma unroll
      for (int j = 0; j < kMaxAxes - 1; ++j) axis += i >= plan.ends[j];
      const int64_t p = __ldg(pos + axis * N + t);
      const uint64_t turn = (uint64_t)p * plan.turns[i] + 0x80000000ull;
      // The nearest quarter turn, and the rest: an eighth at most either way.
      const uint32_t whole = (uint32_t)(turn >> 32), quarter = (whole + 0x20000000u) >> 30;
      const int32_t rest = (int32_t)(whole - (quarter << 30));
      float s, c;
      sincospif((float)rest * 0x1p-31f, &s, &c);
      const float a = quarter & 1 ? s : c, b = quarter & 1 ? c : s;
      cs[i] = quarter == 1 || quarter == 2 ? -a : a;
      sn[i] = (quarter & 2 ? -b : b) * sign;
    }
    __syncwarp();
    for (int32_t first = 0; first < items; first += 32 * kFlight) {
      if (first > 0) load(first);
#pragma unroll
      for (int u = 0; u < kFlight; ++u) {
        const int32_t item = first + 32 * u + lane;
        if (item < items) {
          const T* in;
          T* out;
          int32_t i0;
          locate(item, in, out, i0);
          float o1[V], o2[V];
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const float a1 = x1[u].get(v), a2 = x2[u].get(v), c = cs[i0 + v], s = sn[i0 + v];
            o1[v] = a1 * c - a2 * s;
            o2[v] = a2 * c + a1 * s;
          }
          Vec<T, V> y1, y2;
          y1.put(o1);
          y2.put(o2);
          store_vec<T, V>(out, y1);
          store_vec<T, V>(out + half, y2);
        }
      }
    }
    __syncwarp();                              // the table is rewritten for the next token
  }
}

template <typename T, int V>
pe_status launch(const Tensor& q, const Tensor& k, const int32_t* pos, int64_t N, int32_t D,
                 const Plan& plan, float sign, cudaStream_t stream) {
  int64_t blocks = ceil_div(N, kThreads / 32);
  const int64_t most = (int64_t)device_sm_count() * kBlocksPerSm;
  if (blocks > most) blocks = most;
  rope_axes_kernel<T, V, 4>
      <<<(unsigned)blocks, kThreads, 0, stream>>>(q, k, pos, N, D, plan, sign);
  PE_CUDA_TRY(cudaGetLastError());
  return PE_OK;
}

bool by(const Tensor& x, int64_t V, uintptr_t bytes) {
  return x.heads == 0 || (x.in_stride % V == 0 && x.out_stride % V == 0 && aligned(x.in, bytes) &&
                          aligned(x.out, bytes));
}

template <typename T>
pe_status run(const Tensor& q, const Tensor& k, const int32_t* pos, int64_t N, int32_t D,
              const Plan& plan, float sign, cudaStream_t stream) {
  constexpr int V = 16 / sizeof(T);
  if (D / 2 % V == 0 && by(q, V, 16) && by(k, V, 16))
    return launch<T, V>(q, k, pos, N, D, plan, sign, stream);
  if (V > 4 && D / 2 % 4 == 0 && by(q, 4, 8) && by(k, 4, 8))
    return launch<T, 4>(q, k, pos, N, D, plan, sign, stream);
  return launch<T, 1>(q, k, pos, N, D, plan, sign, stream);
}

// Nothing to do, or a tensor whose tokens lie within their strides.
bool tensor_ok(const Tensor& x, int64_t N, int32_t D) {
  if (x.heads == 0) return true;
  const int64_t row = (int64_t)x.heads * D;
  return x.in && x.out && (N <= 1 || (x.in_stride >= row && x.out_stride >= row)) &&
         (x.in != x.out || N <= 1 || x.in_stride == x.out_stride);
}

}  // namespace

}  // namespace pe

using namespace pe;

extern "C" pe_status pe_rope_axes(pe_dtype dtype, const void* q, int64_t q_stride, void* q_out,
                                  int64_t q_out_stride, int32_t q_heads, const void* k,
                                  int64_t k_stride, void* k_out, int64_t k_out_stride,
                                  int32_t k_heads, const int32_t* positions,
                                  const int32_t* sections, int32_t num_axes, int64_t N,
                                  int32_t head_dim, double theta, int per_axis, int inverse,
                                  pe_stream_t stream_) {
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (dtype != PE_BF16 && dtype != PE_FP32) return PE_ERR_UNSUPPORTED;
  if (N < 0 || q_heads < 0 || k_heads < 0 || head_dim < 2 || head_dim % 2 != 0 ||
      head_dim > 2 * kMaxHalf || num_axes < 1 || num_axes > kMaxAxes || !sections ||
      !(theta > 1.0) || !isfinite(theta))
    return PE_ERR_INVALID_ARG;
  const int32_t half = head_dim / 2;
  Plan plan = {};
  int32_t pair = 0;
  for (int axis = 0; axis < kMaxAxes; ++axis) {
    const int32_t size = axis < num_axes ? sections[axis] : 0;
    if (size < 0 || size > half - pair) return PE_ERR_INVALID_ARG;
    for (int32_t j = 0; j < size; ++j, ++pair) {
      const double power = per_axis ? -(double)j / size : -(double)pair / half;
      const double turn = pow(theta, power) / 6.283185307179586476925;
      plan.turns[pair] = (uint64_t)ldexp(turn, 64);               // below 2^64 / 6
    }
    plan.ends[axis] = pair;
  }
  if (pair != half) return PE_ERR_INVALID_ARG;
  if ((int64_t)(q_heads > k_heads ? q_heads : k_heads) * head_dim > (1 << 28))
    return PE_ERR_OVERFLOW;
  if (N == 0 || (q_heads == 0 && k_heads == 0)) return PE_OK;
  const Tensor tq = {q, q_out, q_stride, q_out_stride, q_heads};
  const Tensor tk = {k, k_out, k_stride, k_out_stride, k_heads};
  if (!positions || !tensor_ok(tq, N, head_dim) || !tensor_ok(tk, N, head_dim))
    return PE_ERR_INVALID_ARG;
  if ((q_heads && !by_elements(dtype, q, q_out)) || (k_heads && !by_elements(dtype, k, k_out)) ||
      !by_elements(PE_FP32, positions))
    return PE_ERR_UNSUPPORTED;
  if (!device_is_sm103()) return PE_ERR_UNSUPPORTED;
  const float sign = inverse ? -1.f : 1.f;
  if (dtype == PE_FP32)
    return run<float>(tq, tk, positions, N, head_dim, plan, sign, stream);
  return run<__nv_bfloat16>(tq, tk, positions, N, head_dim, plan, sign, stream);
}
