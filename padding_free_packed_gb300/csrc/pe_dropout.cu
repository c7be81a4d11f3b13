// Dropout from a counter-based generator: y[e] = x[e] / (1 - p) where element e is kept, 0
// where it is not (plus residual[e]). Element e is kept iff word e % 4 of
// Philox4x32-10(key = seed, counter = (e / 4, offset)) is at least p 2^32 (J. Salmon et al.,
// Parallel random numbers: as easy as 1, 2, 3, SC 2011: ten rounds of two 32 x 32 bit
// products), so the backward draws the same numbers again instead of reading a mask.
// A bandwidth kernel; the generator is 40 integer instructions for four elements, the round
// keys are launch parameters, and every thread keeps several 16-byte loads in flight.
// Measured (GB300, device time): 169151 x 1024 bf16 with residual in 158 us (6.6 TB/s, 0.97 of
// the measured copy rate), without 146 us (0.70: the generator's integer products are the
// bound), 90487 x 512 fp32 with residual 82 us (1.0). Four loads in flight a thread instead
// of two took 3 % more; products and comparisons one element at a time 9 %. Tensors that do not
// start at multiples of 16 bytes go one element a thread, each with a whole block of four
// words: 169151 x 1024 bf16 without residual 610 us (0.17), 90487 x 512 fp32 163 (0.33).
#include <math.h>

#include "pe_vec.cuh"

namespace pe {

namespace {

constexpr int kThreads = 256;
constexpr int kBlocksPerSm = 16;       // three turns: a stride short enough for DRAM's pages, and
                                       // the last turn short (4: 169 us, 8: 163, 16: 158, one
                                       // turn's worth of work a block: 187)
constexpr int kRounds = 10;

struct Keys {
  uint32_t k[kRounds][2];
};

struct Draw {
  Keys keys;
  uint64_t offset;
  const uint64_t* device_offset;     // added to offset, or null
  uint32_t most_dropped;             // kept iff word > most_dropped (all are where p = 0)
  float scale;
};

__device__ __forceinline__ void philox(const Keys& keys, uint64_t block, uint32_t o0, uint32_t o1,
                                       uint32_t (&c)[4]) {
  c[0] = (uint32_t)block;
  c[1] = (uint32_t)(block >> 32);
  c[2] = o0;
  c[3] = o1;
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    const uint64_t p0 = (uint64_t)c[0] * 0xD2511F53u, p1 = (uint64_t)c[2] * 0xCD9E8D57u;
    c[0] = (uint32_t)(p1 >> 32) ^ c[1] ^ keys.k[i][0];
    c[2] = (uint32_t)(p0 >> 32) ^ c[3] ^ keys.k[i][1];
    c[1] = (uint32_t)p1;
    c[3] = (uint32_t)p0;
  }
}

template <typename T>
struct Args {
  const T* x;            // x and res may be y: not read through the read-only path
  const T* res;
  int64_t count;
  T* y;
  Draw d;
};

// V consecutive elements (a multiple of 4, or 1) a thread and step, kSteps steps in flight.
// kAll: p = 0, no numbers are drawn.
template <typename T, int V, int kSteps, bool kAll>
__global__ void __launch_bounds__(kThreads)
dropout_kernel(const Args<T> a) {
  uint64_t offset = a.d.offset;
  if (a.d.device_offset) offset += *a.d.device_offset;
  const uint32_t o0 = (uint32_t)offset, o1 = (uint32_t)(offset >> 32);
  const uint32_t dropped = a.d.most_dropped;
  const int64_t units = a.count / V, stride = (int64_t)gridDim.x * kThreads;
  for (int64_t i0 = (int64_t)blockIdx.x * kThreads + threadIdx.x; i0 < units;
       i0 += kSteps * stride) {
    Vec<T, V> x[kSteps], r[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int64_t i = i0 + s * stride;
      if (i < units) {
        x[s] = load_vec<T, V>(a.x + i * V);
        if (a.res) r[s] = load_vec<T, V>(a.res + i * V);
      }
    }
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int64_t i = i0 + s * stride;
      if (i < units) {
        float o[V];
        if constexpr (V == 1) {
          o[0] = x[s].get(0) * a.d.scale;
          if constexpr (!kAll) {
            uint32_t w[4];
            philox(a.d.keys, (uint64_t)i >> 2, o0, o1, w);
            const int at = (int)(i & 3);
            const uint32_t word = at == 0 ? w[0] : at == 1 ? w[1] : at == 2 ? w[2] : w[3];
            if (word <= dropped) o[0] = 0.f;
          }
          if (a.res) o[0] += r[s].get(0);
        } else {
          const uint64_t scale = sm103::f2(a.d.scale, a.d.scale);
#pragma unroll
          for (int v = 0; v < V; v += 4) {
#pragma unroll
            for (int j = v; j < v + 4; j += 2)
              sm103::f2_split(sm103::fmul2(x[s].pair(j / 2), scale), o[j], o[j + 1]);
            if constexpr (!kAll) {
              uint32_t w[4];
              philox(a.d.keys, (uint64_t)(i * V + v) >> 2, o0, o1, w);
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (w[j] <= dropped) o[v + j] = 0.f;
            }
          }
          if (a.res) {
#pragma unroll
            for (int j = 0; j < V; j += 2)
              sm103::f2_split(sm103::fadd2(sm103::f2(o[j], o[j + 1]), r[s].pair(j / 2)), o[j],
                              o[j + 1]);
          }
        }
        Vec<T, V> out;
        out.put(o);
        store_vec<T, V>(a.y + i * V, out);
      }
    }
  }
  if constexpr (V > 1) {               // the last count % V elements, one a thread
    const int64_t e = units * V + threadIdx.x;
    if (blockIdx.x == 0 && e < a.count) {
      float o = to_f32(a.x[e]) * a.d.scale;
      if constexpr (!kAll) {
        uint32_t w[4];
        philox(a.d.keys, (uint64_t)e >> 2, o0, o1, w);
        const int at = (int)(e & 3);
        const uint32_t word = at == 0 ? w[0] : at == 1 ? w[1] : at == 2 ? w[2] : w[3];
        if (word <= dropped) o = 0.f;
      }
      if (a.res) o += to_f32(a.res[e]);
      a.y[e] = from_f32<T>(o);
    }
  }
}

template <typename T, int V, int kSteps>
pe_status launch(const Args<T>& a, bool all, cudaStream_t stream) {
  const auto kernel =
      all ? dropout_kernel<T, V, kSteps, true> : dropout_kernel<T, V, kSteps, false>;
  int64_t blocks = ceil_div(ceil_div(a.count, V), kThreads);
  const int64_t most = (int64_t)device_sm_count() * kBlocksPerSm;
  if (blocks > most) blocks = most;
  kernel<<<(unsigned)blocks, kThreads, 0, stream>>>(a);
  PE_CUDA_TRY(cudaGetLastError());
  return PE_OK;
}

template <typename T>
pe_status run(const void* x, const void* res, int64_t count, void* y, const Draw& d,
              bool all, cudaStream_t stream) {
  const Args<T> a = {static_cast<const T*>(x), static_cast<const T*>(res), count,
                     static_cast<T*>(y), d};
  constexpr int V = 16 / sizeof(T);
  if (aligned(x, 16) && aligned(y, 16) && aligned(res, 16)) return launch<T, V, 2>(a, all, stream);
  return launch<T, 1, 4>(a, all, stream);
}

}  // namespace

}  // namespace pe

using namespace pe;

extern "C" pe_status pe_dropout(pe_dtype dtype, const void* x, const void* residual,
                                int64_t count, double p, uint64_t seed, uint64_t offset,
                                const uint64_t* device_offset, void* y, pe_stream_t stream_) {
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (dtype != PE_BF16 && dtype != PE_FP32) return PE_ERR_UNSUPPORTED;
  if (count < 0 || !(p >= 0.0 && p < 1.0)) return PE_ERR_INVALID_ARG;
  if (count > (1LL << 60)) return PE_ERR_OVERFLOW;
  if (count == 0) return PE_OK;
  if (!x || !y) return PE_ERR_INVALID_ARG;
  if (!aligned(device_offset, 8) || !by_elements(dtype, x, residual, y))
    return PE_ERR_UNSUPPORTED;
  if (!device_is_sm103()) return PE_ERR_UNSUPPORTED;
  Draw d;
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
  for (int i = 0; i < kRounds; ++i, k0 += 0x9E3779B9u, k1 += 0xBB67AE85u) {
    d.keys.k[i][0] = k0;
    d.keys.k[i][1] = k1;
  }
  d.offset = offset;
  d.device_offset = device_offset;
  // word >= p 2^32 <=> word > ceil(p 2^32) - 1, a number below 2^32 for p > 0.
  const bool all = p == 0.0;
  d.most_dropped = all ? 0u : (uint32_t)((uint64_t)ceil(p * 4294967296.0) - 1);
  d.scale = (float)(1.0 / (1.0 - p));
  if (dtype == PE_FP32) return run<float>(x, residual, count, y, d, all, stream);
  return run<__nv_bfloat16>(x, residual, count, y, d, all, stream);
}
