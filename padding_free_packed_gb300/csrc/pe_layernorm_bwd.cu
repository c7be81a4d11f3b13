// Backward of LayerNorm over packed token rows. h is the normalised input as the forward
// stored it; with n = (h - mean) rstd and g = w dy,
//   dx = rstd (g - mean(g) - n mean(g n)) (+ dresidual),
//   dweight = sum over rows of dy n, dbias = sum over rows of dy.
// A bandwidth kernel: a row of h and dy is read once into the registers of 1 to 8 warps, its
// statistics are formed again from there (mean first, then squares of what is left, so a
// large mean costs no precision), and dx is written once. The weight's and bias's sums of a
// thread's own channels stay in fp32 registers until the block's last row; a second kernel
// adds the blocks' lines in a fixed order. The next row's loads are in flight while a row is
// worked on. Rows wider than 4096 channels take a block each and keep those sums in shared
// memory.
// Measured (GB300, device time, with the residual's gradient): 32299 x 768 bf16 in 41 us (4.8
// TB/s, 0.71 of the measured copy rate; some 5 us are the start, the last rows and the second
// kernel), 169151 x 1024 bf16 220 us (0.93), 32299 x 2304 bf16 125 us (0.70), 90487 x 512
// fp32 114 us (0.96). What bounds it is bytes in flight: the sums a thread keeps (two for
// each of its channels) leave 16 to 24 warps an SM. In paired arithmetic 768 channels took 42
// us where single fp32 operations took 45. bf16 rows of odd width move two bytes at a time
// (20000 x 777 51 us, 0.36).
#include <math.h>

#include "pe_vec.cuh"

namespace pe {

namespace {

constexpr int kThreads = 256;
constexpr int32_t kMaxChannels = 16384;
constexpr int32_t kWide = 4096;                 // wider rows: one block of 1024 threads a row
constexpr int kMaxBlocks = 608, kMaxWideBlocks = 152;

template <typename T>
struct Args {
  const T* dy;           // dy, h and dres may be dx: not read through the read-only path
  const T* h;
  const T* w;
  const T* dres;
  int64_t N;
  int32_t C;
  float inv_c;           // 1 / C
  float eps;
  T* dx;
  float* part;           // [gridDim.x][2 C]: this block's sums for the weight, the bias, or
                         // null: one cluster, which writes the gradients itself
  float* dweight;
  float* dbias;
};

// Sums of kSums numbers a thread over the kGroup threads of a row, the same in all of them.
template <int kSums, int kGroup>
__device__ __forceinline__ void group_sum(float (&x)[kSums], float* red, int group) {
#pragma unroll
  for (int i = 0; i < kSums; ++i) x[i] = warp_sum(x[i]);
  if constexpr (kGroup > 32) {
    constexpr int kWarps = kGroup / 32;
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int i = 0; i < kSums; ++i) red[i * 32 + warp] = x[i];
    }
    group_sync<kGroup>(group);
#pragma unroll
    for (int i = 0; i < kSums; ++i) {
      x[i] = 0.f;
#pragma unroll
      for (int j = 0; j < kWarps; ++j) x[i] += red[i * 32 + group * kWarps + j];
    }
  }
}

// Blocks an SM that the registers are to allow: more of them spill, fewer leave too few rows
// in flight (169151 x 1024 bf16, 16 channels a thread: 1 block 284 us, 2 blocks 220, 3 blocks
// 495; 90487 x 512 fp32, 8 channels: 2 blocks 116 us, 3 blocks 184).
template <int V, int kIter, int kGroup>
constexpr int kMinBlocks =
    V == 8 ? (kIter > 1 ? 2 : kGroup == 96 ? 4 : 3) : V * kIter > 8 ? 1 : 2;

// kGroup threads a row, each with kIter vectors of V channels, the same for all of its rows.
template <typename T, int V, int kIter, int kGroup>
__global__ void __launch_bounds__(kGroup > kThreads ? kGroup : kThreads / kGroup * kGroup,
                                  kGroup > kThreads ? 1 : kMinBlocks<V, kIter, kGroup>)
layernorm_bwd_kernel(const Args<T> a) {
  constexpr bool kIsWide = kGroup > kThreads;
  constexpr int kGroups = kIsWide ? 1 : kThreads / kGroup;
  constexpr int kBlock = kGroup * kGroups;
  extern __shared__ float sums[];            // wide: [2][C]; else every group's, at the end
  __shared__ float red[2][4 * 32];           // two sets: a row's writes miss the last's reads
  const int g = threadIdx.x % kGroup, group = threadIdx.x / kGroup;
  const int64_t step = (int64_t)gridDim.x * kGroups;
  int64_t t = (int64_t)blockIdx.x * kGroups + group;

  // A thread's channels in pairs: half as many instructions, which is what bounds rows in
  // flight here. Single channels (rows that start anywhere) go one at a time.
  constexpr bool kPaired = V > 1 && !kIsWide;
  constexpr int kKept = kIsWide ? 1 : kIter * V;
  float dw[kPaired ? 1 : kKept], db[kPaired ? 1 : kKept];
  uint64_t dw2[kPaired ? kKept / 2 : 1], db2[kPaired ? kKept / 2 : 1];
#pragma unroll
  for (int i = 0; i < (kPaired ? 1 : kKept); ++i) dw[i] = db[i] = 0.f;
#pragma unroll
  for (int i = 0; i < (kPaired ? kKept / 2 : 1); ++i) dw2[i] = db2[i] = 0ull;
  if constexpr (kIsWide) {
    for (int32_t c = threadIdx.x; c < 2 * a.C; c += kBlock) sums[c] = 0.f;
    __syncthreads();
  }
  Vec<T, V> wv[kPaired ? kIter : 1];             // the weight of this thread's channels
  if constexpr (kPaired) {
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
      const int32_t c = (it * kGroup + g) * V;
      wv[it].zero();
      if (c < a.C) wv[it] = load_vec<T, V>(a.w + c);
    }
  }

  Vec<T, V> dyv[kIter], hv[kIter], rv[kIter];
  auto load = [&](int64_t row) {
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
      const int32_t c = (it * kGroup + g) * V;
      dyv[it].zero();
      hv[it].zero();
      if (c < a.C && row < a.N) {
        dyv[it] = load_vec<T, V>(a.dy + row * a.C + c);
        hv[it] = load_vec<T, V>(a.h + row * a.C + c);
        if (!kIsWide && a.dres) rv[it] = load_vec<T, V>(a.dres + row * a.C + c);
      }
    }
  };
  load(t);
  int phase = 0;
  for (; t < a.N; t += step) {
    if constexpr (kPaired) {
      using namespace sm103;
      Vec<T, V> dyn[kIter], hn[kIter], rn[kIter];
      uint64_t total = 0ull;
#pragma unroll
      for (int it = 0; it < kIter; ++it) {
        dyn[it] = dyv[it];
        hn[it] = hv[it];
        rn[it] = rv[it];
#pragma unroll
        for (int j = 0; j < V / 2; ++j) total = fadd2(total, hn[it].pair(j));
      }
      load(t + step);
      float first[1], other;
      f2_split(total, first[0], other);
      first[0] += other;
      group_sum<1, kGroup>(first, red[phase], group);
      const float mean = first[0] * a.inv_c;
      // Squares of d = h - mean, and the sums of g and g d.
      uint64_t s0 = 0ull, s1 = 0ull, s2 = 0ull;
      const uint64_t minus_mean = f2(-mean, -mean);
#pragma unroll
      for (int it = 0; it < kIter; ++it) {
        if ((it * kGroup + g) * V < a.C) {
#pragma unroll
          for (int j = 0; j < V / 2; ++j) {
            const uint64_t d = fadd2(hn[it].pair(j), minus_mean);
            const uint64_t gv = fmul2(dyn[it].pair(j), wv[it].pair(j));
            s0 = ffma2(d, d, s0);
            s1 = fadd2(s1, gv);
            s2 = ffma2(gv, d, s2);
          }
        }
      }
      float s[3], t0, t1, t2;
      f2_split(s0, s[0], t0);
      f2_split(s1, s[1], t1);
      f2_split(s2, s[2], t2);
      s[0] += t0;
      s[1] += t1;
      s[2] += t2;
      group_sum<3, kGroup>(s, red[phase] + 32, group);
      phase ^= 1;
      const float rstd = rsqrtf(fmaf(s[0], a.inv_c, a.eps));
      const float mean_g = s[1] * a.inv_c, along = rstd * (s[2] * a.inv_c) * rstd;
      const uint64_t rstd2 = f2(rstd, rstd), minus_g = f2(-mean_g, -mean_g);
      const uint64_t minus_along = f2(-along, -along);      // -mean(g n) rstd
#pragma unroll
      for (int it = 0; it < kIter; ++it) {
        const int32_t c = (it * kGroup + g) * V;
        if (c < a.C) {
          Vec<T, V> o;
#pragma unroll
          for (int j = 0; j < V / 2; ++j) {
            const int e = it * (V / 2) + j;
            const uint64_t dy = dyn[it].pair(j), d = fadd2(hn[it].pair(j), minus_mean);
            uint64_t x = ffma2(d, minus_along, ffma2(dy, wv[it].pair(j), minus_g));
            x = a.dres ? ffma2(x, rstd2, rn[it].pair(j)) : fmul2(x, rstd2);
            o.put_pair(j, x);
            dw2[e] = ffma2(dy, fmul2(d, rstd2), dw2[e]);
            db2[e] = fadd2(db2[e], dy);
          }
          store_vec<T, V>(a.dx + t * a.C + c, o);
        }
      }
    } else {
      Vec<T, V> dyn[kIter], hn[kIter], rn[kIter];
#pragma unroll
      for (int it = 0; it < kIter; ++it) {
        dyn[it] = dyv[it];
        hn[it] = hv[it];
        if constexpr (!kIsWide) rn[it] = rv[it];
      }
      if constexpr (!kIsWide) load(t + step);
      float first[1] = {0.f};
#pragma unroll
      for (int it = 0; it < kIter; ++it)
#pragma unroll
        for (int v = 0; v < V; ++v) first[0] += hn[it].get(v);
      group_sum<1, kGroup>(first, red[phase], group);
      const float mean = first[0] * a.inv_c;
      float s[3] = {0.f, 0.f, 0.f};            // as above
#pragma unroll
      for (int it = 0; it < kIter; ++it) {
        const int32_t c = (it * kGroup + g) * V;
        if (c < a.C) {
          const Vec<T, V> w = load_vec<T, V>(a.w + c);   // from the caches, here and below
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const float d = hn[it].get(v) - mean, gv = dyn[it].get(v) * w.get(v);
            s[0] = fmaf(d, d, s[0]);
            s[1] += gv;
            s[2] = fmaf(gv, d, s[2]);
          }
        }
      }
      group_sum<3, kGroup>(s, red[phase] + 32, group);
      phase ^= 1;
      const float rstd = rsqrtf(fmaf(s[0], a.inv_c, a.eps));
      const float mean_g = s[1] * a.inv_c, along = rstd * (s[2] * a.inv_c) * rstd;
#pragma unroll
      for (int it = 0; it < kIter; ++it) {
        const int32_t c = (it * kGroup + g) * V;
        if (c < a.C) {
          const Vec<T, V> w = load_vec<T, V>(a.w + c);
          if constexpr (kIsWide) {
            if (a.dres) rn[it] = load_vec<T, V>(a.dres + t * a.C + c);
          }
          float dx[V];
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const float dy = dyn[it].get(v), d = hn[it].get(v) - mean;
            dx[v] = rstd * (fmaf(dy, w.get(v), -mean_g) - d * along);
            if (a.dres) dx[v] += rn[it].get(v);
            if constexpr (kIsWide) {
              sums[c + v] = fmaf(dy, d * rstd, sums[c + v]);
              sums[a.C + c + v] += dy;
            } else {
              dw[it * V + v] = fmaf(dy, d * rstd, dw[it * V + v]);
              db[it * V + v] += dy;
            }
          }
          Vec<T, V> o;
          o.put(dx);
          store_vec<T, V>(a.dx + t * a.C + c, o);
        }
      }
      if constexpr (kIsWide) load(t + step);
    }
  }
  auto kept = [&](bool bias, int i) {            // this thread's sum i
    if constexpr (kPaired) {
      float lo, hi;
      sm103::f2_split(bias ? db2[i / 2] : dw2[i / 2], lo, hi);
      return i % 2 ? hi : lo;
    } else {
      return bias ? db[i] : dw[i];
    }
  };

  griddep_launch_dependents();               // the second kernel may come to wait for this one
  constexpr int kOwnSums = kGroups > 1 ? kGroups * kKept * (kGroup + 1) : 0;
  float* part = a.part ? a.part + (int64_t)blockIdx.x * 2 * a.C : sums + kOwnSums;
  if constexpr (kIsWide) {
    __syncthreads();
    for (int32_t c = threadIdx.x; c < 2 * a.C; c += kBlock) part[c] = sums[c];
  } else if constexpr (kGroups == 1) {
#pragma unroll
    for (int it = 0; it < kIter; ++it)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int32_t c = (it * kGroup + g) * V + v;
        if (c < a.C) {
          part[c] = kept(false, it * V + v);
          part[a.C + c] = kept(true, it * V + v);
        }
      }
  } else {
    // [group][vector element][thread], a row padded so that neither access conflicts; the
    // weight's sums, then the bias's.
    constexpr int kLine = kGroup + 1;
    float* mine = sums + group * (kIter * V * kLine);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kIter * V; ++i) mine[i * kLine + g] = kept(which, i);
      __syncthreads();
      for (int32_t c = threadIdx.x; c < a.C; c += kBlock) {
        const int vec = c / V, i = vec / kGroup * V + c % V;
        float total = 0.f;
#pragma unroll
        for (int w = 0; w < kGroups; ++w) total += sums[(w * kIter * V + i) * kLine + vec % kGroup];
        part[which * a.C + c] = total;
      }
    }
  }
  if constexpr (!kIsWide) {
    if (!a.part)
      sum_lines_of_cluster(part, (int32_t)gridDim.x, a.C, a.dweight, a.C, a.dbias);
  }
}

// Rows that one cluster takes: six for each group of threads of its eight blocks, 16 channels
// a thread. That saves a launch and a workspace, which cost the host more than the rows in
// turn cost the device (320 x 500 fp32: 7.8 us on the device, with two launches 4.6; calls
// in a row from Python 15.4 us, four less than with two launches).
int32_t few_threads(int32_t C) {
  return C <= 512 ? 32 : C <= 1024 ? 64 : C <= 2048 ? 128 : 256;
}
int64_t few_rows(int32_t C) {
  return C > kWide ? 0 : 6 * kClusterLines * (kThreads / few_threads(C));
}

template <typename T, int V, int kIter, int kGroup>
pe_status launch(const Args<T>& a, cudaStream_t stream) {
  constexpr bool wide = kGroup > kThreads;
  constexpr int kGroups = wide ? 1 : kThreads / kGroup;
  static_assert(!wide || kIter * kGroup * V >= kMaxChannels, "a block holds the widest row");
  size_t smem = wide ? 2 * (size_t)a.C * sizeof(float)
                : kGroups > 1 ? (size_t)kGroups * kIter * V * (kGroup + 1) * sizeof(float)
                              : 0;
  const auto kernel = layernorm_bwd_kernel<T, V, kIter, kGroup>;
  if (a.N <= few_rows(a.C)) {
    smem += 2 * (size_t)a.C * sizeof(float);
    static_assert(wide || kGroups * kIter * V * (kGroup + 1) + 2 * kWide <= 56 * 256,
                  "the sums and a line fit the opt-in below");
    static std::atomic<uint64_t> done{0};
    PE_TRY(allow_shared_memory(kernel, 56 << 10, done));
    Args<T> few = a;
    few.part = nullptr;
    const int64_t need = ceil_div(a.N, kGroups);
    const dim3 blocks((unsigned)(need < kClusterLines ? need : kClusterLines));
    return launch_clusters(kernel, blocks, blocks, kGroup * kGroups, smem, stream, few);
  }
  if (wide) {
    static std::atomic<uint64_t> done{0};
    PE_TRY(allow_shared_memory(kernel, 2 * kMaxChannels * (int)sizeof(float), done));
  }
  static const int resident =
      resident_blocks(kernel, kGroup * kGroups, wide ? 2 * kMaxChannels * sizeof(float) : smem);
  if (resident < 1) return PE_ERR_CUDA;
  int64_t blocks = ceil_div(a.N, kGroups), most = (int64_t)resident * device_sm_count();
  if (most > (wide ? kMaxWideBlocks : kMaxBlocks)) most = wide ? kMaxWideBlocks : kMaxBlocks;
  if (blocks > most) blocks = most;
  kernel<<<(unsigned)blocks, kGroup * kGroups, smem, stream>>>(a);
  PE_CUDA_TRY(cudaGetLastError());
  return launch_sum_parts(a.part, (int32_t)blocks, a.C, a.dweight, a.C, a.dbias, stream);
}

// The form for V neighbouring channels per access: vectors a thread and threads a row, by the
// row's width. 16 channels a thread of bf16, 8 of fp32 (which take twice the registers); with
// the residual's gradient:
//   bf16 32299 x 768    16 channels of 64 threads 43.2 us, 8 of 96 41.6, 24 of 32 51
//   bf16 169151 x 1024  16 of 64 220 us, 8 of 128 236;   90487 x 512  16 of 32 64, 8 of 64 68
template <typename T, int V>
pe_status launch_rows(const Args<T>& a, cudaStream_t stream) {
  const int32_t C = a.C;
  if (C > kWide) return launch<T, V, 16 / V, 1024>(a, stream);
  if (a.N <= few_rows(C)) {
    if (few_threads(C) == 32) return launch<T, V, 16 / V, 32>(a, stream);
    if (few_threads(C) == 64) return launch<T, V, 16 / V, 64>(a, stream);
    if (few_threads(C) == 128) return launch<T, V, 16 / V, 128>(a, stream);
    return launch<T, V, 16 / V, 256>(a, stream);
  }
  if constexpr (V == 8) {
    if (C <= 256) return launch<T, V, 1, 32>(a, stream);
    if (C <= 512) return launch<T, V, 2, 32>(a, stream);
    if (C <= 768) return launch<T, V, 1, 96>(a, stream);
    if (C <= 1024) return launch<T, V, 2, 64>(a, stream);
    if (C <= 2048) return launch<T, V, 2, 128>(a, stream);
    return launch<T, V, 2, 256>(a, stream);
  } else {
    constexpr int kIter = 8 / V;               // eight channels a thread
    if (C <= 256) return launch<T, V, kIter, 32>(a, stream);
    if (C <= 512) return launch<T, V, kIter, 64>(a, stream);
    if (C <= 1024) return launch<T, V, kIter, 128>(a, stream);
    if (C <= 2048) return launch<T, V, kIter, 256>(a, stream);
    return launch<T, V, 2 * kIter, 256>(a, stream);
  }
}

template <typename T>
pe_status run(const void* dy, const void* h, const void* w, const void* dres, int64_t N,
              int32_t C, float eps, void* dx, float* dweight, float* dbias, void* ws,
              cudaStream_t stream) {
  const Args<T> a = {static_cast<const T*>(dy),
                     static_cast<const T*>(h),
                     static_cast<const T*>(w),
                     static_cast<const T*>(dres),
                     N,
                     C,
                     1.f / (float)C,
                     eps,
                     static_cast<T*>(dx),
                     static_cast<float*>(ws),
                     dweight,
                     dbias};
  constexpr int V = 16 / sizeof(T);
  if (vectors<V>(C, a.dy, a.w, a.h, a.dx, a.dres))
    return launch_rows<T, V>(a, stream);
  if (V > 4 && vectors<4>(C, a.dy, a.w, a.h, a.dx, a.dres))
    return launch_rows<T, 4>(a, stream);
  if (vectors<2>(C, a.dy, a.w, a.h, a.dx, a.dres))
    return launch_rows<T, 2>(a, stream);
  return launch_rows<T, 1>(a, stream);
}

}  // namespace

}  // namespace pe

using namespace pe;

extern "C" size_t pe_layernorm_bwd_workspace_size(int64_t N, int32_t C) {
  if (N < 1 || C < 1 || C > kMaxChannels || N <= few_rows(C)) return 0;
  return (size_t)(C > kWide ? kMaxWideBlocks : kMaxBlocks) * 2 * (size_t)C * sizeof(float);
}

extern "C" pe_status pe_layernorm_bwd(pe_dtype dtype, const void* dy, const void* h,
                                      const void* weight, const void* dresidual, int64_t N,
                                      int32_t C, float eps, void* dx, float* dweight,
                                      float* dbias, void* workspace, size_t workspace_bytes,
                                      pe_stream_t stream_) {
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (dtype != PE_BF16 && dtype != PE_FP32) return PE_ERR_UNSUPPORTED;
  if (N < 0 || C < 1 || !(eps > 0.f) || !isfinite(eps) || !dweight) return PE_ERR_INVALID_ARG;
  if (C > kMaxChannels) return PE_ERR_UNSUPPORTED;
  if (N > 0) {
    if (!dy || !h || !weight || !dx) return PE_ERR_INVALID_ARG;
    const size_t need = pe_layernorm_bwd_workspace_size(N, C);
    if (need && (!workspace || !aligned(workspace, 16) || workspace_bytes < need))
      return PE_ERR_WORKSPACE;
  }
  if (!device_is_sm103()) return PE_ERR_UNSUPPORTED;
  if (N == 0) {
    PE_CUDA_TRY(cudaMemsetAsync(dweight, 0, (size_t)C * sizeof(float), stream));
    if (dbias) PE_CUDA_TRY(cudaMemsetAsync(dbias, 0, (size_t)C * sizeof(float), stream));
    return PE_OK;
  }
  if (dtype == PE_FP32)
    return run<float>(dy, h, weight, dresidual, N, C, eps, dx, dweight, dbias, workspace, stream);
  return run<__nv_bfloat16>(dy, h, weight, dresidual, N, C, eps, dx, dweight, dbias, workspace,
                            stream);
}
