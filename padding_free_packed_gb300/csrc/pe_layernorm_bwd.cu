// Backward of LayerNorm over packed token rows. h is the normalised input as the forward
// stored it; with n = (h - mean) rstd and g = w dy,
//   dx = rstd (g - mean(g) - n mean(g n)) (+ dresidual),
//   dweight = sum over rows of dy n, dbias = sum over rows of dy.
// A bandwidth kernel: a row of h and dy is read once into the registers of 1 to 8 warps, its
// statistics are formed again from there (mean first, then squares of what is left, so a
// large mean costs no precision), and dx is written once. The weight's and bias's sums of a
// thread's own channels stay in fp32 registers until the block's last row; a second kernel
// adds the blocks' lines in a fixed order. The next row's loads are in flight while a row is
// worked on, in registers or, for wider rows, in a ring in shared memory. Rows wider than 4096
// channels take a block each and keep those sums in shared memory.
// Measured (GB300, device time, with the residual's gradient): 32299 x 768 bf16 in 36 us (5.5
// TB/s, 0.81 of the measured copy rate; some 5 us are the start, the last rows and the second
// kernel), 169151 x 1024 bf16 207 us (0.99), 32299 x 2304 bf16 94 us (0.93), 90487 x 512
// fp32 113 us (0.97). What bounds the narrower ones is a row's chain of two joint sums, with
// the 8 to 24 warps an SM that the registers of a thread's own sums (two for each of its
// channels) leave. In paired arithmetic 768 channels took 42 us where single fp32 operations
// took 45. Further from the bound: fp32 rows past 2304 channels, without the ring (20000 x 3000
// 174 us, 0.81, x 4096 207, 0.93), bf16 rows of odd width, which move two bytes at a time (20000
// x 777 50 us, 0.37), and rows past 4096 channels, a block each with nothing in flight beside its
// joint sums (10000 x 5120 bf16 353 us, 0.17, x 8192 468, 0.21; 5000 x 8192 fp32 213, 0.45).
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
    V == 8 ? (kIter > 1 ? 2 : 3) : V * kIter > 8 ? 1 : 2;

// With a ring of rows in shared memory no registers wait for loads, so a thread can have 24
// channels of bf16 (or 12 of fp32) and a row fewer threads, whose sums take fewer steps: 768
// channels of one warp, without a barrier, 36 us, of two 38, of three with 8 each 39. One
// block an SM, of as many threads as the registers allow.
constexpr int kRing = 3;                       // the row at work and two more
template <int V, int kIter>
constexpr int kRingThreads = V * kIter > 8 ? 384 : 512;
template <int V, int kIter, int kGroup, bool kByRing>
constexpr int kGroupsOf = kGroup > kThreads ? 1
                          : kByRing         ? kRingThreads<V, kIter> / kGroup
                                            : kThreads / kGroup;

// 16 bytes into shared memory, in the thread's open group of copies.
__device__ __forceinline__ void copy_16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// Waits for this thread's copies but those of its last kLeft groups.
template <int kLeft>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// kGroup threads a row, each with kIter vectors of V channels, the same for all of its rows.
// kByRing: every thread copies into the ring what it will read itself, so that its own wait is
// enough.
template <typename T, int V, int kIter, int kGroup, bool kByRing>
__global__ void __launch_bounds__(kGroup * kGroupsOf<V, kIter, kGroup, kByRing>,
                                  kGroup > kThreads || kByRing ? 1 : kMinBlocks<V, kIter, kGroup>)
layernorm_bwd_kernel(const Args<T> a) {
  constexpr bool kIsWide = kGroup > kThreads;
  constexpr int kGroups = kGroupsOf<V, kIter, kGroup, kByRing>;
  constexpr int kBlock = kGroup * kGroups;
  // wide: [2][C]; else the ring, then every group's at the end
  extern __shared__ __align__(16) float sums[];
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
  // The ring: [row][dy, h, dres][vector][thread], 16 bytes each.
  static_assert(!kByRing || (kPaired && sizeof(T) * V == 16), "the ring holds 16 bytes a vector");
  constexpr uint32_t kPlane = kBlock * 16, kSlot = 3 * kIter * kPlane;
  [[maybe_unused]] char* const mine_in_ring = reinterpret_cast<char*>(sums) + threadIdx.x * 16;
  [[maybe_unused]] uint32_t slot = 0;          // of the row at work
  [[maybe_unused]] auto fetch = [&](int64_t row, uint32_t into) {
    const uint32_t at = sm103::smem_u32(mine_in_ring) + into * kSlot;
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
      const int32_t c = (it * kGroup + g) * V;
      if (c < a.C && row < a.N) {
        copy_16(at + it * kPlane, a.dy + row * a.C + c);
        copy_16(at + (kIter + it) * kPlane, a.h + row * a.C + c);
        if (a.dres) copy_16(at + (2 * kIter + it) * kPlane, a.dres + row * a.C + c);
      }
    }
    copy_commit();                             // a group for every row, copied or not
  };
  [[maybe_unused]] auto fetched = [&](int plane) {
    return load_vec<T, V>(
        reinterpret_cast<const T*>(mine_in_ring + slot * kSlot + plane * kPlane));
  };
  if constexpr (kByRing) {
#pragma unroll
    for (int i = 0; i < kRing - 1; ++i) fetch(t + i * step, i);
  } else {
    load(t);
  }
  int phase = 0;
  for (; t < a.N; t += step) {
    if constexpr (kPaired) {
      using namespace sm103;
      Vec<T, V> dyn[kIter], hn[kIter], rn[kIter];
      uint64_t total = 0ull;
      if constexpr (kByRing) {
        // Over the row before, whose numbers have all been used.
        fetch(t + (kRing - 1) * step, slot == 0 ? kRing - 1 : slot - 1);
        copy_wait<kRing - 1>();
      }
#pragma unroll
      for (int it = 0; it < kIter; ++it) {
        if constexpr (kByRing) {
          dyn[it].zero();
          hn[it].zero();
          if ((it * kGroup + g) * V < a.C) {
            dyn[it] = fetched(it);
            hn[it] = fetched(kIter + it);
          }
        } else {
          dyn[it] = dyv[it];
          hn[it] = hv[it];
          rn[it] = rv[it];
        }
#pragma unroll
        for (int j = 0; j < V / 2; ++j) total = fadd2(total, hn[it].pair(j));
      }
      if constexpr (!kByRing) load(t + step);
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
          if constexpr (kByRing) {
            if (a.dres) rn[it] = fetched(2 * kIter + it);
          }
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
      if constexpr (kByRing) slot = slot + 1 == kRing ? 0 : slot + 1;
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
// in a row from Python 16 us, four less than with two launches).
int32_t few_threads(int32_t C) {
  return C <= 512 ? 32 : C <= 1024 ? 64 : C <= 2048 ? 128 : 256;
}
int64_t few_rows(int32_t C) {
  return C > kWide ? 0 : 6 * kClusterLines * (kThreads / few_threads(C));
}

// `resident` blocks an SM (or as many as there are rows for), and the sum of their lines.
template <typename T, typename K>
pe_status launch_blocks(K* kernel, const Args<T>& a, int groups, int threads, size_t smem,
                        int resident, int most_blocks, cudaStream_t stream) {
  if (resident < 1) return PE_ERR_CUDA;
  int64_t blocks = ceil_div(a.N, groups), most = (int64_t)resident * device_sm_count();
  if (most > most_blocks) most = most_blocks;
  if (blocks > most) blocks = most;
  kernel<<<(unsigned)blocks, threads, smem, stream>>>(a);
  PE_CUDA_TRY(cudaGetLastError());
  return launch_sum_parts(a.part, (int32_t)blocks, a.C, a.dweight, a.C, a.dbias, stream);
}

template <typename T, int V, int kIter, int kGroup>
pe_status launch_ring(const Args<T>& a, cudaStream_t stream) {
  constexpr int kGroups = kGroupsOf<V, kIter, kGroup, true>, kBlock = kGroup * kGroups;
  constexpr size_t join = (size_t)kGroups * kIter * V * (kGroup + 1) * sizeof(float);
  constexpr size_t ring = (size_t)kRing * 3 * kIter * 16 * kBlock;
  constexpr size_t smem = join > ring ? join : ring;
  static_assert(smem <= 226 << 10, "the ring fits an SM's shared memory");
  const auto kernel = layernorm_bwd_kernel<T, V, kIter, kGroup, true>;
  static std::atomic<uint64_t> done{0};
  PE_TRY(allow_shared_memory(kernel, (int)smem, done));
  return launch_blocks(kernel, a, kGroups, kBlock, smem, 1, kMaxBlocks, stream);
}

template <typename T, int V, int kIter, int kGroup>
pe_status launch(const Args<T>& a, cudaStream_t stream) {
  constexpr bool wide = kGroup > kThreads;
  constexpr int kGroups = kGroupsOf<V, kIter, kGroup, false>;
  static_assert(!wide || kIter * kGroup * V >= kMaxChannels, "a block holds the widest row");
  size_t smem = wide ? 2 * (size_t)a.C * sizeof(float)
                : kGroups > 1 ? (size_t)kGroups * kIter * V * (kGroup + 1) * sizeof(float)
                              : 0;
  const auto kernel = layernorm_bwd_kernel<T, V, kIter, kGroup, false>;
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
  static DeviceNumber known;
  const int resident = resident_blocks(
      kernel, kGroup * kGroups, wide ? 2 * kMaxChannels * sizeof(float) : smem, known);
  return launch_blocks(kernel, a, kGroups, kGroup * kGroups, smem, resident,
                       wide ? kMaxWideBlocks : kMaxBlocks, stream);
}

// The form for V neighbouring channels per access: vectors a thread and threads a row, by the
// row's width. With the residual's gradient, channels of threads by registers / by the ring:
//   bf16 90487 x 512    16 of 32 61 us, 8 of 64 68       / 24 of 32 59, 16 of 32 61
//        20000 x 256    8 of 32 12.8                     / 24 of 32 14.6, 8 of 32 12.8
//        32299 x 768    8 of 96 41, 16 of 64 43          / 24 of 32 36, 16 of 64 38
//        169151 x 1024  16 of 64 218, 8 of 128 236       / 24 of 64 207, 16 of 64 209
//        20000 x 1536   16 of 128 52                     / 24 of 64 43
//        32299 x 2304   16 of 256 124                    / 24 of 96 94
//        20000 x 4096   16 of 256 112                    / 24 of 192 100
//   fp32 90487 x 512    8 of 64 113                      / 8 of 96 110
//        20000 x 768    8 of 128 45                      / 8 of 128 40, 12 of 64 42
//        20000 x 1140   8 of 256 73                      / 12 of 192 70, 8 of 160 66
//        20000 x 2304   16 of 256 147                    / 12 of 192 111
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
    if (C <= 768) return launch_ring<T, V, 3, 32>(a, stream);
    if (C <= 1536) return launch_ring<T, V, 3, 64>(a, stream);
    if (C <= 2304) return launch_ring<T, V, 3, 96>(a, stream);
    return launch_ring<T, V, 3, 192>(a, stream);
  } else {
    constexpr int kIter = 8 / V;               // eight channels a thread
    if (C <= 256) return launch<T, V, kIter, 32>(a, stream);
    if (C <= 512) return launch<T, V, kIter, 64>(a, stream);
    if constexpr (V * sizeof(T) == 16) {
      if (C <= 1024) return launch_ring<T, V, 2, 128>(a, stream);
      if (C <= 2304) return launch_ring<T, V, 3, 192>(a, stream);
    } else {
      if (C <= 1024) return launch<T, V, kIter, 128>(a, stream);
      if (C <= 2048) return launch<T, V, kIter, 256>(a, stream);
    }
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
  if (C > kMaxChannels || !by_elements(PE_FP32, dweight, dbias)) return PE_ERR_UNSUPPORTED;
  if (N > 0) {
    if (!dy || !h || !weight || !dx) return PE_ERR_INVALID_ARG;
    if (!by_elements(dtype, dy, h, weight, dresidual, dx)) return PE_ERR_UNSUPPORTED;
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
