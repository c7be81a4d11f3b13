// Matrix product of 8-bit operands with a scale for each block of 128, few rows:
// out[i, j] = sum over c of sa[c, i] sb[c, j / 128] (sum over block c of
// a[i, l] b[j, l]).
//
// Few rows of a leave few tiles, and a tile's time is the latency of its loads.
// So the tile is narrow (128 rows of b, which is the MMA's M, by kT = 16, 32 or 64 rows
// of a, its N), several blocks of k are in flight in a CTA, and a cluster of up to 8 CTAs
// shares the sum over k, joined through distributed shared memory in the order of
// k (no workspace, no second launch). A thread holds one row of b, i.e. one column
// of out, so stores of a warp are consecutive for any n; the scale of b is one
// number a block, those of a one for each of the thread's kT sums.
//
// Measured (GB300, device time): 1 x 2304 x 768 in 4.4 us and 320 x 1001 x 1140 in
// 6.4 us, of which a launch that does nothing is 2.3 us and each block of k 0.29 us
// (kT = 16) to 0.43 us (64); the pair kernel takes 8.9 and 14 us. 128 rows a CTA lost
// to 64 wherever the pair kernel did too (320 x 2304 x 768: 9.0 against 6.7 us).
//
//   warps 0-3   scaling and sums
//   warp 4      TMA producer
//   warp 5      MMA issue
//   warp 6      looks for scales that are far: where it finds one, the CTA sums its
//               blocks again, each in two steps (a test in the loop of warps 0-3 took
//               768 x 768 x 9001 from 20.6 us to 24 and more, one before it to 22)
#include <type_traits>

#include "pe_matmul_fp8.cuh"

namespace pe {

namespace {

using namespace sm103;

constexpr int kThreads = 224;
constexpr int kBufs = 4;                  // accumulators in flight
constexpr int kScaleAhead = 6;            // blocks of k that scales are copied ahead
constexpr int kScaleSlots = 8;
constexpr int kMaxSplit = 8;

// Blocks in flight: two CTAs share an SM.
template <int kT>
constexpr int kStages = kT == 64 ? 4 : 5;

template <int kT>
struct alignas(1024) Smem {
  union {
    struct {
      uint8_t b[kStages<kT>][128 * kFp8Block];
      uint8_t a[kStages<kT>][kT * kFp8Block];
    } in;
    float sums[kT][128];                  // this CTA's part, once its loads are done
  };
  alignas(16) float scale[4][kScaleSlots][kT + 4];   // each warp's own copy; [kT]: of b
  uint64_t full[kStages<kT>], empty[kStages<kT>];
  uint64_t acc_full[kBufs], acc_empty[kBufs];
  uint64_t drain;
  uint32_t tmem_base;
  WaitGuard guard;
};

struct Params {
  const float* a_scales;
  const float* b_scales;
  int32_t m, n;
  int32_t blocks;            // of k
  int32_t split;
  int32_t out_fp32;
  int32_t out_by_four;       // rows of out start at multiples of four elements
  uint32_t idesc;
  void* out;
  DeviceStatus* status;
  uint64_t wait_limit_ns;
};

enum WaitSite { kSiteProducer = 81, kSiteMma = 82, kSiteEpilogue = 83 };

__device__ __forceinline__ void mma_fp8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b32 r;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "elect.sync r|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 16 consecutive 32-bit columns of this thread's tensor-memory lane, waited for.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ float4 load_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Four consecutive elements of out (the first `left` of them), in one store where
// rows of out start at multiples of four elements.
__device__ __forceinline__ void store4(const Params& p, int64_t at, int32_t left,
                                       const float4& v) {
  if (p.out_fp32) {
    float* o = static_cast<float*>(p.out) + at;
    if (p.out_by_four) {
      *reinterpret_cast<float4*>(o) = v;
    } else {
      o[0] = v.x;
      if (left > 1) o[1] = v.y;
      if (left > 2) o[2] = v.z;
      if (left > 3) o[3] = v.w;
    }
  } else {
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + at;
    if (p.out_by_four) {
      *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    } else {
      o[0] = __float2bfloat16_rn(v.x);
      if (left > 1) o[1] = __float2bfloat16_rn(v.y);
      if (left > 2) o[2] = __float2bfloat16_rn(v.z);
      if (left > 3) o[3] = __float2bfloat16_rn(v.w);
    }
  }
}

template <int kT>
__global__ void __launch_bounds__(kThreads)
matmul_rows_kernel(const __grid_constant__ CUtensorMap tm_a,
                   const __grid_constant__ CUtensorMap tm_b, const Params p) {
  constexpr int S = kStages<kT>;
  constexpr uint32_t kTmemCols = kBufs * kT < 32 ? 32 : kBufs * kT;
  extern __shared__ uint8_t raw[];
  Smem<kT>& s =
      *reinterpret_cast<Smem<kT>*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int32_t col_tile = blockIdx.x / p.split, part = blockIdx.x - col_tile * p.split;
  const int32_t col0 = col_tile * 128, row0 = blockIdx.y * kT;
  const int32_t lo = (int32_t)((int64_t)p.blocks * part / p.split);
  const int32_t count = (int32_t)((int64_t)p.blocks * (part + 1) / p.split) - lo;
  volatile WaitGuard* guard = &s.guard;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(smem_u32(&s.full[i]), 1);
      mbar_init(smem_u32(&s.empty[i]), 1);
    }
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(smem_u32(&s.acc_full[i]), 1);
      mbar_init(smem_u32(&s.acc_empty[i]), 4);
    }
    mbar_init(smem_u32(&s.drain), 1);
    s.guard.abort = 0;
    s.guard.limit_ns = p.wait_limit_ns;
    fence_mbarrier_init();
  }
  if (warp == 5) {
    tmem_alloc(smem_u32(&s.tmem_base), kTmemCols);
    tmem_relinquish();
  }
  if (warp == 4 && lane == 0) {
    prefetch_tensormap(&tm_a);
    prefetch_tensormap(&tm_b);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;

  float sum[kT];
  const int32_t col_blocks = (p.n + kFp8Block - 1) / kFp8Block;

  // All blocks of this CTA. `from` counts the blocks of earlier calls, so that barriers go
  // on in their phases; `far` is whether the blocks are added in two steps. Returns, in
  // warp 6, whether they have to be.
  auto add_blocks = [&](int32_t from, auto far) {
    bool found = false;
    if (warp == 4) {
      if (lane == 0) {
        // ---------------------------------------------------------- producer
        int32_t issued = from;
        for (; issued < from + count; ++issued) {
          const int stage = issued % S;
          if (!mbar_wait(smem_u32(&s.empty[stage]), ((issued / S) & 1) ^ 1, guard, p.status,
                         kSiteProducer))
            break;
          const uint32_t bar = smem_u32(&s.full[stage]);
          const int32_t x = (lo + issued - from) * kFp8Block;
          mbar_arrive_expect_tx(bar, (128 + kT) * kFp8Block);
          tma_load_2d(smem_u32(s.in.b[stage]), &tm_b, bar, x, col0);
          tma_load_2d(smem_u32(s.in.a[stage]), &tm_a, bar, x, row0);
        }
        // No load is in flight past this (all have been waited for unless a wait gave up).
        for (int32_t i = issued > S ? issued - S : 0; i < issued; ++i)
          mbar_drain_wait(smem_u32(&s.full[i % S]), (i / S) & 1);
      }
      __syncwarp();
    } else if (warp == 5) {
      // ------------------------------------------------------------ MMA issue
      for (int32_t i = from; i < from + count; ++i) {
        const int stage = i % S, buf = i % kBufs;
        if (!warp_wait(smem_u32(&s.full[stage]), (i / S) & 1, guard, p.status, kSiteMma)) break;
        if (!warp_wait(smem_u32(&s.acc_empty[buf]), ((i / kBufs) & 1) ^ 1, guard, p.status,
                       kSiteMma))
          break;
        tc_fence_after();
        const uint64_t db = smem_desc_sw128(smem_u32(s.in.b[stage]), 16, 1024);
        const uint64_t da = smem_desc_sw128(smem_u32(s.in.a[stage]), 16, 1024);
#pragma unroll
        for (int k = 0; k < 4; ++k)          // 32 bytes of k each: 2 units of 16 bytes
          mma_fp8(tmem + buf * kT, db + 2 * k, da + 2 * k, p.idesc, k > 0);
        tc_commit_warp(smem_u32(&s.acc_full[buf]));
        tc_commit_warp(smem_u32(&s.empty[stage]));
      }
      tc_commit_warp(smem_u32(&s.drain));    // no MMA is in flight past this
      mbar_drain_wait(smem_u32(&s.drain), from ? 1 : 0);
    } else if (warp == 6) {
      // ------------------------------------------------------------ far scales
      if constexpr (!decltype(far)::value) {
        constexpr int kFlight = 8;           // loads; past the end, the last one again
        for (int32_t e = lane; e < count * kT; e += 32 * kFlight) {
          float v[kFlight];
#pragma unroll
          for (int u = 0; u < kFlight; ++u) {
            const int32_t at = e + 32 * u < count * kT ? e + 32 * u : count * kT - 1;
            const int32_t row = row0 + at % kT;
            v[u] = __ldg(p.a_scales + (int64_t)(lo + at / kT) * p.m + (row < p.m ? row : row0));
          }
#pragma unroll
          for (int u = 0; u < kFlight; ++u) found |= scale_is_far(v[u]);
        }
        for (int32_t i = lane; i < count; i += 32)
          found |= scale_is_far(__ldg(p.b_scales + (int64_t)(lo + i) * col_blocks + col_tile));
        __syncwarp();
      }
    } else {
      // ------------------------------------------------------------ scaling and sums
#pragma unroll
      for (int c = 0; c < kT; ++c) sum[c] = 0.f;
      const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
      auto copy_scales = [&](int32_t i) {    // of block i, into this warp's ring
        if (i < count) {
          float* slot = s.scale[warp][i % kScaleSlots];
          const float* src = p.a_scales + (int64_t)(lo + i) * p.m + row0;
#pragma unroll
          for (int c = 0; c < kT; c += 32) {
            const int at = c + lane;
            if (kT >= 32 || at < kT)
              copy_async4(&slot[at], src + (row0 + at < p.m ? at : 0), row0 + at < p.m);
          }
          if (lane == 0)
            copy_async4(&slot[kT], p.b_scales + (int64_t)(lo + i) * col_blocks + col_tile, true);
        }
        copy_async_commit();
      };
      // 16 or 32 columns of tensor memory, scaled, to the sums of rows h ...
      auto add = [&](const auto& d, int h, const float* slot, float sb) {
        constexpr int kCols = sizeof(d) / sizeof(d[0]);
#pragma unroll
        for (int c = 0; c < kCols; c += 4) {
          const float4 sa = *reinterpret_cast<const float4*>(slot + h + c);
          const float a[4] = {sa.x, sa.y, sa.z, sa.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float& to = sum[h + c + j];
            const float v = __uint_as_float(d[c + j]);
            if constexpr (decltype(far)::value) {
              const float2 f = far_factors(a[j], sb);
              to = fmaf(v * f.x, f.y, to);
            } else {
              to = fmaf(a[j] * sb, v, to);
            }
          }
        }
      };
      for (int32_t i = 0; i < kScaleAhead; ++i) copy_scales(i);
      for (int32_t i = 0; i < count; ++i) {
        copy_scales(i + kScaleAhead);        // the slot's block has been read (syncwarp below)
        copy_async_wait<kScaleAhead>();
        __syncwarp();
        const float* slot = s.scale[warp][i % kScaleSlots];
        const float sb = slot[kT];
        const int buf = (from + i) % kBufs;
        if (!warp_wait(smem_u32(&s.acc_full[buf]), ((from + i) / kBufs) & 1, guard, p.status,
                       kSiteEpilogue))
          break;
        tc_fence_after();
        const uint32_t src = lane_base + buf * kT;
        if constexpr (kT == 16) {
          uint32_t d[16];
          tmem_ld16(src, d);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&s.acc_empty[buf]));
          add(d, 0, slot, sb);
        } else {
#pragma unroll
          for (int h = 0; h < kT; h += 32) {
            uint32_t d[32];
            tmem_ld32(src + h, d);
            tmem_wait_ld(d);
            if (h + 32 == kT) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(smem_u32(&s.acc_empty[buf]));
            }
            add(d, h, slot, sb);
          }
        }
      }
      copy_async_wait<0>();
    }
    // Every load and MMA of this CTA is done.
    tc_fence_before();
    return __syncthreads_or(found);
  };
  if (add_blocks(0, std::false_type())) {
    const bool gave_up = guard->abort;       // the same in all threads until the barrier
    __syncthreads();
    tc_fence_after();
    if (!gave_up) add_blocks(count, std::true_type());
  }
  // This CTA's stages may hold its sums now.
  if (p.split == 1) {
    const int32_t col = col0 + threadIdx.x;
    if (warp < 4 && col < p.n) {
#pragma unroll
      for (int c = 0; c < kT; ++c) {
        if (row0 + c < p.m) {
          const int64_t at = (int64_t)(row0 + c) * p.n + col;
          if (p.out_fp32)
            static_cast<float*>(p.out)[at] = sum[c];
          else
            static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(sum[c]);
        }
      }
    }
  } else {
    if (warp < 4) {
#pragma unroll
      for (int c = 0; c < kT; ++c) s.sums[c][threadIdx.x] = sum[c];
    }
    cluster_sync();
    // The cluster's CTAs deal the kT rows of out among them, their warps each CTA's;
    // a lane adds four columns, with the parts of two rows in flight.
    const int32_t col = col0 + 4 * lane;
    if (warp < 4 && col < p.n) {
      const int32_t step = 4 * p.split;
      const int32_t rows = p.m - row0 < kT ? p.m - row0 : kT;
      for (int32_t c = (int32_t)cluster_rank() + p.split * warp; c < rows; c += 2 * step) {
        const bool two = c + step < rows;
        const uint32_t at0 = smem_u32(&s.sums[c][4 * lane]);
        const uint32_t at1 = two ? smem_u32(&s.sums[c + step][4 * lane]) : at0;
        float4 v[2][kMaxSplit];
#pragma unroll
        for (int r = 0; r < kMaxSplit; ++r) {
          if (r < p.split) {
            v[0][r] = load_cluster_f32x4(peer_address(at0, r));
            v[1][r] = load_cluster_f32x4(peer_address(at1, r));
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h == 1 && !two) break;
          float4 t = v[h][0];
#pragma unroll
          for (int r = 1; r < kMaxSplit; ++r) {
            if (r < p.split) {
              t.x += v[h][r].x;
              t.y += v[h][r].y;
              t.z += v[h][r].z;
              t.w += v[h][r].w;
            }
          }
          store4(p, (int64_t)(row0 + c + h * step) * p.n + col, p.n - col, t);
        }
      }
    }
    cluster_sync();                        // the sums have been read by the whole cluster
  }
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int kT>
pe_status launch(const MatmulFp8& q, int32_t split, DeviceStatus* status, cudaStream_t stream) {
  CUtensorMap ma, mb;
  PE_TRY(matmul_map(&ma, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, q.a, q.m, q.k, q.a_ld, kT));
  PE_TRY(matmul_map(&mb, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, q.b, q.n, q.k, q.b_ld, 128));
  Params p;
  p.a_scales = q.a_scales;
  p.b_scales = q.b_scales;
  p.m = q.m;
  p.n = q.n;
  p.blocks = (int32_t)ceil_div(q.k, kFp8Block);
  p.split = split;
  p.out_fp32 = q.out_fp32 ? 1 : 0;
  p.out_by_four = q.n % 4 == 0 && aligned(q.out, q.out_fp32 ? 16 : 8) ? 1 : 0;
  p.idesc = idesc_fp8(128, kT, q.b_e5m2, q.a_e5m2);     // b is the MMA's first operand
  p.out = q.out;
  p.status = status;
  p.wait_limit_ns = wait_limit_ns();
  const size_t smem = sizeof(Smem<kT>) + 1024;
  static_assert(sizeof(Smem<kT>) + 1024 <= 227 * 1024, "shared memory exceeds the per-CTA limit");
  PE_CUDA_TRY(cudaFuncSetAttribute(matmul_rows_kernel<kT>,
                                   cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   static_cast<int>(smem)));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(ceil_div(q.n, 128) * split), (unsigned)ceil_div(q.m, kT));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  PE_CUDA_TRY(cudaLaunchKernelEx(&cfg, matmul_rows_kernel<kT>, ma, mb, p));
  return PE_OK;
}

}  // namespace

pe_status matmul_rows(const MatmulFp8& p, int32_t rows, int32_t split, DeviceStatus* status,
                      cudaStream_t stream) {
  switch (rows) {
    case 16: return launch<16>(p, split, status, stream);
    case 32: return launch<32>(p, split, status, stream);
    default: return launch<64>(p, split, status, stream);
  }
}

}  // namespace pe
