// Matrix product with bias, activation and residual, few rows:
// out = act(a b^T + bias) + residual.
//
// Few rows of a leave few tiles, and a tile's time is the latency of its loads. So the tile
// is narrow (128 rows of b, which is the MMA's M, by kT = 16, 32 or 64 rows of a, its N),
// several blocks of k are in flight in a CTA, and a cluster of up to 8 CTAs shares the sum
// over k, joined through distributed shared memory in the order of k (no workspace, no
// second launch). An accumulator sums four blocks of k (of fp32 operands' parts of one size),
// which four warps then add to fp32 sums in registers (the tensor cores cut a sum off after
// every 16 products); at the end they copy them to shared memory, and the cluster's CTAs deal
// out the rows among them: a lane adds four neighbouring columns, finishes and writes them. That part is one warp a
// scheduler or two, so it is bound by its instructions, not by memory: the activation is a
// template's, and all eight warps take part.
// With geglu the tile's rows of b are 64 of the gate's and the same 64 of the up part's.
//
// Measured (GB300, device time, K = 768, bf16): 1 x 2304 in 5.6 us, 64 x 768 in 5.8, 128 x 2304
// in 6.6, 320 x 2304 in 8.4, 320 x 1001 (K = 1140) in 8.0, of which a launch that does nothing is 2.3. A block
// of k takes 0.28 us in turn, the latency of its load through six stages.
//
//   warps 0-3   sums to shared memory
//   warp 4      TMA producer
//   warp 5      MMA issue
//   all         join and epilogue
#include "pe_matmul.cuh"

namespace pe {

namespace {

using namespace sm103;

constexpr int kThreads = 256;
constexpr int kMaxSplit = 8;
constexpr int kChunk = 4;                 // blocks of k that one accumulator sums
constexpr uint32_t kBBytes = 128 * 128;

// Blocks in flight: two CTAs share an SM.
template <int kT>
constexpr int kStages = kT == 64 ? 4 : kT == 32 ? 5 : 6;

template <int kT>
struct alignas(1024) Smem {
  union {
    struct {
      uint8_t b[kStages<kT>][kBBytes];
      uint8_t a[kStages<kT>][kT * 128];
    } in;
    float sums[kT][128];                  // this CTA's part, once its loads are done
  };
  uint64_t full[kStages<kT>], empty[kStages<kT>];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  WaitGuard guard;
};

struct Params {
  MatmulEpilogue e;
  int32_t blocks;            // of k, of all terms
  int32_t term_blocks;       // of one term
  int32_t terms;
  int32_t split;
  Chains chains;
  int32_t a_transposed, b_transposed;
  int32_t up_row;            // geglu: b's first up row
  uint32_t idesc;
  DeviceStatus* status;
  uint64_t wait_limit_ns;
};

enum WaitSite { kSiteProducer = 101, kSiteMma = 102, kSiteEpilogue = 103 };

__device__ __forceinline__ float4 load_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
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

template <int kT, int kAct>
__global__ void __launch_bounds__(kThreads, 2)
matmul_narrow_kernel(const __grid_constant__ CUtensorMap tm_a,
                     const __grid_constant__ CUtensorMap tm_b, const __grid_constant__ Params p) {
  constexpr int S = kStages<kT>;
  constexpr bool kGeglu = kAct == PE_ACT_GEGLU;
  constexpr uint32_t kTmemCols = 2 * kT;
  constexpr int32_t kOutCols = kGeglu ? 64 : 128;          // of a tile
  extern __shared__ uint8_t raw[];
  Smem<kT>& s =
      *reinterpret_cast<Smem<kT>*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int32_t col_tile = blockIdx.x / p.split, part = blockIdx.x - col_tile * p.split;
  const int32_t col0 = col_tile * kOutCols, row0 = blockIdx.y * kT;
  const int32_t lo = (int32_t)((int64_t)p.blocks * part / p.split);
  const int32_t count = (int32_t)((int64_t)p.blocks * (part + 1) / p.split) - lo;
  volatile WaitGuard* guard = &s.guard;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(smem_u32(&s.full[i]), 1);
      mbar_init(smem_u32(&s.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
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
  griddep_wait();                          // what the kernel before this one wrote is read below
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;

  if (warp == 4) {
    if (lane == 0) {
      // ---------------------------------------------------------- producer
      int32_t term = lo / p.term_blocks, kb = lo - term * p.term_blocks;
      int32_t issued = 0;
      for (; issued < count; ++issued) {
        const int stage = issued % S;
        if (!mbar_wait(smem_u32(&s.empty[stage]), ((issued / S) & 1) ^ 1, guard, p.status,
                       kSiteProducer))
          break;
        const uint32_t bar = smem_u32(&s.full[stage]);
        const uint32_t sb = smem_u32(s.in.b[stage]), sa = smem_u32(s.in.a[stage]);
        const int32_t x = kb * kMatmulBlock;
        const int32_t pa = term_a(term, p.terms), pb = term_b(term, p.terms);
        mbar_arrive_expect_tx(bar, kBBytes + kT * 128);
        // b in two boxes of 64 rows (or, stored transposed, 64 columns).
        const int32_t second = kGeglu ? p.up_row + col0 : col0 + 64;
        if (p.b_transposed) {
          tma_load_3d(sb, &tm_b, bar, col0, x, pb);
          tma_load_3d(sb + kBBytes / 2, &tm_b, bar, second, x, pb);
        } else {
          tma_load_3d(sb, &tm_b, bar, x, col0, pb);
          tma_load_3d(sb + kBBytes / 2, &tm_b, bar, x, second, pb);
        }
        if (p.a_transposed)
          tma_load_3d(sa, &tm_a, bar, row0, x, pa);
        else
          tma_load_3d(sa, &tm_a, bar, x, row0, pa);
        if (++kb == p.term_blocks) {
          kb = 0;
          ++term;
        }
      }
      // No load is in flight past this (all have been waited for unless a wait gave up).
      for (int32_t i = issued > S ? issued - S : 0; i < issued; ++i)
        mbar_drain_wait(smem_u32(&s.full[i % S]), (i / S) & 1);
    }
    __syncwarp();
  } else if (warp == 5) {
    // ------------------------------------------------------------ MMA issue
    const uint32_t step_a = p.a_transposed ? 128 : 2, step_b = p.b_transposed ? 128 : 2;
    bool ok = true;
    int32_t turn = -1, end = 0, buf = 0;
    for (int32_t i = 0; i < count; ++i) {
      const int stage = i % S;
      ok = warp_wait(smem_u32(&s.full[stage]), (i / S) & 1, guard, p.status, kSiteMma);
      if (!ok) break;
      const bool fresh = i == end;         // a chain begins
      if (fresh) {
        end = p.chains.end(lo + i, lo + count, kChunk) - lo;
        buf = ++turn & 1;
        ok = warp_wait(smem_u32(&s.acc_empty[buf]), ((turn >> 1) & 1) ^ 1, guard, p.status,
                       kSiteMma);
        if (!ok) break;
      }
      tc_fence_after();
      const uint64_t db =
          smem_desc_sw128(smem_u32(s.in.b[stage]), p.b_transposed ? 8192 : 16, 1024);
      const uint64_t da = smem_desc_sw128(smem_u32(s.in.a[stage]), 16, 1024);
#pragma unroll
      for (int k = 0; k < 4; ++k)          // 16 elements of k each
        mma_ss_warp(tmem + buf * kT, db + k * step_b, da + k * step_a, p.idesc,
                    !fresh || k > 0);
      tc_commit_warp(smem_u32(&s.empty[stage]));
      if (i == end - 1) tc_commit_warp(smem_u32(&s.acc_full[buf]));
    }
    tc_commit_warp(smem_u32(&s.drain));    // no MMA is in flight past this
    mbar_drain_wait(smem_u32(&s.drain), 0);
  } else if (warp < 4) {
    // ------------------------------------------------------------ sums
    float sum[kT];
#pragma unroll
    for (int c = 0; c < kT; ++c) sum[c] = 0.f;
    bool ok = true;
    int32_t turn = 0;
    for (int32_t block = lo; block < lo + count;
         block = p.chains.end(block, lo + count, kChunk), ++turn) {
      const int buf = turn & 1;
      const float weight = p.chains.weight(block);
      ok = warp_wait(smem_u32(&s.acc_full[buf]), (turn >> 1) & 1, guard, p.status,
                     kSiteEpilogue);
      if (!ok) break;
      tc_fence_after();
      const uint32_t src = tmem + ((uint32_t)(warp * 32) << 16) + buf * kT;
      auto hand_back = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s.acc_empty[buf]));
      };
      if constexpr (kT == 16) {
        uint32_t d[16];
        tmem_ld16(src, d);
        hand_back();
#pragma unroll
        for (int c = 0; c < 16; ++c) sum[c] = fmaf(__uint_as_float(d[c]), weight, sum[c]);
      } else {
#pragma unroll
        for (int h = 0; h < kT; h += 32) {
          uint32_t d[32];
          tmem_ld32(src + h, d);
          tmem_wait_ld(d);
          if (h + 32 == kT) hand_back();
#pragma unroll
          for (int c = 0; c < 32; ++c)
            sum[h + c] = fmaf(__uint_as_float(d[c]), weight, sum[h + c]);
        }
      }
    }
    // The stages may hold the sums now: the last commit says that every MMA has read its
    // operands, and every load has arrived.
    if (ok) {
#pragma unroll
      for (int c = 0; c < kT; ++c) s.sums[c][threadIdx.x] = sum[c];
    }
  }
  griddep_launch_dependents();             // the next kernel may come to wait for this one
  tc_fence_before();
  if (p.split == 1)
    __syncthreads();
  else
    cluster_sync();
  // ---------------------------------------------------------------- join and epilogue
  constexpr int kLanes = kOutCols / 4;                     // of a row
  constexpr int kRowsWarp = 32 / kLanes;                   // rows of a warp at a time
  constexpr int kFlight = 4;                               // of them in flight
  const int at = 4 * (lane % kLanes);
  const int32_t col = col0 + at;
  if (col < p.e.n) {
    const Finish4<kAct> finish(p.e, col);
    const int32_t rank = p.split == 1 ? 0 : (int32_t)cluster_rank();
    const int32_t rows = p.e.m - row0 < kT ? p.e.m - row0 : kT;
    const int32_t step = 8 * kRowsWarp * p.split;
    for (int32_t c0 = (rank * 8 + warp) * kRowsWarp + lane / kLanes; c0 < rows;
         c0 += kFlight * step) {
      float residual[kFlight][4];
      float4 z[kFlight], u[kFlight];
#pragma unroll
      for (int i = 0; i < kFlight; ++i) {
        const int32_t c = c0 + i * step;
        z[i] = u[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c < rows && p.e.residual) finish.residual(row0 + c, residual[i]);
      }
      // The cluster's parts in the order of k, those of all rows in flight.
#pragma unroll 2
      for (int32_t r = 0; r < p.split; ++r) {
        float4 v[kFlight], w[kFlight];
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
          const int32_t c = c0 + i * step;
          if (c < rows) {
            if (p.split == 1) {
              v[i] = *reinterpret_cast<const float4*>(&s.sums[c][at]);
              if constexpr (kGeglu) w[i] = *reinterpret_cast<const float4*>(&s.sums[c][64 + at]);
            } else {
              const uint32_t there = peer_address(smem_u32(&s.sums[c][at]), r);
              v[i] = load_cluster_f32x4(there);
              if constexpr (kGeglu) w[i] = load_cluster_f32x4(there + 256);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
          if (c0 + i * step < rows) {
            z[i].x += v[i].x;
            z[i].y += v[i].y;
            z[i].z += v[i].z;
            z[i].w += v[i].w;
            if constexpr (kGeglu) {
              u[i].x += w[i].x;
              u[i].y += w[i].y;
              u[i].z += w[i].z;
              u[i].w += w[i].w;
            }
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kFlight; ++i)
        if (c0 + i * step < rows) finish.row(row0 + c0 + i * step, z[i], u[i], residual[i]);
    }
  }
  if (p.split > 1) cluster_sync();         // the sums have been read by the whole cluster
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int kT, int kAct>
pe_status launch(const Matmul& q, int32_t split, DeviceStatus* status, cudaStream_t stream) {
  constexpr bool kGeglu = kAct == PE_ACT_GEGLU;
  CUtensorMap ma, mb;
  auto map = [&](CUtensorMap* to, const MatmulOperand& x, int32_t rows, uint32_t box) {
    const auto bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    return x.transposed ? matmul_map_planes(to, bf16, 2, x.base, q.k, rows, x.ld * 2, 64, q.planes)
                        : matmul_map_planes(to, bf16, 2, x.base, rows, q.k, x.ld * 2, box,
                                            q.planes);
  };
  PE_TRY(map(&ma, q.a, q.m, kT));
  PE_TRY(map(&mb, q.b, q.n, 64));
  Params p = {};
  p.e = q.e;
  p.term_blocks = (int32_t)ceil_div(q.k, kMatmulBlock);
  p.terms = q.planes == 3 ? kMaxMatmulTerms : 1;
  p.blocks = p.term_blocks * p.terms;
  p.chains = Chains::of(p.term_blocks, p.terms);
  p.split = split;
  p.a_transposed = q.a.transposed ? 1 : 0;
  p.b_transposed = q.b.transposed ? 1 : 0;
  p.up_row = kGeglu ? q.e.n : 0;
  p.idesc = idesc_bf16(128, kT, q.b.transposed, q.a.transposed);   // b is the first operand
  p.status = status;
  p.wait_limit_ns = wait_limit_ns();
  const size_t smem = sizeof(Smem<kT>) + 1024;
  static_assert(2 * (sizeof(Smem<kT>) + 2048) <= 227 * 1024, "two CTAs share an SM");
  const auto kernel = matmul_narrow_kernel<kT, kAct>;
  static std::atomic<uint64_t> done{0};
  PE_TRY(allow_shared_memory(kernel, static_cast<int>(smem), done));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(ceil_div(q.e.n, kGeglu ? 64 : 128) * split),
                     (unsigned)ceil_div(q.m, kT));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  PE_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, ma, mb, p));
  return PE_OK;
}

template <int kT>
pe_status launch_rows(const Matmul& q, int32_t split, DeviceStatus* status, cudaStream_t stream) {
  switch (q.e.act) {
    case PE_ACT_GEGLU: return launch<kT, PE_ACT_GEGLU>(q, split, status, stream);
    case PE_ACT_GELU: return launch<kT, PE_ACT_GELU>(q, split, status, stream);
    case PE_ACT_RELU: return launch<kT, PE_ACT_RELU>(q, split, status, stream);
    default: return launch<kT, PE_ACT_NONE>(q, split, status, stream);
  }
}

}  // namespace

pe_status matmul_narrow(const Matmul& p, int32_t rows, int32_t split, DeviceStatus* status,
                        cudaStream_t stream) {
  switch (rows) {
    case 16: return launch_rows<16>(p, split, status, stream);
    case 32: return launch_rows<32>(p, split, status, stream);
    default: return launch_rows<64>(p, split, status, stream);
  }
}

}  // namespace pe
