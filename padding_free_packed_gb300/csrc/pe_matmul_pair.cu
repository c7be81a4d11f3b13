// Matrix product of 8-bit operands with a scale for each block of 128, many
// rows: out[i, j] = sum over c of sa[c, i] sb[c, j / 128] (sum over block c of
// a[i, l] b[j, l]).
//
// A pair of CTAs (tcgen05 cta_group::2) works on a 256 x 256 tile: each CTA
// loads 128 rows of a and 128 rows of b, one 128-byte block of k at a time, and
// the pair's MMAs (M = 256, N = 256, K = 32) leave a 128 x 256 half of the
// block's product in each CTA's tensor memory. The scales change with every
// block of k, so a block's product cannot stay in the accumulator: eight
// epilogue warps read it from tensor memory and add it, scaled, to fp32 sums in
// registers (one thread: one row, 128 columns, so one scale a thread and block)
// while the MMAs of the next block fill the other half of tensor memory.
//
//   warp 0       TMA producer (both CTAs), a ring of kStages blocks
//   warp 1       MMA issue (first CTA of the pair)
//   warp 2       the blocks' scales, copied ahead into a ring in shared memory
//   warps 4-11   scaling and sums; warps 4-7 columns 0-127, 8-11 128-255
//
// Work: whole tiles in turn, or, where few tiles have long sums, equal runs of
// consecutive blocks of k (a run may start and end inside a tile); a tile that
// several pairs share is then summed from their fp32 parts, in the order of k,
// by a second kernel.
#include <cudaTypedefs.h>

#include "pe_matmul_fp8.cuh"
#include "pe_sm103.cuh"

namespace pe {

namespace {

using namespace sm103;

constexpr int kTile = 256;
constexpr int kRows = 128;                               // rows of a (and of b) per CTA
constexpr int kStages = 4;
constexpr int kScaleSlots = 8;                           // blocks of k whose scales are in flight
constexpr int kThreads = 384;
constexpr uint32_t kOperandBytes = kRows * kFp8Block;    // 16 KiB
constexpr uint32_t kPairBytes = 4 * kOperandBytes;       // both CTAs' a and b of one block
constexpr uint32_t kRegsLaunch = 168;
constexpr uint32_t kRegsLow = 56, kRegsHigh = 224;
static_assert(128 * (kRegsLow + 2 * kRegsHigh) <= kThreads * kRegsLaunch,
              "register split exceeds the launch allocation");
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kBoxBytes = 32 * 128;                 // 32 rows of 128 bytes, swizzled
constexpr int kMaxPairs = 80;
constexpr size_t kPartFloats = (size_t)kTile * kTile;

struct alignas(1024) Smem {
  uint8_t a[kStages][kOperandBytes];
  uint8_t b[kStages][kOperandBytes];
  alignas(1024) uint8_t out[8][2 * kBoxBytes];
  float a_scale[kScaleSlots][kRows];
  float b_scale[kScaleSlots][2];
  uint64_t full[kStages], empty[kStages];    // full: the first CTA's serve the pair
  uint64_t acc_full[2], acc_empty[2];        // acc_empty: likewise
  uint64_t scale_full[kScaleSlots], scale_empty[kScaleSlots];
  uint64_t drain;
  int32_t issued[2];                         // blocks each CTA's producer loaded (first CTA)
  int32_t aborted[2];
  uint32_t tmem_base;
  WaitGuard guard;
};
static_assert(sizeof(Smem) + 1024 <= 227 * 1024, "shared memory exceeds the per-CTA limit");

struct Params {
  const float* a_scales;
  const float* b_scales;
  int32_t m, n;
  int32_t blocks;            // of k
  int32_t col_tiles;
  int32_t tiles;
  int32_t shared_tiles;      // 1: runs of blocks, partial tiles through `parts`
  int32_t tma_store;         // out rows start at 16-byte multiples
  int32_t out_fp32;
  uint32_t idesc;
  void* out;
  float* parts;              // [2 * pairs][2 CTAs][64 column groups][128 rows] float4
  DeviceStatus* status;
  uint64_t wait_limit_ns;
};

enum WaitSite { kSiteProducer = 71, kSiteMma = 72, kSiteEpilogue = 73, kSiteScales = 74 };

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
// Address, in the cluster's shared window, of the same variable in CTA `rank`.
__device__ __forceinline__ uint32_t peer_address(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
__device__ __forceinline__ void store_cluster_i32(uint32_t addr, int32_t v) {
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr)
               : "memory");
}
__device__ __forceinline__ void mbar_complete_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
// Tile load into this CTA, counted on a barrier of the pair's first CTA.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                              int32_t x, int32_t y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void mma_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                         uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives once on this barrier in both CTAs when the MMAs issued so far complete.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}

// Four bytes to shared memory without a register on the way (zero unless `in`),
// and an arrival on `bar` when this thread's copies so far have landed.
__device__ __forceinline__ void copy_async4(uint32_t dst, const float* src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
               "r"(in ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void copy_async_wait_all() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// kind::f8f6f4, fp32 accumulator, both operands K-major.
constexpr uint32_t idesc_fp8(int M, int N, bool a_e5m2, bool b_e5m2) {
  return (1u << 4) | ((a_e5m2 ? 1u : 0u) << 7) | ((b_e5m2 ? 1u : 0u) << 10) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// First block of pair `p`'s run when `total` blocks are dealt to `pairs`.
__host__ __device__ __forceinline__ int64_t run_start(int64_t total, int32_t pairs, int32_t p) {
  return total / pairs * p + (total % pairs) * p / pairs;
}

// The blocks a pair works on, in order: (tile, block of k) pairs.
struct Walk {
  int32_t tile, block, last;      // last: one past the segment's last block
  int32_t stride;
  int64_t left;                   // blocks after this segment (runs), or tiles

  // The pair's first segment; false when it has none.
  __device__ bool start(const Params& p, int32_t pair, int32_t pairs) {
    if (p.shared_tiles) {
      const int64_t total = (int64_t)p.tiles * p.blocks;
      const int64_t lo = run_start(total, pairs, pair), hi = run_start(total, pairs, pair + 1);
      if (lo >= hi) return false;
      tile = (int32_t)(lo / p.blocks);
      block = (int32_t)(lo - (int64_t)tile * p.blocks);
      const int64_t room = hi - lo;
      last = room < p.blocks - block ? block + (int32_t)room : p.blocks;
      left = room - (last - block);
      return true;
    }
    stride = pairs;
    tile = pair;
    block = 0;
    last = p.blocks;
    return tile < p.tiles;
  }
  // Moves to the next block; false at the end of the work.
  __device__ bool next(const Params& p) {
    if (++block < last) return true;
    if (p.shared_tiles) {
      if (left <= 0) return false;
      ++tile;
      block = 0;
      last = left < p.blocks ? (int32_t)left : p.blocks;
      left -= last;
      return true;
    }
    tile += stride;
    block = 0;
    return tile < p.tiles;
  }
};

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
matmul_pair_kernel(const __grid_constant__ CUtensorMap tm_a,
                   const __grid_constant__ CUtensorMap tm_b,
                   const __grid_constant__ CUtensorMap tm_out, const Params p) {
  extern __shared__ uint8_t raw[];
  Smem& s = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int32_t pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  volatile WaitGuard* guard = &s.guard;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&s.full[i]), 1);
      mbar_init(smem_u32(&s.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s.acc_full[i]), 1);
      mbar_init(smem_u32(&s.acc_empty[i]), 16);
    }
    for (int i = 0; i < kScaleSlots; ++i) {
      mbar_init(smem_u32(&s.scale_full[i]), 32);
      mbar_init(smem_u32(&s.scale_empty[i]), 8);
    }
    mbar_init(smem_u32(&s.drain), 1);
    s.guard.abort = 0;
    s.guard.limit_ns = p.wait_limit_ns;
    fence_mbarrier_init();
    prefetch_tensormap(&tm_a);
    prefetch_tensormap(&tm_b);
    prefetch_tensormap(&tm_out);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&s.tmem_base)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();                          // barriers of both CTAs exist before any arrival
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;

  if (warp < 4) {
    regs_release<kRegsLow>();
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------------- producer
      int32_t issued = 0;
      Walk w;
      for (bool more = w.start(p, pair, pairs); more; more = w.next(p)) {
        const int stage = issued % kStages;
        const uint32_t turn = issued / kStages;
        if (!mbar_wait(smem_u32(&s.empty[stage]), (turn & 1) ^ 1, guard, p.status, kSiteProducer))
          break;
        const int32_t rt = w.tile / p.col_tiles, ct = w.tile - rt * p.col_tiles;
        const uint32_t bar = peer_address(smem_u32(&s.full[stage]), 0);
        if (rank == 0) mbar_arrive_expect_tx(smem_u32(&s.full[stage]), kPairBytes);
        tma_load_pair(smem_u32(s.a[stage]), &tm_a, bar, w.block * kFp8Block,
                      rt * kTile + (int32_t)rank * kRows);
        tma_load_pair(smem_u32(s.b[stage]), &tm_b, bar, w.block * kFp8Block,
                      ct * kTile + (int32_t)rank * kRows);
        ++issued;
      }
      store_cluster_i32(peer_address(smem_u32(&s.issued[rank]), 0), issued);
    } else if (warp == 1 && lane == 0 && rank == 0) {
      // ---------------------------------------------------------- MMA issue
      int32_t done = 0;
      Walk w;
      for (bool more = w.start(p, pair, pairs); more; more = w.next(p)) {
        const int stage = done % kStages, buf = done & 1;
        if (!mbar_wait(smem_u32(&s.acc_empty[buf]), ((done >> 1) & 1) ^ 1, guard, p.status,
                       kSiteMma))
          break;
        if (!mbar_wait(smem_u32(&s.full[stage]), (done / kStages) & 1, guard, p.status, kSiteMma))
          break;
        tc_fence_after();
        const uint64_t da = smem_desc_sw128(smem_u32(s.a[stage]), 16, 1024);
        const uint64_t db = smem_desc_sw128(smem_u32(s.b[stage]), 16, 1024);
#pragma unroll
        for (int i = 0; i < 4; ++i)        // 32 bytes of k each: 2 units of 16 bytes
          mma_pair(tmem + buf * kTile, da + 2 * i, db + 2 * i, p.idesc, i > 0);
        commit_pair(smem_u32(&s.empty[stage]));
        commit_pair(smem_u32(&s.acc_full[buf]));
        ++done;
      }
      if (s.guard.abort) {                 // let the MMAs in flight finish
        commit_pair(smem_u32(&s.drain));
        mbar_drain_wait(smem_u32(&s.drain), 0);
      }
    } else if (warp == 2) {
      // ---------------------------------------------------------- scales
      const int32_t col_blocks = (p.n + kFp8Block - 1) / kFp8Block;
      int32_t done = 0;
      Walk w;
      for (bool more = w.start(p, pair, pairs); more; more = w.next(p)) {
        const int slot = done % kScaleSlots;
        if (!warp_wait(smem_u32(&s.scale_empty[slot]), ((done / kScaleSlots) & 1) ^ 1, guard,
                       p.status, kSiteScales))
          break;
        const int32_t rt = w.tile / p.col_tiles, ct = w.tile - rt * p.col_tiles;
        const int32_t row0 = rt * kTile + (int32_t)rank * kRows;
        const float* src = p.a_scales + (int64_t)w.block * p.m;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int32_t row = row0 + i * 32 + lane;
          copy_async4(smem_u32(&s.a_scale[slot][i * 32 + lane]), src + (row < p.m ? row : 0),
                      row < p.m);
        }
        if (lane < 2) {
          const int32_t cb = ct * 2 + lane;
          copy_async4(smem_u32(&s.b_scale[slot][lane]),
                      p.b_scales + (int64_t)w.block * col_blocks + (cb < col_blocks ? cb : 0),
                      cb < col_blocks);
        }
        copy_async_arrive(smem_u32(&s.scale_full[slot]));
        ++done;
      }
      copy_async_wait_all();
    }
    __syncwarp();
  } else {
    regs_claim<kRegsHigh>();
    // ------------------------------------------------------------ scaling and sums
    const int quad = warp & 3, half = (warp - 4) >> 2;
    const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16) + half * 128;
    const int32_t row_in = (int32_t)rank * kRows + quad * 32;   // this warp's rows in the tile
    uint8_t* stage_out = s.out[warp - 4];
    const uint32_t empty0 = peer_address(smem_u32(&s.acc_empty[0]), 0);
    const uint32_t empty1 = peer_address(smem_u32(&s.acc_empty[1]), 0);

    uint64_t acc[64];
#pragma unroll
    for (int i = 0; i < 64; ++i) acc[i] = 0ull;
    int32_t done = 0;
    Walk w;
    int32_t first_block = 0;
    bool more = w.start(p, pair, pairs);
    bool begins = true;                    // the segment is the pair's first
    if (more) first_block = w.block;
    while (more) {
      const int buf = done & 1;
      const int slot = done % kScaleSlots;
      if (!warp_wait(smem_u32(&s.scale_full[slot]), (done / kScaleSlots) & 1, guard, p.status,
                     kSiteEpilogue))
        break;
      const float scale = s.a_scale[slot][quad * 32 + lane] * s.b_scale[slot][half];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&s.scale_empty[slot]));
      if (!warp_wait(smem_u32(&s.acc_full[buf]), (done >> 1) & 1, guard, p.status, kSiteEpilogue))
        break;
      tc_fence_after();
      const uint64_t scale2 = f2(scale, scale);
      uint32_t d[2][32];
      tmem_ld32(lane_base + buf * kTile, d[0]);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        tmem_wait_ld(d[c & 1]);
        if (c < 3) {
          tmem_ld32(lane_base + buf * kTile + 32 * (c + 1), d[(c + 1) & 1]);
        } else {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(buf ? empty1 : empty0);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i)
          acc[c * 16 + i] = ffma2(f2(__uint_as_float(d[c & 1][2 * i]),
                                     __uint_as_float(d[c & 1][2 * i + 1])),
                                  scale2, acc[c * 16 + i]);
      }
      ++done;
      const int32_t tile = w.tile, block = w.block;
      const bool ends = block + 1 == w.last;
      more = w.next(p);
      if (!ends) continue;

      // The segment's sums: a whole tile goes to out, a part to the workspace.
      const int32_t rt = tile / p.col_tiles, ct = tile - rt * p.col_tiles;
      const int32_t row0 = rt * kTile + row_in, col0 = ct * kTile + half * 128;
      if (first_block != 0 || block + 1 != p.blocks) {
        const int32_t slot = 2 * pair + (begins ? 0 : 1);
        float4* part = reinterpret_cast<float4*>(p.parts + slot * kPartFloats) +
                       (rank * 64 + half * 32) * 128 + quad * 32 + lane;
#pragma unroll
        for (int g = 0; g < 32; ++g) {
          float4 v;
          f2_split(acc[2 * g], v.x, v.y);
          f2_split(acc[2 * g + 1], v.z, v.w);
          part[g * 128] = v;
        }
      } else if (row0 < p.m && col0 < p.n) {
        if (p.tma_store) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {    // 64 columns: one bf16 box or two fp32 boxes
            if (lane == 0 && (h == 0 || p.out_fp32)) bulk_wait_read();
            __syncwarp();
#pragma unroll
            for (int g = 0; g < 16; ++g) { // 4 columns
              float x0, x1, x2, x3;
              f2_split(acc[h * 32 + 2 * g], x0, x1);
              f2_split(acc[h * 32 + 2 * g + 1], x2, x3);
              if (p.out_fp32) {
                *reinterpret_cast<float4*>(stage_out + (g >> 3) * kBoxBytes + lane * 128 +
                                           (((g & 7) ^ (lane & 7)) << 4)) =
                    make_float4(x0, x1, x2, x3);
              } else {
                *reinterpret_cast<uint2*>(stage_out + h * kBoxBytes + lane * 128 +
                                          (((g >> 1) ^ (lane & 7)) << 4) + (g & 1) * 8) =
                    make_uint2(pack_bf16x2(x0, x1), pack_bf16x2(x2, x3));
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              if (p.out_fp32) {
                for (int b = 0; b < 2; ++b)
                  if (col0 + h * 64 + b * 32 < p.n)
                    tma_store_2d(&tm_out, smem_u32(stage_out + b * kBoxBytes),
                                 col0 + h * 64 + b * 32, row0);
              } else if (col0 + h * 64 < p.n) {
                tma_store_2d(&tm_out, smem_u32(stage_out + h * kBoxBytes), col0 + h * 64, row0);
              }
              bulk_commit();
            }
          }
        } else {
          // Rows that start anywhere: 64 columns at a time through the stage, then
          // a row at a time in runs of 32 columns.
          const int32_t rows = p.m - row0 < 32 ? p.m - row0 : 32;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            __syncwarp();
#pragma unroll
            for (int g = 0; g < 16; ++g) {
              float4 v;
              f2_split(acc[h * 32 + 2 * g], v.x, v.y);
              f2_split(acc[h * 32 + 2 * g + 1], v.z, v.w);
              *reinterpret_cast<float4*>(stage_out + (g >> 3) * kBoxBytes + lane * 128 +
                                         (((g & 7) ^ (lane & 7)) << 4)) = v;
            }
            __syncwarp();
            for (int32_t r = 0; r < rows; ++r) {
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                const int32_t col = col0 + h * 64 + b * 32 + lane;
                const float v = *reinterpret_cast<const float*>(
                    stage_out + b * kBoxBytes + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) +
                    (lane & 3) * 4);
                if (col < p.n) {
                  const int64_t at = (int64_t)(row0 + r) * p.n + col;
                  if (p.out_fp32)
                    static_cast<float*>(p.out)[at] = v;
                  else
                    static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(v);
                }
              }
            }
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = 0ull;
      begins = false;
      if (more) first_block = w.block;
    }
    bulk_wait_all();
  }

  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) store_cluster_i32(peer_address(smem_u32(&s.aborted[rank]), 0),
                                          s.guard.abort);
  __syncthreads();
  cluster_sync();
  if (rank == 0 && threadIdx.x == 0 && (s.aborted[0] || s.aborted[1])) {
    // Both producers have stopped. Blocks that only one CTA loaded are put right
    // on their barrier, then every load that may be in flight is waited for.
    const int32_t n0 = s.issued[0], n1 = s.issued[1];
    const int32_t both = n0 < n1 ? n0 : n1, any = n0 < n1 ? n1 : n0;
    for (int32_t i = both; i < any; ++i) {
      const uint32_t bar = smem_u32(&s.full[i % kStages]);
      if (n0 > n1)
        mbar_complete_tx(bar, kPairBytes / 2);
      else
        mbar_arrive_expect_tx(bar, kPairBytes / 2);
    }
    for (int32_t i = any > kStages ? any - kStages : 0; i < any; ++i)
      mbar_drain_wait(smem_u32(&s.full[i % kStages]), (i / kStages) & 1);
  }
  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTmemCols)
                 : "memory");
  }
}

// Sums the parts of every tile that several pairs share, in the order of k. One
// block per 32 x 128 piece of a tile; parts are column-group-major.
__global__ void __launch_bounds__(256)
matmul_parts_kernel(const Params p, int32_t pairs) {
  __shared__ float tile[32][129];
  const int piece = blockIdx.x & 15;                     // 2 CTAs x 4 row quarters x 2 halves
  const int32_t t = blockIdx.x >> 4;
  const int rank = piece >> 3, quad = (piece >> 1) & 3, half = piece & 1;
  const int32_t rt = t / p.col_tiles, ct = t - rt * p.col_tiles;
  const int32_t row0 = rt * kTile + rank * kRows + quad * 32, col0 = ct * kTile + half * 128;
  const int64_t total = (int64_t)p.tiles * p.blocks;
  const int64_t lo = (int64_t)t * p.blocks, hi = lo + p.blocks;
  // The pair that holds block `lo`: run_start(q) <= lo < run_start(q + 1).
  int32_t q = (int32_t)(lo / (total / pairs + 1));
  while (q + 1 < pairs && run_start(total, pairs, q + 1) <= lo) ++q;
  if (run_start(total, pairs, q + 1) >= hi) return;      // one pair wrote the whole tile
  if (row0 >= p.m || col0 >= p.n) return;
  const int row = threadIdx.x & 31, g0 = threadIdx.x >> 5;
  griddep_wait();
  float4 sum[4] = {};
  for (; q < pairs; ++q) {
    const int64_t start = run_start(total, pairs, q);
    if (start >= hi) break;
    if (start == run_start(total, pairs, q + 1)) continue;
    const int32_t slot = 2 * q + (start >= lo ? 0 : 1);
    const float4* part = reinterpret_cast<const float4*>(p.parts + slot * kPartFloats) +
                         (rank * 64 + half * 32) * 128 + quad * 32 + row;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = part[(g0 + 8 * i) * 128];
      sum[i].x += v.x;
      sum[i].y += v.y;
      sum[i].z += v.z;
      sum[i].w += v.w;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = 4 * (g0 + 8 * i);
    tile[row][c] = sum[i].x;
    tile[row][c + 1] = sum[i].y;
    tile[row][c + 2] = sum[i].z;
    tile[row][c + 3] = sum[i].w;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < 32 * 128; e += 256) {
    const int r = e >> 7, c = e & 127;
    if (row0 + r < p.m && col0 + c < p.n) {
      const int64_t at = (int64_t)(row0 + r) * p.n + col0 + c;
      if (p.out_fp32)
        static_cast<float*>(p.out)[at] = tile[r][c];
      else
        static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(tile[r][c]);
    }
  }
}

// ---------------------------------------------------------------- host side
PFN_cuTensorMapEncodeTiled_v12000 g_encode_matmul = nullptr;

pe_status get_encoder_matmul() {
  if (g_encode_matmul) return PE_OK;
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult qres;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                       &qres) != cudaSuccess ||
      qres != cudaDriverEntryPointSuccess || !fn)
    return PE_ERR_CUDA;
  g_encode_matmul = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  return PE_OK;
}

// Row-major [rows, cols] of `type`, rows `pitch` bytes apart, boxes of box_rows
// rows of 128 bytes, 128-byte swizzle.
pe_status make_map(CUtensorMap* map, CUtensorMapDataType type, int size, const void* base,
                   int64_t rows, int64_t cols, int64_t pitch, uint32_t box_rows) {
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch)};
  cuuint32_t box[2] = {128u / size, box_rows};
  cuuint32_t elem_strides[2] = {1, 1};
  CUresult r = g_encode_matmul(map, type, 2, const_cast<void*>(base), dims, strides, box,
                               elem_strides, CU_TENSOR_MAP_INTERLEAVE_NONE,
                               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? PE_OK : PE_ERR_CUDA;
}

int32_t pair_count() {
  const int32_t n = device_sm_count() / 2;
  return n < kMaxPairs ? n : kMaxPairs;
}

// Runs of blocks instead of whole tiles: when the busiest pair then saves more
// blocks than the parts and the second kernel cost.
bool use_runs(int64_t tiles, int64_t blocks, int64_t pairs) {
  const int64_t whole = ceil_div(tiles, pairs) * blocks;
  return whole - ceil_div(tiles * blocks, pairs) > 24;
}

}  // namespace

size_t matmul_pair_workspace(int64_t m, int64_t n, int64_t k) {
  // The size must not depend on the device at hand: parts for the most pairs any
  // device runs whenever some number of pairs would use runs.
  const int64_t tiles = ceil_div(m, kTile) * ceil_div(n, kTile), blocks = ceil_div(k, kFp8Block);
  for (int64_t pairs = 1; pairs <= kMaxPairs; ++pairs)
    if (use_runs(tiles, blocks, pairs)) return 2 * kMaxPairs * kPartFloats * sizeof(float);
  return 0;
}

pe_status matmul_pair(const MatmulFp8& q, void* workspace, DeviceStatus* status,
                      cudaStream_t stream) {
  PE_TRY(get_encoder_matmul());
  CUtensorMap ma, mb, mo;
  PE_TRY(make_map(&ma, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, q.a, q.m, q.k, q.a_ld, kRows));
  PE_TRY(make_map(&mb, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, q.b, q.n, q.k, q.b_ld, kRows));
  const int size = q.out_fp32 ? 4 : 2;
  const bool tma_store = aligned(q.out, 16) && (int64_t)q.n * size % 16 == 0;
  mo = ma;
  if (tma_store)
    PE_TRY(make_map(&mo, q.out_fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                    : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                    size, q.out, q.m, q.n, (int64_t)q.n * size, 32));
  const size_t smem = sizeof(Smem) + 1024;
  PE_CUDA_TRY(cudaFuncSetAttribute(matmul_pair_kernel,
                                   cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   static_cast<int>(smem)));
  cudaFuncAttributes attr;
  PE_CUDA_TRY(cudaFuncGetAttributes(&attr, matmul_pair_kernel));
  if (static_cast<uint32_t>(attr.numRegs) * kThreads < 128u * (kRegsLow + 2 * kRegsHigh))
    return PE_ERR_UNSUPPORTED;
  Params p;
  p.a_scales = q.a_scales;
  p.b_scales = q.b_scales;
  p.m = q.m;
  p.n = q.n;
  p.blocks = (int32_t)ceil_div(q.k, kFp8Block);
  p.col_tiles = (int32_t)ceil_div(q.n, kTile);
  const int64_t tiles = ceil_div(q.m, kTile) * p.col_tiles;
  if (tiles >= (1LL << 27)) return PE_ERR_OVERFLOW;
  p.tiles = (int32_t)tiles;
  int32_t pairs = pair_count();
  p.shared_tiles = use_runs(tiles, p.blocks, pairs) ? 1 : 0;
  if (!p.shared_tiles && tiles < pairs) pairs = (int32_t)tiles;
  p.tma_store = tma_store ? 1 : 0;
  p.out_fp32 = q.out_fp32 ? 1 : 0;
  p.idesc = idesc_fp8(256, kTile, q.a_e5m2, q.b_e5m2);
  p.out = q.out;
  p.parts = static_cast<float*>(workspace);
  p.status = status;
  p.wait_limit_ns = wait_limit_ns();
  matmul_pair_kernel<<<2 * pairs, kThreads, smem, stream>>>(ma, mb, mo, p);
  PE_CUDA_TRY(cudaGetLastError());
  if (p.shared_tiles)
    return launch_after_previous(matmul_parts_kernel, dim3((unsigned)(16 * tiles)), dim3(256), 0,
                                 stream, p, pairs);
  return PE_OK;
}

}  // namespace pe
