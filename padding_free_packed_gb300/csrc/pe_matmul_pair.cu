// Matrix product of 8-bit operands with a scale for each block of 128, many
// rows: out[i, j] = sum over c of sa[c, i] sb[c, j / 128] (sum over block c of
// a[i, l] b[j, l]).
//
// A pair of CTAs (tcgen05 cta_group::2) works on a 256 x 256 tile: each CTA
// loads 128 rows of a and 128 rows of b, one 128-byte block of k at a time, and
// the pair's MMAs (M = 256, N = 128, K = 32) leave two 128 x 128 products of the
// block in each CTA's tensor memory, one for each 128 columns. The scales change
// with every block of k, so a block's product cannot stay in the accumulator:
// eight epilogue warps read it from tensor memory and add it, scaled, to fp32
// sums in registers (one thread: one row, 128 columns, so one scale a thread and
// block) while the MMAs of the next block fill the other half of tensor memory.
//
//   warp 0       TMA producer (both CTAs), a ring of kStages blocks
//   warps 1, 2   MMA issue for columns 0-127 and 128-255 (first CTA of the pair)
//   warp 3       the blocks' scales, copied ahead into a ring in shared memory
//   warps 4-11   scaling and sums; warps 4-7 columns 0-127, 8-11 128-255
//
// The two column halves are separate pipelines (accumulators, barriers, issuing
// warp) so that a half's tensor memory is handed back as soon as its four warps
// in both CTAs have read it: the way back through the other CTA is long, and four
// small accumulators in flight cover it better than two large ones.
//
// Work: whole tiles in turn, or, where few tiles have long sums, equal runs of
// consecutive blocks of k (a run may start and end inside a tile); a tile that
// several pairs share is then summed from their fp32 parts, in the order of k,
// by a second kernel.
//
// Measured (GB300, device time of a burst): 169151 x 1024 x 1024 to bf16 in 155 us (2.29
// PFLOP/s, 1.20 of the measured dense bf16 rate; the floor at twice that rate is
// 93 us; 169 us for seconds on end, when the power cap holds the clock at 1.85 GHz),
// 32299 x 2304 x 768 in 57 us, 2304 x 768 x 32299 to fp32 in 62 us. A block's MMAs take
// 517 of the 900 cycles between blocks, in two halves of N = 128 as in one of 256. The
// epilogue's part in the first: 142 us without its multiply-adds, 134 without the
// stores, 109 with neither; what is left then is the chain of hand-overs (MMAs,
// commit, read, arrival from the other CTA some 250 cycles away, next MMAs) over the
// two accumulators of a half. Tried and slower there: sixteen epilogue warps of 64
// columns 189 us; one N = 256 accumulator a block 163 us; 256 x 128 tiles with four
// accumulators 190 us; rows of out straight from registers in 32-byte pieces 230 us
// (187 us through boxes then). Asking for the next block's barrier and scales before
// the last sums changed nothing (155 us).
#include "pe_matmul_fp8.cuh"

namespace pe {

namespace {

using namespace sm103;

constexpr int kTile = 256;
constexpr int kRows = 128;                               // rows of a (and of b) per CTA
constexpr int kStages = 4;
constexpr int kIssueWarps = 2;
constexpr int kScaleAhead = 8;                           // blocks of k that scales are copied ahead
constexpr int kScaleSlots = 16;
constexpr int kThreads = 384;
constexpr uint32_t kOperandBytes = kRows * kFp8Block;    // 16 KiB
constexpr uint32_t kPairBytes = 4 * kOperandBytes;       // both CTAs' a and b of one block
constexpr uint32_t kRegsLaunch = 168;
constexpr uint32_t kRegsLow = 40, kRegsHigh = 232;
static_assert(128 * (kRegsLow + 2 * kRegsHigh) <= kThreads * kRegsLaunch,
              "register split exceeds the launch allocation");
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kBoxBytes = 32 * 128;                 // 32 rows of 128 bytes
constexpr int kMaxPairs = 80;
constexpr size_t kPartFloats = (size_t)kTile * kTile;

struct alignas(1024) Smem {
  uint8_t a[kStages][kOperandBytes];
  uint8_t b[kStages][kOperandBytes];
  alignas(1024) uint8_t out[8][2 * kBoxBytes];
  float a_scale[kScaleSlots][kRows];
  float b_scale[kScaleSlots][2];
  uint64_t full[kStages], empty[kStages];    // full: the first CTA's serve the pair
  uint64_t acc_full[2][2], acc_empty[2][2];  // [column half][buffer]; acc_empty: likewise.
                                             // acc_full counts the MMAs and the scales
  uint64_t drain[kIssueWarps];
  int32_t issued[2];                         // blocks each CTA's producer loaded (first CTA)
  int32_t aborted[2];
  uint32_t tmem_base;
  WaitGuard guard;
};
static_assert(kScaleSlots >= kScaleAhead + 5, "a slot is reused only after its last reader");
static_assert(sizeof(Smem) + 1024 <= 227 * 1024, "shared memory exceeds the per-CTA limit");

struct Params {
  const float* a_scales;
  const float* b_scales;
  int32_t m, n;
  int32_t blocks;            // of k
  int32_t col_tiles;
  int32_t tiles;
  int32_t shared_tiles;      // 1: runs of blocks, partial tiles through `parts`
  int32_t run_blocks;        // blocks of every pair's run, and
  int32_t run_more;          // how many pairs get one more
  int32_t out_fp32;
  uint32_t idesc;
  void* out;
  float* parts;              // [2 * pairs][2 CTAs][64 column groups][128 rows] float4
  DeviceStatus* status;
  uint64_t wait_limit_ns;
};

enum WaitSite { kSiteProducer = 71, kSiteMma = 72, kSiteEpilogue = 73, kSiteScales = 74 };

__device__ __forceinline__ void store_cluster_i32(uint32_t addr, int32_t v) {
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
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
// Both are executed by a whole warp with the same operands; one lane issues.
__device__ __forceinline__ void mma_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                         uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b32 r;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "elect.sync r|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives once on this barrier in both CTAs when the MMAs issued so far complete.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b32 r;\n\telect.sync r|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;\n\t}" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}

// First block of pair `q`'s run: the blocks are dealt evenly, the first pairs get one
// more each.
__device__ __forceinline__ int32_t run_start(const Params& p, int32_t q) {
  return p.run_blocks * q + (q < p.run_more ? q : p.run_more);
}

// The work of a pair as segments (a tile and a run of its blocks of k), in order.
struct Walk {
  int32_t tile, first, last;      // last: one past the segment's last block
  int32_t stride;
  int32_t left;                   // blocks after this segment (shared tiles)

  // The pair's first segment; false when it has none.
  __device__ bool start(const Params& p, int32_t pair, int32_t pairs) {
    if (p.shared_tiles) {
      const int32_t lo = run_start(p, pair), hi = run_start(p, pair + 1);
      if (lo >= hi) return false;
      tile = lo / p.blocks;
      first = lo - tile * p.blocks;
      const int32_t room = hi - lo;
      last = room < p.blocks - first ? first + room : p.blocks;
      left = room - (last - first);
      return true;
    }
    stride = pairs;
    tile = pair;
    first = 0;
    last = p.blocks;
    return tile < p.tiles;
  }
  __device__ bool next(const Params& p) {
    first = 0;
    if (p.shared_tiles) {
      if (left <= 0) return false;
      ++tile;
      last = left < p.blocks ? left : p.blocks;
      left -= last;
      return true;
    }
    tile += stride;
    return tile < p.tiles;
  }
};

// Blocks of all of the pair's segments.
__device__ __forceinline__ int32_t pair_blocks(const Params& p, int32_t pair, int32_t pairs) {
  if (p.shared_tiles) return run_start(p, pair + 1) - run_start(p, pair);
  return pair < p.tiles ? ((p.tiles - 1 - pair) / pairs + 1) * p.blocks : 0;
}

// The registers of the epilogue's inner loop have names of their own (four groups of
// 32 sums, two of 32 loaded columns): loads of the next columns are then in flight
// while the columns before them are added, without a copy of either. The same loop
// on C++ variables took a move for every second column, and paired fp32 arithmetic
// (two columns an instruction, at half the rate) one for almost every column.
#define PE_DECLARE_SUMS()                                                                   \
  asm volatile(                                                                             \
      ".reg .b32 pe_s0_<32>, pe_s1_<32>, pe_s2_<32>, pe_s3_<32>, pe_d0_<32>, pe_d1_<32>;")
#define PE_EACH32(OP, q, h)                                                                  \
  OP(q, h, 0) OP(q, h, 1) OP(q, h, 2) OP(q, h, 3) OP(q, h, 4) OP(q, h, 5) OP(q, h, 6)        \
  OP(q, h, 7) OP(q, h, 8) OP(q, h, 9) OP(q, h, 10) OP(q, h, 11) OP(q, h, 12) OP(q, h, 13)    \
  OP(q, h, 14) OP(q, h, 15) OP(q, h, 16) OP(q, h, 17) OP(q, h, 18) OP(q, h, 19) OP(q, h, 20) \
  OP(q, h, 21) OP(q, h, 22) OP(q, h, 23) OP(q, h, 24) OP(q, h, 25) OP(q, h, 26)              \
  OP(q, h, 27) OP(q, h, 28) OP(q, h, 29) OP(q, h, 30) OP(q, h, 31)
#define PE_FMA(q, h, i) "fma.rn.f32 pe_s" #q "_" #i ", pe_d" #h "_" #i ", f, pe_s" #q "_" #i ";\n\t"
#define PE_D8(h, a, b, c, d, e, f, g, i)                                                    \
  "pe_d" #h "_" #a ", pe_d" #h "_" #b ", pe_d" #h "_" #c ", pe_d" #h "_" #d ", pe_d" #h "_" #e \
  ", pe_d" #h "_" #f ", pe_d" #h "_" #g ", pe_d" #h "_" #i
// 32 columns of this thread's lane, from column `off` on, into group h.
#define PE_LOAD(h, off)                                                                   \
  "add.u32 a, %2, " #off ";\n\ttcgen05.ld.sync.aligned.32x32b.x32.b32 {" PE_D8(            \
      h, 0, 1, 2, 3, 4, 5, 6, 7) ", " PE_D8(h, 8, 9, 10, 11, 12, 13, 14, 15) ", " PE_D8(    \
      h, 16, 17, 18, 19, 20, 21, 22, 23) ", " PE_D8(h, 24, 25, 26, 27, 28, 29, 30, 31)      \
      "}, [a];\n\t"
#define PE_WAIT_LOADS "tcgen05.wait::ld.sync.aligned;\n\t"
// One block of k: the 128 columns at tensor-memory address `src`, scaled, added to
// the sums. The accumulator is handed back as soon as it has been read, by the lane
// with `first` set, on the barrier `back` of the pair's first CTA. Where the scale of
// some lane is not a normal number (the two scales' product may have left the range of
// fp32), such lanes add zero times the block, the accumulator is kept, and the return
// value asks for add_far (zero and infinite scales come that way too). Looked at while
// the loads are in flight, which costs nothing: 169151 x 1024 x 1024 153 us with and
// without (171 with multiply-adds that such lanes skip).
__device__ __forceinline__ uint32_t add_block(float scale, uint32_t src, uint32_t back,
                                              uint32_t first) {
  uint32_t far;
  asm volatile("{\n\t.reg .b32 a;\n\t.reg .f32 f;\n\t.reg .pred p, q;\n\t"
                   PE_LOAD(0, 0) PE_LOAD(1, 32)
               "abs.f32 f, %1;\n\tsetp.lt.f32 p, f, 0f00800000;\n\t"
               "setp.gt.or.f32 p, f, 0f7F7FFFFF, p;\n\tselp.f32 f, 0f00000000, %1, p;\n\t"
               "vote.sync.any.pred p, p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t"
                   PE_WAIT_LOADS PE_EACH32(PE_FMA, 0, 0) PE_LOAD(0, 64) PE_EACH32(PE_FMA, 1, 1)
                       PE_LOAD(1, 96) PE_WAIT_LOADS
               "tcgen05.fence::before_thread_sync;\n\tbar.warp.sync 0xffffffff;\n\t"
               "setp.ne.and.b32 q, %4, 0, !p;\n\t"
               "@q mbarrier.arrive.shared::cluster.b64 _, [%3];\n\t"
               PE_EACH32(PE_FMA, 2, 0) PE_EACH32(PE_FMA, 3, 1) "}" : "=r"(far) : "f"(scale),
               "r"(src), "r"(back), "r"(first)
               : "memory");
  return far;
}
#define PE_ZERO(q, h, i) "mov.b32 pe_s" #q "_" #i ", 0;\n\t"
__device__ __forceinline__ void clear_sums() {
  asm volatile(PE_EACH32(PE_ZERO, 0, 0) PE_EACH32(PE_ZERO, 1, 0) PE_EACH32(PE_ZERO, 2, 0)
                   PE_EACH32(PE_ZERO, 3, 0)::
                       : "memory");
}
#define PE_GET8(q, i0, i1, i2, i3, i4, i5, i6, i7)                                         \
  asm volatile("mov.b32 %0, pe_s" #q "_" #i0 ";\n\tmov.b32 %1, pe_s" #q "_" #i1              \
               ";\n\tmov.b32 %2, pe_s" #q "_" #i2 ";\n\tmov.b32 %3, pe_s" #q "_" #i3          \
               ";\n\tmov.b32 %4, pe_s" #q "_" #i4 ";\n\tmov.b32 %5, pe_s" #q "_" #i5          \
               ";\n\tmov.b32 %6, pe_s" #q "_" #i6 ";\n\tmov.b32 %7, pe_s" #q "_" #i7 ";"      \
               : "=f"(x[i0]), "=f"(x[i1]), "=f"(x[i2]), "=f"(x[i3]), "=f"(x[i4]),           \
                 "=f"(x[i5]), "=f"(x[i6]), "=f"(x[i7]))
#define PE_GET32(q)                             \
  PE_GET8(q, 0, 1, 2, 3, 4, 5, 6, 7);           \
  PE_GET8(q, 8, 9, 10, 11, 12, 13, 14, 15);     \
  PE_GET8(q, 16, 17, 18, 19, 20, 21, 22, 23);   \
  PE_GET8(q, 24, 25, 26, 27, 28, 29, 30, 31)
// The sums of columns 32 q .. 32 q + 31.
template <int q>
__device__ __forceinline__ void get_sums(float (&x)[32]) {
  if constexpr (q == 0) {
    PE_GET32(0);
  } else if constexpr (q == 1) {
    PE_GET32(1);
  } else if constexpr (q == 2) {
    PE_GET32(2);
  } else {
    PE_GET32(3);
  }
}

__device__ __forceinline__ float load_shared(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// The lanes that add_block left out: their products with the factors of far_factors are
// summed in memory, so that this rare path leaves the registers of the block loop alone
// (as a second form of add_block it made that loop a tenth slower).
__device__ __forceinline__ void add_far(float (&far)[kRows], bool begun, bool left_out, float2 f,
                                        uint32_t src) {
#pragma unroll 1
  for (int c = 0; c < kRows; c += 8) {
    uint32_t d[8];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3]), "=r"(d[4]), "=r"(d[5]), "=r"(d[6]),
          "=r"(d[7])
        : "r"(src + c)
        : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float before = begun ? far[c + i] : 0.f;
      far[c + i] = left_out ? fmaf(__uint_as_float(d[i]) * f.x, f.y, before) : before;
    }
  }
}

#define PE_ADD(q, h, i)                                                                     \
  asm volatile("add.rn.f32 pe_s" #q "_" #i ", pe_s" #q "_" #i ", %0;" ::"f"(far[32 * q + i]));
__device__ __forceinline__ void merge_far(const float (&far)[kRows]) {
  PE_EACH32(PE_ADD, 0, 0) PE_EACH32(PE_ADD, 1, 0) PE_EACH32(PE_ADD, 2, 0) PE_EACH32(PE_ADD, 3, 0)
}

// How rows of out are written: bf16 or fp32 boxes by TMA, or, where rows start
// anywhere, either type element by element.
enum Out { kOutBf16 = 0, kOutFp32 = 1, kOutAnywhere = 2 };

// Columns 32 q .. of a warp's 32 rows x 128 columns at (row0, col0) of out. `stage`:
// this warp's two boxes of 32 rows x 128 bytes.
template <int kOut, int q>
__device__ __forceinline__ void store_quarter(const Params& p, const CUtensorMap& tm_out,
                                              uint32_t stage, int lane, int32_t row0,
                                              int32_t col0) {
  float x[32];
  get_sums<q>(x);
  if constexpr (kOut == kOutBf16) {        // two quarters fill a box
    const uint32_t box = stage + (q >> 1) * kBoxBytes;
    const uint32_t row = box + lane * 128 + ((lane & 7) << 4);
#pragma unroll
    for (int g = 0; g < 4; ++g)
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(row ^ ((q % 2 * 4 + g) << 4)),
                   "r"(pack_bf16x2(x[8 * g], x[8 * g + 1])),
                   "r"(pack_bf16x2(x[8 * g + 2], x[8 * g + 3])),
                   "r"(pack_bf16x2(x[8 * g + 4], x[8 * g + 5])),
                   "r"(pack_bf16x2(x[8 * g + 6], x[8 * g + 7]))
                   : "memory");
    if constexpr (q % 2 == 1) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0 && col0 + q / 2 * 64 < p.n) {
        tma_store_2d(&tm_out, box, col0 + q / 2 * 64, row0);
        bulk_commit();
      }
    }
  } else if constexpr (kOut == kOutFp32) {
    const uint32_t box = stage + (q & 1) * kBoxBytes;
    const uint32_t row = box + lane * 128 + ((lane & 7) << 4);
    if constexpr (q == 2) {                // both boxes are in use
      if (lane == 0) bulk_wait_read();
      __syncwarp();
    }
#pragma unroll
    for (int g = 0; g < 8; ++g)
      asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(row ^ (g << 4)),
                   "f"(x[4 * g]), "f"(x[4 * g + 1]), "f"(x[4 * g + 2]), "f"(x[4 * g + 3])
                   : "memory");
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0 && col0 + q * 32 < p.n) {
      tma_store_2d(&tm_out, box, col0 + q * 32, row0);
      bulk_commit();
    }
  } else {
    // Through the stage, then row by row: a row's 32 columns are consecutive.
    __syncwarp();
    const uint32_t row = stage + lane * 128 + ((lane & 7) << 4);
#pragma unroll
    for (int g = 0; g < 8; ++g)
      asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(row ^ (g << 4)),
                   "f"(x[4 * g]), "f"(x[4 * g + 1]), "f"(x[4 * g + 2]), "f"(x[4 * g + 3])
                   : "memory");
    __syncwarp();
    const int32_t col = col0 + q * 32 + lane;
    const int32_t rows = col >= p.n ? 0 : p.m - row0;
    int64_t at = (int64_t)row0 * p.n + col;
#pragma unroll
    for (int32_t r0 = 0; r0 < 32; r0 += 8, at += 8 * (int64_t)p.n) {   // eight reads in flight
      float v[8];
#pragma unroll
      for (int32_t r = 0; r < 8; ++r)
        v[r] = load_shared(stage + (r0 + r) * 128 + (((lane >> 2) ^ r) << 4) + (lane & 3) * 4);
      if (p.out_fp32) {
#pragma unroll
        for (int32_t r = 0; r < 8; ++r)
          if (r0 + r < rows) static_cast<float*>(p.out)[at + r * (int64_t)p.n] = v[r];
      } else {
#pragma unroll
        for (int32_t r = 0; r < 8; ++r)
          if (r0 + r < rows)
            static_cast<__nv_bfloat16*>(p.out)[at + r * (int64_t)p.n] = __float2bfloat16_rn(v[r]);
      }
    }
  }
}

// A quarter of a part: [column group][row] float4, so that a warp's stores are
// consecutive.
template <int q>
__device__ __forceinline__ void store_part(float4* part) {
  float x[32];
  get_sums<q>(x);
#pragma unroll
  for (int g = 0; g < 8; ++g)
    part[(8 * q + g) * 128] = make_float4(x[4 * g], x[4 * g + 1], x[4 * g + 2], x[4 * g + 3]);
}

template <int kOut>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
matmul_pair_kernel(const __grid_constant__ CUtensorMap tm_a,
                   const __grid_constant__ CUtensorMap tm_b,
                   const __grid_constant__ CUtensorMap tm_out, const Params p) {
  PE_DECLARE_SUMS();
  extern __shared__ uint8_t raw[];
  Smem& s = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int32_t pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  volatile WaitGuard* guard = &s.guard;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&s.full[i]), 1);
      mbar_init(smem_u32(&s.empty[i]), 2);
    }
    for (int i = 0; i < 2; ++i) {
      for (int j = 0; j < 2; ++j) {
        mbar_init(smem_u32(&s.acc_full[i][j]), 2);
        mbar_init(smem_u32(&s.acc_empty[i][j]), 8);
      }
    }
    for (int i = 0; i < kIssueWarps; ++i) mbar_init(smem_u32(&s.drain[i]), 1);
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
      const uint32_t full0 = peer_address(smem_u32(&s.full[0]), 0);
      int32_t issued = 0, stage = 0;
      uint32_t parity = 1;
      bool ok = true;
      Walk w;
      for (bool more = w.start(p, pair, pairs); more && ok; more = w.next(p)) {
        const int32_t rt = w.tile / p.col_tiles, ct = w.tile - rt * p.col_tiles;
        const int32_t row = rt * kTile + (int32_t)rank * kRows;
        const int32_t col = ct * kTile + (int32_t)rank * 64;   // 64 rows of each column half
        for (int32_t block = w.first; block < w.last; ++block) {
          ok = eager_wait(smem_u32(&s.empty[stage]), parity, guard, p.status, kSiteProducer);
          if (!ok) break;
          const uint32_t bar = full0 + stage * 8;
          if (rank == 0) mbar_arrive_expect_tx(smem_u32(&s.full[stage]), kPairBytes);
          tma_load_pair(smem_u32(s.a[stage]), &tm_a, bar, block * kFp8Block, row);
          tma_load_pair(smem_u32(s.b[stage]), &tm_b, bar, block * kFp8Block, col);
          tma_load_pair(smem_u32(s.b[stage]) + kOperandBytes / 2, &tm_b, bar, block * kFp8Block,
                        col + 128);
          ++issued;
          if (++stage == kStages) {
            stage = 0;
            parity ^= 1;
          }
        }
      }
      store_cluster_i32(peer_address(smem_u32(&s.issued[rank]), 0), issued);
    } else if ((warp == 1 || warp == 2) && rank == 0) {
      // ---------------------------------------------------------- MMA issue
      const int half = warp - 1;
      const int32_t blocks = pair_blocks(p, pair, pairs);
      const uint32_t full0 = smem_u32(&s.full[0]), empty0 = smem_u32(&s.empty[0]);
      const uint32_t acc_full = smem_u32(&s.acc_full[half][0]);
      const uint32_t acc_empty = smem_u32(&s.acc_empty[half][0]);
      const uint64_t desc_a0 = smem_desc_sw128(smem_u32(s.a[0]), 16, 1024);
      const uint64_t desc_b0 =
          smem_desc_sw128(smem_u32(s.b[0]) + half * (kOperandBytes / 2), 16, 1024);
      uint32_t stage = 0, parity = 0;
      // Both barriers of a block are asked for while the one before is issued.
      bool free = true, loaded = false;
      for (int32_t i = 0; i < blocks; ++i) {
        const uint32_t buf = i & 1;
        if (!__all_sync(0xffffffffu, free && loaded)) {
          if (!eager_warp_wait(acc_empty + buf * 8, ((i >> 1) & 1) ^ 1, guard, p.status, kSiteMma))
            break;
          if (!eager_warp_wait(full0 + stage * 8, parity, guard, p.status, kSiteMma)) break;
        }
        tc_fence_after();
        const uint64_t da = desc_a0 + stage * (kOperandBytes / 16);
        const uint64_t db = desc_b0 + stage * (kOperandBytes / 16);
        const uint32_t d = tmem + buf * kTile + half * 128;
#pragma unroll
        for (int k = 0; k < 4; ++k)        // 32 bytes of k each: 2 units of 16 bytes
          mma_pair(d, da + 2 * k, db + 2 * k, p.idesc, k > 0);
        commit_pair(acc_full + buf * 8);
        commit_pair(empty0 + stage * 8);
        if (++stage == kStages) {
          stage = 0;
          parity ^= 1;
        }
        free = mbar_test_wait(acc_empty + (buf ^ 1) * 8, (((i + 1) >> 1) & 1) ^ 1);
        loaded = mbar_test_wait(full0 + stage * 8, parity);
      }
      commit_pair(smem_u32(&s.drain[warp - 1]));   // no MMA is in flight past this
      mbar_drain_wait(smem_u32(&s.drain[warp - 1]), 0);
    } else if (warp == 3) {
      // ---------------------------------------------------------- scales
      const int32_t col_blocks = (p.n + kFp8Block - 1) / kFp8Block;
      const int32_t blocks = pair_blocks(p, pair, pairs);
      Walk w;
      bool more = w.start(p, pair, pairs);
      const float* a_src = nullptr;
      const float* b_src = nullptr;
      uint32_t a_step[4];                  // to this lane's rows 32, 64 and 96 further
      auto locate = [&]() {                // this lane's rows (and columns) in w's tile
        // Rows and columns outside the matrix take row or column 0's scale: their sums are
        // zeros (operands outside are) or NaN, and not stored.
        const int32_t rt = w.tile / p.col_tiles, cb = 2 * (w.tile - rt * p.col_tiles) + (lane & 1);
        const int32_t row = rt * kTile + (int32_t)rank * kRows + lane;
        a_src = p.a_scales + (int64_t)w.first * p.m + (row < p.m ? row : 0);
        b_src = p.b_scales + (int64_t)w.first * col_blocks + (cb < col_blocks ? cb : 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) a_step[i] = row + 32 * i < p.m ? 32 * i : 0;
      };
      if (more) locate();
      for (int32_t i = -kScaleAhead; i < blocks; ++i) {
        if (more) {
          // The slot held block i - 8, and both CTAs are done with it: the MMAs of block
          // i - 3, which have completed, waited for block i - 5 to be read.
          const int slot = (i + kScaleAhead) % kScaleSlots;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            copy_async4(&s.a_scale[slot][j * 32 + lane], a_src + a_step[j], true);
          if (lane < 2) copy_async4(&s.b_scale[slot][lane], b_src, true);
          a_src += p.m;
          b_src += col_blocks;
          if (++w.first == w.last) {
            more = w.next(p);
            if (more) locate();
          }
        }
        copy_async_commit();
        if (i < 0) continue;
        copy_async_wait<kScaleAhead>();    // block i's scales are here
        const uint32_t bar = smem_u32(&s.acc_full[0][i & 1]);
        if (i >= 2) {                      // its turn of the barriers has begun
          const uint32_t before = (uint32_t)((i >> 1) - 1) & 1;
          if (!eager_warp_wait(bar, before, guard, p.status, kSiteScales) ||
              !eager_warp_wait(bar + 16, before, guard, p.status, kSiteScales))
            break;
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar);
          mbar_arrive(bar + 16);
        }
      }
      copy_async_wait<0>();
    }
    __syncwarp();
  } else {
    regs_claim<kRegsHigh>();
    // ------------------------------------------------------------ scaling and sums
    const int quad = warp & 3, half = (warp - 4) >> 2;
    const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16) + half * 128;
    const int32_t row_in = (int32_t)rank * kRows + quad * 32;   // this warp's rows in the tile
    const uint32_t stage_out = smem_u32(s.out[warp - 4]);
    const uint32_t acc_empty = peer_address(smem_u32(&s.acc_empty[half][0]), 0);

    const uint32_t acc_full = smem_u32(&s.acc_full[half][0]);
    const uint32_t first = lane == 0 ? 1u : 0u;
    const uint32_t a_scale = smem_u32(&s.a_scale[0][quad * 32 + lane]);
    const uint32_t b_scale = smem_u32(&s.b_scale[0][half]);

    uint32_t buf = 0, parity = 0, slot = 0;
    bool ok = true;
    Walk w;
    if (w.start(p, pair, pairs)) {
      for (bool begins = true;; begins = false) {       // begins: the pair's first segment
        clear_sums();
        float far[kRows];                               // what add_block leaves out,
        bool any_far = false;                           // if anything
        for (int32_t block = w.first; block < w.last; ++block) {
          if (!eager_warp_wait(acc_full + buf * 8, parity, guard, p.status, kSiteEpilogue)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const float sa = load_shared(a_scale + slot * (kRows * 4));
          const float sb = load_shared(b_scale + slot * 8);
          const float scale = sa * sb;
          if (add_block(scale, lane_base + buf * kTile, acc_empty + buf * 8, first)) {
            const bool left_out = fabsf(scale) < 0x1p-126f || fabsf(scale) > 3.402823466e38f;
            add_far(far, any_far, left_out, far_factors(sa, sb), lane_base + buf * kTile);
            any_far = true;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(acc_empty + buf * 8);
          }
          slot = (slot + 1) % kScaleSlots;
          parity ^= buf;
          buf ^= 1;
        }
        if (!ok) break;
        if (any_far) merge_far(far);
        // The segment's sums: a whole tile goes to out, a part to the workspace.
        const int32_t rt = w.tile / p.col_tiles, ct = w.tile - rt * p.col_tiles;
        const int32_t row0 = rt * kTile + row_in, col0 = ct * kTile + half * 128;
        if (w.first != 0 || w.last != p.blocks) {
          float4* part =
              reinterpret_cast<float4*>(p.parts + (2 * pair + (begins ? 0 : 1)) * kPartFloats) +
              (rank * 64 + half * 32) * 128 + quad * 32 + lane;
          store_part<0>(part);
          store_part<1>(part);
          store_part<2>(part);
          store_part<3>(part);
        } else if (row0 < p.m && col0 < p.n) {
          if (lane == 0) bulk_wait_read();              // the tile before has left the stage
          __syncwarp();
          store_quarter<kOut, 0>(p, tm_out, stage_out, lane, row0, col0);
          store_quarter<kOut, 1>(p, tm_out, stage_out, lane, row0, col0);
          store_quarter<kOut, 2>(p, tm_out, stage_out, lane, row0, col0);
          store_quarter<kOut, 3>(p, tm_out, stage_out, lane, row0, col0);
        }
        if (!w.next(p)) break;
      }
    }
    bulk_wait_all();
  }

  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) store_cluster_i32(peer_address(smem_u32(&s.aborted[rank]), 0),
                                          s.guard.abort);
  __syncthreads();
  cluster_sync();
  // The issuing warps' last commits arrive in both CTAs: the second stays until they,
  // and so every arrival before them, have reached its barriers.
  if (rank == 1 && threadIdx.x == 0)
    for (int i = 0; i < kIssueWarps; ++i) mbar_drain_wait(smem_u32(&s.drain[i]), 0);
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
  griddep_wait();                                        // before any block may leave
  const int piece = blockIdx.x & 15;                     // 2 CTAs x 4 row quarters x 2 halves
  const int32_t t = blockIdx.x >> 4;
  const int rank = piece >> 3, quad = (piece >> 1) & 3, half = piece & 1;
  const int32_t rt = t / p.col_tiles, ct = t - rt * p.col_tiles;
  const int32_t row0 = rt * kTile + rank * kRows + quad * 32, col0 = ct * kTile + half * 128;
  if (row0 >= p.m || col0 >= p.n) return;
  const int32_t lo = t * p.blocks, hi = lo + p.blocks;   // the tile's blocks
  // Pair q holds block `lo`: run_start(q) <= lo < run_start(q + 1).
  const int32_t long_end = p.run_more * (p.run_blocks + 1);
  int32_t q = lo < long_end ? lo / (p.run_blocks + 1)
                            : p.run_more + (lo - long_end) / p.run_blocks;
  if (run_start(p, q + 1) >= hi) return;                 // one pair wrote the whole tile
  const int row = threadIdx.x & 31, g0 = threadIdx.x >> 5;
  const float4* parts = reinterpret_cast<const float4*>(p.parts) +
                        (rank * 64 + half * 32) * 128 + quad * 32 + row + g0 * 128;
  float4 sum[4] = {};
  // Four parts in flight, added in the order of k. A pair's part of the tile is its
  // first segment unless its run began before the tile.
  constexpr int kAhead = 4;
  while (q < pairs && run_start(p, q) < hi) {
    float4 v[kAhead][4];
    bool in[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int32_t start = run_start(p, q + j);
      in[j] = q + j < pairs && start < hi;
      const int64_t slot = 2 * (q + j) + (start >= lo ? 0 : 1);
      if (in[j]) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[j][i] = parts[slot * (int64_t)(kPartFloats / 4) + 8 * i * 128];
      }
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (in[j]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sum[i].x += v[j][i].x;
          sum[i].y += v[j][i].y;
          sum[i].z += v[j][i].z;
          sum[i].w += v[j][i].w;
        }
      }
    }
    q += kAhead;
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
int32_t pair_count() {
  const int32_t n = device_sm_count() / 2;
  return n < kMaxPairs ? n : kMaxPairs;
}

}  // namespace

size_t matmul_pair_workspace() { return 2 * kMaxPairs * kPartFloats * sizeof(float); }

pe_status matmul_pair(const MatmulFp8& q, bool runs, void* workspace, DeviceStatus* status,
                      cudaStream_t stream) {
  CUtensorMap ma, mb, mo;
  PE_TRY(matmul_map(&ma, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, q.a, q.m, q.k, q.a_ld, kRows));
  PE_TRY(matmul_map(&mb, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, q.b, q.n, q.k, q.b_ld, kRows / 2));
  const int size = q.out_fp32 ? 4 : 2;
  const bool tma_store = aligned(q.out, 16) && (int64_t)q.n * size % 16 == 0;
  mo = ma;
  if (tma_store)
    PE_TRY(matmul_map(&mo, q.out_fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                    : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                    size, q.out, q.m, q.n, (int64_t)q.n * size, 32));
  const auto kernel = !tma_store  ? matmul_pair_kernel<kOutAnywhere>
                      : q.out_fp32 ? matmul_pair_kernel<kOutFp32>
                                   : matmul_pair_kernel<kOutBf16>;
  const size_t smem = sizeof(Smem) + 1024;
  PE_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   static_cast<int>(smem)));
  cudaFuncAttributes attr;
  PE_CUDA_TRY(cudaFuncGetAttributes(&attr, kernel));
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
  p.tiles = (int32_t)tiles;
  int32_t pairs = pair_count();
  p.shared_tiles = runs ? 1 : 0;
  p.run_blocks = (int32_t)(tiles * p.blocks / pairs);
  p.run_more = (int32_t)(tiles * p.blocks % pairs);
  if (!p.shared_tiles && tiles < pairs) pairs = (int32_t)tiles;
  p.out_fp32 = q.out_fp32 ? 1 : 0;
  p.idesc = idesc_fp8(256, 128, q.a_e5m2, q.b_e5m2);
  p.out = q.out;
  p.parts = static_cast<float*>(workspace);
  p.status = status;
  p.wait_limit_ns = wait_limit_ns();
  kernel<<<2 * pairs, kThreads, smem, stream>>>(ma, mb, mo, p);
  PE_CUDA_TRY(cudaGetLastError());
  if (p.shared_tiles)
    return launch_after_previous(matmul_parts_kernel, dim3((unsigned)(16 * tiles)), dim3(256), 0,
                                 stream, p, pairs);
  return PE_OK;
}

}  // namespace pe
