// Matrix product with bias, activation and residual, many rows:
// out = act(a b^T + bias) + residual.
//
// A pair of CTAs (tcgen05 cta_group::2) works on a 256 x 256 tile: each CTA loads 128 rows of
// a and 128 rows of b, 64 elements of k at a time, and the pair's MMAs (M = 256, N = 256, K =
// 16) sum a tile in tensor memory, over the whole of k or a chain of its blocks. Two accumulators take turns, so the
// epilogue of a tile runs under the next tile's MMAs. An operand stored with k as its rows is
// loaded in boxes of 64 columns by 64 rows and read by the MMA as it lies there.
//
// Every CTA loads its own rows by itself: no load writes into another CTA's shared memory, so
// that the kernel can run in any process, one of several GPUs' among them.
//
//   warps 0, 2   loads of a and of b (every CTA), a ring of kStages blocks
//   warp 1       MMA issue (first CTA of each pair)
//   warps 4-11   epilogue; warps 4-7 the tile's left half, 8-11 its right half: bias, z into
//                pre, activation, residual (loaded by TMA into the box that the result then
//                leaves from), rounding, TMA stores of 32 rows x 128 bytes
//
// With geglu the tile is 128 columns of out: the first CTA loads their gate rows of b, the
// second their up rows, so that a thread finds both in its row of tensor memory.
//
// fp32 operands come as three bf16 parts each, and six products of parts, the smallest
// first, are summed like six times as many blocks of k, what parts of one size give in chains of
// its own.
//
// Work: whole tiles in turn, or, where few tiles have long sums, slices of k, all tiles of a
// slice before the next (so that the pairs read the same blocks of k at about the same
// time); the slices' fp32 sums are then added, in the order of k, by a second kernel, which
// also does the epilogue.
//
// What bounds it: a block of 64 is 512 cycles of MMAs, and every other cycle is one in which
// the tensor cores wait for an instruction. Measured, in cycles a block (32299 x 2304 x 768;
// the same with geglu; with gelu; 19456 x 2304 x 8192):
//   loads and MMAs by one thread each, in branches of one thread   767  767  1040   608
//   loads of a and of b by a warp each                             655  827  1020   546
//   MMAs issued by a whole warp, one elected lane                  569  708   917   518
//   loads likewise, gelu in paired arithmetic                      548  542   690   519
// A branch of one thread keeps its operands out of the uniform registers that these
// instructions read, and the epilogue's warps, whose independent multiply-adds never stall,
// take the issue slots of the scheduler that the MMA warp is on (one such warp beside it
// made 589 cycles 982; on another scheduler it changed nothing). With gelu that is what is
// left: its own instructions are some 500 cycles a block on each scheduler.
//
// Measured (GB300, device time of a burst): 32299 x 2304 x 768 bf16 in 66.6 us (1.72 PFLOP/s,
// 0.89 of the measured dense bf16 rate), with geglu and pre 81 (1.41), 169151 x 1024 x 1024
// with bias and residual 214 to 221 us (1.65; the tensor cores are busy for 0.905 of the
// cycles), the input gradient 32299 x 768 x 2304 71 to 73 (1.6), 2304 x 768 x 32299 to fp32 78.5
// (1.46), 90487 x 512 x 512 of fp32 180 beside the 73 that cut its operands into parts; with
// results in fp32 gelu is 32 calls out of line for a thread and unit, 90487 x 1024 x 512 637 us
// for 400. For seconds on end the power cap rules:
// 77 us for the first, 238 for 169151 x 1024 x 1024, at 1.6 to 1.8 GHz.
#include <type_traits>

#include "pe_matmul.cuh"

namespace pe {

namespace {

using namespace sm103;

constexpr int kTile = 256;
constexpr int kRows = 128;                               // rows of a (and of b) per CTA
constexpr int kStages = 6;
constexpr int kThreads = 384;
constexpr uint32_t kOperandBytes = kRows * 128;          // 16 KiB
constexpr uint32_t kPairBytes = 4 * kOperandBytes;       // both CTAs' a and b of one block
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kBoxBytes = 32 * 128;                 // 32 rows of 128 bytes
// How rows of out, residual and pre move between a warp's box and memory: by TMA or, where
// rows start anywhere, by the warp's lanes.
enum Out {
  kOutBf16 = 0,
  kOutFp32 = 1,
  kOutBf16Anywhere = 2,
  kOutFp32Anywhere = 3,
  kOutBf16Long = 4,                    // sums of more than kLongest blocks, or of parts
  kOutBf16AnywhereLong = 6,
  kOutSlices = 8                       // sums of slices, finished elsewhere to fp32
};
constexpr bool is_fp32(int out) { return out & 1; }
constexpr bool by_tma(int out) { return !(out & 2); }

constexpr uint32_t kRegsLaunch = 168;
constexpr uint32_t kRegsLow = 40, kRegsHigh = 232;
static_assert(128 * (kRegsLow + 2 * kRegsHigh) <= kThreads * kRegsLaunch,
              "register split exceeds the launch allocation");
// Blocks of k that one accumulator sums. The tensor cores align 16 products and the sum so far
// to the largest of them and cut them off towards zero, so a chain of additions of numbers of
// one sign loses a share that grows with its length: k = 4096 1.1e-5 of the sum, 8192 3.2e-5,
// 2^17 8e-4, 2^19 3.3e-3, which a result rounded to bf16 (2e-3 to 4e-3) shows. So results
// rounded to bf16 have chains of kLongest blocks at most; fp32 results, and longer sums, add
// chains of eight in fp32 registers: 1.1e-7 of the sum of magnitudes lost in the mean, 3.5e-7 at
// most, whatever k (elementary fp32 operations: 1.1e-5 at most over 32299). Of one accumulator
// a block takes 516 cycles, of chains of eight 532 (32299 x 768 x 2304 to fp32 82 us), of four
// 560 (89). The slices of fp32 results, weights' gradients, have an epilogue short enough for
// chains of four: 2304 x 768 x 32299 in 78.5 us for 77.7, off by 2.5e-7 of the result's size for
// 4.7e-7 (elementary fp32 operations 2.7e-7).
constexpr int32_t kLongest = 128;
constexpr bool by_chunks(int out) { return out & (kOutFp32 | kOutBf16Long | kOutSlices); }
constexpr int32_t chunk_of(int out) { return out & kOutSlices ? 4 : 8; }
constexpr size_t kPartFloats = (size_t)kTile * kTile;
constexpr int kPartsAhead = 5, kPartBlocks = 4;          // parts in flight; blocks an SM

struct alignas(1024) Smem {
  uint8_t a[kStages][kOperandBytes];
  uint8_t b[kStages][kOperandBytes];
  alignas(1024) uint8_t box[8][kBoxBytes];     // of each epilogue warp
  alignas(16) float bias[2][kRows];            // of each half of the tile
  uint64_t full[kStages], empty[kStages];      // full: the first CTA's serve the pair
  uint64_t acc_full[2], acc_empty[2];          // acc_empty: likewise
  uint64_t residual[8];                        // the box's residual has arrived
  uint64_t drain;
  int32_t loaded[2];                           // blocks of a, of b that this CTA loaded
  int32_t issued[2][2];                        // the same of both CTAs, and whether one of
  int32_t aborted[2];                          // their waits gave up
  uint32_t tmem_base;
  WaitGuard guard;
};
static_assert(sizeof(Smem) + 1024 <= 227 * 1024, "shared memory exceeds the per-CTA limit");

// Quotients by a number known at launch, of 0 <= x < 2^31: with 2^(l-1) < d <= 2^l and m =
// floor(2^(31+l) / d) + 1, x / d is the upper word of x m shifted right by l - 1 (T.
// Granlund and P. Montgomery, Division by invariant integers using multiplication, 1994).
// The warps that feed the tensor cores divide between two tiles.
struct Divisor {
  uint32_t d, m;
  int32_t shift;             // -1: d = 1

  __host__ static Divisor of(int32_t d) {
    int32_t l = 0;
    while ((1ll << l) < d) ++l;
    return {(uint32_t)d, d == 1 ? 0u : (uint32_t)((1ull << (31 + l)) / (uint32_t)d + 1), l - 1};
  }
  __device__ int32_t quotient(int32_t x) const {
    return shift < 0 ? x : (int32_t)(__umulhi((uint32_t)x, m) >> shift);
  }
};

struct Params {
  MatmulEpilogue e;
  int32_t blocks;            // of k, of all terms
  int32_t term_blocks;       // of one term
  int32_t terms;
  Chains chains;
  int32_t a_transposed, b_transposed;
  int32_t up_row;            // geglu: b's first up row
  int32_t row_tiles;
  int32_t col_tiles;
  int32_t tiles;             // row_tiles * col_tiles
  int32_t slices;            // of k; more than one: sums through `parts`
  int32_t slice_blocks;      // blocks of a slice; the first slices
  int32_t slice_more;        // have one more
  Divisor by_band, by_tiles; // quotients by a band's tiles, by all tiles
  uint32_t idesc;
  float* parts;              // [slices][tiles][2 CTAs][2 halves][32 column groups][128 rows] float4
  DeviceStatus* status;
  uint64_t wait_limit_ns;
};

struct Maps {
  CUtensorMap a, b, out, residual, pre, pre_up;
};

enum WaitSite { kSiteProducer = 91, kSiteMma = 92, kSiteEpilogue = 93, kSiteResidual = 94 };

__device__ __forceinline__ void store_cluster_i32(uint32_t addr, int32_t v) {
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void mbar_complete_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// The loads and MMAs below are executed by a whole warp with the same operands, and one lane
// issues: a warp that runs together keeps them in uniform registers, where these instructions
// take their operands from; in a branch of one thread each of them first costs several moves.

// Box load into this CTA, counted on a barrier of the pair's first CTA.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                              int32_t x, int32_t y, int32_t z) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b32 r;\n\telect.sync r|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
// The same box into the L2 cache only.
__device__ __forceinline__ void tma_prefetch(const CUtensorMap* map, int32_t x, int32_t y,
                                             int32_t z) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b32 r;\n\telect.sync r|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];\n\t}" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(x), "r"(y), "r"(z)
      : "memory");
}
// Announces a block's bytes on its barrier.
__device__ __forceinline__ void expect_pair(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b32 r;\n\t.reg .b64 st;\n\telect.sync r|e, 0xffffffff;\n\t"
      "@e mbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n\t}" ::"r"(bar),
      "r"(kPairBytes)
      : "memory");
}
// The four MMAs of a block: operands at the descriptors' low words (the high
// ones are the same for all), kA and kB units of 16 bytes from 16 elements of k to the next.
template <uint32_t kA, uint32_t kB>
__device__ __forceinline__ void mma_block(uint32_t d_tmem, uint32_t a_low, uint32_t a_high,
                                          uint32_t b_low, uint32_t b_high, uint32_t idesc,
                                          uint32_t accumulate) {
#define PE_MMA "@e tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %5, "
#define PE_NEXT(i, j)                                                                \
  "add.u32 a, %1, %" #i ";\n\tadd.u32 b, %3, %" #j ";\n\tmov.b64 da, {a, %2};\n\t" \
  "mov.b64 db, {b, %4};\n\t"
  asm volatile(
      "{\n\t.reg .pred p, t, e;\n\t.reg .b32 a, b, r;\n\t.reg .b64 da, db;\n\t"
      "setp.ne.b32 p, %6, 0;\n\tsetp.eq.b32 t, 0, 0;\n\telect.sync r|e, 0xffffffff;\n\t"
      "mov.b64 da, {%1, %2};\n\tmov.b64 db, {%3, %4};\n\t" PE_MMA "p;\n\t" PE_NEXT(7, 8)
          PE_MMA "t;\n\t" PE_NEXT(9, 10) PE_MMA "t;\n\t" PE_NEXT(11, 12) PE_MMA "t;\n\t}" ::"r"(
              d_tmem),
      "r"(a_low), "r"(a_high), "r"(b_low), "r"(b_high), "r"(idesc), "r"(accumulate), "n"(kA),
      "n"(kB), "n"(2 * kA), "n"(2 * kB), "n"(3 * kA), "n"(3 * kB)
      : "memory");
#undef PE_MMA
#undef PE_NEXT
}
// Arrives once on this barrier of both CTAs when the MMAs issued so far complete.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b32 r;\n\telect.sync r|e, 0xffffffff;\n\t@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;\n\t}" ::"r"(bar),
      "h"(uint16_t{3})
      : "memory");
}
// Tiles are dealt in bands of four rows, down the rows first, so that the pairs at work
// share operands in L2 both ways.
constexpr int32_t kBand = 4;
__device__ __forceinline__ void place(const Params& p, int32_t tile, int32_t& row, int32_t& col) {
  const int32_t band = p.by_band.quotient(tile), rest = tile - band * (int32_t)p.by_band.d;
  const int32_t left = p.row_tiles - band * kBand;
  col = left >= kBand ? rest / kBand : left == 1 ? rest : left == 2 ? rest / 2 : rest / 3;
  row = band * kBand + rest - col * (left < kBand ? left : kBand);
}

// The work of a pair: units, of a tile and a slice of its blocks of k, slice by slice.
struct Walk {
  int32_t unit, tile;
  int32_t first, last;            // last: one past the unit's last block

  __device__ bool at(const Params& p, int32_t u) {
    unit = tile = u;
    first = 0;
    last = p.blocks;
    if (p.slices > 1) {
      const int32_t slice = p.by_tiles.quotient(u);
      tile = u - slice * p.tiles;
      first = slice * p.slice_blocks + (slice < p.slice_more ? slice : p.slice_more);
      last = first + p.slice_blocks + (slice < p.slice_more ? 1 : 0);
    }
    return u < p.tiles * p.slices;
  }
};

// 32 columns of a row, rounded, into the box's 16-byte chunks from `chunk` on.
template <int kOut>
__device__ __forceinline__ void put_row(uint32_t row, int chunk, const float (&x)[32]) {
  if constexpr (!is_fp32(kOut)) {
#pragma unroll
    for (int g = 0; g < 4; ++g)
      store_shared_v4(row ^ ((chunk + g) << 4),
                      make_uint4(pack_bf16x2(x[8 * g], x[8 * g + 1]),
                                 pack_bf16x2(x[8 * g + 2], x[8 * g + 3]),
                                 pack_bf16x2(x[8 * g + 4], x[8 * g + 5]),
                                 pack_bf16x2(x[8 * g + 6], x[8 * g + 7])));
  } else {
#pragma unroll
    for (int g = 0; g < 8; ++g)
      store_shared_v4(row ^ (g << 4),
                      make_uint4(__float_as_uint(x[4 * g]), __float_as_uint(x[4 * g + 1]),
                                 __float_as_uint(x[4 * g + 2]), __float_as_uint(x[4 * g + 3])));
  }
}
// Adds the residual that lies in the box.
template <int kOut>
__device__ __forceinline__ void add_row(uint32_t row, int chunk, float (&x)[32]) {
  if constexpr (!is_fp32(kOut)) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const uint4 r = load_shared_v4(row ^ ((chunk + g) << 4));
      const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[8 * g + 2 * j] += __uint_as_float(w[j] << 16);
        x[8 * g + 2 * j + 1] += __uint_as_float(w[j] & 0xffff0000u);
      }
    }
  } else {
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      const uint4 r = load_shared_v4(row ^ (g << 4));
      x[4 * g] += __uint_as_float(r.x);
      x[4 * g + 1] += __uint_as_float(r.y);
      x[4 * g + 2] += __uint_as_float(r.z);
      x[4 * g + 3] += __uint_as_float(r.w);
    }
  }
}

// A box to rows that start anywhere: a row's 128 bytes are 32 consecutive words, one a lane.
// Where a bf16 row starts in the middle of a word, lane l writes columns 2 l - 1 and 2 l in
// one word, and the first and last columns go alone. `rows` and `cols` of the box exist.
template <bool kFp32>
__device__ __forceinline__ void box_to_rows(uint32_t box, int lane, void* out, int64_t ld,
                                            int64_t row0, int64_t col0, int32_t rows,
                                            int32_t cols) {
  if (cols <= 0) return;
#pragma unroll 1
  for (int r0 = 0; r0 < 32 && r0 < rows; r0 += 8) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      w[i] = __float_as_uint(
          load_shared_f32(box + (r0 + i) * 128 + (((lane >> 2) ^ i) << 4) + (lane & 3) * 4));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (r0 + i >= rows) break;
      const int64_t at = (row0 + r0 + i) * ld + col0;
      if constexpr (kFp32) {
        if (lane < cols) static_cast<uint32_t*>(out)[at + lane] = w[i];
      } else {
        uint16_t* to = static_cast<uint16_t*>(out) + at;
        const int shift = (int)(reinterpret_cast<uintptr_t>(to) >> 1 & 1);   // the warp's
        const uint32_t before = __shfl_up_sync(0xffffffffu, w[i], 1);
        const uint32_t word = shift ? (before >> 16) | (w[i] << 16) : w[i];
        const int32_t c = 2 * lane - shift;              // the word's first column
        if (c >= 0 && c + 1 < cols) {
          *reinterpret_cast<uint32_t*>(to + c) = word;
        } else {
          if (c >= 0 && c < cols) to[c] = (uint16_t)word;
          if (c < 0) to[0] = (uint16_t)(word >> 16);
        }
        if (shift && lane == 31 && cols > 63) to[63] = (uint16_t)(w[i] >> 16);
      }
    }
  }
}
// The same the other way: the residual's rows into a box.
template <bool kFp32>
__device__ __forceinline__ void rows_to_box(uint32_t box, int lane, const void* in, int64_t ld,
                                            int64_t row0, int64_t col0, int32_t rows,
                                            int32_t cols) {
#pragma unroll 1
  for (int r0 = 0; r0 < 32 && r0 < rows; r0 += 8) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[i] = 0;
      if (r0 + i < rows) {
        const int64_t at = (row0 + r0 + i) * ld + col0;
        if constexpr (kFp32) {
          if (lane < cols) w[i] = static_cast<const uint32_t*>(in)[at + lane];
        } else {
          const uint16_t* from = static_cast<const uint16_t*>(in) + at + 2 * lane;
          if (2 * lane + 1 < cols && (reinterpret_cast<uintptr_t>(from) & 2) == 0) {
            w[i] = *reinterpret_cast<const uint32_t*>(from);
          } else {
            if (2 * lane < cols) w[i] = from[0];
            if (2 * lane + 1 < cols) w[i] |= (uint32_t)from[1] << 16;
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      asm volatile("st.shared.b32 [%0], %1;" ::"r"(box + (r0 + i) * 128 +
                                                   (((lane >> 2) ^ i) << 4) + (lane & 3) * 4),
                   "r"(w[i])
                   : "memory");
  }
}

// 32 columns of this thread's lane from tensor memory.
__device__ __forceinline__ void load_acc(uint32_t src, float (&z)[32]) {
  uint32_t r[32];
  tmem_ld32(src, r);
  tmem_wait_ld(r);
#pragma unroll
  for (int i = 0; i < 32; ++i) z[i] = __uint_as_float(r[i]);
}
// Two columns an instruction, here and in gelu: every instruction of the epilogue takes an
// issue slot from the warps that feed the tensor cores.
__device__ __forceinline__ void add_bias(const float* bias, float (&z)[32]) {
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    const float4 b = *reinterpret_cast<const float4*>(bias + 4 * g);
    f2_split(fadd2(f2(z[4 * g], z[4 * g + 1]), f2(b.x, b.y)), z[4 * g], z[4 * g + 1]);
    f2_split(fadd2(f2(z[4 * g + 2], z[4 * g + 3]), f2(b.z, b.w)), z[4 * g + 2], z[4 * g + 3]);
  }
}

template <int kOut>
__device__ __forceinline__ void apply_gelu(float (&z)[32]) {
  if constexpr (is_fp32(kOut)) {
#pragma unroll
    for (int i = 0; i < 32; ++i) z[i] = gelu_fp32(z[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 32; i += 2)
      f2_split(GeluPair(z[i], z[i + 1]).value(z[i], z[i + 1]), z[i], z[i + 1]);
  }
}

template <int kOut, bool kGeglu>
__global__ void __launch_bounds__(kThreads, 1)
matmul_tiles_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
  extern __shared__ uint8_t raw[];
  Smem& s = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int32_t rank = (int32_t)cluster_rank();           // in the pair
  const int32_t pair = blockIdx.x / 2, pairs = gridDim.x / 2;
  volatile WaitGuard* guard = &s.guard;
  constexpr int32_t kOutCols = kGeglu ? kTile / 2 : kTile;   // of a tile

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&s.full[i]), 1);
      mbar_init(smem_u32(&s.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s.acc_full[i]), 1);
      mbar_init(smem_u32(&s.acc_empty[i]), 16);
    }
    for (int i = 0; i < 8; ++i) mbar_init(smem_u32(&s.residual[i]), 1);
    mbar_init(smem_u32(&s.drain), 1);
    s.guard.abort = 0;
    s.guard.limit_ns = p.wait_limit_ns;
    fence_mbarrier_init();
    prefetch_tensormap(&maps.a);
    prefetch_tensormap(&maps.b);
    prefetch_tensormap(&maps.out);
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
  griddep_wait();                          // what the kernel before this one wrote is read below
  cluster_sync();                          // every CTA's barriers exist before any arrival
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;

  if (by_chunks(kOut) && warp < 4) regs_release<kRegsLow>();
  if (warp == 0 || warp == 2) {
    // ---------------------------------------------------------- loads
    auto load = [&](auto of_b, auto is_transposed) {
      constexpr bool kB = decltype(of_b)::value, kTransposed = decltype(is_transposed)::value;
      const CUtensorMap* map = kB ? &maps.b : &maps.a;
      const uint32_t to0 = smem_u32(kB ? s.b[0] : s.a[0]);
      const uint32_t full0 = peer_address(smem_u32(&s.full[0]), 0);
      const uint32_t full_own = smem_u32(&s.full[0]), empty0 = smem_u32(&s.empty[0]);
      const int32_t x_end = p.term_blocks * kMatmulBlock;
      int32_t issued = 0;
      uint32_t stage = 0, parity = 1;
      bool ok = true;
      Walk w;
      int32_t next_row, next_col;                      // of tiles
      bool more = w.at(p, pair);
      place(p, w.tile, next_row, next_col);
      for (; more && ok; more = w.at(p, w.unit + pairs)) {
        const int32_t at = !kB      ? next_row * kTile + rank * kRows
                           : kGeglu ? next_col * kOutCols + (rank ? p.up_row : 0)
                                    : next_col * kTile + rank * kRows;
        int32_t term = p.terms == 1 ? 0 : w.first / p.term_blocks;
        int32_t x = (w.first - term * p.term_blocks) * kMatmulBlock;
        int32_t z = kB ? term_b(term, p.terms) : term_a(term, p.terms);
        // The rows of a that this CTA's next tile reads, which the pairs on its row of
        // tiles share out, go to L2 under this tile: from HBM a block takes longer than
        // the ring is deep (169151 x 1024 x 1024 222 us without, 217 with; with residual
        // 253, 243).
        Walk next;
        const bool ahead = next.at(p, w.unit + pairs) && p.slices == 1;
        place(p, next.tile, next_row, next_col);
        const int32_t ahead_at = next_row * kTile + rank * kRows;
        int32_t until = !kB && !kTransposed && ahead ? next_col : 0x7fffffff;
        for (int32_t left = w.last - w.first; left > 0; --left) {
          ok = eager_warp_wait(empty0 + stage * 8, parity, guard, p.status, kSiteProducer);
          if (!ok) break;
          const uint32_t bar = full0 + stage * 8, to = to0 + stage * kOperandBytes;
          if (!kB && rank == 0) expect_pair(full_own + stage * 8);
          if constexpr (kTransposed) {                 // 64 columns by 64 rows a box
            tma_load_pair(to, map, bar, at, x, z);
            tma_load_pair(to + kOperandBytes / 2, map, bar, at + 64, x, z);
          } else {
            tma_load_pair(to, map, bar, x, at, z);
          }
          if constexpr (!kB && !kTransposed) {
            if (until-- == 0) {
              tma_prefetch(map, x, ahead_at, z);
              until = p.col_tiles - 1;
            }
          }
          ++issued;
          if (++stage == kStages) {
            stage = 0;
            parity ^= 1;
          }
          x += kMatmulBlock;
          if (x == x_end) {
            x = 0;
            ++term;
            z = kB ? term_b(term, p.terms) : term_a(term, p.terms);
          }
        }
      }
      if (lane == 0) s.loaded[kB] = issued;
    };
    if (warp == 0) {
      if (p.a_transposed)
        load(std::false_type(), std::true_type());
      else
        load(std::false_type(), std::false_type());
    } else {
      if (p.b_transposed)
        load(std::true_type(), std::true_type());
      else
        load(std::true_type(), std::false_type());
    }
  } else if (warp == 1 && rank == 0) {
    // ---------------------------------------------------------- MMA issue
    // 16 elements of k: 32 bytes along rows of k, or 16 rows of 128 bytes; an operand's
    // next 64 columns, where k runs along its rows, are the stage's second half.
    auto issue = [&](auto a_is_transposed, auto b_is_transposed) {
      constexpr bool kAT = decltype(a_is_transposed)::value;
      constexpr bool kBT = decltype(b_is_transposed)::value;
      const uint64_t desc_a = smem_desc_sw128(smem_u32(s.a[0]), kAT ? 8192 : 16, 1024);
      const uint64_t desc_b = smem_desc_sw128(smem_u32(s.b[0]), kBT ? 8192 : 16, 1024);
      const uint32_t full0 = smem_u32(&s.full[0]), empty0 = smem_u32(&s.empty[0]);
      uint32_t stage = 0, parity = 0;
      int32_t turn = 0;                  // of the accumulators
      bool ok = true;
      Walk w;
      for (bool more = w.at(p, pair); more && ok; more = w.at(p, w.unit + pairs)) {
        for (int32_t block = w.first; block < w.last && ok; ++turn) {
          const uint32_t buf = turn & 1, d = tmem + buf * kTile;
          const int32_t end = by_chunks(kOut) ? p.chains.end(block, w.last, chunk_of(kOut)) : w.last;
          uint32_t accumulate = 0;
          ok = eager_warp_wait(smem_u32(&s.acc_empty[buf]), ((turn >> 1) & 1) ^ 1, guard, p.status,
                          kSiteMma);
          for (; block < end && ok; ++block) {
            ok = eager_warp_wait(full0 + stage * 8, parity, guard, p.status, kSiteMma);
            if (!ok) break;
            tc_fence_after();
            mma_block<kAT ? 128 : 2, kBT ? 128 : 2>(
                d, (uint32_t)desc_a + stage * (kOperandBytes / 16), (uint32_t)(desc_a >> 32),
                (uint32_t)desc_b + stage * (kOperandBytes / 16), (uint32_t)(desc_b >> 32),
                p.idesc, accumulate);
            commit_pair(empty0 + stage * 8);
            accumulate = 1;
            if (++stage == kStages) {
              stage = 0;
              parity ^= 1;
            }
          }
          if (ok) commit_pair(smem_u32(&s.acc_full[buf]));
        }
      }
    };
    if (p.a_transposed) {
      if (p.b_transposed)
        issue(std::true_type(), std::true_type());
      else
        issue(std::true_type(), std::false_type());
    } else {
      if (p.b_transposed)
        issue(std::false_type(), std::true_type());
      else
        issue(std::false_type(), std::false_type());
    }
    commit_pair(smem_u32(&s.drain));         // waited for below: no MMA in flight past that
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    if constexpr (by_chunks(kOut)) regs_claim<kRegsHigh>();
    const int quad = warp & 3, half = (warp - 4) >> 2;
    const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16);
    const int32_t row_in = rank * kRows + quad * 32;            // this warp's rows in the tile
    const uint32_t acc_empty = peer_address(smem_u32(&s.acc_empty[0]), 0);
    // This warp's box, this thread's row of it, and the barrier that counts its residuals.
    const uint32_t box = smem_u32(s.box[warp - 4]);
    const uint32_t box_row = box + lane * 128 + ((lane & 7) << 4);
    const uint32_t box_bar = smem_u32(&s.residual[warp - 4]);
    uint32_t box_parity = 0;
    constexpr int kUnits = kGeglu ? 2 : 4;                      // of 32 columns of out
    constexpr int kPerBox = is_fp32(kOut) ? 1 : 2;              // units in a box
    const bool ahead = by_tma(kOut) && p.e.residual && !p.e.pre;
    int32_t turn = 0;                      // of the accumulators
    bool ok = true;
    Walk w;
    for (bool more = w.at(p, pair); more; more = w.at(p, w.unit + pairs)) {
      int32_t tile_row, tile_col;
      place(p, w.tile, tile_row, tile_col);
      const int32_t row0 = tile_row * kTile + row_in;
      const int32_t col0 = tile_col * kOutCols + half * (kOutCols / 2);
      const bool whole = kOut != kOutSlices && p.slices == 1;
      const bool stored = whole && row0 < p.e.m && col0 < p.e.n;
      bool loading = false;                // the box's residual is on its way
      auto load_residual = [&](int32_t col) {
        if (lane == 0) {
          mbar_arrive_expect_tx(box_bar, kBoxBytes);
          tma_load_2d(box, &maps.residual, box_bar, col, row0);
        }
        loading = true;
      };
      auto take = [&]() {                  // the box that left before has been read
        if (by_tma(kOut) && lane == 0) bulk_wait_read();
        __syncwarp();
      };
      if (stored && ok && ahead) {
        take();
        load_residual(col0);
      }
      // The bias of this half's 128 columns of the accumulator: with geglu 64 of the gate's,
      // then 64 of the up part's. The half's warps meet here for every segment, after a wait
      // that gave up too.
      [[maybe_unused]] float* bias = s.bias[half];
      if constexpr (kOut != kOutSlices) {
        named_barrier(1 + half, 128);        // the segment before has read its own
        {
          const int i = quad * 32 + lane;
          float v = 0.f;
          if (p.e.bias) {
            const int32_t c = kGeglu ? col0 + (i & 63) : col0 + i;
            if (c < p.e.n)
              v = io_get(p.e.bias, kGeglu && i >= 64 ? (int64_t)p.up_row + c : c, is_fp32(kOut));
          }
          bias[i] = v;
        }
        named_barrier(1 + half, 128);
      }
      if (!ok) continue;
      // Columns of accumulator `buf`: 32 u .. of this half (with geglu u = 2, 3 are up's).
      auto columns = [&](uint32_t buf, int u) {
        return lane_base + buf * kTile +
               (kGeglu ? half * 64 + (u & 1) * 32 + (u >> 1) * 128 : half * 128 + u * 32);
      };
      auto hand_back = [&](uint32_t buf) {  // the accumulator has been read
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(acc_empty + buf * 8);
      };
      float sum[by_chunks(kOut) ? kRows : 1];
      uint32_t buf = turn & 1;
      if constexpr (by_chunks(kOut)) {
#pragma unroll
        for (int i = 0; i < kRows; ++i) sum[i] = 0.f;
        for (int32_t block = w.first; block < w.last;
             block = p.chains.end(block, w.last, chunk_of(kOut)), ++turn) {
          buf = turn & 1;
          const float weight = p.chains.weight(block);
          ok = eager_warp_wait(smem_u32(&s.acc_full[buf]), (turn >> 1) & 1, guard, p.status,
                               kSiteEpilogue);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            float z[32];
            load_acc(columns(buf, u), z);
            if (u == 3) hand_back(buf);
#pragma unroll
            for (int i = 0; i < 32; ++i) sum[32 * u + i] = fmaf(z[i], weight, sum[32 * u + i]);
          }
        }
      } else {
        ok = eager_warp_wait(smem_u32(&s.acc_full[buf]), (turn >> 1) & 1, guard, p.status,
                             kSiteEpilogue);
        tc_fence_after();
        ++turn;
      }
      if (!ok) {
        if (loading && lane == 0) mbar_drain_wait(box_bar, box_parity);
        box_parity ^= loading ? 1u : 0u;
        continue;
      }
      auto load = [&](int u, float (&z)[32]) {
        if constexpr (by_chunks(kOut)) {
#pragma unroll
          for (int i = 0; i < 32; ++i) z[i] = sum[32 * u + i];
        } else {
          load_acc(columns(buf, u), z);
        }
      };
      if (!stored) {
        if (!whole) {
          float4* part =
              reinterpret_cast<float4*>(p.parts + (int64_t)w.unit * kPartFloats) +
              (rank * 64 + half * 32) * 128 + quad * 32 + lane;
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            float z[32];
            load(u, z);
#pragma unroll
            for (int g = 0; g < 8; ++g)
              part[(8 * u + g) * 128] =
                  make_float4(z[4 * g], z[4 * g + 1], z[4 * g + 2], z[4 * g + 3]);
          }
        }
        if (!by_chunks(kOut)) hand_back(buf);
        continue;
      }
      // The box to columns `col` .. of a tensor (its map; its address and rows, of p.e.n
      // columns from there on).
      auto leave = [&](const CUtensorMap* map, void* to, int64_t ld, int32_t col) {
        if constexpr (by_tma(kOut)) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && col < p.e.n) {
            tma_store_2d(map, box, col, row0);
            bulk_commit();
          }
        } else {
          __syncwarp();
          box_to_rows<is_fp32(kOut)>(box, lane, to, ld, row0, col, p.e.m - row0, p.e.n - col);
        }
      };
      // Loops over the accumulator's columns stay loops where the sums are not in registers:
      // unrolled, their code pushed the MMA warp's out of the instruction cache.
      if (p.e.pre) {                       // z, before anything else
#pragma unroll(by_chunks(kOut) ? 2 : 1)
        for (int part = 0; part < (kGeglu ? 2 : 1); ++part) {
#pragma unroll(by_chunks(kOut) ? 4 : 1)
          for (int u = 0; u < kUnits; ++u) {
            float z[32];
            load(part * 2 + u, z);
            add_bias(bias + part * 64 + u * 32, z);
            if (u % kPerBox == 0) take();
            put_row<kOut>(box_row, u % kPerBox * 4, z);
            if (u % kPerBox == kPerBox - 1)
              leave(part ? &maps.pre_up : &maps.pre,
                    static_cast<char*>(p.e.pre) + (int64_t)part * p.e.n * (is_fp32(kOut) ? 4 : 2),
                    p.e.pre_ld, col0 + u / kPerBox * kPerBox * 32);
          }
        }
      }
#pragma unroll(by_chunks(kOut) ? 4 : 1)
      for (int u = 0; u < kUnits; ++u) {
        const int32_t col = col0 + u * 32;
        float y[32];
        load(u, y);
        add_bias(bias + u * 32, y);
        if constexpr (kGeglu) {
          apply_gelu<kOut>(y);
          float up[32];
          load(2 + u, up);
          add_bias(bias + 64 + u * 32, up);
#pragma unroll
          for (int i = 0; i < 32; ++i) y[i] *= up[i];
        }
        if (!by_chunks(kOut) && u == kUnits - 1) hand_back(buf);
        if constexpr (!kGeglu) {
          if (p.e.act == PE_ACT_GELU) {
            apply_gelu<kOut>(y);
          } else if (p.e.act == PE_ACT_RELU) {
#pragma unroll
            for (int i = 0; i < 32; ++i) y[i] = y[i] < 0.f ? 0.f : y[i];
          }
        }
        if (u % kPerBox == 0) {
          if (!loading) take();
          if (p.e.residual && col < p.e.n) {
            if constexpr (by_tma(kOut)) {
              if (!loading) load_residual(col);
              ok = eager_warp_wait(box_bar, box_parity, guard, p.status, kSiteResidual);
              if (!ok) break;
              loading = false;
              box_parity ^= 1;
            } else {
              rows_to_box<is_fp32(kOut)>(box, lane, p.e.residual, p.e.residual_ld, row0, col,
                                         p.e.m - row0, p.e.n - col);
              __syncwarp();
            }
          }
        }
        if (p.e.residual) add_row<kOut>(box_row, u % kPerBox * 4, y);
        put_row<kOut>(box_row, u % kPerBox * 4, y);
        if (u % kPerBox == kPerBox - 1)
          leave(&maps.out, p.e.out, p.e.out_ld, col0 + u / kPerBox * kPerBox * 32);
      }
      if (!ok) {                           // the residual did not come in time
        if (lane == 0) mbar_drain_wait(box_bar, box_parity);
        box_parity ^= 1;
      }
    }
    bulk_wait_all();
  }

  griddep_launch_dependents();             // the next kernel may come to wait for this one
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) {
    for (uint32_t to = 0; to < 2; ++to) {
      for (int i = 0; i < 2; ++i)
        store_cluster_i32(peer_address(smem_u32(&s.issued[i][rank]), to), s.loaded[i]);
      store_cluster_i32(peer_address(smem_u32(&s.aborted[rank]), to), s.guard.abort);
    }
  }
  __syncthreads();
  cluster_sync();
  if (threadIdx.x == 0) {
    // The issuing warp's last commit arrives in both CTAs, which stay until it, and so every
    // arrival before it, has reached their barriers.
    mbar_drain_wait(smem_u32(&s.drain), 0);
    bool aborted = false;
    int32_t fewest = s.loaded[0], most = s.loaded[0];
    for (int i = 0; i < 2; ++i) {
      aborted |= s.aborted[i] != 0;
      for (int j = 0; j < 2; ++j) {
        fewest = s.issued[j][i] < fewest ? s.issued[j][i] : fewest;
        most = s.issued[j][i] > most ? s.issued[j][i] : most;
      }
    }
    if (rank == 0 && aborted) {
      // All loading warps have stopped. Blocks that only some of them loaded are put right
      // on this pair's barrier, then every load that may be in flight is waited for.
      for (int32_t i = fewest; i < most; ++i) {
        uint32_t bytes = 0;                // into the pair's CTAs
        for (int j = 0; j < 2; ++j) {
          if (s.issued[0][j] > i) bytes += kOperandBytes;
          if (s.issued[1][j] > i) bytes += kOperandBytes;
        }
        const uint32_t bar = smem_u32(&s.full[i % kStages]);
        if (s.loaded[0] <= i)              // nothing was expected yet
          mbar_arrive_expect_tx(bar, bytes);
        else if (bytes < kPairBytes)
          mbar_complete_tx(bar, kPairBytes - bytes);
      }
      for (int32_t i = most > kStages ? most - kStages : 0; i < most; ++i)
        mbar_drain_wait(smem_u32(&s.full[i % kStages]), (i / kStages) & 1);
    }
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

// Adds the slices' sums of every tile, in the order of k, and finishes them; without slices,
// finishes zeros. One block per 32 rows x 64 columns of the accumulator (32 of the gate, 32
// of the up part with geglu); parts are column-group-major. Small blocks with few sums a
// thread, since what it waits for is L2: 27 tiles of 5 slices in 7 us, in blocks of 128
// columns 9.7.
template <int kAct>
__global__ void __launch_bounds__(256, kPartBlocks)
matmul_parts_kernel(const __grid_constant__ Params p) {
  constexpr bool kGeglu = kAct == PE_ACT_GEGLU;
  constexpr int32_t kOutCols = kGeglu ? kTile / 2 : kTile;
  __shared__ float tile[32][68];
  griddep_wait();                                        // before any block may leave
  const int piece = blockIdx.x & 31;       // 2 CTAs x 4 row quarters x 2 halves x 2 parts
  const int32_t t = blockIdx.x >> 5;
  const int rank = piece >> 4, quad = (piece >> 2) & 3, half = (piece >> 1) & 1;
  const int sub = piece & 1;
  int32_t rt, ct;
  place(p, t, rt, ct);
  const int32_t row0 = rt * kTile + rank * kRows + quad * 32;
  const int32_t col0 = ct * kOutCols + half * (kOutCols / 2) + sub * (kOutCols / 4);
  if (row0 >= p.e.m || col0 >= p.e.n) return;
  const int row = threadIdx.x & 31, g0 = threadIdx.x >> 5;
  // Two groups of four columns: neighbours by 32 columns, or the gate's and the up part's.
  constexpr int kApart = kGeglu ? 16 : 8;
  float4 sum[2] = {};
  const float4* parts = reinterpret_cast<const float4*>(p.parts + (int64_t)t * kPartFloats) +
                        (rank * 64 + half * 32 + sub * (kGeglu ? 8 : 16) + g0) * 128 +
                        quad * 32 + row;
  for (int32_t q = 0; q < p.slices; q += kPartsAhead) {
    float4 v[kPartsAhead][2];
#pragma unroll
    for (int j = 0; j < kPartsAhead; ++j) {
      if (q + j < p.slices) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          v[j][i] = parts[(int64_t)(q + j) * p.tiles * (int64_t)(kPartFloats / 4) +
                          i * kApart * 128];
      }
    }
#pragma unroll
    for (int j = 0; j < kPartsAhead; ++j) {
      if (q + j < p.slices) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          sum[i].x += v[j][i].x;
          sum[i].y += v[j][i].y;
          sum[i].z += v[j][i].z;
          sum[i].w += v[j][i].w;
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) *reinterpret_cast<float4*>(&tile[row][4 * (g0 + 8 * i)]) = sum[i];
  __syncthreads();
  // Four columns of out a thread, the same in all of its rows.
  constexpr int kGroups = kGeglu ? 8 : 16, kStep = 256 / kGroups, kFlight = 32 / kStep;
  const int c = 4 * (threadIdx.x % kGroups), r0 = threadIdx.x / kGroups;
  if (col0 + c >= p.e.n) return;
  const Finish4<kAct> finish(p.e, col0 + c);
  float residual[kFlight][4];
  if (p.e.residual) {
#pragma unroll
    for (int i = 0; i < kFlight; ++i)
      if (row0 + r0 + i * kStep < p.e.m) finish.residual(row0 + r0 + i * kStep, residual[i]);
  }
#pragma unroll
  for (int i = 0; i < kFlight; ++i) {
    const int r = r0 + i * kStep;
    if (row0 + r < p.e.m)
      finish.row(row0 + r, *reinterpret_cast<const float4*>(&tile[r][c]),
                 *reinterpret_cast<const float4*>(&tile[r][kGeglu ? c + 32 : c]), residual[i]);
  }
}

// ---------------------------------------------------------------- host side
Params base_params(const Matmul& q) {
  Params p = {};
  p.e = q.e;
  p.term_blocks = (int32_t)ceil_div(q.k, kMatmulBlock);
  p.terms = q.planes == 3 ? kMaxMatmulTerms : 1;
  p.blocks = p.term_blocks * p.terms;
  p.chains = Chains::of(p.term_blocks, p.terms);
  p.a_transposed = q.a.transposed ? 1 : 0;
  p.b_transposed = q.b.transposed ? 1 : 0;
  const bool geglu = q.e.act == PE_ACT_GEGLU;
  p.up_row = geglu ? q.e.n : 0;
  p.row_tiles = (int32_t)ceil_div(q.m, kTile);
  p.col_tiles = (int32_t)ceil_div(q.e.n, geglu ? kTile / 2 : kTile);
  p.tiles = p.row_tiles * p.col_tiles;
  p.by_band = Divisor::of(kBand * p.col_tiles);
  p.by_tiles = Divisor::of(p.tiles);
  p.idesc = idesc_bf16(256, 256, q.a.transposed, q.b.transposed);
  p.wait_limit_ns = wait_limit_ns();
  return p;
}

pe_status launch_parts(const Params& p, cudaStream_t stream) {
  const auto kernel = p.e.act == PE_ACT_GEGLU  ? matmul_parts_kernel<PE_ACT_GEGLU>
                      : p.e.act == PE_ACT_GELU ? matmul_parts_kernel<PE_ACT_GELU>
                      : p.e.act == PE_ACT_RELU ? matmul_parts_kernel<PE_ACT_RELU>
                                               : matmul_parts_kernel<PE_ACT_NONE>;
  return launch_after_previous(kernel, dim3((unsigned)(32 * p.tiles)), dim3(256), 0, stream, p);
}

pe_status operand_map(CUtensorMap* map, const MatmulOperand& x, int32_t rows, int32_t k,
                      int32_t planes) {
  const auto bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  return x.transposed
             ? matmul_map_planes(map, bf16, 2, x.base, k, rows, x.ld * 2, 64, planes)
             : matmul_map_planes(map, bf16, 2, x.base, rows, k, x.ld * 2, kRows, planes);
}

template <int kOut, bool kGeglu>
pe_status launch_kernel(const Maps& maps, const Params& p, cudaStream_t stream) {
  const auto kernel = matmul_tiles_kernel<kOut, kGeglu>;
  const size_t smem = sizeof(Smem) + 1024;
  static std::atomic<uint64_t> done{0};
  PE_TRY(allow_shared_memory(kernel, static_cast<int>(smem), done));
  if (by_chunks(kOut)) {                     // the register split needs its registers
    static DeviceNumber known;
    const int registers = known.of_current([&] {
      cudaFuncAttributes attr;
      return cudaFuncGetAttributes(&attr, kernel) == cudaSuccess ? attr.numRegs : 0;
    });
    if (registers < 1) return PE_ERR_CUDA;
    if (static_cast<uint32_t>(registers) * kThreads < 128u * (kRegsLow + 2 * kRegsHigh))
      return PE_ERR_UNSUPPORTED;
  }
  const int64_t work = (int64_t)p.tiles * p.slices, fit = device_sm_count() / 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * (work < fit ? work : fit)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  PE_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, maps, p));
  return PE_OK;
}

template <bool kGeglu>
pe_status launch_out(bool boxes, const Maps& maps, const Params& p, cudaStream_t stream) {
  if (p.e.out_fp32 && p.slices > 1) return launch_kernel<kOutSlices, kGeglu>(maps, p, stream);
  if (p.e.out_fp32)
    return boxes ? launch_kernel<kOutFp32, kGeglu>(maps, p, stream)
                 : launch_kernel<kOutFp32Anywhere, kGeglu>(maps, p, stream);
  if (p.terms > 1 || p.slice_blocks + (p.slice_more ? 1 : 0) > kLongest)
    return boxes ? launch_kernel<kOutBf16Long, kGeglu>(maps, p, stream)
                 : launch_kernel<kOutBf16AnywhereLong, kGeglu>(maps, p, stream);
  return boxes ? launch_kernel<kOutBf16, kGeglu>(maps, p, stream)
               : launch_kernel<kOutBf16Anywhere, kGeglu>(maps, p, stream);
}

}  // namespace

size_t matmul_tiles_workspace(int64_t tiles, int32_t slices) {
  return slices > 1 ? (size_t)tiles * (size_t)slices * kPartFloats * sizeof(float) : 0;
}

pe_status matmul_no_sum(const Matmul& q, cudaStream_t stream) {
  return launch_parts(base_params(q), stream);
}

pe_status matmul_tiles(const Matmul& q, int32_t slices, void* workspace,
                       DeviceStatus* status, cudaStream_t stream) {
  Maps maps;
  PE_TRY(operand_map(&maps.a, q.a, q.m, q.k, q.planes));
  PE_TRY(operand_map(&maps.b, q.b, q.n, q.k, q.planes));
  const MatmulEpilogue& e = q.e;
  const bool geglu = e.act == PE_ACT_GEGLU;
  const int size = e.out_fp32 ? 4 : 2;
  auto boxes = [&](const void* x, int64_t ld) {
    return !x || (aligned(x, 16) && ld * size % 16 == 0);
  };
  char* pre_up = static_cast<char*>(e.pre) + (geglu ? (int64_t)e.n * size : 0);
  const bool tma = boxes(e.out, e.out_ld) && boxes(e.residual, e.residual_ld) &&
                   boxes(e.pre, e.pre_ld) && (!e.pre || aligned(pre_up, 16));
  maps.out = maps.residual = maps.pre = maps.pre_up = maps.a;
  if (tma) {
    const auto type = e.out_fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    auto map = [&](CUtensorMap* to, const void* x, int64_t ld) {
      return x ? matmul_map(to, type, size, x, e.m, e.n, ld * size, 32) : PE_OK;
    };
    PE_TRY(map(&maps.out, e.out, e.out_ld));
    PE_TRY(map(&maps.residual, e.residual, e.residual_ld));
    PE_TRY(map(&maps.pre, e.pre, e.pre_ld));
    PE_TRY(map(&maps.pre_up, e.pre ? pre_up : nullptr, e.pre_ld));
  }
  Params p = base_params(q);
  p.slices = slices;
  p.slice_blocks = p.blocks / slices;
  p.slice_more = p.blocks % slices;
  p.status = status;
  p.parts = static_cast<float*>(workspace);
  PE_TRY(geglu ? launch_out<true>(tma, maps, p, stream)
               : launch_out<false>(tma, maps, p, stream));
  return slices == 1 ? PE_OK : launch_parts(p, stream);
}

}  // namespace pe
