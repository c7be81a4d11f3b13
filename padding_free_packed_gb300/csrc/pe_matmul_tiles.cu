// Matrix product with bias, activation and residual, many rows:
// out = act(a b^T + bias) + residual.
//
// A pair of CTAs (tcgen05 cta_group::2) works on a 256 x 256 tile: each CTA loads 128 rows of
// a and 128 rows of b, 64 elements of k at a time, and the pair's MMAs (M = 256, N = 256, K =
// 16) sum a tile over the whole of k in tensor memory. Two accumulators take turns, so the
// epilogue of a tile runs under the next tile's MMAs. An operand stored with k as its rows is
// loaded in boxes of 64 columns by 64 rows and read by the MMA as it lies there.
//
//   warp 0       TMA producer (both CTAs), a ring of kStages blocks
//   warp 1       MMA issue (first CTA of the pair)
//   warps 4-11   epilogue; warps 4-7 the tile's left half, 8-11 its right half: bias, z into
//                pre, activation, residual (loaded by TMA into the box that the result then
//                leaves from), rounding, TMA stores of 32 rows x 128 bytes
//
// With geglu the tile is 128 columns of out: the first CTA loads their gate rows of b, the
// second their up rows, so that a thread finds both in its row of tensor memory.
//
// fp32 operands come as three bf16 parts each, and six products of parts, the smallest
// first, are summed in the same accumulator, as six times as many blocks of k.
//
// Work: whole tiles in turn, or, where few tiles have long sums, equal runs of consecutive
// blocks of k (a run may start and end inside a tile); a tile that several pairs share is
// then summed from their fp32 parts, in the order of k, by a second kernel, which also does
// the epilogue.
#include "pe_matmul.cuh"

namespace pe {

namespace {

using namespace sm103;

constexpr int kTile = 256;
constexpr int kRows = 128;                               // rows of a (and of b) per CTA
constexpr int kStages = 5;
constexpr int kThreads = 384;
constexpr uint32_t kOperandBytes = kRows * 128;          // 16 KiB
constexpr uint32_t kPairBytes = 4 * kOperandBytes;       // both CTAs' a and b of one block
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kBoxBytes = 32 * 128;                 // 32 rows of 128 bytes
// How rows of out, residual and pre are moved: boxes by TMA or, where rows start anywhere,
// element by element.
enum Out { kOutBf16 = 0, kOutFp32 = 1, kOutBf16Anywhere = 2, kOutFp32Anywhere = 3 };
constexpr bool is_fp32(int out) { return out & 1; }
constexpr bool by_boxes(int out) { return out < 2; }

constexpr uint32_t kRegsLaunch = 168;
constexpr uint32_t kRegsLow = 40, kRegsHigh = 232;
static_assert(128 * (kRegsLow + 2 * kRegsHigh) <= kThreads * kRegsLaunch,
              "register split exceeds the launch allocation");
// Blocks of k that one accumulator sums: all of them for results rounded to bf16; for fp32
// results a few, whose sums are then added in fp32 registers. The tensor cores cut the sum
// off after every 16 products (1.7e-8 of it a time, always towards zero, measured), which a
// chain of 11500 products turned into 1.2e-5 of the result; this way it stays at 3e-7.
constexpr int32_t kChunk = 4;
constexpr int32_t chunk_of(int out) { return is_fp32(out) ? kChunk : 0x7fffffff; }
constexpr int kMaxPairs = 80;
constexpr size_t kPartFloats = (size_t)kTile * kTile;

struct alignas(1024) Smem {
  uint8_t a[kStages][kOperandBytes];
  uint8_t b[kStages][kOperandBytes];
  alignas(1024) uint8_t box[8][2][kBoxBytes];  // of each epilogue warp
  alignas(16) float bias[2][kRows];            // of each half of the tile
  uint64_t full[kStages], empty[kStages];      // full: the first CTA's serve the pair
  uint64_t acc_full[2], acc_empty[2];          // acc_empty: likewise
  uint64_t residual[8][2];                     // a box's residual has arrived
  uint64_t drain;
  int32_t issued[2];                           // blocks each CTA's producer loaded (first CTA)
  int32_t aborted[2];
  uint32_t tmem_base;
  WaitGuard guard;
};
static_assert(sizeof(Smem) + 1024 <= 227 * 1024, "shared memory exceeds the per-CTA limit");

struct Params {
  MatmulEpilogue e;
  int32_t blocks;            // of k, of all terms
  int32_t term_blocks;       // of one term
  int32_t terms;
  int32_t a_transposed, b_transposed;
  int32_t up_row;            // geglu: b's first up row
  int32_t col_tiles;
  int32_t tiles;
  int32_t shared_tiles;      // 1: runs of blocks, partial tiles through `parts`
  int32_t run_blocks;        // blocks of every pair's run, and
  int32_t run_more;          // how many pairs get one more
  uint32_t idesc;
  float* parts;              // [2 * pairs][2 CTAs][2 halves][32 column groups][128 rows] float4
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
// Tile load into this CTA, counted on a barrier of the pair's first CTA.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                              int32_t x, int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
// Both are executed by a whole warp with the same operands; one lane issues.
__device__ __forceinline__ void mma_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                         uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b32 r;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "elect.sync r|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
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
__device__ __forceinline__ void bulk_wait_read_but_one() {
  asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
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

// An epilogue warp's boxes: two in turn. A box is filled by the warp's threads (or first by
// a load of the residual) and leaves by a TMA store of its own bulk group.
struct Boxes {
  uint32_t base;                  // of this warp's two boxes
  uint32_t bars;                  // their barriers
  uint32_t phases;                // bit s: parity of slot s's next arrival
  int lane;

  __device__ uint32_t at(int slot) const { return base + slot * kBoxBytes; }
  // This thread's row of a box.
  __device__ uint32_t row(int slot) const { return at(slot) + lane * 128 + ((lane & 7) << 4); }
  __device__ void load(int slot, const CUtensorMap* map, int32_t x, int32_t y) const {
    mbar_arrive_expect_tx(bars + slot * 8, kBoxBytes);
    tma_load_2d(at(slot), map, bars + slot * 8, x, y);
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

// 32 columns of the warp's 32 rows through a box, then row by row, element by element: a
// row's 32 columns are consecutive. `cols` of them exist.
template <bool kFp32>
__device__ __forceinline__ void put_anywhere(const Params& p, uint32_t box, int lane,
                                             const float (&x)[32], const void* residual,
                                             int64_t residual_ld, void* out, int64_t out_ld,
                                             int32_t row0, int64_t col0, int32_t cols) {
  __syncwarp();
  put_row<kOutFp32>(box + lane * 128 + ((lane & 7) << 4), 0, x);
  __syncwarp();
  const int32_t rows = lane < cols ? p.e.m - row0 : 0;
#pragma unroll 1
  for (int32_t r0 = 0; r0 < 32; r0 += 8) {               // eight reads in flight
    float v[8];
#pragma unroll
    for (int32_t r = 0; r < 8; ++r) {
      v[r] = load_shared_f32(box + (r0 + r) * 128 + (((lane >> 2) ^ r) << 4) + (lane & 3) * 4);
      if (residual && r0 + r < rows)
        v[r] += io_get(residual, (int64_t)(row0 + r0 + r) * residual_ld + col0 + lane, kFp32);
    }
#pragma unroll
    for (int32_t r = 0; r < 8; ++r)
      if (r0 + r < rows)
        io_put(out, (int64_t)(row0 + r0 + r) * out_ld + col0 + lane, kFp32, v[r]);
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
__device__ __forceinline__ void add_bias(const float* bias, float (&z)[32]) {
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    const float4 b = *reinterpret_cast<const float4*>(bias + 4 * g);
    z[4 * g] += b.x;
    z[4 * g + 1] += b.y;
    z[4 * g + 2] += b.z;
    z[4 * g + 3] += b.w;
  }
}

template <int kOut>
__device__ __forceinline__ void apply_gelu(float (&z)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) z[i] = is_fp32(kOut) ? gelu_fp32(z[i]) : gelu<__nv_bfloat16>(z[i]);
}

template <int kOut, bool kGeglu>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
matmul_tiles_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
  extern __shared__ uint8_t raw[];
  Smem& s = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int32_t pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
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
    for (int i = 0; i < 16; ++i) mbar_init(smem_u32(&s.residual[i >> 1][i & 1]), 1);
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
  cluster_sync();                          // barriers of both CTAs exist before any arrival
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;

  if (is_fp32(kOut) && warp < 4) regs_release<kRegsLow>();
  if (warp == 0) {
    if (lane == 0) {
      // ---------------------------------------------------------- producer
      const uint32_t full0 = peer_address(smem_u32(&s.full[0]), 0);
      int32_t issued = 0, stage = 0;
      uint32_t parity = 1;
      bool ok = true;
      Walk w;
      for (bool more = w.start(p, pair, pairs); more && ok; more = w.next(p)) {
        const int32_t rt = w.tile / p.col_tiles, ct = w.tile - rt * p.col_tiles;
        const int32_t row = rt * kTile + (int32_t)rank * kRows;
        const int32_t col = kGeglu ? ct * kOutCols + (rank ? p.up_row : 0)
                                   : ct * kTile + (int32_t)rank * kRows;
        int32_t term = w.first / p.term_blocks;
        int32_t x = (w.first - term * p.term_blocks) * kMatmulBlock;
        const int32_t x_end = p.term_blocks * kMatmulBlock;
        for (int32_t block = w.first; block < w.last; ++block) {
          ok = eager_wait(smem_u32(&s.empty[stage]), parity, guard, p.status, kSiteProducer);
          if (!ok) break;
          const uint32_t bar = full0 + stage * 8;
          const uint32_t sa = smem_u32(s.a[stage]), sb = smem_u32(s.b[stage]);
          const int32_t pa = term_a(term, p.terms), pb = term_b(term, p.terms);
          if (rank == 0) mbar_arrive_expect_tx(smem_u32(&s.full[stage]), kPairBytes);
          if (p.a_transposed) {
            tma_load_pair(sa, &maps.a, bar, row, x, pa);
            tma_load_pair(sa + kOperandBytes / 2, &maps.a, bar, row + 64, x, pa);
          } else {
            tma_load_pair(sa, &maps.a, bar, x, row, pa);
          }
          if (p.b_transposed) {
            tma_load_pair(sb, &maps.b, bar, col, x, pb);
            tma_load_pair(sb + kOperandBytes / 2, &maps.b, bar, col + 64, x, pb);
          } else {
            tma_load_pair(sb, &maps.b, bar, x, col, pb);
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
          }
        }
      }
      store_cluster_i32(peer_address(smem_u32(&s.issued[rank]), 0), issued);
    }
    __syncwarp();
  } else if (warp == 1 && rank == 0) {
    // ------------------------------------------------------------ MMA issue
    // 16 elements of k: 32 bytes along rows of k, or 16 rows of 128 bytes; an operand's next
    // 64 columns, where k runs along its rows, are the stage's second half.
    const uint64_t desc_a0 = smem_desc_sw128(smem_u32(s.a[0]), p.a_transposed ? 8192 : 16, 1024);
    const uint64_t desc_b0 = smem_desc_sw128(smem_u32(s.b[0]), p.b_transposed ? 8192 : 16, 1024);
    const uint32_t step_a = p.a_transposed ? 128 : 2, step_b = p.b_transposed ? 128 : 2;
    uint32_t stage = 0, parity = 0;
    int32_t turn = 0;                      // of the accumulators
    bool ok = true;
    Walk w;
    for (bool more = w.start(p, pair, pairs); more && ok; more = w.next(p)) {
      for (int32_t block = w.first; block < w.last && ok; ++turn) {
        const uint32_t buf = turn & 1, d = tmem + buf * kTile;
        const int32_t first = block;
        const int32_t end = w.last - first < chunk_of(kOut) ? w.last : first + chunk_of(kOut);
        ok = eager_warp_wait(smem_u32(&s.acc_empty[buf]), ((turn >> 1) & 1) ^ 1, guard, p.status,
                             kSiteMma);
        for (; block < end && ok; ++block) {
          ok = eager_warp_wait(smem_u32(&s.full[stage]), parity, guard, p.status, kSiteMma);
          if (!ok) break;
          tc_fence_after();
          const uint64_t da = desc_a0 + stage * (kOperandBytes / 16);
          const uint64_t db = desc_b0 + stage * (kOperandBytes / 16);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_pair(d, da + k * step_a, db + k * step_b, p.idesc, k > 0 || block > first);
          commit_pair(smem_u32(&s.empty[stage]));
          if (++stage == kStages) {
            stage = 0;
            parity ^= 1;
          }
        }
        if (ok) commit_pair(smem_u32(&s.acc_full[buf]));
      }
    }
    commit_pair(smem_u32(&s.drain));       // no MMA is in flight past this
    mbar_drain_wait(smem_u32(&s.drain), 0);
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    if constexpr (is_fp32(kOut)) regs_claim<kRegsHigh>();
    const int quad = warp & 3, half = (warp - 4) >> 2;
    const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16);
    const int32_t row_in = (int32_t)rank * kRows + quad * 32;   // this warp's rows in the tile
    const uint32_t acc_empty = peer_address(smem_u32(&s.acc_empty[0]), 0);
    Boxes boxes = {smem_u32(s.box[warp - 4][0]), smem_u32(&s.residual[warp - 4][0]), 0, lane};
    constexpr int kUnits = kGeglu ? 2 : 4;                      // of 32 columns of out
    constexpr int kPerBox = is_fp32(kOut) ? 1 : 2;              // units in a box
    const bool ahead = by_boxes(kOut) && p.e.residual && !p.e.pre;
    int32_t turn = 0;                      // of the accumulators
    bool begins = true;                    // the pair's first segment
    bool ok = true;
    Walk w;
    for (bool more = w.start(p, pair, pairs); more; more = w.next(p), begins = false) {
      const int32_t rt = w.tile / p.col_tiles, ct = w.tile - rt * p.col_tiles;
      const int32_t row0 = rt * kTile + row_in;
      const int32_t col0 = ct * kOutCols + half * (kOutCols / 2);
      const bool whole = w.first == 0 && w.last == p.blocks;
      const bool stored = whole && row0 < p.e.m && col0 < p.e.n;
      uint32_t loading = 0;                // bit s: slot s's residual is on its way
      if (stored && ok) {
        if (by_boxes(kOut)) {
          if (lane == 0) bulk_wait_read();                      // the tile before has left
          __syncwarp();
        }
        if (ahead) {
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const int32_t col = col0 + b * kPerBox * 32;
            if (b * kPerBox < kUnits && col < p.e.n) {
              if (lane == 0) boxes.load(b, &maps.residual, col, row0);
              loading |= 1u << b;
            }
          }
        }
      }
      // The bias of this half's 128 columns of the accumulator: with geglu 64 of the gate's,
      // then 64 of the up part's. The half's warps meet here for every segment, after a wait
      // that gave up too.
      float* bias = s.bias[half];
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
      float sum[is_fp32(kOut) ? kRows : 1];
      uint32_t buf = turn & 1;
      if constexpr (is_fp32(kOut)) {
#pragma unroll
        for (int i = 0; i < kRows; ++i) sum[i] = 0.f;
        for (int32_t block = w.first; block < w.last; block += kChunk, ++turn) {
          buf = turn & 1;
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
            for (int i = 0; i < 32; ++i) sum[32 * u + i] += z[i];
          }
        }
      } else {
        ok = eager_warp_wait(smem_u32(&s.acc_full[buf]), (turn >> 1) & 1, guard, p.status,
                             kSiteEpilogue);
        tc_fence_after();
        ++turn;
      }
      if (!ok) {
        if (lane == 0) {
#pragma unroll
          for (int b = 0; b < 2; ++b)
            if (loading >> b & 1) mbar_drain_wait(boxes.bars + b * 8, boxes.phases >> b & 1);
        }
        continue;
      }
      auto load = [&](int u, float (&z)[32]) {
        if constexpr (is_fp32(kOut)) {
#pragma unroll
          for (int i = 0; i < 32; ++i) z[i] = sum[32 * u + i];
        } else {
          load_acc(columns(buf, u), z);
        }
      };
      if (!stored) {
        if (!whole) {
          float4* part =
              reinterpret_cast<float4*>(p.parts + (2 * pair + (begins ? 0 : 1)) * kPartFloats) +
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
        if (!is_fp32(kOut)) hand_back(buf);
        continue;
      }
      int box = 0;                         // of this tile: slots in turn
      auto take = [&]() {                  // waits until the box's slot has been read
        if (by_boxes(kOut) && box >= 2) {
          if (lane == 0) bulk_wait_read_but_one();
          __syncwarp();
        }
      };
      auto leave = [&](const CUtensorMap* map, int32_t col, int32_t cols) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (col < cols) tma_store_2d(map, boxes.at(box & 1), col, row0);
          bulk_commit();                   // a group for every box, so that take() counts them
        }
        ++box;
      };
      if (p.e.pre) {                       // z, before anything else
#pragma unroll
        for (int part = 0; part < (kGeglu ? 2 : 1); ++part) {
#pragma unroll
          for (int u = 0; u < kUnits; ++u) {
            float z[32];
            load(part * 2 + u, z);
            add_bias(bias + part * 64 + u * 32, z);
            const int32_t col = col0 + u * 32;
            if constexpr (!by_boxes(kOut)) {
              put_anywhere<is_fp32(kOut)>(p, boxes.at(0), lane, z, nullptr, 0, p.e.pre, p.e.pre_ld, row0,
                           (int64_t)part * p.e.n + col, p.e.n - col);
            } else {
              if (u % kPerBox == 0) take();
              put_row<kOut>(boxes.row(box & 1), u % kPerBox * 4, z);
              if (u % kPerBox == kPerBox - 1)
                leave(part ? &maps.pre_up : &maps.pre, col0 + u / kPerBox * kPerBox * 32, p.e.n);
            }
          }
        }
      }
#pragma unroll
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
        if (!is_fp32(kOut) && u == kUnits - 1) hand_back(buf);
        if constexpr (!kGeglu) {
          if (p.e.act == PE_ACT_GELU) {
            apply_gelu<kOut>(y);
          } else if (p.e.act == PE_ACT_RELU) {
#pragma unroll
            for (int i = 0; i < 32; ++i) y[i] = y[i] < 0.f ? 0.f : y[i];
          }
        }
        if constexpr (!by_boxes(kOut)) {
          put_anywhere<is_fp32(kOut)>(p, boxes.at(0), lane, y, p.e.residual, p.e.residual_ld, p.e.out,
                       p.e.out_ld, row0, col, p.e.n - col);
        } else {
          const int slot = box & 1;
          if (u % kPerBox == 0) {
            take();
            const int32_t box_col = col;
            if (p.e.residual && box_col < p.e.n) {
              if (!(loading >> slot & 1) && lane == 0)
                boxes.load(slot, &maps.residual, box_col, row0);
              loading &= ~(1u << slot);
              ok = eager_warp_wait(boxes.bars + slot * 8, boxes.phases >> slot & 1, guard,
                                   p.status, kSiteResidual);
              boxes.phases ^= 1u << slot;
              if (!ok) break;
            }
          }
          if (p.e.residual) add_row<kOut>(boxes.row(slot), u % kPerBox * 4, y);
          put_row<kOut>(boxes.row(slot), u % kPerBox * 4, y);
          if (u % kPerBox == kPerBox - 1)
            leave(&maps.out, col0 + u / kPerBox * kPerBox * 32, p.e.n);
        }
      }
      if (!ok) {                           // the residual did not come in time
        if (lane == 0) {
          // This slot's arrival was counted above; the other's may be on its way too.
          const int slot = box & 1;
          mbar_drain_wait(boxes.bars + slot * 8, (boxes.phases >> slot & 1) ^ 1);
          if (loading >> (slot ^ 1) & 1)
            mbar_drain_wait(boxes.bars + (slot ^ 1) * 8, boxes.phases >> (slot ^ 1) & 1);
        }
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
  // The issuing warp's last commits arrive in both CTAs: the second stays until they,
  // and so every arrival before them, have reached its barriers.
  if (rank == 1 && threadIdx.x == 0) mbar_drain_wait(smem_u32(&s.drain), 0);
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

// Sums the parts of every tile that several pairs share, in the order of k, and finishes
// them; without blocks of k, finishes zeros. One block per 32 rows x 128 columns of the
// accumulator (64 of the gate, 64 of the up part with geglu); parts are column-group-major.
template <bool kGeglu>
__global__ void __launch_bounds__(256)
matmul_parts_kernel(const __grid_constant__ Params p, int32_t pairs) {
  constexpr int32_t kOutCols = kGeglu ? kTile / 2 : kTile;
  __shared__ float tile[32][132];
  griddep_wait();                                        // before any block may leave
  const int piece = blockIdx.x & 15;                     // 2 CTAs x 4 row quarters x 2 halves
  const int32_t t = blockIdx.x >> 4;
  const int rank = piece >> 3, quad = (piece >> 1) & 3, half = piece & 1;
  const int32_t rt = t / p.col_tiles, ct = t - rt * p.col_tiles;
  const int32_t row0 = rt * kTile + rank * kRows + quad * 32;
  const int32_t col0 = ct * kOutCols + half * (kOutCols / 2);
  if (row0 >= p.e.m || col0 >= p.e.n) return;
  const int row = threadIdx.x & 31, g0 = threadIdx.x >> 5;
  float4 sum[4] = {};
  if (p.blocks) {
    const int32_t lo = t * p.blocks, hi = lo + p.blocks; // the tile's blocks
    // Pair q holds block `lo`: run_start(q) <= lo < run_start(q + 1).
    const int32_t long_end = p.run_more * (p.run_blocks + 1);
    int32_t q = lo < long_end ? lo / (p.run_blocks + 1)
                              : p.run_more + (lo - long_end) / p.run_blocks;
    if (run_start(p, q + 1) >= hi) return;               // one pair wrote the whole tile
    const float4* parts = reinterpret_cast<const float4*>(p.parts) +
                          (rank * 64 + half * 32) * 128 + quad * 32 + row + g0 * 128;
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
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) *reinterpret_cast<float4*>(&tile[row][4 * (g0 + 8 * i)]) = sum[i];
  __syncthreads();
  // Four columns of out a thread.
  constexpr int kGroups = kGeglu ? 16 : 32;
  for (int e = threadIdx.x; e < 32 * kGroups; e += 256) {
    const int r = e / kGroups, c = 4 * (e % kGroups);
    if (row0 + r < p.e.m && col0 + c < p.e.n) {
      const float4 z = *reinterpret_cast<const float4*>(&tile[r][c]);
      const float4 u = *reinterpret_cast<const float4*>(&tile[r][kGeglu ? c + 64 : c]);
      const float zs[4] = {z.x, z.y, z.z, z.w}, us[4] = {u.x, u.y, u.z, u.w};
      finish4(p.e, row0 + r, col0 + c, p.e.n - col0 - c, zs, us);
    }
  }
}

// ---------------------------------------------------------------- host side
int32_t pair_count() {
  const int32_t n = device_sm_count() / 2;
  return n < kMaxPairs ? n : kMaxPairs;
}

Params base_params(const Matmul& q) {
  Params p = {};
  p.e = q.e;
  p.term_blocks = (int32_t)ceil_div(q.k, kMatmulBlock);
  p.terms = q.planes == 3 ? kMaxMatmulTerms : 1;
  p.blocks = p.term_blocks * p.terms;
  p.a_transposed = q.a.transposed ? 1 : 0;
  p.b_transposed = q.b.transposed ? 1 : 0;
  const bool geglu = q.e.act == PE_ACT_GEGLU;
  p.up_row = geglu ? q.e.n : 0;
  p.col_tiles = (int32_t)ceil_div(q.e.n, geglu ? kTile / 2 : kTile);
  p.tiles = (int32_t)(ceil_div(q.m, kTile) * p.col_tiles);
  p.idesc = idesc_bf16(256, 256, q.a.transposed, q.b.transposed);
  p.wait_limit_ns = wait_limit_ns();
  return p;
}

template <bool kGeglu>
pe_status launch_parts(const Params& p, int32_t pairs, cudaStream_t stream) {
  return launch_after_previous(matmul_parts_kernel<kGeglu>, dim3((unsigned)(16 * p.tiles)),
                               dim3(256), 0, stream, p, pairs);
}

pe_status operand_map(CUtensorMap* map, const MatmulOperand& x, int32_t rows, int32_t k,
                      int32_t planes) {
  if (x.transposed)
    return matmul_map_planes(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, x.base, k, rows, x.ld * 2,
                             64, planes);
  return matmul_map_planes(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, x.base, rows, k, x.ld * 2,
                           kRows, planes);
}

template <int kOut, bool kGeglu>
pe_status launch_tiles(const Maps& maps, const Params& p, int32_t pairs, cudaStream_t stream) {
  const auto kernel = matmul_tiles_kernel<kOut, kGeglu>;
  const size_t smem = sizeof(Smem) + 1024;
  PE_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   static_cast<int>(smem)));
  if (is_fp32(kOut)) {
    cudaFuncAttributes attr;
    PE_CUDA_TRY(cudaFuncGetAttributes(&attr, kernel));
    if (static_cast<uint32_t>(attr.numRegs) * kThreads < 128u * (kRegsLow + 2 * kRegsHigh))
      return PE_ERR_UNSUPPORTED;
  }
  PE_TRY(launch_after_previous(kernel, dim3((unsigned)(2 * pairs)), dim3(kThreads), smem, stream,
                               maps, p));
  return p.shared_tiles ? launch_parts<kGeglu>(p, pairs, stream) : PE_OK;
}

template <bool kGeglu>
pe_status launch_out(bool boxes, const Maps& maps, const Params& p, int32_t pairs,
                     cudaStream_t stream) {
  if (p.e.out_fp32)
    return boxes ? launch_tiles<kOutFp32, kGeglu>(maps, p, pairs, stream)
                 : launch_tiles<kOutFp32Anywhere, kGeglu>(maps, p, pairs, stream);
  return boxes ? launch_tiles<kOutBf16, kGeglu>(maps, p, pairs, stream)
               : launch_tiles<kOutBf16Anywhere, kGeglu>(maps, p, pairs, stream);
}

}  // namespace

size_t matmul_tiles_workspace() { return 2 * kMaxPairs * kPartFloats * sizeof(float); }

pe_status matmul_no_sum(const Matmul& q, cudaStream_t stream) {
  const Params p = base_params(q);
  return q.e.act == PE_ACT_GEGLU ? launch_parts<true>(p, 0, stream)
                                 : launch_parts<false>(p, 0, stream);
}

pe_status matmul_tiles(const Matmul& q, bool runs, void* workspace, DeviceStatus* status,
                       cudaStream_t stream) {
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
  p.status = status;
  p.parts = static_cast<float*>(workspace);
  int32_t pairs = pair_count();
  p.shared_tiles = runs ? 1 : 0;
  p.run_blocks = (int32_t)((int64_t)p.tiles * p.blocks / pairs);
  p.run_more = (int32_t)((int64_t)p.tiles * p.blocks % pairs);
  if (!p.shared_tiles && p.tiles < pairs) pairs = p.tiles;
  return geglu ? launch_out<true>(tma, maps, p, pairs, stream)
               : launch_out<false>(tma, maps, p, pairs, stream);
}

}  // namespace pe
