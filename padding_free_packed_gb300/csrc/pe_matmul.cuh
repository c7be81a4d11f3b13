// Internal interface of the 16- and 32-bit matrix product's kernels:
//   z = a b^T + bias, out = act(z) + residual, and z itself as pre.
#pragma once

#include "pe_act.cuh"
#include "pe_matmul_fp8.cuh"
#include "pe_sm103.cuh"

namespace pe {

constexpr int kMatmulBlock = 64;           // k's elements in 128 bytes, the swizzle's width

// A product's operand in bf16: `planes` matrices one after the other (three parts of an fp32
// matrix, largest first, or the matrix itself).
struct MatmulOperand {
  const void* base;
  int64_t ld;              // elements
  bool transposed;         // stored [k, rows] instead of [rows, k]
};

// What follows the product. n counts the columns of out; with geglu z has twice as many.
struct MatmulEpilogue {
  const void* bias;        // in out's type, as residual and pre are
  const void* residual;
  void* out;
  void* pre;
  int64_t residual_ld, out_ld, pre_ld;     // elements
  int32_t m, n;
  int32_t act;
  int32_t out_fp32;
  int32_t by_four;         // rows of all of them start at multiples of four elements
};

struct Matmul {
  MatmulOperand a, b;
  int32_t m, n, k;         // n: rows of b
  int32_t planes;          // 1, or 3 with six products of parts
  MatmulEpilogue e;
};

// How a product runs. The choice depends on the sizes alone (the workspace size follows it);
// it counts the 152 SMs of the device these kernels are built for.
struct LinearPlan {
  int32_t rows;            // of a per CTA of the narrow kernel: 16, 32 or 64; 0: tiles
  int32_t split;           // narrow: CTAs of a cluster that share a tile's sum
  int32_t slices;          // tiles: of k, their sums added by a second kernel (1: none)
};

constexpr int kMaxMatmulTerms = 6;
// Products of parts of x = h + m / 2^7 + l / 2^14, the smallest first: l h, h l, m m, m h, h m,
// h h. What a part stands for is at most 2^-8 of the one before it, so what is left out is below
// 2^-23 of |a| |b|.
__host__ __device__ __forceinline__ int32_t term_a(int32_t term, int32_t terms) {
  return (0x001102 >> (4 * (terms == 1 ? 5 : term))) & 3;
}
__host__ __device__ __forceinline__ int32_t term_b(int32_t term, int32_t terms) {
  return (0x010120 >> (4 * (terms == 1 ? 5 : term))) & 3;
}

// The blocks of k that one accumulator sums, a chain: `most` of them, and products of parts that
// count for 2^-14, for 2^-7 and for 1 in chains of their own.
struct Chains {
  int32_t small_end, middle_end;     // one past the blocks that count for 2^-14, for 2^-7

  __host__ static Chains of(int32_t term_blocks, int32_t terms) {
    return terms == 1 ? Chains{0, 0} : Chains{3 * term_blocks, 5 * term_blocks};
  }
  // One past the last block of the chain from `block` on, in a sum that ends before `last`.
  __device__ __forceinline__ int32_t end(int32_t block, int32_t last, int32_t most) const {
    const int32_t end = last - block < most ? last : block + most;
    const int32_t kind = block < small_end ? small_end : block < middle_end ? middle_end : end;
    return kind < end ? kind : end;
  }
  __device__ __forceinline__ float weight(int32_t block) const {
    return block < small_end ? 0x1p-14f : block < middle_end ? 0x1p-7f : 1.f;
  }
};

// Tiles of 256 x 256 (or slices of their sums) on pairs of CTAs.
size_t matmul_tiles_workspace(int64_t tiles, int32_t slices);
pe_status matmul_tiles(const Matmul& p, int32_t slices, void* workspace, DeviceStatus* status,
                       cudaStream_t stream);
// What is left of a product without a sum: z = bias.
pe_status matmul_no_sum(const Matmul& p, cudaStream_t stream);
// Few rows: 128 rows of b by 16, 32 or 64 rows of a per CTA, the sum over k split over a
// cluster.
pe_status matmul_narrow(const Matmul& p, int32_t rows, int32_t split, DeviceStatus* status,
                        cudaStream_t stream);
// fp32 operands as they are, neither transposed, few products.
pe_status matmul_few(const Matmul& p, cudaStream_t stream);

namespace sm103 {

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int32_t x, int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

__device__ __forceinline__ float load_shared_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint4 load_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void store_shared_v4(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
}

// An element of a tensor in out's type.
__device__ __forceinline__ float io_get(const void* p, int64_t at, int32_t fp32) {
  return fp32 ? static_cast<const float*>(p)[at]
              : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[at]);
}
__device__ __forceinline__ void io_put(void* p, int64_t at, int32_t fp32, float v) {
  if (fp32)
    static_cast<float*>(p)[at] = v;
  else
    static_cast<__nv_bfloat16*>(p)[at] = __float2bfloat16_rn(v);
}

// gelu where the result is rounded to fp32; out of line, as it is long.
static __device__ __noinline__ float gelu_fp32(float z) { return gelu<float>(z); }

// Four neighbouring columns of out from their sums (with geglu: gate and up), `count` of them
// inside the matrix; the columns' bias is read once for all rows.
template <int kAct>
struct Finish4 {
  static constexpr bool kGeglu = kAct == PE_ACT_GEGLU;
  const MatmulEpilogue& e;
  int32_t col, count;
  bool four;                 // accesses of four elements
  float bias[4], up_bias[4];

  __device__ Finish4(const MatmulEpilogue& epilogue, int32_t first) : e(epilogue), col(first) {
    count = e.n - col < 4 ? e.n - col : 4;
    four = e.by_four && count == 4;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      bias[j] = up_bias[j] = 0.f;
      if (e.bias && j < count) {
        bias[j] = io_get(e.bias, col + j, e.out_fp32);
        if (kGeglu) up_bias[j] = io_get(e.bias, (int64_t)e.n + col + j, e.out_fp32);
      }
    }
  }
  __device__ void put(void* p, int64_t at, const float (&v)[4], bool by_four) const {
    if (by_four) {
      if (e.out_fp32)
        *reinterpret_cast<float4*>(static_cast<float*>(p) + at) =
            make_float4(v[0], v[1], v[2], v[3]);
      else
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p) + at) =
            make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < count) io_put(p, at + j, e.out_fp32, v[j]);
    }
  }
  // The residual of a row, to be read ahead of the sums.
  __device__ void residual(int64_t row, float (&r)[4]) const {
    const int64_t at = row * e.residual_ld + col;
    if (four) {
      if (e.out_fp32) {
        const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(e.residual) + at);
        r[0] = v.x, r[1] = v.y, r[2] = v.z, r[3] = v.w;
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(
            static_cast<const __nv_bfloat16*>(e.residual) + at);
        r[0] = __uint_as_float(v.x << 16), r[1] = __uint_as_float(v.x & 0xffff0000u);
        r[2] = __uint_as_float(v.y << 16), r[3] = __uint_as_float(v.y & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) r[j] = j < count ? io_get(e.residual, at + j, e.out_fp32) : 0.f;
    }
  }
  __device__ void row(int64_t row, const float4& sum, const float4& up_sum,
                      const float (&r)[4]) const {
    const float z[4] = {sum.x + bias[0], sum.y + bias[1], sum.z + bias[2], sum.w + bias[3]};
    const float u[4] = {up_sum.x + up_bias[0], up_sum.y + up_bias[1], up_sum.z + up_bias[2],
                        up_sum.w + up_bias[3]};
    float y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = z[j];
    if constexpr (kAct == PE_ACT_RELU) {
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = z[j] < 0.f ? 0.f : z[j];
    } else if constexpr (kAct >= PE_ACT_GELU) {
      if (e.out_fp32) {
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = gelu_fp32(z[j]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; j += 2)
          f2_split(GeluPair(z[j], z[j + 1]).value(z[j], z[j + 1]), y[j], y[j + 1]);
      }
      if constexpr (kGeglu) {
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] *= u[j];
      }
    }
    if (e.residual) {
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] += r[j];
    }
    if (e.pre) {
      put(e.pre, row * e.pre_ld + col, z, four);
      if (kGeglu) put(e.pre, row * e.pre_ld + e.n + col, u, four && e.n % 4 == 0);
    }
    put(e.out, row * e.out_ld + col, y, four);
  }
};

}  // namespace sm103
}  // namespace pe
