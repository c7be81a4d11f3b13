// Matrix product with bias, activation and residual in 16 and 32 bits: the C entry, the
// choice among the kernels, and the parts of fp32 operands.
#include <math.h>

#include "pe_matmul.cuh"

namespace pe {

namespace {

// The kernels hold row, column and k coordinates of whole tiles in int32, and count blocks of
// 256 x 128 (columns of out with geglu) x 64 in int32, six times with fp32 operands; 32 thread
// blocks a tile of 256 columns stay below 2^31, since three blocks of 128 make two tiles.
constexpr int64_t kMaxSize = (1LL << 31) - 1024;
bool sizes_ok(int64_t m, int64_t n, int64_t k) {
  constexpr int64_t kMaxBlocks = 1LL << 29;
  if (m >= kMaxSize || n >= kMaxSize || k >= kMaxSize / kMaxMatmulTerms) return false;
  if (m == 0 || n == 0) return true;
  const int64_t blocks = k == 0 ? 1 : ceil_div(k, kMatmulBlock);
  return ceil_div(m, 256) * ceil_div(n, 128) <= (kMaxBlocks - 1) / (blocks * kMaxMatmulTerms);
}

// ---------------------------------------------------------------- parts of fp32 operands
// x = h + m / 2^7 + l / 2^14 with h, m and l in bf16: h is x rounded to bf16 (cut off where that
// would leave the range), m the rest rounded, l what is left of that. All differences are exact,
// and l holds the last of x's 24 bits. The rest is up to 2^-8 of x, and what is left up to 2^-17,
// so held as they are they would lose bits below 2^-133, the last bit of bf16, from |x| = 2^-110
// on; held that much larger none is above |x|, an |x| of 2^-124 or more loses nothing, and a
// smaller one at most 2^-148. An infinity or a NaN has NaN for all three, since the products of
// an infinite h with another operand's parts of zero would be NaN in any case.
__device__ __forceinline__ void parts_of(float x, float& h, float& m, float& l) {
  const float r = __bfloat162float(__float2bfloat16_rn(x));
  h = fabsf(r) <= 3.3895314e38f ? r : __uint_as_float(__float_as_uint(x) & 0xffff0000u);
  m = __bfloat162float(__float2bfloat16_rn((x - h) * 0x1p7f));
  l = ((x - h) - m * 0x1p-7f) * 0x1p14f;
  if (!(fabsf(x) <= 3.402823466e38f)) h = m = l = __uint_as_float(0x7fc00000u);
}

struct SplitOperand {
  const float* x;
  int64_t ld;                // elements
  int64_t rows, cols;        // as stored
  __nv_bfloat16* parts;      // [3][rows][part_ld]
  int64_t part_ld;           // cols rounded up to 8
  int32_t vector;            // rows of x start at multiples of 16 bytes
};

constexpr int kSplitThreads = 256;

// Eight neighbouring columns a thread: a bandwidth kernel, 4 bytes read and 6 written an
// element. The first `a_blocks` blocks take a, the others b.
__global__ void __launch_bounds__(kSplitThreads)
split_kernel(const SplitOperand a, const SplitOperand b, unsigned a_blocks) {
  const bool second = blockIdx.x >= a_blocks;
  const SplitOperand& o = second ? b : a;
  const int64_t block = second ? blockIdx.x - a_blocks : blockIdx.x;
  const int64_t blocks = second ? gridDim.x - a_blocks : a_blocks;
  const int64_t groups = o.part_ld / 8, total = o.rows * groups;
  griddep_wait();
  griddep_launch_dependents();             // the product may come to wait for this kernel
  for (int64_t i = block * kSplitThreads + threadIdx.x; i < total; i += blocks * kSplitThreads) {
    const int64_t row = i / groups;
    const int64_t c = (i - row * groups) * 8;
    const float* src = o.x + row * o.ld + c;
    float v[8];
    if (o.vector && c + 8 <= o.cols) {
      const float4 p = *reinterpret_cast<const float4*>(src);
      const float4 q = *reinterpret_cast<const float4*>(src + 4);
      v[0] = p.x, v[1] = p.y, v[2] = p.z, v[3] = p.w;
      v[4] = q.x, v[5] = q.y, v[6] = q.z, v[7] = q.w;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = c + j < o.cols ? src[j] : 0.f;
    }
    uint32_t w[3][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float h[2], m[2], l[2];
      parts_of(v[2 * j], h[0], m[0], l[0]);
      parts_of(v[2 * j + 1], h[1], m[1], l[1]);
      w[0][j] = sm103::pack_bf16x2(h[0], h[1]);
      w[1][j] = sm103::pack_bf16x2(m[0], m[1]);
      w[2][j] = sm103::pack_bf16x2(l[0], l[1]);
    }
    const int64_t to = row * o.part_ld + c, plane = o.rows * o.part_ld;
#pragma unroll
    for (int j = 0; j < 3; ++j)
      *reinterpret_cast<uint4*>(o.parts + j * plane + to) =
          make_uint4(w[j][0], w[j][1], w[j][2], w[j][3]);
  }
}

int64_t round_up(int64_t x, int64_t to) { return ceil_div(x, to) * to; }
// Bytes of a matrix's three parts, each matrix starting at a multiple of 16.
int64_t part_bytes(int64_t rows, int64_t cols) { return 3 * rows * round_up(cols, 8) * 2; }
int64_t split_bytes(int64_t m, int64_t n, int64_t k, bool a_t, bool b_t) {
  return (a_t ? part_bytes(k, m) : part_bytes(m, k)) + (b_t ? part_bytes(k, n) : part_bytes(n, k));
}

pe_status split(Matmul& p, void* parts, cudaStream_t stream) {
  char* at = static_cast<char*>(parts);
  SplitOperand s[2];
  unsigned blocks[2];
  for (int i = 0; i < 2; ++i) {
    MatmulOperand& x = i ? p.b : p.a;
    const int64_t rows = i ? p.n : p.m;
    s[i].x = static_cast<const float*>(x.base);
    s[i].ld = x.ld;
    s[i].rows = x.transposed ? p.k : rows;
    s[i].cols = x.transposed ? rows : p.k;
    s[i].parts = reinterpret_cast<__nv_bfloat16*>(at);
    s[i].part_ld = round_up(s[i].cols, 8);
    s[i].vector = x.ld % 4 == 0 && aligned(x.base, 16);
    at += part_bytes(s[i].rows, s[i].cols);
    const int64_t need = ceil_div(s[i].rows * s[i].part_ld / 8, kSplitThreads);
    const int64_t most = (int64_t)device_sm_count() * 8;
    blocks[i] = (unsigned)(need < most ? need : most);
    x.base = s[i].parts;
    x.ld = s[i].part_ld;
  }
  p.planes = 3;
  return launch_after_previous(split_kernel, dim3(blocks[0] + blocks[1]), dim3(kSplitThreads), 0,
                               stream, s[0], s[1], blocks[0]);
}

// ---------------------------------------------------------------- the choice
int64_t tile_count(int64_t m, int64_t n) { return ceil_div(m, 256) * ceil_div(n, 256); }

// Estimated microseconds of every way, from times measured on a GB300 (m x n x k, bf16; T:
// rows of a per CTA, S: split; tiles: on pairs of CTAs):
//   1 x 2304 x 768     T16 S1 6.8, S2 5.9, S4 5.2, S8 5.7   T64 S4 5.4      tiles 8.4
//   1 x 768 x 2304     T16 S1 13.6, S4 6.9, S8 6.5          T64 S8 6.5      tiles 14.7
//   64 x 768 x 768     T16 S4 5.7   T32 S4 5.9              T64 S2 6.9      tiles 8.9
//   128 x 2304 x 768   T16 S2 7.7   T32 S2 6.3, S4 7.0      T64 S4 6.6      tiles 9.1
//   320 x 1001 x 1140  T16 S1 10.9  T32 S1 9.7              T64 S2 8.4
//   320 x 2304 x 768   T16 S1 14.1  T32 S1 8.1, S2 12.7     T64 S1 8.6      tiles 9.3
//   640 x 2304 x 768                T32 S1 14.5             T64 S1 9.4      tiles 9.5
//   2500 x 768 x 768                T32 S1 15.7             T64 S1 9.8      tiles 9.5
//   20000 x 64 x 768                T32 S1 24.9             T64 S1 18.3     tiles 13.3
// A narrow CTA takes 0.28 for each block of k beside its start and its rows, half as much
// again where two share an SM, and what is left over after 304 takes a second turn. A tile
// takes 0.26 for each block with up to 136 SMs at work, 0.27 with all, and 0.5 between two.
// Slices pay for parts that are written and read:
//   2304 x 768 x 32299 to fp32, 27 tiles   1: 142, 2: 84, 4: 92, 5: 82, 8: 85, 12: 101
//   768 x 768 x 32299, 9 tiles             1: 142, 2: 79, 4: 47, 6: 39, 8: 37, 9: 52, 16: 43
//   1024 x 1024 x 169151, 16 tiles         2: 361, 4: 212, 5: 331, 8: 220, 9: 208, 12: 230
LinearPlan linear_plan(int64_t m, int64_t n, int64_t k, bool fp32, bool geglu,
                       bool a_transposed) {
  constexpr int64_t kSms = 152, kPairs = kSms / 2;
  const int64_t blocks = ceil_div(k, kMatmulBlock) * (fp32 ? kMaxMatmulTerms : 1);
  const int64_t tiles = tile_count(m, n);
  LinearPlan plan = {0, 1, 1};
  double best = 5.5 + (double)ceil_div(tiles, kPairs) *
                          ((tiles <= 68 ? 0.26 : 0.27) * (double)blocks + 0.5);
  // Slices of eight blocks at least.
  for (int32_t slices = 2; slices <= 16 && slices * 8 <= blocks && tiles <= 4 * kPairs; ++slices) {
    const int64_t units = tiles * slices;
    const double t = 9 + (double)ceil_div(units, kPairs) *
                             ((units <= 68 ? 0.26 : 0.27) * (double)ceil_div(blocks, slices) + 0.5) +
                     0.1 * (double)units;
    if (t < best) {
      best = t;
      plan.slices = slices;
    }
  }
  constexpr int32_t kRows[3] = {16, 32, 64};
  constexpr double kStart[3] = {3.6, 4.2, 5.1};
  const int64_t col_tiles = ceil_div(geglu ? n / 2 : n, geglu ? 64 : 128);
  for (int i = a_transposed ? 2 : 0; i < 3; ++i) {
    const int64_t ctas = ceil_div(m, kRows[i]) * col_tiles;
    if (ctas > 8 * kSms || ceil_div(m, kRows[i]) > 65535) continue;
    for (int32_t split = 1; split <= 8 && (split == 1 || split * 2 <= blocks);
         split += split < 2 ? 1 : 2) {
      const int64_t units = ctas * split;
      const bool shared = units > kSms;
      double t = kStart[i] + (shared ? 0.42 : 0.28) * (double)ceil_div(blocks, split);
      if (split > 1) t += 0.6 + 0.13 * split;
      if (shared) t += split > 1 ? 1.5 : 0.2;
      t += (double)(ceil_div(units, 2 * kSms) - 1) * (t - 2);
      if (t < best) {
        best = t;
        plan = {kRows[i], split, 1};
      }
    }
  }
  return plan;
}

// Products of fp32 operands that are not worth their parts (m x n x k, us as they lie; by
// parts): 4 x 8192 x 8192 111; 213, 8 x 2304 x 768 6.9; 12.0, 16 x 768 x 768 6.6; 9.8, 33 x 333
// x 1001 10.9; 10.8, 64 x 64 x 64 2.4; 6.7, but 16 x 8192 x 8192 309; 214, 33 x 2304 x 768 21;
// 13, 56 x 333 x 1001 12.7; 10.8, 5000 x 64 x 100 31; 11.8. By parts costs a launch and a
// workspace more: 20 us a call from Python for 12.
bool few(bool fp32, int64_t m, int64_t n, int64_t k, bool a_t, bool b_t) {
  return fp32 && !a_t && !b_t &&
         (m <= 4 || (m <= 64 && (double)m * (double)n * (double)k <= (double)(1 << 24)));
}

// Parts of slices, then parts of fp32 operands.
size_t workspace_bytes_of(const LinearPlan& plan, bool fp32, int64_t m, int64_t n, int64_t k,
                          bool a_t, bool b_t) {
  return matmul_tiles_workspace(tile_count(m, n), plan.slices) +
         (fp32 ? (size_t)split_bytes(m, n, k, a_t, b_t) : 0);
}

// A matrix of bf16 that TMA can read.
bool operand_ok(const void* x, int64_t ld) { return aligned(x, 16) && ld % 8 == 0; }

bool io_dtype(int dtype) { return dtype == PE_BF16 || dtype == PE_FP32; }

}  // namespace

}  // namespace pe

using namespace pe;

extern "C" size_t pe_matmul_workspace_size(pe_dtype dtype, int a_transposed, int b_transposed,
                                           int64_t m, int64_t n, int64_t k,
                                           pe_activation activation) {
  if (!io_dtype(dtype) || !activation_ok(activation) || m <= 0 || n <= 0 || k <= 0 ||
      !sizes_ok(m, n, k))
    return 0;
  const bool fp32 = dtype == PE_FP32;
  if (few(fp32, m, n, k, a_transposed != 0, b_transposed != 0)) return 0;
  const LinearPlan plan =
      linear_plan(m, n, k, fp32, activation == PE_ACT_GEGLU, a_transposed != 0);
  return workspace_bytes_of(plan, fp32, m, n, k, a_transposed != 0, b_transposed != 0);
}

extern "C" pe_status pe_matmul(pe_dtype dtype, const void* a, int64_t a_ld, int a_transposed,
                               const void* b, int64_t b_ld, int b_transposed, int64_t m,
                               int64_t n, int64_t k, const void* bias, pe_activation activation,
                               const void* residual, int64_t residual_ld, pe_dtype out_dtype,
                               void* out, int64_t out_ld, void* pre, int64_t pre_ld,
                               void* workspace, size_t workspace_bytes, pe_stream_t stream_) {
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (!io_dtype(dtype) || !io_dtype(out_dtype)) return PE_ERR_UNSUPPORTED;
  if (!activation_ok(activation) || m < 0 || n < 0 || k < 0) return PE_ERR_INVALID_ARG;
  const bool geglu = activation == PE_ACT_GEGLU;
  if (geglu && n % 2 != 0) return PE_ERR_INVALID_ARG;
  if (!sizes_ok(m, n, k)) return PE_ERR_OVERFLOW;
  if (m == 0 || n == 0) return PE_OK;
  const int64_t cols = geglu ? n / 2 : n;
  if (!out || (k > 0 && (!a || !b))) return PE_ERR_INVALID_ARG;
  if (out_ld < cols || (residual && residual_ld < cols) || (pre && pre_ld < n) ||
      (k > 0 && (a_ld < (a_transposed ? m : k) || b_ld < (b_transposed ? n : k))))
    return PE_ERR_INVALID_ARG;
  if (pre && (pre == out || pre == residual)) return PE_ERR_INVALID_ARG;
  if (out == residual && out_ld != residual_ld) return PE_ERR_INVALID_ARG;
  constexpr int64_t kMaxLd = 1LL << 36;      // a row's bytes stay below TMA's 2^40
  if (out_ld > kMaxLd || (residual && residual_ld > kMaxLd) || (pre && pre_ld > kMaxLd) ||
      (k > 0 && (a_ld > kMaxLd || b_ld > kMaxLd)))
    return PE_ERR_OVERFLOW;
  const bool fp32 = dtype == PE_FP32;
  if (k > 0 && !fp32 && (!operand_ok(a, a_ld) || !operand_ok(b, b_ld))) return PE_ERR_UNSUPPORTED;
  if (k > 0 && fp32 && (!aligned(a, 4) || !aligned(b, 4))) return PE_ERR_UNSUPPORTED;
  // TMA reads the up part's columns from a multiple of 16 bytes on.
  if (geglu && b_transposed && cols % 8 != 0) return PE_ERR_UNSUPPORTED;
  const uintptr_t size = out_dtype == PE_FP32 ? 4 : 2;
  if (!aligned(out, size) || !aligned(bias, size) || !aligned(residual, size) ||
      !aligned(pre, size))
    return PE_ERR_UNSUPPORTED;
  const bool direct = k == 0 || few(fp32, m, n, k, a_transposed != 0, b_transposed != 0);
  const LinearPlan plan = direct ? LinearPlan{0, 1, 1}
                                 : linear_plan(m, n, k, fp32, geglu, a_transposed != 0);
  const size_t need =
      direct ? 0 : workspace_bytes_of(plan, fp32, m, n, k, a_transposed != 0, b_transposed != 0);
  if (need && (!workspace || !aligned(workspace, 16) || workspace_bytes < need))
    return PE_ERR_WORKSPACE;
  if (!device_is_sm103()) return PE_ERR_UNSUPPORTED;
  auto four = [&](const void* x, int64_t ld) { return !x || (aligned(x, 4 * size) && ld % 4 == 0); };
  Matmul p;
  p.a = {a, a_ld, a_transposed != 0};
  p.b = {b, b_ld, b_transposed != 0};
  p.m = (int32_t)m;
  p.n = (int32_t)n;
  p.k = (int32_t)k;
  p.planes = 1;
  p.e = {bias,
         residual,
         out,
         pre,
         residual_ld,
         out_ld,
         pre_ld,
         (int32_t)m,
         (int32_t)cols,
         activation,
         out_dtype == PE_FP32 ? 1 : 0,
         four(out, out_ld) && four(residual, residual_ld) && four(pre, pre_ld) ? 1 : 0};
  if (k == 0) return matmul_no_sum(p, stream);
  if (direct) return matmul_few(p, stream);
  DeviceStatus* status = nullptr;
  PE_TRY(matmul_status_word(&status));
  if (fp32)
    PE_TRY(split(p,
                 static_cast<char*>(workspace) +
                     matmul_tiles_workspace(tile_count(m, n), plan.slices),
                 stream));
  if (plan.rows) return matmul_narrow(p, plan.rows, plan.split, status, stream);
  return matmul_tiles(p, plan.slices, workspace, status, stream);
}
