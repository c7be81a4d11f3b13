// Quantisation of a matrix to 8 bits with a scale for each 1 x 128 or 128 x 128
// block, as it is and (or) transposed, from one read.
//
// One block of threads per 128 x 128 tile: a tile holds whole scale blocks of
// both outputs, so nothing is shared between tiles. A warp takes 16 rows, a
// lane 4 of the 128 columns, and the 64 values stay in registers. Row maxima are
// warp shuffles, column maxima and the tile's maximum go through shared memory.
// The transposed bytes are packed along a lane's 16 rows and exchanged through
// shared memory so that every output row is written in runs of 128 bytes.
#include "pe_fp8.cuh"

namespace pe {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 128;
constexpr int kRowsPerWarp = kTile / kWarps;       // 16: one 16-byte run of a transposed row
constexpr unsigned kFull = 0xffffffffu;
static_assert(kTile == kFp8Block && kRowsPerWarp == 16, "tile layout");

struct QuantizeArgs {
  const void* x;
  int64_t rows, cols;
  int64_t col_tiles;
  uint8_t* y;
  int64_t y_ld;
  float* scales;       // [col_tiles][rows], or [col_tiles][row tiles]
  uint8_t* yt;
  int64_t yt_ld;
  float* scales_t;     // [row tiles][cols], or [row tiles][col_tiles]
};

// kVec: a lane's 4 columns are adjacent (rows of x start at multiples of 4
// elements); otherwise they are 32 apart and move one element at a time.
template <typename T, bool kVec, bool kE5M2, bool kSquare>
__global__ void __launch_bounds__(kThreads)
quantize_kernel(const QuantizeArgs a) {
  __shared__ float colmax[kWarps][kTile];
  __shared__ uint4 exchange[kTile][kWarps];        // [column][16-row run], runs swizzled
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t rt = blockIdx.x / a.col_tiles, ct = blockIdx.x - rt * a.col_tiles;
  const int64_t r0 = rt * kTile, c0 = ct * kTile;
  const int row_count = (int)(a.rows - r0 < kTile ? a.rows - r0 : kTile);
  const int col_count = (int)(a.cols - c0 < kTile ? a.cols - c0 : kTile);
  const int64_t row_tiles = (a.rows + kTile - 1) / kTile;
  const int wr = warp * kRowsPerWarp;              // this warp's first row in the tile
  auto col = [&](int j) { return kVec ? lane * 4 + j : j * 32 + lane; };

  float x[kRowsPerWarp][4];
  const T* src = static_cast<const T*>(a.x) + (r0 + wr) * a.cols + c0;
#pragma unroll
  for (int i = 0; i < kRowsPerWarp; ++i) {
#pragma unroll
    for (int j = 0; j < 4; ++j) x[i][j] = 0.f;
    if (wr + i < row_count) {
      if constexpr (kVec) {
        if (col(0) < col_count) {                  // cols is a multiple of 4
          if constexpr (sizeof(T) == 2) {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(src + i * a.cols + col(0)));
            x[i][0] = __uint_as_float(v.x << 16);
            x[i][1] = __uint_as_float(v.x & 0xffff0000u);
            x[i][2] = __uint_as_float(v.y << 16);
            x[i][3] = __uint_as_float(v.y & 0xffff0000u);
          } else {
            const float4 v = __ldg(reinterpret_cast<const float4*>(src + i * a.cols + col(0)));
            x[i][0] = v.x;
            x[i][1] = v.y;
            x[i][2] = v.z;
            x[i][3] = v.w;
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (col(j) < col_count) x[i][j] = to_f32(src[i * a.cols + col(j)]);
      }
    }
  }

  float cmax[4] = {0.f, 0.f, 0.f, 0.f};            // over this warp's rows, then over the tile
  if (kSquare || a.yt) {
#pragma unroll
    for (int i = 0; i < kRowsPerWarp; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) cmax[j] = max_nan(cmax[j], fabsf(x[i][j]));
    if constexpr (kSquare) {
      float m = max_nan(max_nan(cmax[0], cmax[1]), max_nan(cmax[2], cmax[3]));
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) m = max_nan(m, __shfl_xor_sync(kFull, m, off));
      if (lane == 0) colmax[0][warp] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = max_nan(m, colmax[0][w]);
      cmax[0] = m;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) colmax[warp][col(j)] = cmax[j];
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int w = 0; w < kWarps; ++w) cmax[j] = max_nan(cmax[j], colmax[w][col(j)]);
    }
  }
  float tile_factor = 0.f, tile_scale = 0.f;
  if constexpr (kSquare) tile_scale = fp8_scale<kE5M2>(cmax[0], tile_factor);

  if (a.y) {
    if (kSquare && threadIdx.x == 0) a.scales[ct * row_tiles + rt] = tile_scale;
#pragma unroll
    for (int i = 0; i < kRowsPerWarp; ++i) {
      float f = tile_factor;
      if constexpr (!kSquare) {
        float m = max_nan(max_nan(fabsf(x[i][0]), fabsf(x[i][1])),
                          max_nan(fabsf(x[i][2]), fabsf(x[i][3])));
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) m = max_nan(m, __shfl_xor_sync(kFull, m, off));
        const float scale = fp8_scale<kE5M2>(m, f);
        if (lane == 0 && wr + i < row_count) a.scales[ct * a.rows + r0 + wr + i] = scale;
      }
      if (wr + i < row_count) {
        uint8_t* dst = a.y + (r0 + wr + i) * a.y_ld + c0;
        const uint32_t q = fp8x4<kE5M2>(x[i][0] * f, x[i][1] * f, x[i][2] * f, x[i][3] * f);
        if constexpr (kVec) {
          if (col(0) < col_count) *reinterpret_cast<uint32_t*>(dst + col(0)) = q;
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (col(j) < col_count) dst[col(j)] = (uint8_t)(q >> (8 * j));
        }
      }
    }
  }

  if (a.yt) {
    if (kSquare && threadIdx.x == 0) a.scales_t[rt * a.col_tiles + ct] = tile_scale;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float f = tile_factor;
      if constexpr (!kSquare) {
        const float scale = fp8_scale<kE5M2>(cmax[j], f);
        if (warp == 0 && col(j) < col_count) a.scales_t[rt * a.cols + c0 + col(j)] = scale;
      }
      uint32_t q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        q[i] = fp8x4<kE5M2>(x[4 * i][j] * f, x[4 * i + 1][j] * f, x[4 * i + 2][j] * f,
                            x[4 * i + 3][j] * f);
      exchange[col(j)][warp ^ ((col(j) >> (kVec ? 2 : 0)) & 7)] =
          make_uint4(q[0], q[1], q[2], q[3]);
    }
    __syncthreads();
    // 8 threads per transposed row, 32 rows at a time.
    const int run = threadIdx.x & 7;
    const int run_rows = row_count - run * 16;     // valid bytes of this run
#pragma unroll
    for (int i = 0; i < kTile / 32; ++i) {
      const int c = i * 32 + (threadIdx.x >> 3);
      if (c >= col_count) continue;
      const uint4 v = exchange[c][run ^ ((c >> (kVec ? 2 : 0)) & 7)];
      uint8_t* dst = a.yt + (c0 + c) * a.yt_ld + r0 + run * 16;
      if (run_rows >= 16) {
        *reinterpret_cast<uint4*>(dst) = v;
      } else {
        const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int b = 0; b < 16; ++b)
          if (b < run_rows) dst[b] = (uint8_t)(q[b >> 2] >> (8 * (b & 3)));
      }
    }
  }
}

template <typename T, bool kVec, bool kE5M2>
pe_status launch(const QuantizeArgs& a, bool square, unsigned grid, cudaStream_t stream) {
  if (square)
    quantize_kernel<T, kVec, kE5M2, true><<<grid, kThreads, 0, stream>>>(a);
  else
    quantize_kernel<T, kVec, kE5M2, false><<<grid, kThreads, 0, stream>>>(a);
  PE_CUDA_TRY(cudaGetLastError());
  return PE_OK;
}

template <typename T>
pe_status run(const QuantizeArgs& a, bool e5m2, bool square, unsigned grid, cudaStream_t stream) {
  const bool vec = a.cols % 4 == 0 && aligned(a.x, 4 * sizeof(T));
  if (vec)
    return e5m2 ? launch<T, true, true>(a, square, grid, stream)
                : launch<T, true, false>(a, square, grid, stream);
  return e5m2 ? launch<T, false, true>(a, square, grid, stream)
              : launch<T, false, false>(a, square, grid, stream);
}

}  // namespace

}  // namespace pe

using namespace pe;

extern "C" pe_status pe_quantize_fp8(pe_dtype dtype, pe_fp8_type fp8_type, const void* x,
                                     int64_t rows, int64_t cols, int32_t block_rows, void* y,
                                     int64_t y_ld, float* scales, void* yt, int64_t yt_ld,
                                     float* scales_t, pe_stream_t stream_) {
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if ((dtype != PE_BF16 && dtype != PE_FP32) || !fp8_type_ok(fp8_type)) return PE_ERR_UNSUPPORTED;
  if (rows < 0 || cols < 0 || (block_rows != 1 && block_rows != kFp8Block))
    return PE_ERR_INVALID_ARG;
  if (rows >= (1LL << 31) || cols >= (1LL << 31)) return PE_ERR_OVERFLOW;
  if (rows == 0 || cols == 0) return PE_OK;
  if (!x || (!y && !yt) || (y && !scales) || (yt && !scales_t)) return PE_ERR_INVALID_ARG;
  if ((y && !fp8_layout_ok(y, y_ld, cols)) || (yt && !fp8_layout_ok(yt, yt_ld, rows)))
    return PE_ERR_UNSUPPORTED;
  if (!device_is_sm103()) return PE_ERR_UNSUPPORTED;
  const int64_t col_tiles = ceil_div(cols, kTile), tiles = col_tiles * ceil_div(rows, kTile);
  if (tiles >= (1LL << 31)) return PE_ERR_OVERFLOW;
  const QuantizeArgs a = {x,      rows, cols,
                          col_tiles, static_cast<uint8_t*>(y), y_ld, scales,
                          static_cast<uint8_t*>(yt), yt_ld, scales_t};
  if (dtype == PE_FP32)
    return run<float>(a, fp8_type == PE_E5M2, block_rows != 1, (unsigned)tiles, stream);
  return run<__nv_bfloat16>(a, fp8_type == PE_E5M2, block_rows != 1, (unsigned)tiles, stream);
}
