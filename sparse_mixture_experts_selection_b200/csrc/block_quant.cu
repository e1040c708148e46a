// e4m3 codes with one power-of-two scale for each 1 x 128 tile of a row
// (activations) or each 128 x 128 block of a matrix (weights): the smallest s
// with max |x| / s <= 448, each x / s rounded to the nearest code.  Dividing by
// a power of two is exact, so the codes depend on the values alone.
#include "api.h"
#include "common.cuh"
#include "e4m3.cuh"
#include "kernels.h"

namespace moe {
namespace {

// Eight values from 16-byte loads.
__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
  const uint4 q = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

__device__ __forceinline__ float top8(const float (&v)[8]) {
  float t = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) t = fmaxf(t, fabsf(v[i]));
  return t;
}

__device__ __forceinline__ uint2 codes8(const float (&v)[8], float inv) {
  return make_uint2(e4m3_pack4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                    e4m3_pack4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
}

// Eight lanes per tile, 16 values each: two 16-byte loads (bf16) and one of codes
// out, no shared memory; two tiles a time, their loads in flight together.  Bound by
// memory and, nearly as much, by the instructions: 16 values a lane share one
// maximum and its exponent (32768 x 7168 bf16: 118 us, 6.0 TB/s; eight values a lane took
// 1.4 times as long).
constexpr int kTiles = 2;
template <typename TIn>
__global__ void __launch_bounds__(256) quantize_tiles_kernel(const TIn* __restrict__ src, int64_t n_tiles, int tiles,
                                                             int cols, uint8_t* __restrict__ codes,
                                                             float* __restrict__ scales) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x % 8;
  // whole warps walk together, four tiles each time: their shuffles name all lanes
  const int64_t step = (int64_t)gridDim.x * (blockDim.x / 8);
  const int mine = threadIdx.x / 8 % 4;
  int64_t t0 = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) / 32 * 4;
  // row and tile in the row, carried along: a 64-bit division a tile would take longer than its memory
  int64_t row = (t0 + mine) / tiles;
  int in_row = (int)((t0 + mine) - row * tiles);
  const int64_t rows_step = step / tiles;
  const int tiles_step = (int)(step - rows_step * tiles);
  for (; t0 < n_tiles; t0 += kTiles * step) {
    float v[kTiles][2][8];
    int64_t at[kTiles];                              // -1: no values there
#pragma unroll
    for (int k = 0; k < kTiles; ++k) {
      const int c = in_row * 128 + lane * 16;        // cols is a multiple of 16: 16 values or none
      at[k] = t0 + k * step + mine < n_tiles && c < cols ? row * cols + c : -1;
      row += rows_step;
      in_row += tiles_step;
      if (in_row >= tiles) { in_row -= tiles; ++row; }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[k][h][j] = 0.0f;
        if (at[k] >= 0) load8(src + at[k] + 8 * h, v[k][h]);
      }
    }
#pragma unroll
    for (int k = 0; k < kTiles; ++k) {
      float top = fmaxf(top8(v[k][0]), top8(v[k][1]));
#pragma unroll
      for (int off = 4; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
      const int e = e4m3_scale_exponent(top);
      if (at[k] >= 0) {
        const uint2 lo = codes8(v[k][0], pow2(-e)), hi = codes8(v[k][1], pow2(-e));
        *reinterpret_cast<uint4*>(codes + at[k]) = make_uint4(lo.x, lo.y, hi.x, hi.y);
        if (lane == 0) scales[t0 + k * step + mine] = pow2(e);
      }
    }
  }
}

// A block of 256 threads per 128 x 128 block: 16 threads across a row, eight
// rows each, all values in registers between the maximum and the codes.  32 matrices of
// 2048 x 7168: bf16 257 us (5.5 TB/s), fp32 328 us (7.2 TB/s, most of it reads).
template <typename TIn>
__global__ void __launch_bounds__(256) quantize_blocks_kernel(const TIn* __restrict__ src, int rows, int cols,
                                                              int row_blocks, int col_blocks,
                                                              uint8_t* __restrict__ codes, float* __restrict__ scales) {
  __shared__ float tops[8];
  const int64_t b = blockIdx.x;
  const int cb = (int)(b % col_blocks);
  const int rb = (int)(b / col_blocks % row_blocks);
  const int64_t m = b / col_blocks / row_blocks;
  const int c = cb * 128 + threadIdx.x % 16 * 8;
  const int64_t base = m * rows * cols + c;
  float v[8][8];
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = rb * 128 + threadIdx.x / 16 + 16 * i;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
    if (r < rows && c < cols) load8(src + base + (int64_t)r * cols, v[i]);
    top = fmaxf(top, top8(v[i]));
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
  if (threadIdx.x % kWarp == 0) tops[threadIdx.x / kWarp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) top = fmaxf(top, tops[w]);
  const int e = e4m3_scale_exponent(top);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = rb * 128 + threadIdx.x / 16 + 16 * i;
    if (r < rows && c < cols) *reinterpret_cast<uint2*>(codes + base + (int64_t)r * cols) = codes8(v[i], pow2(-e));
  }
  if (threadIdx.x == 0) scales[b] = pow2(e);
}

constexpr int kMaxSide = 1 << 30;        // rounding up to blocks stays within 32 bits
constexpr int64_t kMaxRows = (int64_t)1 << 32;     // of tiles: values are counted in 64 bits

moe_status check_source(const void* src, int dtype, int cols, const void* codes, const void* scales, bool empty) {
  if (dtype != MOE_DTYPE_F32 && dtype != MOE_DTYPE_BF16) return fail(MOE_ERR_INVALID_ARG, "src_dtype=%d", dtype);
  if (cols < 16 || cols % 16) return fail(MOE_ERR_INVALID_ARG, "cols=%d must be a positive multiple of 16", cols);
  if (cols > kMaxSide) return fail(MOE_ERR_UNSUPPORTED, "cols=%d > 2^30", cols);
  if (empty) return MOE_OK;
  MOE_NONNULL(src); MOE_NONNULL(codes); MOE_NONNULL4(scales);
  return MOE_OK;
}

cudaError_t launch_quantize_tiles(const void* src, int src_dtype, int64_t n_rows, int cols, uint8_t* codes,
                                  float* scales, cudaStream_t st) {
  const int tiles = (cols + 127) / 128;
  const int64_t n_tiles = n_rows * tiles;
  const int64_t want = (n_tiles + 31) / 32;
  const dim3 grid((unsigned)(want < 148 * 4 ? want : 148 * 4));      // all resident
  if (src_dtype == MOE_DTYPE_BF16)
    return launch_pdl(quantize_tiles_kernel<uint16_t>, grid, dim3(256), 0, st, static_cast<const uint16_t*>(src),
                      n_tiles, tiles, cols, codes, scales);
  return launch_pdl(quantize_tiles_kernel<float>, grid, dim3(256), 0, st, static_cast<const float*>(src), n_tiles,
                    tiles, cols, codes, scales);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_quantize_tiles(const void* src, int32_t src_dtype, int64_t n_rows, int32_t cols,
                                         uint8_t* codes, float* scales, void* stream) {
  if (n_rows < 0) return fail(MOE_ERR_INVALID_ARG, "n_rows=%lld < 0", (long long)n_rows);
  if (n_rows > kMaxRows) return fail(MOE_ERR_UNSUPPORTED, "n_rows=%lld > 2^32", (long long)n_rows);
  MOE_CHECK(check_source(src, src_dtype, cols, codes, scales, n_rows == 0));
  if (n_rows == 0) return MOE_OK;
  const cudaError_t e = launch_quantize_tiles(src, src_dtype, n_rows, cols, codes, scales,
                                              static_cast<cudaStream_t>(stream));
  return launch_status(e, "quantize");
}

extern "C" moe_status moe_quantize_blocks(const void* src, int32_t src_dtype, int32_t n_mats, int32_t rows,
                                          int32_t cols, uint8_t* codes, float* scales, void* stream) {
  if (n_mats < 0 || rows < 0) return fail(MOE_ERR_INVALID_ARG, "n_mats=%d rows=%d", n_mats, rows);
  if (rows > kMaxSide) return fail(MOE_ERR_UNSUPPORTED, "rows=%d > 2^30", rows);
  const bool empty = n_mats == 0 || rows == 0;
  MOE_CHECK(check_source(src, src_dtype, cols, codes, scales, empty));
  if (empty) return MOE_OK;
  const int rb = (rows + 127) / 128, cb = (cols + 127) / 128;
  const int64_t each = (int64_t)rb * cb;           // below 2^47; times n_mats it may pass 64 bits
  if (each > 0x7FFFFFFF / n_mats) return fail(MOE_ERR_UNSUPPORTED, "%d matrices of %lld blocks", n_mats, (long long)each);
  const int64_t n = n_mats * each;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (src_dtype == MOE_DTYPE_BF16)
    quantize_blocks_kernel<uint16_t><<<(unsigned)n, 256, 0, st>>>(static_cast<const uint16_t*>(src), rows, cols, rb,
                                                                  cb, codes, scales);
  else
    quantize_blocks_kernel<float><<<(unsigned)n, 256, 0, st>>>(static_cast<const float*>(src), rows, cols, rb, cb,
                                                               codes, scales);
  return cuda_status();
}
