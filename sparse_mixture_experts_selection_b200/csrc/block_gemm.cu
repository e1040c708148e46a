// Grouped matrix products of block-scaled e4m3 operands, and the SwiGLU experts
// made of them:
//   out[r, j] = row_scale[r] * sum_b xs[r, b] * ws[g, j / 128, b] * sum_{k in b} x[r, k] * w[g, j, k]
#include "api.h"
#include "common.cuh"
#include "e4m3.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kBlock = 128;              // values per scale
constexpr int kMaxGroups = 1024;
constexpr int kTile = 64;

int blocks_of(int n) { return (n + kBlock - 1) / kBlock; }

struct BlockArgs {
  int G, N, K, max_rows;
  const int* offsets;
  const uint8_t *x, *w;
  const float *xs, *wsc, *row_scale;
  int out_f32;
  void* out;
  int* err;
};

__device__ __forceinline__ float e4m3_value(uint8_t c) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

// A block of 256 threads computes 64 rows x 64 columns of one group, 4 x 4 a
// thread, one block of 128 of the reduction at a time.
__global__ void __launch_bounds__(256) block_product_kernel(const BlockArgs a) {
  __shared__ float sx[kTile][33], sw[kTile][33];
  // the group and row tile of this block: groups in order, each rounded up to whole tiles
  int tile = blockIdx.x, g = 0, r0 = 0, r1 = 0;
  for (; g < a.G; ++g) {
    r0 = a.offsets ? a.offsets[g] : 0;
    r1 = a.offsets ? a.offsets[g + 1] : a.max_rows;
    if (r0 < 0 || r1 < r0 || r1 > a.max_rows) {
      if (threadIdx.x == 0) set_device_error(a.err, MOE_DEVERR_INDEX);
      continue;
    }
    const int n = (r1 - r0 + kTile - 1) / kTile;
    if (tile < n) break;
    tile -= n;
  }
  if (g == a.G) return;
  const int m0 = r0 + tile * kTile, n0 = blockIdx.y * kTile;
  const int KB = (a.K + kBlock - 1) / kBlock, NB = (a.N + kBlock - 1) / kBlock;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float acc[4][4] = {};
  for (int b = 0; b < KB; ++b) {
    float part[4][4] = {};
    for (int k0 = b * kBlock; k0 < min(a.K, (b + 1) * kBlock); k0 += 32) {
      for (int i = threadIdx.x; i < kTile * 32; i += 256) {
        const int r = i / 32, k = k0 + i % 32;
        sx[r][i % 32] = m0 + r < r1 && k < a.K ? e4m3_value(a.x[(size_t)(m0 + r) * a.K + k]) : 0.0f;
        sw[r][i % 32] = n0 + r < a.N && k < a.K ? e4m3_value(a.w[((size_t)g * a.N + n0 + r) * a.K + k]) : 0.0f;
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 32; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) part[i][j] = fmaf(sx[ty + 16 * i][k], sw[tx + 16 * j][k], part[i][j]);
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = m0 + ty + 16 * i, c = n0 + tx + 16 * j;
        if (r < r1 && c < a.N)
          acc[i][j] = fmaf(a.xs[(size_t)r * KB + b] * a.wsc[((size_t)g * NB + c / kBlock) * KB + b], part[i][j], acc[i][j]);
      }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = m0 + ty + 16 * i, c = n0 + tx + 16 * j;
      if (r >= r1 || c >= a.N) continue;
      const float v = a.row_scale ? acc[i][j] * a.row_scale[r] : acc[i][j];
      if (a.out_f32) static_cast<float*>(a.out)[(size_t)r * a.N + c] = v;
      else static_cast<bf16*>(a.out)[(size_t)r * a.N + c] = from_f32<bf16>(v);
    }
}

// u[r, c] <- SiLU(u) * v for the rows of all groups.
__global__ void __launch_bounds__(256) swiglu_kernel(float* u, const float* v, int64_t n) {
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x)
    u[i] = u[i] / (1.0f + expf(-u[i])) * v[i];
}

void product(const BlockArgs& a, cudaStream_t st) {
  block_product_kernel<<<dim3(a.max_rows / kTile + a.G, (a.N + kTile - 1) / kTile), 256, 0, st>>>(a);
}

moe_status check_product(int n_groups, int n_cols, int k, int max_rows) {
  if (n_groups < 1) return fail(MOE_ERR_INVALID_ARG, "n_groups=%d < 1", n_groups);
  if (n_groups > kMaxGroups) return fail(MOE_ERR_UNSUPPORTED, "n_groups=%d > %d", n_groups, kMaxGroups);
  if (n_cols < 1) return fail(MOE_ERR_INVALID_ARG, "n_cols=%d < 1", n_cols);
  if (k < 16 || k % 16) return fail(MOE_ERR_INVALID_ARG, "k=%d must be a positive multiple of 16", k);
  if (max_rows < 0) return fail(MOE_ERR_INVALID_ARG, "max_rows=%d < 0", max_rows);
  if (n_cols > 1 << 20 || k > 1 << 20) return fail(MOE_ERR_UNSUPPORTED, "n_cols=%d k=%d above 2^20", n_cols, k);
  if ((int64_t)n_groups * n_cols > 0x7FFFFFFF) return fail(MOE_ERR_UNSUPPORTED, "n_groups * n_cols above 2^31");
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_block_matmul_workspace_size(int32_t n_groups, int32_t n_cols, int32_t k, int32_t max_rows,
                                                      size_t* bytes) {
  MOE_CHECK(check_product(n_groups, n_cols, k, max_rows));
  if (!bytes) return fail(MOE_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = kAlign;
  return MOE_OK;
}

extern "C" moe_status moe_block_matmul(int32_t n_groups, int32_t n_cols, int32_t k, int32_t max_rows,
                                       const int32_t* offsets, const uint8_t* x, const float* x_scale,
                                       const uint8_t* w, const float* w_scale, const float* row_scale,
                                       int32_t out_dtype, void* out, void* ws, size_t ws_bytes, void* stream) {
  size_t need = 0;
  MOE_CHECK(moe_block_matmul_workspace_size(n_groups, n_cols, k, max_rows, &need));
  if (out_dtype != MOE_DTYPE_F32 && out_dtype != MOE_DTYPE_BF16) return fail(MOE_ERR_INVALID_ARG, "out_dtype=%d", out_dtype);
  if (!offsets && n_groups != 1) return fail(MOE_ERR_INVALID_ARG, "offsets is NULL with n_groups=%d", n_groups);
  MOE_ALIGNED4(offsets); MOE_ALIGNED4(row_scale);
  MOE_CHECK(check_ws(ws, ws_bytes, need));
  if (max_rows == 0) return MOE_OK;
  MOE_NONNULL(x); MOE_NONNULL4(x_scale); MOE_NONNULL(w); MOE_NONNULL4(w_scale); MOE_NONNULL(out);
  BlockArgs a{n_groups, n_cols, k, max_rows, offsets, x, w, x_scale, w_scale, row_scale,
              out_dtype == MOE_DTYPE_F32, out, at<int>(ws, 0)};
  product(a, static_cast<cudaStream_t>(stream));
  return cuda_status();
}

namespace {

// workspace of the experts: the error word, U, V, the codes of their product and its scales
struct FfnLayout {
  size_t u, v, codes, scales, total;
};

FfnLayout ffn_layout(int f, int max_rows) {
  FfnLayout L{};
  const size_t rows = max_rows > 0 ? max_rows : 1;
  size_t o = kAlign;
  L.u = o; o = align_up(o + rows * f * 4);
  L.v = o; o = align_up(o + rows * f * 4);
  L.codes = o; o = align_up(o + rows * f);
  L.scales = o; o = align_up(o + rows * blocks_of(f) * 4);
  L.total = o;
  return L;
}

}  // namespace

extern "C" moe_status moe_block_ffn_workspace_size(int32_t n_experts, int32_t d_model, int32_t d_ffn, int32_t max_rows,
                                                   size_t* bytes) {
  MOE_CHECK(check_product(n_experts, d_ffn, d_model, max_rows));
  MOE_CHECK(check_product(n_experts, d_model, d_ffn, max_rows));
  if (!bytes) return fail(MOE_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = ffn_layout(d_ffn, max_rows).total;
  return MOE_OK;
}

extern "C" moe_status moe_block_ffn(int32_t n_experts, int32_t d_model, int32_t d_ffn, int32_t max_rows,
                                    const int32_t* offsets, const uint8_t* x, const float* x_scale,
                                    const uint8_t* w_gate, const float* s_gate, const uint8_t* w_up, const float* s_up,
                                    const uint8_t* w_down, const float* s_down, const float* row_scale,
                                    int32_t out_dtype, void* out, void* ws, size_t ws_bytes, void* stream) {
  size_t need = 0;
  MOE_CHECK(moe_block_ffn_workspace_size(n_experts, d_model, d_ffn, max_rows, &need));
  if (out_dtype != MOE_DTYPE_F32 && out_dtype != MOE_DTYPE_BF16) return fail(MOE_ERR_INVALID_ARG, "out_dtype=%d", out_dtype);
  if (!offsets && n_experts != 1) return fail(MOE_ERR_INVALID_ARG, "offsets is NULL with n_experts=%d", n_experts);
  MOE_ALIGNED4(offsets); MOE_ALIGNED4(row_scale);
  MOE_CHECK(check_ws(ws, ws_bytes, need));
  if (max_rows == 0) return MOE_OK;
  MOE_NONNULL(x); MOE_NONNULL4(x_scale); MOE_NONNULL(w_gate); MOE_NONNULL4(s_gate); MOE_NONNULL(w_up);
  MOE_NONNULL4(s_up); MOE_NONNULL(w_down); MOE_NONNULL4(s_down); MOE_NONNULL(out);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const FfnLayout L = ffn_layout(d_ffn, max_rows);
  float *u = at<float>(ws, L.u), *v = at<float>(ws, L.v);
  uint8_t* codes = at<uint8_t>(ws, L.codes);
  float* scales = at<float>(ws, L.scales);
  int* err = at<int>(ws, 0);
  product({n_experts, d_ffn, d_model, max_rows, offsets, x, w_gate, x_scale, s_gate, nullptr, 1, u, err}, st);
  product({n_experts, d_ffn, d_model, max_rows, offsets, x, w_up, x_scale, s_up, nullptr, 1, v, err}, st);
  swiglu_kernel<<<148 * 8, 256, 0, st>>>(u, v, (int64_t)max_rows * d_ffn);
  const cudaError_t e = launch_quantize_tiles(u, MOE_DTYPE_F32, max_rows, d_ffn, codes, scales, st);
  if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "quantize launch: %s", cudaGetErrorString(e));
  product({n_experts, d_model, d_ffn, max_rows, offsets, codes, w_down, scales, s_down, row_scale,
           out_dtype == MOE_DTYPE_F32, out, err}, st);
  return cuda_status();
}
