// Dropout with the residual behind the experts, and its backward:
//   out_i = res_i + (u_i >= p ? x_i / (1 - p) : 0)
// u_i = word / 2^32 of Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel
// random numbers: as easy as 1, 2, 3", 2011): block i / 4 of the counter,
// word i % 4.  The mask is drawn again in the backward and never stored, so a
// pass moves x, res and out and nothing else.  Drawing 32 bits takes about 30
// instructions a value; they hide behind the memory traffic of a 2-byte value
// only because one block serves four values and nothing is drawn twice.
#include <cmath>

#include "api.h"
#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

// The four 32-bit words of counter block (c, n) under the key.
__device__ __forceinline__ uint4 philox(uint64_t c, uint64_t n, uint64_t key) {
  uint32_t c0 = (uint32_t)c, c1 = (uint32_t)(c >> 32), c2 = (uint32_t)n, c3 = (uint32_t)(n >> 32);
  uint32_t k0 = (uint32_t)key, k1 = (uint32_t)(key >> 32);
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// word < cut drops the value: u < p exactly when word < ceil(p * 2^32)
__device__ __forceinline__ float dropped(float x, float res, uint32_t word, uint64_t cut, float scale) {
  return (uint64_t)word >= cut ? fmaf(x, scale, res) : res;
}

// x and out may be the same array: a thread reads its values before it writes them.
template <typename T>
__global__ void __launch_bounds__(256) dropout_kernel(const T* x, const T* res, T* out, int64_t n, uint64_t cut,
                                                      float scale, const uint64_t* rng) {
  pdl_wait();
  pdl_trigger();
  const uint64_t key = rng[0], draw = rng[1];
  const int64_t blocks = (n + 3) / 4;
  for (int64_t q = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; q < blocks; q += (int64_t)gridDim.x * blockDim.x) {
    const uint4 w = philox((uint64_t)q, draw, key);
    const uint32_t word[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t i = 4 * q + j;
      if (i < n) out[i] = from_f32<T>(dropped(to_f32<T>(x[i]), res ? to_f32<T>(res[i]) : 0.0f, word[j], cut, scale));
    }
  }
}

moe_status run_dropout(const void* x, const void* res, int32_t dtype, int64_t n, double p, const uint64_t* rng,
                       void* out, void* stream) {
  if (dtype != MOE_DTYPE_F32 && dtype != MOE_DTYPE_BF16) return fail(MOE_ERR_INVALID_ARG, "dtype=%d", dtype);
  if (n < 0) return fail(MOE_ERR_INVALID_ARG, "n=%lld < 0", (long long)n);
  if (!(p >= 0.0 && p <= 1.0)) return fail(MOE_ERR_INVALID_ARG, "p=%g outside [0, 1]", p);
  if (n == 0) return MOE_OK;
  MOE_NONNULL(x); MOE_ALIGNED(res); MOE_NONNULL(out);
  if (!rng) return fail(MOE_ERR_INVALID_ARG, "rng is NULL");
  if (reinterpret_cast<uintptr_t>(rng) & 7u) return fail(MOE_ERR_INVALID_ARG, "rng is not 8-byte aligned");
  const uint64_t cut = (uint64_t)std::ceil(p * 4294967296.0);
  const float scale = p < 1.0 ? (float)(1.0 / (1.0 - p)) : 0.0f;
  const int64_t want = ((n + 3) / 4 + 255) / 256;
  const dim3 grid((unsigned)(want < 148 * 8 ? want : 148 * 8));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == MOE_DTYPE_F32)
    e = launch_pdl(dropout_kernel<float>, grid, dim3(256), 0, st, static_cast<const float*>(x),
                   static_cast<const float*>(res), static_cast<float*>(out), n, cut, scale, rng);
  else
    e = launch_pdl(dropout_kernel<bf16>, grid, dim3(256), 0, st, static_cast<const bf16*>(x),
                   static_cast<const bf16*>(res), static_cast<bf16*>(out), n, cut, scale, rng);
  return e != cudaSuccess ? fail(MOE_ERR_CUDA, "dropout launch: %s", cudaGetErrorString(e)) : MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" moe_status moe_dropout_add(const void* x, const void* res, int32_t dtype, int64_t n, double p,
                                      const uint64_t* rng, void* out, void* stream) {
  return moe::run_dropout(x, res, dtype, n, p, rng, out, stream);
}

extern "C" moe_status moe_dropout_backward(const void* dy, int32_t dtype, int64_t n, double p, const uint64_t* rng,
                                           void* dx, void* stream) {
  return moe::run_dropout(dy, nullptr, dtype, n, p, rng, dx, stream);
}
