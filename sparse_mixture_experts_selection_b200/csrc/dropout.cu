// Dropout with the residual behind the experts, and its backward:
//   out_i = res_i + (u_i >= p ? x_i / (1 - p) : 0)
// u_i = word / 2^32 of Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel
// random numbers: as easy as 1, 2, 3", 2011): block i / 4 of the counter,
// word i % 4.  The mask is drawn again in the backward and never stored, so a
// pass moves x, res and out and nothing else: 4096 x 7168 bf16 with a residual 32 to
// 34 us (5.2 to 5.5 TB/s; torch's add of that size 28.8 us), 8191 x 2048 fp32 without 22.5 us
// (6.0 TB/s).  2-byte values are bound by the instructions of the draw as much as by
// memory, hence one block for four values and the keys made once.
#include <cmath>

#include "api.h"
#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

// The ten rounds' keys, made once per thread: the compiler would rather add them up
// again in every block, and the instructions are what bounds 2-byte values.
struct Keys {
  uint32_t k0[10], k1[10];
  __device__ __forceinline__ explicit Keys(uint64_t key) {
#pragma unroll
    for (int i = 0; i < 10; ++i) {
      k0[i] = (uint32_t)key + i * 0x9E3779B9u;
      k1[i] = (uint32_t)(key >> 32) + i * 0xBB67AE85u;
      asm volatile("" : "+r"(k0[i]), "+r"(k1[i]));
    }
  }
};

// The four 32-bit words of counter block (c, n).
__device__ __forceinline__ uint4 philox(uint64_t c, uint64_t n, const Keys& k) {
  uint32_t c0 = (uint32_t)c, c1 = (uint32_t)(c >> 32), c2 = (uint32_t)n, c3 = (uint32_t)(n >> 32);
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k.k0[i];
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k.k1[i];
    c3 = (uint32_t)a;
  }
  return make_uint4(c0, c1, c2, c3);
}

// u < p exactly when word < ceil(p * 2^32), and that when word <= last, one less;
// `all` (p = 0) keeps every value.
__device__ __forceinline__ float dropped(float x, float res, uint32_t word, uint32_t last, bool all, float scale) {
  return word > last || all ? fmaf(x, scale, res) : res;
}

// 16 bytes of a thread: 4 or 8 values and the counter blocks that cover them.
__device__ __forceinline__ void unpack(const uint4& q, float (&v)[4]) {
  v[0] = __uint_as_float(q.x); v[1] = __uint_as_float(q.y); v[2] = __uint_as_float(q.z); v[3] = __uint_as_float(q.w);
}
__device__ __forceinline__ void unpack(const uint4& q, float (&v)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack(const float (&v)[4]) {
  return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}
__device__ __forceinline__ uint4 pack(const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Whole 16-byte vectors, U of them a thread with their loads in flight together
// while the words are drawn; the last block also takes the n % V values behind them.
// x and out may be the same array: a thread reads its values before it writes them.
constexpr int U = 4;
template <typename T, bool RES>
__global__ void __launch_bounds__(256) dropout_kernel(const T* x, const T* res, T* out, int64_t n, uint32_t last, bool all,
                                                      float scale, const uint64_t* rng) {
  constexpr int V = 16 / (int)sizeof(T);
  pdl_wait();
  pdl_trigger();
  const uint64_t draw = rng[1];
  const int64_t vecs = n / V;
  const int64_t first = (int64_t)blockIdx.x * (256 * U) + threadIdx.x;
  uint4 qx[U], qr[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t i = first + u * 256;
    qx[u] = qr[u] = make_uint4(0, 0, 0, 0);
    if (i < vecs) {
      qx[u] = reinterpret_cast<const uint4*>(x)[i];
      if (RES) qr[u] = reinterpret_cast<const uint4*>(res)[i];
    }
  }
  const Keys key(rng[0]);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t i = first + u * 256;
    if (i >= vecs) break;
    float v[V], r[V];
    unpack(qx[u], v);
    unpack(qr[u], r);
#pragma unroll
    for (int q = 0; q < V / 4; ++q) {
      const uint4 w = philox((uint64_t)(i * (V / 4) + q), draw, key);
      v[4 * q] = dropped(v[4 * q], r[4 * q], w.x, last, all, scale);
      v[4 * q + 1] = dropped(v[4 * q + 1], r[4 * q + 1], w.y, last, all, scale);
      v[4 * q + 2] = dropped(v[4 * q + 2], r[4 * q + 2], w.z, last, all, scale);
      v[4 * q + 3] = dropped(v[4 * q + 3], r[4 * q + 3], w.w, last, all, scale);
    }
    reinterpret_cast<uint4*>(out)[i] = pack(v);
  }
  const int64_t i = vecs * V + threadIdx.x;
  if (blockIdx.x == gridDim.x - 1 && i < n) {
    const uint4 w = philox((uint64_t)(i / 4), draw, key);
    const uint32_t word = i % 4 == 0 ? w.x : i % 4 == 1 ? w.y : i % 4 == 2 ? w.z : w.w;
    out[i] = from_f32<T>(dropped(to_f32<T>(x[i]), RES ? to_f32<T>(res[i]) : 0.0f, word, last, all, scale));
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
  const uint32_t last = (uint32_t)(cut - 1);       // cut = 0 keeps all: not looked at
  const float scale = p < 1.0 ? (float)(1.0 / (1.0 - p)) : 0.0f;
  const int64_t vecs = n / (dtype == MOE_DTYPE_F32 ? 4 : 8);
  const int64_t blocks = (vecs + 256 * U - 1) / (256 * U);
  if (blocks > 0x7FFFFFFF) return fail(MOE_ERR_UNSUPPORTED, "n=%lld", (long long)n);
  const dim3 grid((unsigned)(blocks > 0 ? blocks : 1));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto start = [&](auto zero) {
    using T = decltype(zero);
    return launch_pdl(res ? dropout_kernel<T, true> : dropout_kernel<T, false>, grid, dim3(256), 0, st,
                      static_cast<const T*>(x), static_cast<const T*>(res), static_cast<T*>(out), n, last, cut == 0, scale, rng);
  };
  const cudaError_t e = dtype == MOE_DTYPE_F32 ? start(float{}) : start(bf16{});
  return launch_status(e, "dropout");
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
