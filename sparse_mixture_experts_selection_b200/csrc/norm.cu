// Norm of the rows in front of the router and the experts, and its backward.
//
//   c = x - mean(x) (layer) or x (rms);  rstd = 1 / sqrt(mean(c^2) + eps)
//   y = c * rstd * gamma + beta;  optionally y once more as e4m3 tiles of 1 x 128
//   backward, xhat = c * rstd, g = gamma * dy:
//     dx = rstd * (g - mean(g) [layer] - xhat * mean(g * xhat)) + dres
//     dgamma = sum_rows dy * xhat,  dbeta = sum_rows dy
//
// Both are bound by memory: one pass over the data.  A row lives in the registers of W warps
// (NV 16-byte vectors per lane), so the centred sum of squares needs no second
// read and does not cancel for rows with a large mean; sums go lane -> warp
// (shuffles) -> row (shared memory), always in the same order.
#include <algorithm>
#include <cmath>

#include "api.h"
#include "common.cuh"
#include "e4m3.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kMaxNormCols = 16384;
constexpr int kSms = 148;
constexpr int kNormGrid = 2 * kSms;      // blocks of the row-by-row backward: their partial sums are the workspace
// Wide rows run in resident blocks that walk the rows, the next kDepth rows on their way
// to shared memory meanwhile: see ring_norm_kernel.
constexpr int kDepth = 3;
constexpr int grad_depth(int W) { return W == 32 ? 2 : 4; }    // of the backward: 192 KB
constexpr int kRingRows = 3 * kSms, kRingVecs = 128, kRingGradVecs = 64;     // where those run

// How rows map to warps: W warps per row, NV vectors of V elements per lane,
// `slots` rows at a time in a block of `threads`.
struct NormShape {
  int W, NV, threads, slots;
};

NormShape norm_shape(int d, int dtype, int max_nv) {
  const int V = dtype == MOE_DTYPE_F32 ? 4 : 8;
  const int nvec = (d + V - 1) / V;
  NormShape s{};
  s.W = 1;
  while (s.W < 32 && (nvec + 32 * s.W - 1) / (32 * s.W) > max_nv) s.W *= 2;
  const int nv = (nvec + 32 * s.W - 1) / (32 * s.W);
  s.NV = nv <= 1 ? 1 : nv <= 2 ? 2 : 4;
  s.threads = s.W <= 8 ? 256 : 32 * s.W;
  s.slots = s.threads / (32 * s.W);
  return s;
}

template <typename T> struct Vec;
template <> struct Vec<float> {
  static constexpr int N = 4;
  __device__ static void unpack(const uint4& q, float (&v)[4]) {
    v[0] = __uint_as_float(q.x); v[1] = __uint_as_float(q.y);
    v[2] = __uint_as_float(q.z); v[3] = __uint_as_float(q.w);
  }
  __device__ static uint4 pack(const float (&v)[4]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
  __device__ static uint32_t bits(float v) { return __float_as_uint(v); }
  __device__ static float value(uint32_t b) { return __uint_as_float(b); }
};
template <> struct Vec<bf16> {
  static constexpr int N = 8;
  __device__ static void unpack(const uint4& q, float (&v)[8]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ static uint4 pack(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// One lane's share of a row.  VECTOR: slot i of the lane is the 16-byte vector
// i * 32W + lane, when d is a whole number of vectors (every row then starts
// on 16 bytes); otherwise element j of slot i is column (i * N + j) * 32W + lane,
// single loads that neighbouring lanes make side by side.
template <typename T, int W, bool VECTOR>
struct Row {
  static constexpr int N = Vec<T>::N, L = 32 * W;
  __device__ static int col(int i, int j, int lane) { return VECTOR ? (i * L + lane) * N + j : (i * N + j) * L + lane; }
  // whole vectors are inside or outside together
  __device__ static bool inside(int i, int j, int lane, int d) { return col(i, VECTOR ? 0 : j, lane) < d; }
  // columns at or beyond d read as `other`
  __device__ static void load(const T* p, int d, int i, int lane, float other, float (&v)[N]) {
    if (VECTOR) {
      const int c = (i * L + lane) * N;
      if (c < d) {
        Vec<T>::unpack(*reinterpret_cast<const uint4*>(p + c), v);
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = other;
      }
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int c = col(i, j, lane);
        v[j] = c < d ? to_f32<T>(p[c]) : other;
      }
    }
  }
  __device__ static void store(T* p, int d, int i, int lane, const float (&v)[N]) {
    if (VECTOR) {
      const int c = (i * L + lane) * N;
      if (c < d) *reinterpret_cast<uint4*>(p + c) = Vec<T>::pack(v);
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int c = col(i, j, lane);
        if (c < d) p[c] = from_f32<T>(v[j]);
      }
    }
  }
  // the same columns of an fp32 array (null: `other`)
  __device__ static void load_f32(const float* p, int d, int i, int lane, float other, float (&v)[N]) {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = other;
    if (!p) return;
    if (VECTOR) {
      const int c = (i * L + lane) * N;
      if (c >= d) return;
      if ((reinterpret_cast<uintptr_t>(p) & 15u) == 0) {       // gains are only promised 4-byte alignment
#pragma unroll
        for (int j = 0; j < N; j += 4) {
          const float4 q = *reinterpret_cast<const float4*>(p + c + j);
          v[j] = q.x; v[j + 1] = q.y; v[j + 2] = q.z; v[j + 3] = q.w;
        }
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = p[c + j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int c = col(i, j, lane);
        if (c < d) v[j] = p[c];
      }
    }
  }
};

// Sums of K values over the W warps of a row, the same in every lane.  Called by
// all threads of the block; buf holds two generations so that one barrier per
// call is enough.
template <int W, int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float (*buf)[32 * K], int& gen) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(kFull, v[k], off);
  if (W == 1) return;
  const int warp = threadIdx.x / kWarp;
  float* b = buf[gen];
  if (threadIdx.x % kWarp == 0)
#pragma unroll
    for (int k = 0; k < K; ++k) b[k * 32 + warp] = v[k];
  __syncthreads();
  // lane l takes the sum of warp l % W of the row; W is a power of two
  const int from = warp / W * W + threadIdx.x % W;
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = b[k * 32 + from];
#pragma unroll
  for (int off = W / 2; off > 0; off >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(kFull, v[k], off);
  gen ^= 1;
}

struct NormArgs {
  const void* x;
  const float *gamma, *beta;
  void* out;
  float *mean, *rstd;
  uint8_t* codes;
  float* scales;
  int64_t n_rows;
  int d;
  float eps;
};

// One row, in the registers of its W warps (r >= n_rows: only the barriers are kept).
template <typename T, int W, int NV, bool VECTOR, bool LAYER, bool TILES>
__device__ __forceinline__ void normalize(const NormArgs& a, float (&v)[NV][Vec<T>::N], int64_t r, int lane, float inv_d,
                                          const float (&g)[NV][Vec<T>::N], const float (&b)[NV][Vec<T>::N],
                                          float (*buf)[32], int& gen) {
  using R = Row<T, W, VECTOR>;
  constexpr int N = R::N, L = R::L;
  const int d = a.d;
  const bool valid = r < a.n_rows;
  float mean = 0.0f;
  if (LAYER) {
    float s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < N; ++j) s[0] += v[i][j];
    row_sum<W, 1>(s, buf, gen);
    mean = s[0] * inv_d;
  }
  float q[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (LAYER) v[i][j] -= R::inside(i, j, lane, d) ? mean : 0.0f;     // beyond the row: 0 - 0
      q[0] = fmaf(v[i][j], v[i][j], q[0]);
    }
  row_sum<W, 1>(q, buf, gen);
  const float rstd = 1.0f / sqrtf(q[0] * inv_d + a.eps);
  if (valid && lane == 0) {
    if (a.mean) a.mean[r] = mean;
    if (a.rstd) a.rstd[r] = rstd;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int j = 0; j < N; ++j) v[i][j] = fmaf(v[i][j] * rstd, g[i][j], b[i][j]);
    if (valid && a.out) R::store(static_cast<T*>(a.out) + r * d, d, i, lane, v[i]);
    if (TILES) {
      // the stored values, in tiles of 128 columns = 128 / N neighbouring lanes
      const int c = (i * L + lane) * N;
      float top = 0.0f;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        v[i][j] = c < d ? to_f32<T>(from_f32<T>(v[i][j])) : 0.0f;
        top = fmaxf(top, fabsf(v[i][j]));
      }
#pragma unroll
      for (int off = 64 / N; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
      const int e = e4m3_scale_exponent(top);
      const float inv = pow2(-e);
      if (valid && c < d) {
        uint32_t w[N / 4];
#pragma unroll
        for (int j = 0; j < N; j += 4)
          w[j / 4] = e4m3_pack4(v[i][j] * inv, v[i][j + 1] * inv, v[i][j + 2] * inv, v[i][j + 3] * inv);
        uint8_t* out = a.codes + r * d + c;
        if (N == 8) *reinterpret_cast<uint2*>(out) = make_uint2(w[0], w[N / 4 - 1]);
        else *reinterpret_cast<uint32_t*>(out) = w[0];
        if (c % 128 == 0) a.scales[r * ((d + 127) / 128) + c / 128] = pow2(e);
      }
    }
  }
}

template <typename T, int W, int NV, bool VECTOR, bool LAYER, bool TILES>
__global__ void __launch_bounds__(W <= 8 ? 256 : 32 * W) norm_kernel(const NormArgs a) {
  using R = Row<T, W, VECTOR>;
  constexpr int N = R::N, L = R::L, SLOTS = (W <= 8 ? 256 : 32 * W) / L;
  __shared__ float buf[2][32];
  int gen = 0;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x % L;
  const int64_t r = (int64_t)blockIdx.x * SLOTS + threadIdx.x / L;
  const int d = a.d;
  const T* x = static_cast<const T*>(a.x) + (r < a.n_rows ? r : 0) * d;
  float v[NV][N], g[NV][N], b[NV][N];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    R::load(x, d, i, lane, 0.0f, v[i]);
    R::load_f32(a.gamma, d, i, lane, 1.0f, g[i]);
    R::load_f32(a.beta, d, i, lane, 0.0f, b[i]);
  }
  normalize<T, W, NV, VECTOR, LAYER, TILES>(a, v, r, lane, 1.0f / (float)d, g, b, buf, gen);
}

struct NormGradArgs {
  const void *dy, *x, *dres;
  const float *gamma, *mean, *rstd;
  void* dx;
  float* part;               // [parts][2][d]: dgamma, dbeta of one block slot's rows
  int64_t n_rows;
  int d, want_sums;
};

// A block walks rows blockIdx * SLOTS + slot, += grid * SLOTS; its lanes keep
// their columns' gains and the running dgamma, dbeta in registers.
template <typename T, int W, int NV, bool VECTOR, bool LAYER>
__global__ void __launch_bounds__(W <= 8 ? 256 : 32 * W) norm_grad_kernel(const NormGradArgs a) {
  using R = Row<T, W, VECTOR>;
  constexpr int N = R::N, L = R::L, SLOTS = (W <= 8 ? 256 : 32 * W) / L;
  __shared__ float buf[2][64];
  int gen = 0;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x % L, slot = threadIdx.x / L;
  const int d = a.d;
  const float inv_d = 1.0f / (float)d;
  float gamma[NV][N], dg[NV][N], db[NV][N];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    R::load_f32(a.gamma, d, i, lane, 1.0f, gamma[i]);
#pragma unroll
    for (int j = 0; j < N; ++j) dg[i][j] = db[i][j] = 0.0f;
  }
  const int64_t step = (int64_t)gridDim.x * SLOTS;
  for (int64_t r0 = (int64_t)blockIdx.x * SLOTS; r0 < a.n_rows; r0 += step) {
    const int64_t r = r0 + slot;
    const bool valid = r < a.n_rows;
    const T* xr = static_cast<const T*>(a.x) + (valid ? r : r0) * d;
    const T* dyr = static_cast<const T*>(a.dy) + (valid ? r : r0) * d;
    float xh[NV][N], dy[NV][N];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      R::load(xr, d, i, lane, 0.0f, xh[i]);
      R::load(dyr, d, i, lane, 0.0f, dy[i]);
    }
    const float rstd = valid ? a.rstd[r] : 0.0f;
    const float mean = LAYER && valid ? a.mean[r] : 0.0f;
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < N; ++j) {
        if (!R::inside(i, j, lane, d)) { xh[i][j] = 0.0f; continue; }
        xh[i][j] = (xh[i][j] - mean) * rstd;
        if (valid) {
          dg[i][j] = fmaf(dy[i][j], xh[i][j], dg[i][j]);
          db[i][j] += dy[i][j];
        }
        dy[i][j] *= gamma[i][j];
        s[0] += dy[i][j];
        s[1] = fmaf(dy[i][j], xh[i][j], s[1]);
      }
    row_sum<W, 2>(s, buf, gen);
    const float m1 = LAYER ? s[0] * inv_d : 0.0f, m2 = s[1] * inv_d;
    if (!valid) continue;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float o[N], res[N];
      if (a.dres) R::load(static_cast<const T*>(a.dres) + r * d, d, i, lane, 0.0f, res);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        o[j] = rstd * (dy[i][j] - m1 - xh[i][j] * m2);
        if (a.dres) o[j] += res[j];
      }
      R::store(static_cast<T*>(a.dx) + r * d, d, i, lane, o);
    }
  }
  if (!a.want_sums) return;
  float* part = a.part + ((size_t)blockIdx.x * SLOTS + slot) * 2 * d;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int c = R::col(i, j, lane);
      if (c < d) { part[c] = dg[i][j]; part[d + c] = db[i][j]; }
    }
}

// ---------------------------------------------------------------------------
// wide rows
// ---------------------------------------------------------------------------
// Each thread copies its own two vectors of a row to its own place in shared
// memory (cp.async, past the L1 cache) kDepth rows ahead, so nothing but the sums is
// shared between threads, the loads in flight do not wait for the sums, and
// gains stay in registers.  One block per row instead reads the gains again with each
// row and has no load in flight while it sums: 47 against 27 us for 4096 x 7168 bf16
// (4.3 TB/s; a plain copy of that size takes 21 us), and depth 4 or 6 takes 31 or 33.
// From three rows an SM on (bf16, 7168 columns, ring and block per row: 296 rows 4.2 and 4.7 us, 444 rows
// 5.8 and 8.0, 1184 rows 9.1 and 15.3) and rows of 128 16-byte vectors (8192 rows of 1024 columns
// 11.8 and 14.2, of 512 columns 10.8 and 6.4: half of the threads have none).
// What it uses most of now are issue slots, 69 % (20 instructions a value; the rms kind, with
// fewer of them and one sum a row instead of two, takes 20 us); neither they nor memory are at
// their limit.  fp32, with half the instructions a byte: 42 us, 5.6 TB/s.
// Times are of calls over inputs in turn, on the device; one by itself with a cold L2 takes 4 to 6 us longer.
__device__ __forceinline__ void copy16(void* smem, const void* global, bool in) {
  const int bytes = in ? 16 : 0;                       // 0: zeros are written
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(smem)), "l"(global), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

constexpr int kRingNV = 2;

template <typename T, int W, bool LAYER, bool TILES>
__global__ void __launch_bounds__(32 * W, W <= 16 ? 32 / W : 1) ring_norm_kernel(const NormArgs a) {
  using R = Row<T, W, true>;
  constexpr int N = R::N, L = R::L, NV = kRingNV;
  extern __shared__ uint4 ring[];                      // [kDepth][NV][L]
  __shared__ float buf[2][32];
  int gen = 0;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x, d = a.d;
  const T* x = static_cast<const T*>(a.x);
  auto fetch = [&](int64_t r, int slot) {
    if (r < a.n_rows) {
      const int64_t at = r * d + lane * N;
      uint4* to = ring + slot * (NV * L) + lane;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const bool in = R::col(i, 0, lane) < d;
        copy16(to + i * L, x + (in ? at + i * L * N : 0), in);
      }
    }
    copy_commit();
  };
#pragma unroll
  for (int k = 0; k < kDepth - 1; ++k) fetch(blockIdx.x + (int64_t)k * gridDim.x, k);
  float g[NV][N], b[NV][N];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    R::load_f32(a.gamma, d, i, lane, 1.0f, g[i]);
    R::load_f32(a.beta, d, i, lane, 0.0f, b[i]);
  }
  const float inv_d = 1.0f / (float)d;
  int slot = 0;
  for (int64_t r = blockIdx.x; r < a.n_rows; r += gridDim.x) {
    fetch(r + (int64_t)(kDepth - 1) * gridDim.x, (slot + kDepth - 1) % kDepth);
    copy_wait<kDepth - 1>();
    float v[NV][N];
#pragma unroll
    for (int i = 0; i < NV; ++i) Vec<T>::unpack(ring[(slot * NV + i) * L + lane], v[i]);
    slot = slot + 1 == kDepth ? 0 : slot + 1;
    normalize<T, W, NV, true, LAYER, TILES>(a, v, r, lane, inv_d, g, b, buf, gen);
  }
}

// The backward: gains, the running dgamma and dbeta and the row in registers, one block
// of 512 threads on an SM: 44 us for 4096 x 7168 bf16 with dres (5.3 TB/s), and 4 for
// the parts' sums.  The row read twice from shared memory with 1024 threads on an SM
// took 41 instructions a value instead of 28 and 64 us, 1024 threads with one vector
// each 73 us.  It wins for any number of rows from 64 vectors a row on, where norm_grad_kernel
// would need a second warp a row (bf16, this and norm_grad_kernel, with the parts' sums: 1 x 7168 6.5 and
// 11.8 us, 64 x 7168 8.7 and 15.5, 444 x 7168 13 and 32, 512 x 512 6.2 and 9.9; with 32 vectors 8192 x 256
// 18 and 21, 32768 x 256 57 and 32).
// Rows of more than 1024 vectors take 1024 threads, whose 64 registers do not hold gains, running sums and the
// row of the widest: bf16 kernels of more than 8192 columns spill 340 to 468 bytes a thread here and in
// norm_grad_kernel, fp32 ones 296 to 404 in norm_grad_kernel; with the parts' sums 4096 x 9000 bf16 142 us,
// 4096 x 16384 bf16 157 (2.6 TB/s), fp32 238 (3.4 TB/s).
template <typename T, int W, bool LAYER>
__global__ void __launch_bounds__(32 * W, W <= 16 ? 16 / W : 1) ring_norm_grad_kernel(const NormGradArgs a) {
  using R = Row<T, W, true>;
  constexpr int N = R::N, L = R::L, NV = kRingNV, DEPTH = grad_depth(W);
  extern __shared__ uint4 ring[];                      // [DEPTH][dy, x, dres][NV][L]
  __shared__ float buf[2][64];
  int gen = 0;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x, d = a.d;
  const int arrays = a.dres ? 3 : 2;
  const T *dy_ = static_cast<const T*>(a.dy), *x_ = static_cast<const T*>(a.x), *dres_ = static_cast<const T*>(a.dres);
  auto fetch = [&](int64_t r, int slot) {
    if (r < a.n_rows) {
      const int64_t at = r * d + lane * N;
      uint4* to = ring + slot * (3 * NV * L) + lane;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const bool in = R::col(i, 0, lane) < d;
        const int64_t c = in ? at + i * L * N : 0;
        copy16(to + i * L, dy_ + c, in);
        copy16(to + (NV + i) * L, x_ + c, in);
        if (arrays == 3) copy16(to + (2 * NV + i) * L, dres_ + c, in);
      }
    }
    copy_commit();
  };
#pragma unroll
  for (int k = 0; k < DEPTH - 1; ++k) fetch(blockIdx.x + (int64_t)k * gridDim.x, k);
  float gamma[NV][N], dg[NV][N], db[NV][N];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    R::load_f32(a.gamma, d, i, lane, 1.0f, gamma[i]);
#pragma unroll
    for (int j = 0; j < N; ++j) dg[i][j] = db[i][j] = 0.0f;
  }
  const float inv_d = 1.0f / (float)d;
  int slot = 0;
  float next_rstd = 0.0f, next_mean = 0.0f;            // a row ahead, like the row itself
  if (blockIdx.x < a.n_rows) {
    next_rstd = a.rstd[blockIdx.x];
    if (LAYER) next_mean = a.mean[blockIdx.x];
  }
  for (int64_t r = blockIdx.x; r < a.n_rows; r += gridDim.x) {
    fetch(r + (int64_t)(DEPTH - 1) * gridDim.x, (slot + DEPTH - 1) % DEPTH);
    const float rstd = next_rstd, mean = next_mean;
    if (r + gridDim.x < a.n_rows) {
      next_rstd = a.rstd[r + gridDim.x];
      if (LAYER) next_mean = a.mean[r + gridDim.x];
    }
    copy_wait<DEPTH - 1>();
    const uint4* from = ring + slot * (3 * NV * L) + lane;
    float dy[NV][N], xh[NV][N], s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      Vec<T>::unpack(from[i * L], dy[i]);              // zeros beyond the row: they add nothing
      Vec<T>::unpack(from[(NV + i) * L], xh[i]);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        xh[i][j] = (xh[i][j] - mean) * rstd;
        dg[i][j] = fmaf(dy[i][j], xh[i][j], dg[i][j]);
        db[i][j] += dy[i][j];
        dy[i][j] *= gamma[i][j];
        s[0] += dy[i][j];
        s[1] = fmaf(dy[i][j], xh[i][j], s[1]);
      }
    }
    row_sum<W, 2>(s, buf, gen);
    // rstd (g - m1 - xhat m2) as (rstd g - rstd m1) - xhat (rstd m2)
    const float m1 = LAYER ? s[0] * inv_d * rstd : 0.0f, m2 = s[1] * inv_d * rstd;
    T* dx = static_cast<T*>(a.dx) + r * d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float o[N];
#pragma unroll
      for (int j = 0; j < N; ++j) o[j] = fmaf(-xh[i][j], m2, LAYER ? fmaf(dy[i][j], rstd, -m1) : dy[i][j] * rstd);
      if (arrays == 3) {
        float res[N];
        Vec<T>::unpack(from[(2 * NV + i) * L], res);
#pragma unroll
        for (int j = 0; j < N; ++j) o[j] += res[j];
      }
      R::store(dx, d, i, lane, o);
    }
    slot = slot + 1 == DEPTH ? 0 : slot + 1;
  }
  if (!a.want_sums) return;
  float* part = a.part + (size_t)blockIdx.x * 2 * d;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = R::col(i, 0, lane);
    if (c >= d) continue;
#pragma unroll
    for (int j = 0; j < N; j += 4) {
      *reinterpret_cast<float4*>(part + c + j) = make_float4(dg[i][j], dg[i][j + 1], dg[i][j + 2], dg[i][j + 3]);
      *reinterpret_cast<float4*>(part + d + c + j) = make_float4(db[i][j], db[i][j + 1], db[i][j + 2], db[i][j + 3]);
    }
  }
}

// dgamma (blockIdx.y = 0) and dbeta (1): the parts summed in a fixed order, 32
// columns per block, 32 interleaved runs of parts joined at the end.
__global__ void __launch_bounds__(1024) norm_grad_sum_kernel(const float* part, int parts, int d, float* dgamma,
                                                             float* dbeta) {
  __shared__ float s[32][33];
  pdl_wait();
  pdl_trigger();
  float* out = blockIdx.y == 0 ? dgamma : dbeta;
  if (!out) return;
  const int cx = threadIdx.x % 32, py = threadIdx.x / 32;
  const int c = blockIdx.x * 32 + cx;
  float v = 0.0f;
  if (c < d)
#pragma unroll 4
    for (int p = py; p < parts; p += 32) v += part[((size_t)p * 2 + blockIdx.y) * d + c];
  s[py][cx] = v;
  __syncthreads();
  // warp py holds column py's runs
  v = s[cx][py];
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
  if (cx == 0 && blockIdx.x * 32 + py < d) out[blockIdx.x * 32 + py] = v;
}

template <typename T, int W, int NV, bool VECTOR, bool LAYER>
cudaError_t start_norm(const NormArgs& a, const NormShape& s, cudaStream_t st) {
  const dim3 grid((unsigned)((a.n_rows + s.slots - 1) / s.slots));
  if constexpr (VECTOR) {
    if (a.codes) return launch_pdl(norm_kernel<T, W, NV, VECTOR, LAYER, true>, grid, dim3(s.threads), 0, st, a);
  }
  return launch_pdl(norm_kernel<T, W, NV, VECTOR, LAYER, false>, grid, dim3(s.threads), 0, st, a);
}

template <typename T, int W, int NV, bool VECTOR, bool LAYER>
cudaError_t start_norm_grad(const NormGradArgs& a, const NormShape& s, int grid, cudaStream_t st) {
  return launch_pdl(norm_grad_kernel<T, W, NV, VECTOR, LAYER>, dim3(grid), dim3(s.threads), 0, st, a);
}

// Warps per row of the resident blocks for rows of at least min_vecs vectors, 0 where one
// block per row (or warp) runs.
int ring_warps(int min_vecs, int d, int dtype) {
  const int V = dtype == MOE_DTYPE_F32 ? 4 : 8;
  if (d % V || d / V < min_vecs || d / V > 32 * 32 * kRingNV) return 0;
  int W = 4;
  while (d / V > 32 * W * kRingNV) W *= 2;
  return W;
}
int ring_grad_grid(int W, int64_t n_rows) {
  return (int)std::min<int64_t>(n_rows, W >= 16 ? kSms : kSms * 16 / W);        // 512 threads of an SM
}

// 48 KB of static and dynamic shared memory need no permission
template <typename K>
cudaError_t allow_smem(K kernel, size_t bytes) {
  return bytes <= 47 * 1024 ? cudaSuccess
                            : cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <typename T, int W, bool LAYER, bool TILES>
cudaError_t start_ring(const NormArgs& a, cudaStream_t st) {
  const size_t smem = (size_t)kDepth * kRingNV * 32 * W * 16;
  const int per_sm = W <= 16 ? 32 / W : 1;             // 1024 threads, 128 KB at most
  const dim3 grid((unsigned)(a.n_rows < kSms * per_sm ? a.n_rows : kSms * per_sm));
  const cudaError_t e = allow_smem(ring_norm_kernel<T, W, LAYER, TILES>, smem);
  return e != cudaSuccess ? e : launch_pdl(ring_norm_kernel<T, W, LAYER, TILES>, grid, dim3(32 * W), smem, st, a);
}
template <typename T, int W, bool LAYER>
cudaError_t start_ring(const NormArgs& a, cudaStream_t st) {
  return a.codes ? start_ring<T, W, LAYER, true>(a, st) : start_ring<T, W, LAYER, false>(a, st);
}
template <typename T, bool LAYER>
cudaError_t start_ring(int W, const NormArgs& a, cudaStream_t st) {
  return W == 4 ? start_ring<T, 4, LAYER>(a, st) : W == 8 ? start_ring<T, 8, LAYER>(a, st)
       : W == 16 ? start_ring<T, 16, LAYER>(a, st) : start_ring<T, 32, LAYER>(a, st);
}

template <typename T, int W, bool LAYER>
cudaError_t start_ring_grad(const NormGradArgs& a, cudaStream_t st) {
  const size_t smem = (size_t)grad_depth(W) * 3 * kRingNV * 32 * W * 16;
  const cudaError_t e = allow_smem(ring_norm_grad_kernel<T, W, LAYER>, smem);
  return e != cudaSuccess ? e : launch_pdl(ring_norm_grad_kernel<T, W, LAYER>, dim3(ring_grad_grid(W, a.n_rows)), dim3(32 * W),
                                           smem, st, a);
}
template <typename T, bool LAYER>
cudaError_t start_ring_grad(int W, const NormGradArgs& a, cudaStream_t st) {
  return W == 4 ? start_ring_grad<T, 4, LAYER>(a, st) : W == 8 ? start_ring_grad<T, 8, LAYER>(a, st)
       : W == 16 ? start_ring_grad<T, 16, LAYER>(a, st) : start_ring_grad<T, 32, LAYER>(a, st);
}

// F(T, W, NV, VECTOR, LAYER) for the shape; one- and two-vector rows take one warp.
#define MOE_NORM_PICK(F, T, ...)                                                        \
  [&]() -> cudaError_t {                                                                \
    auto pick = [&](auto vec, auto layer) -> cudaError_t {                              \
      constexpr bool VEC = decltype(vec)::value, LAY = decltype(layer)::value;          \
      if (s.W == 1) {                                                                   \
        if (s.NV == 1) return F<T, 1, 1, VEC, LAY>(__VA_ARGS__);                        \
        if (s.NV == 2) return F<T, 1, 2, VEC, LAY>(__VA_ARGS__);                        \
      }                                                                                 \
      MOE_NORM_WIDE(F, T, __VA_ARGS__)                                                  \
      return cudaErrorInvalidValue;                                                     \
    };                                                                                  \
    if (vector) return layer ? pick(std::true_type{}, std::true_type{}) : pick(std::true_type{}, std::false_type{});     \
    return layer ? pick(std::false_type{}, std::true_type{}) : pick(std::false_type{}, std::false_type{});               \
  }()

moe_status check_rows(int dtype, int64_t n_rows, int d, int kind) {
  if (dtype != MOE_DTYPE_F32 && dtype != MOE_DTYPE_BF16) return fail(MOE_ERR_INVALID_ARG, "dtype=%d", dtype);
  if (n_rows < 0) return fail(MOE_ERR_INVALID_ARG, "n_rows=%lld < 0", (long long)n_rows);
  if (n_rows > 0x7FFFFFFF) return fail(MOE_ERR_UNSUPPORTED, "n_rows=%lld above 2^31", (long long)n_rows);
  if (d < 1) return fail(MOE_ERR_INVALID_ARG, "d=%d < 1", d);
  if (d > kMaxNormCols) return fail(MOE_ERR_UNSUPPORTED, "d=%d > %d", d, kMaxNormCols);
  if (kind != MOE_NORM_LAYER && kind != MOE_NORM_RMS) return fail(MOE_ERR_INVALID_ARG, "kind=%d", kind);
  return MOE_OK;
}

constexpr int kNormVecs = 4, kNormGradVecs = 2;

int norm_grad_grid(const NormShape& s, int64_t n_rows) {
  const int64_t blocks = (n_rows + s.slots - 1) / s.slots;
  return (int)(blocks < kNormGrid ? blocks : kNormGrid);
}

}  // namespace
}  // namespace moe

using namespace moe;

#define MOE_NORM_WIDE(F, T, ...)                                     \
  if (s.W == 1) return F<T, 1, 4, VEC, LAY>(__VA_ARGS__);            \
  if (s.W == 2) return F<T, 2, 4, VEC, LAY>(__VA_ARGS__);            \
  if (s.W == 4) return F<T, 4, 4, VEC, LAY>(__VA_ARGS__);            \
  if (s.W == 8) return F<T, 8, 4, VEC, LAY>(__VA_ARGS__);            \
  if (s.W == 16) return F<T, 16, 4, VEC, LAY>(__VA_ARGS__);          \
  if constexpr (sizeof(T) == 4) {                                    \
    if (s.W == 32) return F<T, 32, 4, VEC, LAY>(__VA_ARGS__);        \
  }

extern "C" moe_status moe_layer_norm(const void* x, int32_t dtype, int64_t n_rows, int32_t d, int32_t kind,
                                     const float* gamma, const float* beta, float eps, void* out, float* mean,
                                     float* rstd, uint8_t* codes, float* scales, void* stream) {
  MOE_CHECK(check_rows(dtype, n_rows, d, kind));
  if (!(eps > 0.0f) || !std::isfinite(eps)) return fail(MOE_ERR_INVALID_ARG, "eps must be positive and finite");
  if (codes && d % 16) return fail(MOE_ERR_INVALID_ARG, "codes need d=%d to be a multiple of 16", d);
  if (n_rows == 0) return MOE_OK;          // empty arrays have no addresses
  if (!out && !codes) return fail(MOE_ERR_INVALID_ARG, "out and codes are both NULL");
  if (!codes != !scales) return fail(MOE_ERR_INVALID_ARG, "codes and scales go together");
  MOE_NONNULL(x); MOE_ALIGNED(out); MOE_ALIGNED(codes);
  MOE_ALIGNED4(gamma); MOE_ALIGNED4(beta); MOE_ALIGNED4(mean); MOE_ALIGNED4(rstd); MOE_ALIGNED4(scales);
  const NormShape s = norm_shape(d, dtype, kNormVecs);
  NormArgs a{x, gamma, beta, out, mean, rstd, codes, scales, n_rows, d, eps};
  const bool layer = kind == MOE_NORM_LAYER;
  const bool vector = d % (dtype == MOE_DTYPE_F32 ? 4 : 8) == 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int W = n_rows < kRingRows ? 0 : ring_warps(kRingVecs, d, dtype);
  cudaError_t e;
  if (W && dtype == MOE_DTYPE_F32) e = layer ? start_ring<float, true>(W, a, st) : start_ring<float, false>(W, a, st);
  else if (W) e = layer ? start_ring<bf16, true>(W, a, st) : start_ring<bf16, false>(W, a, st);
  else if (dtype == MOE_DTYPE_F32) e = MOE_NORM_PICK(start_norm, float, a, s, st);
  else e = MOE_NORM_PICK(start_norm, bf16, a, s, st);
  return launch_status(e, "norm");
}

extern "C" moe_status moe_layer_norm_backward_workspace_size(int64_t n_rows, int32_t d, size_t* bytes) {
  MOE_CHECK(check_rows(MOE_DTYPE_F32, n_rows, d, MOE_NORM_LAYER));
  if (!bytes) return fail(MOE_ERR_INVALID_ARG, "bytes is NULL");
  size_t parts = 0;
  for (int dtype : {MOE_DTYPE_F32, MOE_DTYPE_BF16}) {
    const NormShape s = norm_shape(d, dtype, kNormGradVecs);
    const int W = ring_warps(kRingGradVecs, d, dtype);
    const size_t p = W ? (size_t)ring_grad_grid(W, n_rows) : (size_t)norm_grad_grid(s, n_rows) * s.slots;
    parts = p > parts ? p : parts;
  }
  *bytes = kAlign + align_up(parts * 2 * d * 4);
  return MOE_OK;
}

#undef MOE_NORM_WIDE
// rows of whole vectors that take more than a warp run in resident blocks, but for the longest
#define MOE_NORM_WIDE(F, T, ...)                                                \
  if constexpr (!VEC) {                                                         \
    if (s.W == 2) return F<T, 2, 2, VEC, LAY>(__VA_ARGS__);                     \
    if (s.W == 4) return F<T, 4, 2, VEC, LAY>(__VA_ARGS__);                     \
    if (s.W == 8) return F<T, 8, 2, VEC, LAY>(__VA_ARGS__);                     \
    if (s.W == 16) return F<T, 16, 2, VEC, LAY>(__VA_ARGS__);                   \
    if (s.W == 32 && s.NV <= 2) return F<T, 32, 2, VEC, LAY>(__VA_ARGS__);      \
  }                                                                             \
  if constexpr (sizeof(T) == 4) {                                               \
    if (s.W == 32) return F<T, 32, 4, VEC, LAY>(__VA_ARGS__);                   \
  }

extern "C" moe_status moe_layer_norm_backward(const void* dy, const void* x, int32_t dtype, int64_t n_rows, int32_t d,
                                              int32_t kind, const float* gamma, const float* mean, const float* rstd,
                                              const void* dres, void* dx, float* dgamma, float* dbeta, void* ws,
                                              size_t ws_bytes, void* stream) {
  MOE_CHECK(check_rows(dtype, n_rows, d, kind));
  size_t need = 0;
  MOE_CHECK(moe_layer_norm_backward_workspace_size(n_rows, d, &need));
  MOE_ALIGNED4(gamma); MOE_ALIGNED4(mean); MOE_ALIGNED4(dgamma); MOE_ALIGNED4(dbeta);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (n_rows == 0) {
    if (dgamma) cudaMemsetAsync(dgamma, 0, (size_t)d * 4, st);
    if (dbeta) cudaMemsetAsync(dbeta, 0, (size_t)d * 4, st);
    return cuda_status();
  }
  MOE_NONNULL(dy); MOE_NONNULL(x); MOE_NONNULL(dx); MOE_NONNULL4(rstd); MOE_ALIGNED(dres);
  if (kind == MOE_NORM_LAYER && !mean) return fail(MOE_ERR_INVALID_ARG, "mean is NULL");
  MOE_CHECK(check_ws(ws, ws_bytes, need));
  const NormShape s = norm_shape(d, dtype, kNormGradVecs);
  const int W = ring_warps(kRingGradVecs, d, dtype);
  const int grid = W ? ring_grad_grid(W, n_rows) : norm_grad_grid(s, n_rows);
  const int parts = W ? grid : grid * s.slots;
  float* part = at<float>(ws, kAlign);
  NormGradArgs a{dy, x, dres, gamma, mean, rstd, dx, part, n_rows, d, dgamma || dbeta};
  const bool layer = kind == MOE_NORM_LAYER;
  const bool vector = d % (dtype == MOE_DTYPE_F32 ? 4 : 8) == 0;
  cudaError_t e;
  if (W && dtype == MOE_DTYPE_F32) e = layer ? start_ring_grad<float, true>(W, a, st) : start_ring_grad<float, false>(W, a, st);
  else if (W) e = layer ? start_ring_grad<bf16, true>(W, a, st) : start_ring_grad<bf16, false>(W, a, st);
  else if (dtype == MOE_DTYPE_F32) e = MOE_NORM_PICK(start_norm_grad, float, a, s, grid, st);
  else e = MOE_NORM_PICK(start_norm_grad, bf16, a, s, grid, st);
  if (e == cudaSuccess && (dgamma || dbeta))
    e = launch_pdl(norm_grad_sum_kernel, dim3((d + 31) / 32, 2), dim3(1024), 0, st, part, parts, d, dgamma, dbeta);
  return launch_status(e, "norm backward");
}
