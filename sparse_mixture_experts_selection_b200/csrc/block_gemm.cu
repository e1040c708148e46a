// Grouped matrix products of block-scaled e4m3 operands, and the SwiGLU experts
// made of them, on the 5th-generation tensor cores:
//   out[r, j] = row_scale[r] * sum_b xs[r, b] * ws[g, j / 128, b] * sum_{k in b} x[r, k] * w[g, j, k]
//
// The scales differ from one block of 128 of the reduction to the next, so the
// tensor cores sum one block (four tcgen05.mma of 32) into tensor memory and
// eight warps add it, times the two scales, to fp32 accumulators in their
// registers, while the tensor cores fill the other tensor-memory buffer with the next block.
//
// Work unit = (group, 128-row tile, tile of 256 weight rows, range of blocks).
// The 256 weight rows are two blocks of 128: columns j .. j + 255 of the plain
// product, or the gate and the up rows of the same 128 columns of the SwiGLU
// product, whose epilogue then holds a whole 1 x 128 tile of each row of
// A = SiLU(U) V and quantizes it on the spot: A never reaches memory but as
// codes and scales.  Units of a group go row tile fastest, so CTAs that run
// together share weight tiles through L2 and weights stream from HBM about once.
//
// Few rows leave few units: the blocks of the reduction are then cut into ranges,
// each unit of a range leaves its accumulators in the workspace, and the last
// unit of a tile to finish adds the ranges in ascending order (so the sum
// does not depend on which one was last) and runs the epilogue.
//
// Warp roles (384 threads): warp 0 = TMA producer (+ tensor memory), warp 1 =
// MMA issuer, warps 4 .. 11 = accumulators and epilogue: warp w reads the tensor
// memory lanes of rows 32 (w % 4) .. + 31 and one half of the columns.  A thread
// of theirs holds 128 accumulators and 32 values on their way; the first four
// warps give up registers for that (setmaxnreg).
#include <algorithm>
#include <cuda.h>

#include "api.h"
#include "common.cuh"
#include "e4m3.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kBlock = 128;              // values per scale; also the k-block of a pipeline stage
constexpr int kMaxGroups = 1024;
constexpr int BM = 128, BN = 256;
constexpr int A_BYTES = BM * kBlock, B_BYTES = BN * kBlock;
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;      // 48 KB
constexpr int STAGES = 4;
constexpr int SUB_ROWS = 32;                        // row box of short row tiles
constexpr int EPI_WARPS = 8;
constexpr int NUM_THREADS = 128 + 32 * EPI_WARPS;
constexpr int EPI_THREAD0 = 128;
// 3 x 128 threads are launched with 168 registers each: 128 x 72 + 256 x 216 are as many
constexpr int FEW_REGS = 72, MANY_REGS = 216;
static_assert(128 * FEW_REGS + 32 * EPI_WARPS * MANY_REGS <= NUM_THREADS * 168, "registers of the launch");
constexpr int TMEM_COLS = 512;
constexpr int MAX_RANGES = 32;
// byte counters of the tiles whose reduction is cut, in the control block of the
// workspace: words 4 .. 63 (word 0 is the error word)
constexpr int COUNTER_WORD0 = 4, MAX_CUT_TILES = 60 * 4;
constexpr int PART_FLOATS = 128 * 32 * EPI_WARPS;   // accumulators of one unit

struct Control {
  uint64_t full[STAGES], empty[STAGES], acc_full[2], acc_empty[2], drain;
  uint32_t tmem;
  int abort, last, total;
  int warp_sum[NUM_THREADS / 32];
  float top[2][BM];                                 // SwiGLU: the two halves' row maxima
  int prefix[kMaxGroups + 1];                       // units of the groups before
};
constexpr size_t SMEM_BYTES = (size_t)STAGES * STAGE_BYTES + sizeof(Control) + 1024;
static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");

int blocks_of(int n) { return (n + kBlock - 1) / kBlock; }

struct BlockArgs {
  CUtensorMap x, x32, w0, w1;       // rows in boxes of 128 and 32; weights in boxes of 128 (gate, up)
  int G, N, K, max_rows;
  int KB, NB, NT;                   // blocks of the reduction and of the columns; column tiles
  int ranges, per;                  // ranges of the reduction, blocks per range
  const int* offsets;
  const float *xs, *ws0, *ws1, *row_scale;
  int out_f32;
  void* out;                        // plain: out; SwiGLU: the codes of A
  float* out_scale;                 // SwiGLU: the scales of A
  float* part;                      // [tiles][ranges][PART_FLOATS]
  int* ctrl;                        // the workspace's control block
};

struct Unit {
  int g, mt, nt, r0, rows;          // rows: of this tile
  int kb0, nk, range, tile;
};

__device__ __forceinline__ Unit decode(const BlockArgs& a, const int* prefix, int u) {
  int lo = 0, hi = a.G;             // prefix[lo] <= u < prefix[lo + 1]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= u) lo = mid; else hi = mid;
  }
  Unit w;
  w.g = lo;
  const int r0 = a.offsets ? __ldg(a.offsets + lo) : 0;
  const int r1 = a.offsets ? __ldg(a.offsets + lo + 1) : a.max_rows;
  const int mts = (r1 - r0 + BM - 1) / BM;
  w.tile = u / a.ranges;            // every group's units are whole tiles of `ranges` units
  int local = u - prefix[lo];
  w.range = local % a.ranges;
  local /= a.ranges;
  w.mt = local % mts;
  w.nt = local / mts;
  w.r0 = r0 + w.mt * BM;
  w.rows = min(BM, r1 - w.r0);
  w.kb0 = w.range * a.per;
  w.nk = min(a.KB, w.kb0 + a.per) - w.kb0;
  return w;
}

// Units before each group (prefix[G] = all) from the offsets; a group whose offsets
// are out of order or out of range has none and sets the error word.
__device__ __forceinline__ void scan_groups(const BlockArgs& a, Control* c) {
  const int t = threadIdx.x, warp = t / kWarp, lane = t % kWarp;
  constexpr int PER = (kMaxGroups + NUM_THREADS - 1) / NUM_THREADS;
  int n[PER], sum = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int g = t * PER + i;
    n[i] = 0;
    if (g < a.G) {
      const int r0 = a.offsets ? __ldg(a.offsets + g) : 0, r1 = a.offsets ? __ldg(a.offsets + g + 1) : a.max_rows;
      if (r0 < 0 || r1 < r0 || r1 > a.max_rows) set_device_error(a.ctrl, MOE_DEVERR_INDEX);
      else n[i] = (r1 - r0 + BM - 1) / BM * a.NT * a.ranges;
    }
    sum += n[i];
  }
  int inc = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int v = __shfl_up_sync(kFull, inc, off);
    if (lane >= off) inc += v;
  }
  if (lane == 31) c->warp_sum[warp] = inc;
  __syncthreads();
  int base = inc - sum;
  for (int w = 0; w < warp; ++w) base += c->warp_sum[w];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int g = t * PER + i;
    if (g <= a.G) c->prefix[g] = base;
    base += n[i];
  }
  __syncthreads();
}

// Wait without giving up on *abort (drains what is in flight before the CTA
// releases its shared and tensor memory).
__device__ __forceinline__ void wait_drain(uint64_t* bar, uint32_t parity, int* err) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity))
    if (global_timer_ns() - t0 > kWaitLimitNs) { set_device_error(err, MOE_DEVERR_WAIT_TIMEOUT); return; }
}

__device__ __forceinline__ uint64_t pack2(float a, float b) {
  return (uint64_t)__float_as_uint(a) | ((uint64_t)__float_as_uint(b) << 32);
}
__device__ __forceinline__ float low(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float high(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }

// acc += v * s, both halves
__device__ __forceinline__ void fma2(uint64_t& acc, uint64_t v, uint64_t s) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(v), "l"(s));
}

__device__ __forceinline__ float silu(float x) { return __fdividef(x, 1.0f + __expf(-x)); }

// Plain epilogue: this thread's row of the output, columns col0 .. col0 + 127.
__device__ __forceinline__ void store_row(const BlockArgs& a, const uint64_t (&acc)[64], int row, int col0) {
  const float rs = a.row_scale ? __ldg(a.row_scale + row) : 1.0f;
  const size_t base = (size_t)row * a.N + col0;
  const bool whole = col0 + 128 <= a.N;
  if (a.out_f32) {
    float* o = static_cast<float*>(a.out) + base;
    if (whole && a.N % 4 == 0) {
#pragma unroll
      for (int j = 0; j < 64; j += 2)
        *reinterpret_cast<float4*>(o + 2 * j) =
            make_float4(low(acc[j]) * rs, high(acc[j]) * rs, low(acc[j + 1]) * rs, high(acc[j + 1]) * rs);
    } else {
#pragma unroll
      for (int j = 0; j < 64; ++j) {
        if (col0 + 2 * j < a.N) o[2 * j] = low(acc[j]) * rs;
        if (col0 + 2 * j + 1 < a.N) o[2 * j + 1] = high(acc[j]) * rs;
      }
    }
    return;
  }
  bf16* o = static_cast<bf16*>(a.out) + base;
  if (whole && a.N % 8 == 0) {
#pragma unroll
    for (int j = 0; j < 64; j += 4) {
      uint32_t p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(low(acc[j + i]) * rs, high(acc[j + i]) * rs);
        p[i] = *reinterpret_cast<const uint32_t*>(&v);
      }
      *reinterpret_cast<uint4*>(o + 2 * j) = make_uint4(p[0], p[1], p[2], p[3]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 64; ++j) {
      if (col0 + 2 * j < a.N) o[2 * j] = from_f32<bf16>(low(acc[j]) * rs);
      if (col0 + 2 * j + 1 < a.N) o[2 * j + 1] = from_f32<bf16>(high(acc[j]) * rs);
    }
  }
}

// SwiGLU epilogue: this thread holds 64 gate (acc[0 .. 31]) and the same 64 up
// columns (acc[32 .. 63]) of its row; the other 64 columns of the 1 x 128 tile are
// with the warp of the other half, which shares the maximum through shared memory.
__device__ __forceinline__ void store_swiglu(const BlockArgs& a, const uint64_t (&acc)[64], const Unit& w, int r,
                                             int half, Control* c) {
  float v[64], top = 0.0f;
  const int col0 = w.nt * kBlock + half * 64;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    v[2 * j] = col0 + 2 * j < a.N ? silu(low(acc[j])) * low(acc[32 + j]) : 0.0f;
    v[2 * j + 1] = col0 + 2 * j + 1 < a.N ? silu(high(acc[j])) * high(acc[32 + j]) : 0.0f;
    top = fmaxf(top, fmaxf(fabsf(v[2 * j]), fabsf(v[2 * j + 1])));
  }
  const int quad = r / 32;
  c->top[half][r] = top;
  asm volatile("bar.sync %0, 64;" ::"r"(1 + quad) : "memory");
  top = fmaxf(top, c->top[half ^ 1][r]);
  asm volatile("bar.sync %0, 64;" ::"r"(1 + quad) : "memory");
  if (r >= w.rows) return;
  const int e = e4m3_scale_exponent(top);
  const float inv = pow2(-e);
  const size_t row = (size_t)(w.r0 + r);
  uint8_t* o = static_cast<uint8_t*>(a.out) + row * a.N + col0;
#pragma unroll
  for (int j = 0; j < 64; j += 16) {
    if (col0 + j >= a.N) break;                       // N is a multiple of 16
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      q[i] = e4m3_pack4(v[j + 4 * i] * inv, v[j + 4 * i + 1] * inv, v[j + 4 * i + 2] * inv, v[j + 4 * i + 3] * inv);
    *reinterpret_cast<uint4*>(o + j) = make_uint4(q[0], q[1], q[2], q[3]);
  }
  if (half == 0) a.out_scale[row * a.NB + w.nt] = pow2(e);
}

template <bool SWIGLU>
__global__ void __launch_bounds__(NUM_THREADS, 1) block_product_kernel(const __grid_constant__ BlockArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* sA = smem;
  uint8_t* sB = smem + STAGES * A_BYTES;
  Control* c = reinterpret_cast<Control*>(smem + STAGES * STAGE_BYTES);
  volatile int* abort_flag = &c->abort;
  int* err = a.ctrl;
  const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) { mbar_init(&c->full[s], 1); mbar_init(&c->empty[s], 1); }
    for (int b = 0; b < 2; ++b) { mbar_init(&c->acc_full[b], 1); mbar_init(&c->acc_empty[b], EPI_WARPS); }
    mbar_init(&c->drain, 1);
    c->abort = 0;
    fence_barrier_init();
  }
  if (warp == 0) tmem_alloc(&c->tmem, TMEM_COLS);
  if (warp == 1 && lane == 0) { prefetch_tmap(&a.x); prefetch_tmap(&a.x32); prefetch_tmap(&a.w0); prefetch_tmap(&a.w1); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  pdl_trigger();
  const uint32_t tmem = c->tmem;
  scan_groups(a, c);
  const int total = c->prefix[a.G];

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(FEW_REGS));
    if (warp == 0 && lane == 0) {
      // ---------------- TMA producer ----------------
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int u = blockIdx.x; u < total && ok; u += gridDim.x) {
        const Unit w = decode(a, c->prefix, u);
        const int sub = w.rows > BM - SUB_ROWS ? 0 : (w.rows + SUB_ROWS - 1) / SUB_ROWS;
        const int by = w.g * a.N + w.nt * (SWIGLU ? kBlock : BN);
        const bool two = SWIGLU || w.nt * BN + kBlock < a.N;
        const uint32_t tx = (uint32_t)(sub ? sub * SUB_ROWS * kBlock : A_BYTES) + (two ? B_BYTES : B_BYTES / 2);
        for (int i = 0; i < w.nk; ++i) {
          if (!mbar_wait(&c->empty[stage], phase ^ 1u, abort_flag, err)) { ok = false; break; }
          const int k = (w.kb0 + i) * kBlock;
          mbar_arrive_expect_tx(&c->full[stage], tx);
          // the weights first: they come from HBM, the rows mostly from L2
          tma_load_2d(sB + stage * B_BYTES, &a.w0, &c->full[stage], k, by);
          if (two) tma_load_2d(sB + stage * B_BYTES + B_BYTES / 2, &a.w1, &c->full[stage], k, SWIGLU ? by : by + kBlock);
          if (sub == 0) tma_load_2d(sA + stage * A_BYTES, &a.x, &c->full[stage], k, w.r0);
          for (int q = 0; q < sub; ++q)
            tma_load_2d(sA + stage * A_BYTES + q * SUB_ROWS * kBlock, &a.x32, &c->full[stage], k, w.r0 + q * SUB_ROWS);
          ++issued;
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      // the last loads must have landed before shared memory is released
      for (int i = 0; i < STAGES && i < issued; ++i) {
        if (--stage < 0) { stage = STAGES - 1; phase ^= 1u; }
        wait_drain(&c->full[stage], phase, err);
      }
    } else if (warp == 1 && lane == 0) {
      // ---------------- MMA issuer ----------------
      int stage = 0;
      uint32_t phase = 0, it = 0;          // it: blocks so far; buffer it % 2
      bool ok = true;
      for (int u = blockIdx.x; u < total && ok; u += gridDim.x) {
        const Unit w = decode(a, c->prefix, u);
        const uint32_t idesc = idesc_e4m3_f32(BM, SWIGLU || w.nt * BN + kBlock < a.N ? BN : kBlock);
        for (int i = 0; i < w.nk; ++i, ++it) {
          const uint32_t buf = it & 1u;
          if (!mbar_wait(&c->acc_empty[buf], ((it >> 1) & 1u) ^ 1u, abort_flag, err) ||
              !mbar_wait(&c->full[stage], phase, abort_flag, err)) { ok = false; break; }
          tc_fence_after();
          const uint32_t a0 = smem_u32(sA + stage * A_BYTES), b0 = smem_u32(sB + stage * B_BYTES);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc_mma_e4m3(tmem + buf * BN, sdesc_kmajor_sw128(a0 + 32 * k), sdesc_kmajor_sw128(b0 + 32 * k), idesc, k != 0);
          tc_commit(&c->empty[stage]);
          tc_commit(&c->acc_full[buf]);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      tc_commit(&c->drain);
      wait_drain(&c->drain, 0, err);
    }
  } else {
    // ---------------- accumulators and epilogue ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(MANY_REGS));
    const int quad = warp & 3, half = (warp - 4) / 4;
    const int r = quad * 32 + lane;
    const int t = threadIdx.x - EPI_THREAD0;
    uint32_t it = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < total && ok; u += gridDim.x) {
      const Unit w = decode(a, c->prefix, u);
      // warps without rows, or without columns, only keep the buffers moving
      const bool idle = quad * 32 >= w.rows || (!SWIGLU && w.nt * BN + half * kBlock >= a.N);
      const float* xs = a.xs + (size_t)(w.r0 + min(r, w.rows - 1)) * a.KB + w.kb0;
      const float* s0 = a.ws0 + ((size_t)w.g * a.NB + (SWIGLU ? w.nt : min(2 * w.nt + half, a.NB - 1))) * a.KB + w.kb0;
      const float* s1 = SWIGLU ? a.ws1 + ((size_t)w.g * a.NB + w.nt) * a.KB + w.kb0 : s0;
      // tensor-memory columns of the thread's 128: gate and up of half the tile, or one half of the columns
      const uint32_t base = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)(half * (SWIGLU ? 64 : 128));
      constexpr int SECOND = SWIGLU ? kBlock : 64;   // the last 64 columns, from `base`
      uint64_t acc[64];
#pragma unroll
      for (int j = 0; j < 64; ++j) acc[j] = 0;
      // scales are loaded two blocks ahead of their use
      float x0 = __ldg(xs), g0 = __ldg(s0), u0 = SWIGLU ? __ldg(s1) : 0.0f;
      float x1 = 0.0f, g1 = 0.0f, u1 = 0.0f;
      if (w.nk > 1) { x1 = __ldg(xs + 1); g1 = __ldg(s0 + 1); if (SWIGLU) u1 = __ldg(s1 + 1); }
      for (int i = 0; i < w.nk; ++i, ++it) {
        float x2 = 0.0f, g2 = 0.0f, u2 = 0.0f;
        if (i + 2 < w.nk) { x2 = __ldg(xs + i + 2); g2 = __ldg(s0 + i + 2); if (SWIGLU) u2 = __ldg(s1 + i + 2); }
        const uint32_t buf = it & 1u;
        if (!mbar_wait(&c->acc_full[buf], (it >> 1) & 1u, abort_flag, err)) { ok = false; break; }
        tc_fence_after();
        if (!idle) {
          const float sg = x0 * g0, su = SWIGLU ? x0 * u0 : sg;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float v[32];
            tmem_ld32(base + buf * BN + (q < 2 ? 32 * q : SECOND + 32 * (q - 2)), v);
            const float s = q < 2 ? sg : su;
            const uint64_t ss = pack2(s, s);
#pragma unroll
            for (int j = 0; j < 16; ++j) fma2(acc[16 * q + j], pack2(v[2 * j], v[2 * j + 1]), ss);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&c->acc_empty[buf]);
        x0 = x1; x1 = x2; g0 = g1; g1 = g2; u0 = u1; u1 = u2;
      }
      if (!ok) break;
      if (a.ranges > 1) {
        // leave the accumulators; the last range of the tile to arrive adds them in order
        float4* mine = reinterpret_cast<float4*>(a.part + ((size_t)w.tile * a.ranges + w.range) * PART_FLOATS);
        if (!idle && r < w.rows)
#pragma unroll
          for (int j = 0; j < 32; ++j)
            __stcg(mine + j * 256 + t, make_float4(low(acc[2 * j]), high(acc[2 * j]), low(acc[2 * j + 1]), high(acc[2 * j + 1])));
        __threadfence();
        asm volatile("bar.sync 5, 256;" ::: "memory");
        if (t == 0) {
          int* word = a.ctrl + COUNTER_WORD0 + w.tile / 4;
          const int shift = 8 * (w.tile % 4);
          const int before = (atomicAdd(word, 1 << shift) >> shift) & 255;
          if (before == a.ranges - 1) atomicSub(word, a.ranges << shift);      // ready for the next call
          c->last = before == a.ranges - 1;
          __threadfence();
        }
        asm volatile("bar.sync 5, 256;" ::: "memory");
        const bool last = c->last != 0;
        asm volatile("bar.sync 5, 256;" ::: "memory");
        if (!last) continue;
        if (!idle && r < w.rows) {
#pragma unroll
          for (int j = 0; j < 64; ++j) acc[j] = 0;
          for (int q = 0; q < a.ranges; ++q) {
            const float4* p = reinterpret_cast<const float4*>(a.part + ((size_t)w.tile * a.ranges + q) * PART_FLOATS);
            const uint64_t one = pack2(1.0f, 1.0f);
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const float4 v = __ldcg(p + j * 256 + t);
              fma2(acc[2 * j], pack2(v.x, v.y), one);
              fma2(acc[2 * j + 1], pack2(v.z, v.w), one);
            }
          }
        }
      }
      if constexpr (SWIGLU) {
        if (!idle) store_swiglu(a, acc, w, r, half, c);
      } else {
        if (!idle && r < w.rows) store_row(a, acc, w.r0 + r, w.nt * BN + half * kBlock);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, TMEM_COLS);
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encoder() {
  static EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess) p = nullptr;
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  return fn;
}

// [rows, cols] bytes in boxes of box_rows x 128, zeros outside
bool tensor_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint32_t box_rows) {
  EncodeTiledFn enc = encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {cols};
  cuuint32_t box[2] = {kBlock, box_rows}, unit[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, unit,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How a product is cut: tiles is an upper bound of the (row, column) tiles of
// any offsets; when they leave more than half of the SMs idle the blocks of the
// reduction are cut into ranges, at least two blocks each.
struct Cut {
  int nt, ranges, per;
  int64_t tiles;
};
constexpr int kSms = 148;

Cut cut_of(int n_groups, int n_cols, int k, int max_rows, bool swiglu) {
  Cut c{};
  const int kb = blocks_of(k);
  c.nt = swiglu ? blocks_of(n_cols) : (n_cols + BN - 1) / BN;
  c.tiles = ((int64_t)max_rows / BM + std::min(n_groups, max_rows)) * c.nt;
  const int64_t want = c.tiles > 0 ? kSms / c.tiles : 1;
  c.per = kb;
  if (want >= 2 && c.tiles <= MAX_CUT_TILES && kb >= 4)
    c.per = std::max({2, (int)((kb + want - 1) / want), (kb + MAX_RANGES - 1) / MAX_RANGES});
  c.ranges = (kb + c.per - 1) / c.per;
  return c;
}

size_t part_bytes(const Cut& c) { return c.ranges > 1 ? (size_t)c.tiles * c.ranges * PART_FLOATS * 4 : 0; }

struct Operands {
  const uint8_t *x, *w0, *w1;
  const float *xs, *ws0, *ws1, *row_scale;
};

// One product (plain: w0; SwiGLU: w0 = gate, w1 = up) over the groups.
cudaError_t product(int G, int N, int K, int max_rows, const int* offsets, const Operands& o, bool swiglu, int out_f32,
                    void* out, float* out_scale, float* part, int* ctrl, cudaStream_t st) {
  const Cut cut = cut_of(G, N, K, max_rows, swiglu);
  BlockArgs a{};
  const void* w1 = swiglu ? o.w1 : o.w0;
  if (!tensor_map(&a.x, o.x, max_rows, K, BM) || !tensor_map(&a.x32, o.x, max_rows, K, SUB_ROWS) ||
      !tensor_map(&a.w0, o.w0, (uint64_t)G * N, K, kBlock) || !tensor_map(&a.w1, w1, (uint64_t)G * N, K, kBlock))
    return cudaErrorInvalidValue;
  a.G = G; a.N = N; a.K = K; a.max_rows = max_rows;
  a.KB = blocks_of(K); a.NB = blocks_of(N); a.NT = cut.nt;
  a.ranges = cut.ranges; a.per = cut.per;
  a.offsets = offsets;
  a.xs = o.xs; a.ws0 = o.ws0; a.ws1 = o.ws1; a.row_scale = o.row_scale;
  a.out_f32 = out_f32; a.out = out; a.out_scale = out_scale; a.part = part; a.ctrl = ctrl;
  static bool attr_done[64] = {};
  int dev = 0, sms = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (dev >= 64 || !attr_done[dev]) {
    cudaError_t e = cudaFuncSetAttribute(block_product_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(block_product_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_done[dev] = true;
  }
  const unsigned grid = (unsigned)std::min<int64_t>(cut.tiles * cut.ranges, sms > 0 ? sms : 1);
  return launch_pdl(swiglu ? block_product_kernel<true> : block_product_kernel<false>, dim3(grid), dim3(NUM_THREADS),
                    SMEM_BYTES, st, a);
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
  *bytes = kAlign + align_up(part_bytes(cut_of(n_groups, n_cols, k, max_rows, false)));
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
  const cudaError_t e = product(n_groups, n_cols, k, max_rows, offsets,
                                {x, w, nullptr, x_scale, w_scale, nullptr, row_scale}, false,
                                out_dtype == MOE_DTYPE_F32, out, nullptr, at<float>(ws, kAlign), at<int>(ws, 0),
                                static_cast<cudaStream_t>(stream));
  return e != cudaSuccess ? fail(MOE_ERR_CUDA, "block product launch: %s", cudaGetErrorString(e)) : MOE_OK;
}

namespace {

// workspace of the experts: the control block, the codes of A and their scales,
// the accumulators of whichever product is cut into ranges
struct FfnLayout {
  size_t codes, scales, part, total;
};

FfnLayout ffn_layout(int n_experts, int d, int f, int max_rows) {
  FfnLayout L{};
  const size_t rows = max_rows > 0 ? max_rows : 1;
  size_t o = kAlign;
  L.codes = o; o = align_up(o + rows * f);
  L.scales = o; o = align_up(o + rows * blocks_of(f) * 4);
  L.part = o;
  o = align_up(o + std::max(part_bytes(cut_of(n_experts, f, d, max_rows, true)),
                            part_bytes(cut_of(n_experts, d, f, max_rows, false))));
  L.total = o;
  return L;
}

}  // namespace

extern "C" moe_status moe_block_ffn_workspace_size(int32_t n_experts, int32_t d_model, int32_t d_ffn, int32_t max_rows,
                                                   size_t* bytes) {
  MOE_CHECK(check_product(n_experts, d_ffn, d_model, max_rows));
  MOE_CHECK(check_product(n_experts, d_model, d_ffn, max_rows));
  if (!bytes) return fail(MOE_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = ffn_layout(n_experts, d_model, d_ffn, max_rows).total;
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
  const FfnLayout L = ffn_layout(n_experts, d_model, d_ffn, max_rows);
  uint8_t* codes = at<uint8_t>(ws, L.codes);
  float *scales = at<float>(ws, L.scales), *part = at<float>(ws, L.part);
  int* ctrl = at<int>(ws, 0);
  cudaError_t e = product(n_experts, d_ffn, d_model, max_rows, offsets,
                          {x, w_gate, w_up, x_scale, s_gate, s_up, nullptr}, true, 0, codes, scales, part, ctrl, st);
  if (e == cudaSuccess)
    e = product(n_experts, d_model, d_ffn, max_rows, offsets, {codes, w_down, nullptr, scales, s_down, nullptr, row_scale},
                false, out_dtype == MOE_DTYPE_F32, out, nullptr, part, ctrl, st);
  return e != cudaSuccess ? fail(MOE_ERR_CUDA, "block experts launch: %s", cudaGetErrorString(e)) : MOE_OK;
}
