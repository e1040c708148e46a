// Grouped matrix products of block-scaled e4m3 operands, and the SwiGLU experts
// made of them, on the 5th-generation tensor cores:
//   out[r, j] = row_scale[r] * sum_b xs[r, b] * ws[g, j / 128, b] * sum_{k in b} x[r, k] * w[g, j, k]
//
// The scales differ from one block of 128 of the reduction to the next, so the
// tensor cores sum one block (four tcgen05.mma of 32) into tensor memory and
// eight warps add it, times the two scales, to fp32 accumulators in their
// registers, while the tensor cores fill the other tensor-memory buffer with the next block.
//
// Work unit = (group, row tile of up to 128, tile of 256 weight rows, range of blocks).
// The 256 weight rows are two blocks of 128: columns j .. j + 255 of the plain
// product, or the gate and the up rows of the same 128 columns of the SwiGLU
// product, whose epilogue then holds whole 1 x 128 tiles of the rows of
// A = SiLU(U) V and quantizes them on the spot: A never reaches memory but as
// codes and scales.  Units of a group go row tile fastest, so CTAs that run
// together share weight tiles through L2 and weights stream from HBM about once.
//
// A row tile of more than kSwapRows = 32 rows is the M = 128 operand and the weights
// are N = 256: a block takes two of the four slots of 128 columns of tensor memory.  A shorter
// tile runs transposed, each block of weights an M = 128 operand and the rows,
// rounded up to 16, N: one slot, so four blocks are on their way, and no padding
// rows in the epilogue (2048 x 7168 weights, one row: 11.1 us, as a plain tile 18.5; 150 experts
// of 4 rows: 353 and 368; 64 experts of 32 rows: 170 and 172).  Tiles of up to 64 rows were no faster
// that way (64 experts of 64 rows, 1400 x 2032: 65 against 58 us a call by itself): the weights
// still pass shared memory whole.
//
// Times here are of calls over inputs in turn, on the device, unless they say "a call by
// itself": that is one with the L2 flushed before it, which takes 5 us longer.
//
// What bounds a block of 128 rows is the way of its sums through the accumulator warps, not the
// tensor cores (512 cycles) nor the loads (20 KB of the 48 left out: 536 instead of 558 us a call
// by itself).  Of about 1220 cycles on a single CTA the warps read tensor memory and add for 445,
// release it and add the last sums for 180, prepare scales and the next wait for 120, wait for the
// tensor cores for 175, and a unit's epilogue comes to 185 for each of its 32 blocks; the other
// 115 were not taken apart.
//
// Groups of many rows run on clusters of two CTAs (cta_group::2) in units of 256 rows:
// each CTA holds its half of the rows and half of the weight rows, so a block takes 32 KB of
// its shared memory, and of the way there from L2, instead of 48.
// 14336 x 4096 weights, single CTAs against pairs: 8 groups of 1024 rows 550 and 499 us, of
// 768 rows 477 and 411, of 512 rows 316 and 291, one of 768 rows 74 and 66.  A tile of 256 that
// is not full costs more than one of 128: one group of 640 rows 51 and 63 us, 256 groups of 128
// rows (2048 x 7168) 702 and 987.  The launch knows the groups' sum alone, and of ragged groups
// the last tiles are half empty: 128 rows a group with pairs, 64 without.  From 768 rows a
// group on pairs' gain of a tenth is more than that.
//
// Few rows leave few units: the blocks of the reduction are then cut into ranges,
// each unit of a range leaves its accumulators in the workspace, and the last
// unit of a tile to finish adds the ranges in ascending order (so the sum
// does not depend on which one was last) and runs the epilogue.  That one CTA has all ranges
// to read, 128 KB each when all rows are there, so few are better than one for every SM.  With at
// most 4, 6, 8 and 12 ranges (us):
//   one row   2048 x 7168: 14.3 12.4 11.0 10.8;  4096 x 14336: 22.5 18.6 17.6 17.5;  256 x 16384: 22.5 17.9 14.6 12.6
//   32 rows   2048 x 7168: 17.3 15.8 15.1 16.2;  4096 x 14336: 26.6 22.7 22.0 22.7;  256 x 16384: 26.6 22.2 18.7 18.0
//   64 rows   2048 x 7168: 20.5 19.8 23.3 24.2;  4096 x 14336: 30.0 27.3 30.4 30.5;  256 x 16384: 29.2 25.7 25.6 26.2
//   300 rows  2048 x 7168: 25.4 26.5 28.4 28.6;  4096 x 14336: 39.8 39.6 41.8 42.7;  256 x 16384: 33.0 32.3 32.0 32.0
// and 7168 x 2048, whose tiles leave room for five at most, 10.1 to 20 with each.
//
// Warp roles (384 threads): warp 0 = TMA producer (+ tensor memory), warp 1 = MMA
// issuer, warps 4 .. 11 = accumulators and epilogue: warp w reads
// the tensor memory lanes 32 (w % 4) .. + 31 and one half of the columns.  A
// thread of theirs holds 128 accumulators and 32 values on their way; the first
// four warps (2 and 3 only fill their warpgroup) give up registers for that (setmaxnreg).
// Each thread fetches the scales of its own row, four blocks at a time and four blocks
// ahead, into registers.  Two warps that staged them in shared memory for all, with a barrier
// each way, cost 8 x 1024 rows 587 us instead of 522 (a call by itself).
#include <algorithm>
#include <type_traits>
#include <cuda.h>

#include "api.h"
#include "common.cuh"
#include "e4m3.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kBlock = 128;              // values per scale; also the k-block of a pipeline stage
constexpr int kMaxGroups = 1024;
constexpr int BM = 128, BN = 256;                   // rows and weight rows of a unit
constexpr int STAGE_RING = 192 * 1024;              // operands on their way
constexpr int A_BYTES = BM * kBlock;
// one CTA loads both blocks of 128 weight rows, a CTA of a pair 64 rows of each
template <bool PAIR> constexpr int w_box() { return PAIR ? kBlock / 2 : kBlock; }
template <bool PAIR> constexpr int w_bytes() { return w_box<PAIR>() * kBlock; }
template <bool PAIR> constexpr int stages() { return STAGE_RING / (A_BYTES + 2 * w_bytes<PAIR>()); }   // 4, 6
constexpr int MAX_STAGES = 6;
constexpr int kPairRows = 768;                      // rows per group from which pairs run
constexpr int SUB_ROWS = 32;                        // row box of short row tiles
constexpr int kSwapRows = 32;                       // row tiles of at most this many rows run transposed
constexpr int SLOTS = 4, SLOT_COLS = 128;           // tensor memory
constexpr int SECOND = SLOT_COLS / 2;               // transposed: columns of the second block of weights in its slot
static_assert(kSwapRows == 32, "a transposed tile's rows: 16 to each half of the accumulator warps");
constexpr int EPI_WARPS = 8;
constexpr int NUM_THREADS = 128 + 32 * EPI_WARPS;
constexpr int EPI_THREAD0 = 128;
// 3 x 128 threads are launched with 168 registers each: 128 x 40 + 256 x 232 are as many
constexpr int FEW_REGS = 40, MANY_REGS = 232;
static_assert(128 * FEW_REGS + 32 * EPI_WARPS * MANY_REGS <= NUM_THREADS * 168, "registers of the launch");
constexpr int TMEM_COLS = 512;
// most ranges of a reduction: of launches of transposed tiles alone, and of others, whose
// sums are longer
constexpr int MAX_RANGES = 8, MAX_RANGES_LONG = 6;
constexpr int CHUNK = 4;                            // blocks whose scales are fetched together
// byte counters of the tiles whose reduction is cut, in the control block of the
// workspace: words 20 .. 63 (word 0 is the error word, 16 and 17 are the unit
// counters of the layer's GEMMs, which may share the workspace)
constexpr int COUNTER_WORD0 = 20, MAX_CUT_TILES = 44 * 4;
constexpr int PART_FLOATS = 128 * 32 * EPI_WARPS;   // accumulators of a unit

struct Control {
  alignas(16) float xs[EPI_WARPS][CHUNK][kSwapRows / 2];   // transposed: scales of a warp's 16 rows
  uint64_t full[MAX_STAGES], done[MAX_STAGES], slot_empty[SLOTS], drain;
  uint32_t tmem;
  int abort, last;
  int warp_sum[NUM_THREADS / 32];
  float top[4][BM];                                 // SwiGLU: maxima of the parts of a row's tile
  int prefix[kMaxGroups + 1];                       // units of the groups before
  alignas(16) uint8_t piece[EPI_WARPS][32 * 64];    // a warp's 32 rows x 64 bytes on their way out
};
constexpr size_t SMEM_BYTES = (size_t)STAGE_RING + sizeof(Control) + 1024;
static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");

int blocks_of(int n) { return (n + kBlock - 1) / kBlock; }

struct BlockArgs {
  CUtensorMap x, x32, w0, w1;       // rows in boxes of 128 and 32; weights in boxes of 128, or 64 for a pair (gate, up)
  int G, N, max_rows;
  int KB, NB, NT;                   // blocks of the reduction and of the columns; column tiles
  int ranges, per;                  // ranges of the reduction, blocks per range
  const int* offsets;
  const float *xs, *ws0, *ws1, *row_scale;
  int out_f32, scales16;            // scales16: scales at 16-byte addresses
  void* out;                        // plain: out; SwiGLU: the codes of A
  float* out_scale;                 // SwiGLU: the scales of A
  float* part;                      // [tiles][ranges][PART_FLOATS]
  int* ctrl;                        // the workspace's control block
};

struct Unit {
  int g, nt, r0, rows;              // first row and rows of this CTA
  int rows_all;                     // rows of the tile: those of both CTAs of a pair
  int kb0, nk, range, tile;
  int n16;                          // transposed: rows rounded up to 16, else 0
  bool two;                         // both blocks of weight rows have columns
};

template <bool SWIGLU, bool PAIR>
__device__ __forceinline__ Unit decode(const BlockArgs& a, const int* prefix, int u, int rank) {
  constexpr int ROWS = PAIR ? 2 * BM : BM;
  int lo = 0, hi = a.G;             // prefix[lo] <= u < prefix[lo + 1]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= u) lo = mid; else hi = mid;
  }
  Unit w;
  w.g = lo;
  const int r0 = a.offsets ? __ldg(a.offsets + lo) : 0;
  const int r1 = a.offsets ? __ldg(a.offsets + lo + 1) : a.max_rows;
  const int mts = (r1 - r0 + ROWS - 1) / ROWS;
  w.tile = u / a.ranges;            // every group's units are whole tiles of `ranges` units
  int local = u - prefix[lo];
  w.range = local % a.ranges;
  local /= a.ranges;
  w.nt = local / mts;
  w.r0 = r0 + local % mts * ROWS;
  w.rows = w.rows_all = min(ROWS, r1 - w.r0);
  if constexpr (PAIR) {
    // the CTAs share the rows in halves of whole warps
    const int half = min(w.rows, (w.rows + 63) / 64 * 32);
    w.r0 += rank ? half : 0;
    w.rows = rank ? w.rows - half : half;
  }
  w.n16 = !PAIR && w.rows <= kSwapRows ? (w.rows + 15) & ~15 : 0;
  w.two = SWIGLU || w.nt * BN + kBlock < a.N;
  w.kb0 = w.range * a.per;
  w.nk = min(a.KB, w.kb0 + a.per) - w.kb0;
  return w;
}

// Units before each group (prefix[G] = all) from the offsets.  Offsets out of order
// or out of range set the error word and leave no units: the tiles of ascending
// offsets are at most those that the launch and the workspace were sized for.
template <bool PAIR>
__device__ __forceinline__ void scan_groups(const BlockArgs& a, Control* c) {
  constexpr int ROWS = PAIR ? 2 * BM : BM;
  const int t = threadIdx.x, warp = t / kWarp, lane = t % kWarp;
  constexpr int PER = (kMaxGroups + NUM_THREADS - 1) / NUM_THREADS;
  int n[PER], sum = 0, bad = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int g = t * PER + i;
    n[i] = 0;
    if (g < a.G) {
      const int r0 = a.offsets ? __ldg(a.offsets + g) : 0, r1 = a.offsets ? __ldg(a.offsets + g + 1) : a.max_rows;
      if (r0 < 0 || r1 < r0 || r1 > a.max_rows) bad = 1;
      else n[i] = (r1 - r0 + ROWS - 1) / ROWS * a.NT * a.ranges;
    }
    sum += n[i];
  }
  if (__syncthreads_or(bad)) {
    if (t == 0) set_device_error(a.ctrl, MOE_DEVERR_INDEX);
    sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) n[i] = 0;
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

// mbar_wait of common.cuh with the clock read only after many tries: these waits
// come several times per block of 128.
// In a pair the other CTA is told to give up too.  What passes between the CTAs is
// tensor memory and the loads' bytes, which order themselves: the barriers are read and, by
// the accumulator warps, arrived on at CTA scope (an acquire or release at
// cluster scope in every block took three times the time).
template <bool PAIR>
__device__ __forceinline__ bool block_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int* err,
                                           uint32_t peer_abort, uint64_t limit_ns = kWaitLimitNs) {
  uint64_t t0 = 0;
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 63u) == 0) {
      if (*abort) return false;
      const uint64_t now = global_timer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > limit_ns) {
        set_device_error(err, MOE_DEVERR_WAIT_TIMEOUT);
        *abort = 1;
        if constexpr (PAIR) st_remote_u32(peer_abort, 1u);
        return false;
      }
    }
  }
}

// Where the next block's sums lie: slots are taken in turn, one block after the
// other, by the MMA issuer and the accumulator warps alike.  A block of two slots takes two
// neighbours (the odd slot before them is passed over); parity holds the phase bit of each slot.
struct SlotWalk {
  uint32_t next = 0, parity = 0;
  // first slot of a block of n slots; its phase bits are flipped for the block after
  __device__ __forceinline__ uint32_t take(uint32_t n, uint32_t& before) {
    uint32_t s = next;
    if (n == 2 && (s & 1u)) s = (s + 1) % SLOTS;
    before = parity >> s;
    parity ^= (n == 2 ? 3u : 1u) << s;
    next = (s + n) % SLOTS;
    return s;
  }
};

// Arrive on a barrier of this CTA or, by its cluster address, of the even one.
__device__ __forceinline__ void arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Wait without giving up on *abort (drains what is in flight before the CTA
// releases its shared and tensor memory).
__device__ __forceinline__ void wait_drain(uint64_t* bar, uint32_t parity, int* err) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity))
    if (global_timer_ns() - t0 > kWaitLimitNs) { set_device_error(err, MOE_DEVERR_WAIT_TIMEOUT); return; }
}

// D (+)= A * B^T, e4m3: over one CTA's operands, or over both CTAs' halves (issued by the even one).
template <bool PAIR>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
  else
    tc_mma_e4m3(d, a, b, idesc, acc);
}

// One lane of the (whole) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t is;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(is));
  return is != 0;
}

// 16 consecutive columns of this thread's tensor-memory lane: the load, and the wait
// through which its values must pass before they are used.
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_wait16(uint32_t (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
               :: "memory");
}

// a += v * s and b += w * s as one packed operation
__device__ __forceinline__ void fma2(float& a, float& b, float v, float w, float s) {
  asm("{\n\t.reg .b64 t, u, x;\n\t"
      "mov.b64 t, {%0, %1};\n\tmov.b64 u, {%2, %3};\n\tmov.b64 x, {%4, %4};\n\t"
      "fma.rn.f32x2 t, u, x, t;\n\t"
      "mov.b64 {%0, %1}, t;\n\t}"
      : "+f"(a), "+f"(b) : "f"(v), "f"(w), "f"(s));
}

// the same with a scale for each
__device__ __forceinline__ void fma2(float& a, float& b, float v, float w, float s, float z) {
  asm("{\n\t.reg .b64 t, u, x;\n\t"
      "mov.b64 t, {%0, %1};\n\tmov.b64 u, {%2, %3};\n\tmov.b64 x, {%4, %5};\n\t"
      "fma.rn.f32x2 t, u, x, t;\n\t"
      "mov.b64 {%0, %1}, t;\n\t}"
      : "+f"(a), "+f"(b) : "f"(v), "f"(w), "f"(s), "f"(z));
}

// Barrier of the 256 accumulator threads; true when all of them bring true.
__device__ __forceinline__ bool all_agree(bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, 6, 256, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all) : "r"((uint32_t)ok) : "memory");
  return all != 0;
}

__device__ __forceinline__ float silu(float x) { return __fdividef(x, 1.0f + __expf(-x)); }

// 16 bytes `v` (0 .. 3) of a row of the piece: turned by the row, so that neither
// the rows written nor those read meet in a bank
__device__ __forceinline__ uint4* piece_at(uint8_t* piece, int row, int v) {
  return reinterpret_cast<uint4*>(piece + row * 64 + ((v ^ (row >> 1)) & 3) * 16);
}

// Plain epilogue: columns col0 .. col0 + 127 of the warp's rows row0 .. row0 + n - 1,
// one row a lane.  Stored as they lie, a 16-byte store of a warp would touch 32
// lines (4000 cycles a tile were measured); so 64 bytes of each row at a time go through
// shared memory and leave four (or, for rows of odd alignment, 16 or 32) lanes to a row.
template <typename T>
__device__ __forceinline__ void store_rows(const BlockArgs& a, const float (&acc)[128], uint8_t* piece, int row0, int n,
                                           int col0) {
  constexpr int PER = 64 / (int)sizeof(T);         // columns of a piece
  const int lane = threadIdx.x % kWarp;
  const float rs = a.row_scale && lane < n ? __ldg(a.row_scale + row0 + lane) : 1.0f;
  T* out = static_cast<T*>(a.out) + (size_t)row0 * a.N + col0;
  const bool vectors = a.N % (16 / (int)sizeof(T)) == 0;
#pragma unroll
  for (int p = 0; p < 128 / PER; ++p) {
    const int cols = min(PER, a.N - col0 - p * PER);
    if (cols <= 0) break;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      uint32_t q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
          q[i] = __float_as_uint(acc[p * PER + 4 * v + i] * rs);
        } else {
          const __nv_bfloat162 b = __floats2bfloat162_rn(acc[p * PER + 8 * v + 2 * i] * rs, acc[p * PER + 8 * v + 2 * i + 1] * rs);
          q[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
      }
      *piece_at(piece, lane, v) = make_uint4(q[0], q[1], q[2], q[3]);
    }
    __syncwarp();
    if (vectors) {
      const int v = lane % 4;                      // whole vectors: cols is a multiple of 16 / sizeof(T)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 8 * i + lane / 4;
        if (r < n && v * (16 / (int)sizeof(T)) < cols)
          *reinterpret_cast<uint4*>(out + (size_t)r * a.N + p * PER + v * (16 / (int)sizeof(T))) = *piece_at(piece, r, v);
      }
    } else {
      constexpr int VALS = 16 / (int)sizeof(T);
      const int j = lane % PER;
#pragma unroll 4
      for (int r = lane / PER; r < n; r += kWarp / PER)
        if (j < cols) out[(size_t)r * a.N + p * PER + j] = reinterpret_cast<const T*>(piece_at(piece, r, j / VALS))[j % VALS];
    }
    __syncwarp();
  }
}

// SwiGLU epilogue: this thread holds 64 gate (acc[0 .. 63]) and the same 64 up
// columns (acc[64 .. 127]) of its row, which become their products; the other 64 columns of
// the 1 x 128 tile are with the warp of the other half, which shares the maximum
// through shared memory.
__device__ __forceinline__ void store_swiglu(const BlockArgs& a, float (&acc)[128], const Unit& w, int row0, int rows,
                                             int r, int half, Control* c) {
  float top = 0.0f;
  const int col0 = w.nt * kBlock + half * 64;
#pragma unroll
  for (int j = 0; j < 64; ++j) {
    acc[j] = col0 + j < a.N ? silu(acc[j]) * acc[64 + j] : 0.0f;
    top = fmaxf(top, fabsf(acc[j]));
  }
  const int quad = r / 32;
  c->top[half][r] = top;
  asm volatile("bar.sync %0, 64;" ::"r"(8 + quad) : "memory");
  top = fmaxf(top, c->top[half ^ 1][r]);
  asm volatile("bar.sync %0, 64;" ::"r"(8 + quad) : "memory");
  if (r >= rows) return;
  const int e = e4m3_scale_exponent(top);
  const float inv = pow2(-e);
  const size_t row = (size_t)(row0 + r);
  uint8_t* o = static_cast<uint8_t*>(a.out) + row * a.N + col0;
#pragma unroll
  for (int j = 0; j < 64; j += 16) {
    if (col0 + j >= a.N) break;                       // N is a multiple of 16
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      q[i] = e4m3_pack4(acc[j + 4 * i] * inv, acc[j + 4 * i + 1] * inv, acc[j + 4 * i + 2] * inv, acc[j + 4 * i + 3] * inv);
    *reinterpret_cast<uint4*>(o + j) = make_uint4(q[0], q[1], q[2], q[3]);
  }
  if (half == 0) a.out_scale[row * a.NB + w.nt] = pow2(e);
}

// Transposed tiles: the thread holds columns col (acc[t]) and col + 128 (acc[16 + t])
// of rows row0 + t, t < n <= 16; a warp writes 32 neighbouring columns of a row at a time.
template <typename T>
__device__ __forceinline__ void store_columns(const BlockArgs& a, const float (&acc)[128], int row0, int n, int col) {
  const int lane = threadIdx.x % kWarp;
  const float rs_lane = a.row_scale && lane < n ? __ldg(a.row_scale + row0 + lane) : 1.0f;    // of row `lane`
  T* out = static_cast<T*>(a.out) + (size_t)row0 * a.N + col;
#pragma unroll
  for (int t = 0; t < 16; ++t) {
    if (t >= n) break;
    const float rs = __shfl_sync(kFull, rs_lane, t);
    if (col < a.N) out[(size_t)t * a.N] = from_f32<T>(acc[t] * rs);
    if (col + kBlock < a.N) out[(size_t)t * a.N + kBlock] = from_f32<T>(acc[16 + t] * rs);
  }
}

// Transposed SwiGLU: acc[t] is the gate and acc[16 + t] the up value of column col
// of row row0 + t; the tile's 128 columns are the 128 lanes of the four warps
// of this half of the rows, which share their maxima through shared memory.
__device__ __forceinline__ void store_swiglu_columns(const BlockArgs& a, float (&acc)[128], const Unit& w, int row0,
                                                     int t0, int n, int r, int half, Control* c) {
  const int col = w.nt * kBlock + r, quad = r / 32;
#pragma unroll
  for (int t = 0; t < 16; ++t) {
    if (t >= n) break;
    acc[t] = col < a.N ? silu(acc[t]) * acc[16 + t] : 0.0f;
    // magnitudes order like their bits; a NaN does not count
    const uint32_t top = __reduce_max_sync(kFull, acc[t] == acc[t] ? __float_as_uint(fabsf(acc[t])) : 0u);
    if (r % 32 == 0) c->top[quad][t0 + t] = __uint_as_float(top);
  }
  asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory");
#pragma unroll
  for (int t = 0; t < 16; ++t) {
    if (t >= n) break;
    float top = 0.0f;
#pragma unroll
    for (int q = 0; q < 4; ++q) top = fmaxf(top, c->top[q][t0 + t]);
    const int e = e4m3_scale_exponent(top);
    const size_t row = (size_t)(row0 + t);
    if (col < a.N)
      static_cast<uint8_t*>(a.out)[row * a.N + col] =
          (uint8_t)__nv_cvt_float_to_fp8(acc[t] * pow2(-e), __NV_SATFINITE, __NV_E4M3);
    if (r == 0) a.out_scale[row * a.NB + w.nt] = pow2(e);
  }
  asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory");   // the maxima are rewritten by the next unit
}

template <bool SWIGLU, bool PAIR>
__global__ void __launch_bounds__(NUM_THREADS, 1) block_product_kernel(const __grid_constant__ BlockArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* sA = smem;
  constexpr int STAGES = stages<PAIR>(), W_BYTES = w_bytes<PAIR>(), B_BYTES = 2 * W_BYTES, CTAS = PAIR ? 2 : 1;
  uint8_t* sB = smem + STAGES * A_BYTES;
  Control* c = reinterpret_cast<Control*>(smem + STAGE_RING);
  volatile int* abort_flag = &c->abort;
  int* err = a.ctrl;
  // the same in all lanes, and known to be: the roles' loops then run on the uniform path
  const int warp = __shfl_sync(kFull, (int)threadIdx.x / kWarp, 0), lane = threadIdx.x % kWarp;
  const uint32_t rank = PAIR ? cluster_rank() : 0u;
  const uint32_t peer_abort = PAIR ? cluster_addr(&c->abort, rank ^ 1u) : 0u;
  auto wait = [&](uint64_t* bar, uint32_t parity) { return block_wait<PAIR>(bar, parity, abort_flag, err, peer_abort); };
  // barriers that both CTAs signal are the even one's
  auto even = [&](uint64_t* bar) { return PAIR ? cluster_addr(bar, 0) : smem_u32(bar); };
  auto commit = [&](uint64_t* bar) {
    if constexpr (PAIR) tc_commit_pair(bar); else tc_commit(bar);
  };
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) { mbar_init(&c->full[s], 1); mbar_init(&c->done[s], 1); }
    for (int b = 0; b < SLOTS; ++b) mbar_init(&c->slot_empty[b], CTAS * EPI_WARPS);
    mbar_init(&c->drain, 1);
    c->abort = 0;
    fence_barrier_init();
  }
  if (warp == 1 && lane == 0) { prefetch_tmap(&a.x); prefetch_tmap(&a.x32); prefetch_tmap(&a.w0); prefetch_tmap(&a.w1); }
  __syncthreads();
  if constexpr (PAIR) {
    cluster_sync_all();        // both CTAs' barriers are initialised before either signals the other
    if (warp == 0) tmem_alloc_pair(&c->tmem, TMEM_COLS);
  } else if (warp == 0) {
    tmem_alloc(&c->tmem, TMEM_COLS);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  pdl_trigger();
  const uint32_t tmem = c->tmem;
  scan_groups<PAIR>(a, c);
  const int total = c->prefix[a.G];
  const int first = (int)blockIdx.x / CTAS, step = (int)gridDim.x / CTAS;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(FEW_REGS));
    if (warp == 0 && lane == 0) {
      // ---------------- TMA producer ----------------
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int u = first; u < total && ok; u += step) {
        const Unit w = decode<SWIGLU, PAIR>(a, c->prefix, u, rank);
        const int sub = (w.rows + SUB_ROWS - 1) / SUB_ROWS;       // four boxes of 32 rows are one of 128
        const int other = PAIR ? (w.rows_all - w.rows + SUB_ROWS - 1) / SUB_ROWS : 0;
        const uint32_t tx = (uint32_t)((sub + other) * SUB_ROWS * kBlock + CTAS * (w.two ? 2 : 1) * W_BYTES);
        // a pair's CTAs: 64 gate and the same 64 up rows each, or each half of the tile's columns
        const int by = w.g * a.N + w.nt * (SWIGLU ? kBlock : BN) +
                       (PAIR ? (int)rank * (SWIGLU || !w.two ? kBlock / 2 : kBlock) : 0);
        const int by1 = SWIGLU ? by : by + w_box<PAIR>();
        for (int i = 0; i < w.nk; ++i) {
          if (!wait(&c->done[stage], phase ^ 1u)) { ok = false; break; }
          const int k = (w.kb0 + i) * kBlock;
          if (rank == 0) mbar_arrive_expect_tx(&c->full[stage], tx);
          const uint32_t bar = even(&c->full[stage]);
          auto load = [&](uint8_t* to, const CUtensorMap* map, int y) {
            if constexpr (PAIR) tma_load_2d_pair(to, map, bar, k, y);
            else tma_load_2d(to, map, &c->full[stage], k, y);
          };
          // the weights first: they come from HBM, the rows mostly from L2
          load(sB + stage * B_BYTES, &a.w0, by);
          if (w.two) load(sB + stage * B_BYTES + W_BYTES, &a.w1, by1);
          if (sub == BM / SUB_ROWS) {
            load(sA + stage * A_BYTES, &a.x, w.r0);
          } else {
            for (int q = 0; q < sub; ++q) load(sA + stage * A_BYTES + q * SUB_ROWS * kBlock, &a.x32, w.r0 + q * SUB_ROWS);
          }
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      // every stage's last release has arrived (the loads have landed and been read)
      // before this CTA may leave
      for (int i = 0; i < STAGES && ok; ++i) {
        ok = wait(&c->done[stage], phase ^ 1u);
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
      }
    } else if (warp == 1 && rank == 0) {
      // ---------------- MMA issuer (of a pair: the even CTA) ----------------
      const uint64_t descA = sdesc_kmajor_sw128(smem_u32(sA)), descB = sdesc_kmajor_sw128(smem_u32(sB));
      int stage = 0;
      uint32_t phase = 0;
      SlotWalk walk;
      bool ok = true;
      for (int u = first; u < total && ok; u += step) {
        const Unit w = decode<SWIGLU, PAIR>(a, c->prefix, u, rank);
        const uint32_t n_slots = w.n16 == 0 ? 2u : 1u;
        const uint32_t idesc = w.n16 ? idesc_e4m3_f32(BM, w.n16) : idesc_e4m3_f32(CTAS * BM, w.two ? BN : kBlock);
        for (int i = 0; i < w.nk; ++i) {
          uint32_t before;
          const uint32_t s = walk.take(n_slots, before);
          ok = wait(&c->full[stage], phase) && wait(&c->slot_empty[s], (before & 1u) ^ 1u) &&
               (n_slots == 1 || wait(&c->slot_empty[s + 1], ((before >> 1) & 1u) ^ 1u));
          if (!__all_sync(kFull, ok)) { ok = false; break; }
          tc_fence_after();
          // descriptors count 16 bytes; a block of 128 is four steps of 32
          const uint64_t da = descA + stage * (A_BYTES / 16), db = descB + stage * (B_BYTES / 16);
          const uint32_t d = tmem + s * SLOT_COLS;
          if (elect_one()) {
            if (w.n16 == 0) {
#pragma unroll
              for (int k = 0; k < 4; ++k) mma<PAIR>(d, da + 2 * k, db + 2 * k, idesc, k != 0);
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k) mma<PAIR>(d, db + 2 * k, da + 2 * k, idesc, k != 0);
              if (w.two) {
#pragma unroll
                for (int k = 0; k < 4; ++k) mma<PAIR>(d + SECOND, db + W_BYTES / 16 + 2 * k, da + 2 * k, idesc, k != 0);
              }
            }
            commit(&c->done[stage]);             // the stage is read and the sums are there
          }
          __syncwarp();
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      // in a pair: the accumulator warps of both CTAs have released all slots
      if constexpr (PAIR) {
        for (int s = 0; s < SLOTS; ++s)
          if (ok && !wait(&c->slot_empty[s], ((walk.parity >> s) & 1u) ^ 1u)) ok = false;
      }
      if (elect_one()) {
        if constexpr (PAIR) tc_commit_local(&c->drain); else tc_commit(&c->drain);
      }
      __syncwarp();
      wait_drain(&c->drain, 0, err);
    }
  } else {
    // ---------------- accumulators and epilogue ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(MANY_REGS));
    const int quad = warp & 3, half = (warp - 4) / 4;
    const int r = quad * 32 + lane;
    const int t = threadIdx.x - EPI_THREAD0;
    const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16);
    const uint32_t release = even(&c->slot_empty[0]);               // slot s: + 8 s
    int stage = 0;
    uint32_t phase = 0;
    SlotWalk walk;
    bool ok = true;
    for (int u = first; u < total && ok; u += step) {
      const Unit w = decode<SWIGLU, PAIR>(a, c->prefix, u, rank);
      const bool swap = !PAIR && w.n16 != 0;
      // transposed: this half's rows t0 .. t0 + n - 1 of the tile
      const int t0 = 16 * half, n = swap ? max(0, min(16, w.rows - t0)) : 0;
      const uint32_t n_slots = swap ? 1u : 2u;
      // warps without rows, or without columns, only keep the slots moving
      const bool idle = swap ? n == 0 : quad * 32 >= w.rows || (half == 1 && !w.two);
      // scales of this thread's row (transposed: of the row that it fetches for its warp) and of the
      // weights' blocks; `vectors`: whole rows of scales are 16-byte vectors
      const float* xp = a.xs + (size_t)(w.r0 + (swap ? min(t0 + lane % 16, w.rows - 1) : min(r, w.rows - 1))) * a.KB + w.kb0;
      const size_t wrow = (size_t)w.g * a.NB;
      const int j1 = SWIGLU ? w.nt : min(2 * w.nt + 1, a.NB - 1), j0 = SWIGLU ? w.nt : !swap && half ? j1 : 2 * w.nt;
      const float *ap = a.ws0 + (wrow + j0) * a.KB + w.kb0, *bp = a.ws1 + (wrow + j1) * a.KB + w.kb0;
      const bool vectors = !((a.KB | w.kb0) & 3) && a.scales16;
      auto fetch = [&](float (&v)[CHUNK], const float* p, int i) {
        if (vectors) {
          const float4 q = __ldg(reinterpret_cast<const float4*>(p + i));
          v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
        } else {
#pragma unroll
          for (int j = 0; j < CHUNK; ++j) v[j] = i + j < w.nk ? __ldg(p + i + j) : 0.0f;
        }
      };
      float nx[CHUNK], na[CHUNK], nb[CHUNK], sa[CHUNK], sb[CHUNK];
#pragma unroll
      for (int j = 0; j < CHUNK; ++j) nx[j] = na[j] = nb[j] = sa[j] = sb[j] = 0.0f;
      auto fetch_all = [&](int i) {
        fetch(nx, xp, i);
        fetch(na, ap, i);
        if (SWIGLU || swap) fetch(nb, bp, i);
      };
      if (!idle) fetch_all(0);
      float acc[128];
#pragma unroll
      for (int j = 0; j < 128; ++j) acc[j] = 0.0f;
      for (int i = 0; i < w.nk; ++i) {
        uint32_t before;
        const uint32_t s = walk.take(n_slots, before);
        if (!idle && i % CHUNK == 0) {
          if (swap) {
            __syncwarp();
#pragma unroll
            for (int j = 0; j < CHUNK; ++j)
              if (lane < 16) c->xs[warp - 4][j][lane] = nx[j];
            __syncwarp();
          }
#pragma unroll
          for (int j = 0; j < CHUNK; ++j) {
            sa[j] = swap ? na[j] : nx[j] * na[j];
            sb[j] = swap ? nb[j] : SWIGLU ? nx[j] * nb[j] : 0.0f;
          }
          if (i + CHUNK < w.nk) fetch_all(i + CHUNK);
        }
        const float w0 = sa[0], w1 = sb[0];
#pragma unroll
        for (int j = 0; j + 1 < CHUNK; ++j) { sa[j] = sa[j + 1]; sb[j] = sb[j + 1]; }
        if (!__all_sync(kFull, wait(&c->done[stage], phase))) { ok = false; break; }
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        tc_fence_after();
        const uint32_t d = lane_base + s * SLOT_COLS;
        auto free_slots = [&] {                       // all values are in registers
          tc_fence_before();
          if (lane == 0) {
            arrive_at(release + 8u * s);
            if (n_slots == 2) arrive_at(release + 8u * s + 8u);
          }
        };
        if (idle) {
          free_slots();
        } else if (!swap) {
          // the thread's row, 128 columns: a block of the plain product, or 64 gate and their 64 up columns
          const uint32_t base = d + (uint32_t)(half * (SWIGLU && !PAIR ? 64 : 128));
          const float s_first = w0, s_last = SWIGLU ? w1 : w0;
          // 16 columns arrive while the 16 before are added
          uint32_t v[2][16];
          tmem_ld16(base, v[0]);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            tmem_wait16(v[q & 1]);
            if (q < 7) tmem_ld16(base + 16 * (q + 1) + (SWIGLU && !PAIR && q + 1 >= 4 ? 64 : 0), v[(q + 1) & 1]);
            else free_slots();
            const float sc = q < 4 ? s_first : s_last;
#pragma unroll
            for (int j = 0; j < 16; j += 2)
              fma2(acc[16 * q + j], acc[16 * q + j + 1], __uint_as_float(v[q & 1][j]), __uint_as_float(v[q & 1][j + 1]), sc);
          }
        } else {
          // one column of each block of weights, 16 rows: acc[t] and acc[16 + t]
          const float* xs = c->xs[warp - 4][i % CHUNK];
          uint32_t v0[16], v1[16];
          tmem_ld16(d + t0, v0);
          tmem_ld16(d + SECOND + t0, v1);
          tmem_wait16(v0);
          tmem_wait16(v1);
          free_slots();
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            const float4 xv = *reinterpret_cast<const float4*>(xs + j);
            fma2(acc[j], acc[j + 1], __uint_as_float(v0[j]), __uint_as_float(v0[j + 1]), xv.x * w0, xv.y * w0);
            fma2(acc[j + 2], acc[j + 3], __uint_as_float(v0[j + 2]), __uint_as_float(v0[j + 3]), xv.z * w0, xv.w * w0);
            fma2(acc[16 + j], acc[17 + j], __uint_as_float(v1[j]), __uint_as_float(v1[j + 1]), xv.x * w1, xv.y * w1);
            fma2(acc[18 + j], acc[19 + j], __uint_as_float(v1[j + 2]), __uint_as_float(v1[j + 3]), xv.z * w1, xv.w * w1);
          }
        }
      }
      // the barriers below want every warp: if a wait gave up in one, all leave here
      if (SWIGLU || (!PAIR && a.ranges > 1)) ok = all_agree(ok);
      if (!ok) break;
      if (!PAIR && a.ranges > 1) {
        // leave the accumulators; the last range of the tile to arrive adds them in order
        const bool mine = !idle && (swap || r < w.rows);
        const size_t tile = (size_t)w.tile * a.ranges;
        float4* here = reinterpret_cast<float4*>(a.part + (tile + w.range) * PART_FLOATS);
        // fours of acc; a transposed tile's are the rows 4 j .. 4 j + 3 of both blocks of weights
        auto used = [&](int j) { return !swap || (j < 8 && 4 * (j % 4) < n); };
        if (mine)
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (used(j))
              __stcg(here + j * 256 + t, make_float4(acc[4 * j], acc[4 * j + 1], acc[4 * j + 2], acc[4 * j + 3]));
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
        if (mine) {
          const float4* p = reinterpret_cast<const float4*>(a.part + tile * PART_FLOATS) + t;
          // two fours of all ranges in flight
          auto join = [&](int j, int k, auto most) {
            constexpr int MOST = decltype(most)::value;
            float4 v[2][MOST];
#pragma unroll
            for (int q = 0; q < MOST; ++q)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                v[h][q] = q < a.ranges ? __ldcg(p + (size_t)q * (PART_FLOATS / 4) + (h ? k : j) * 256)
                                       : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
              for (int q = 0; q < MOST; ++q) { sum.x += v[h][q].x; sum.y += v[h][q].y; sum.z += v[h][q].z; sum.w += v[h][q].w; }
              float* to = acc + 4 * (h ? k : j);
              to[0] = sum.x; to[1] = sum.y; to[2] = sum.z; to[3] = sum.w;
            }
          };
          if (swap) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (4 * j < n) join(j, j + 4, std::integral_constant<int, MAX_RANGES>());
          } else {
#pragma unroll
            for (int j = 0; j < 32; j += 2) join(j, j + 1, std::integral_constant<int, MAX_RANGES_LONG>());
          }
        }
      }
      if constexpr (SWIGLU) {
        if (swap) {
          if (!idle) store_swiglu_columns(a, acc, w, w.r0 + t0, t0, n, r, half, c);
        } else if (!idle) {
          store_swiglu(a, acc, w, w.r0, w.rows, r, half, c);
        }
      } else {
        if (swap) {
          if (!idle) {
            if (a.out_f32) store_columns<float>(a, acc, w.r0 + t0, n, w.nt * BN + r);
            else store_columns<bf16>(a, acc, w.r0 + t0, n, w.nt * BN + r);
          }
        } else if (!idle) {
          uint8_t* piece = c->piece[warp - 4];
          const int row0 = w.r0 + quad * 32, rows = min(32, w.rows - quad * 32), col0 = w.nt * BN + half * kBlock;
          if (a.out_f32) store_rows<float>(a, acc, piece, row0, rows, col0);
          else store_rows<bf16>(a, acc, piece, row0, rows, col0);
        }
      }
    }
  }
  if (*abort_flag) {
    // loads and MMAs may be in flight still: give them time to land before the
    // shared and tensor memory goes
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 1000000ull) {
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync_all();      // neither CTA leaves while the other may still signal it
  tc_fence_after();
  if (warp == 0) {
    if constexpr (PAIR) tmem_dealloc_pair(tmem, TMEM_COLS); else tmem_dealloc(tmem, TMEM_COLS);
  }
}

// Failure-detection self-test: one thread waits on a barrier that nothing arrives on, first
// through the wait of the layer's GEMMs, then through that of the block products; the error
// word is set when both gave up, recorded it and told the other roles.
__global__ void bounded_wait_selftest_kernel(uint64_t limit_ns, int* err) {
  __shared__ uint64_t bar;
  __shared__ int abort_flag, code;
  if (threadIdx.x != 0) return;
  mbar_init(&bar, 1);
  fence_barrier_init();
  bool gave_up = true;
  for (int which = 0; which < 2; ++which) {
    abort_flag = code = 0;
    const bool done = which == 0 ? mbar_wait(&bar, 0, &abort_flag, &code, limit_ns)
                                 : block_wait<false>(&bar, 0, &abort_flag, &code, 0, limit_ns);
    gave_up = gave_up && !done && abort_flag == 1 && code == MOE_DEVERR_WAIT_TIMEOUT;
  }
  if (gave_up) set_device_error(err, MOE_DEVERR_WAIT_TIMEOUT);
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
// any offsets; when they leave more than half of the SMs idle the blocks of
// the reduction are cut into ranges, at least two blocks each.
struct Cut {
  bool pair;
  int nt, ranges, per;
  int64_t tiles;
};
constexpr int kSms = 148;

Cut cut_of(int n_groups, int n_cols, int k, int max_rows, bool swiglu) {
  Cut c{};
  const int kb = blocks_of(k);
  const int64_t some = std::min(n_groups, max_rows);     // at most so many groups have rows
  c.nt = swiglu ? blocks_of(n_cols) : (n_cols + BN - 1) / BN;
  // pairs: groups of many rows, and tiles for two rounds of them at least
  const int64_t pair_tiles = ((int64_t)max_rows + (2 * BM - 1) * some) / (2 * BM) * c.nt;
  c.pair = max_rows >= (int64_t)kPairRows * n_groups && pair_tiles >= kSms;
  if (c.pair) {
    c.tiles = pair_tiles;
    c.per = kb;
    c.ranges = 1;
    return c;
  }
  c.tiles = ((int64_t)max_rows + (BM - 1) * some) / BM * c.nt;
  const int most = max_rows <= kSwapRows ? MAX_RANGES : MAX_RANGES_LONG;
  const int64_t want = c.tiles > 0 ? kSms / c.tiles : 1;
  c.per = kb;
  static_assert(kSms / 2 <= MAX_CUT_TILES, "a counter for every cut tile");
  if (want >= 2 && kb >= 4)
    c.per = std::max({2, (int)((kb + want - 1) / want), (kb + most - 1) / most});
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
  const uint32_t box = cut.pair ? w_box<true>() : w_box<false>();
  if (!tensor_map(&a.x, o.x, max_rows, K, BM) || !tensor_map(&a.x32, o.x, max_rows, K, SUB_ROWS) ||
      !tensor_map(&a.w0, o.w0, (uint64_t)G * N, K, box) || !tensor_map(&a.w1, w1, (uint64_t)G * N, K, box))
    return cudaErrorInvalidValue;
  a.G = G; a.N = N; a.max_rows = max_rows;
  a.KB = blocks_of(K); a.NB = blocks_of(N); a.NT = cut.nt;
  a.ranges = cut.ranges; a.per = cut.per;
  a.offsets = offsets;
  a.xs = o.xs; a.ws0 = o.ws0; a.ws1 = swiglu ? o.ws1 : o.ws0; a.row_scale = o.row_scale;
  a.scales16 = ((reinterpret_cast<uintptr_t>(a.xs) | reinterpret_cast<uintptr_t>(a.ws0) |
                 reinterpret_cast<uintptr_t>(a.ws1)) & 15) == 0;
  a.out_f32 = out_f32; a.out = out; a.out_scale = out_scale; a.part = part; a.ctrl = ctrl;
  static bool attr_done[64] = {};
  int dev = 0, sms = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (dev >= 64 || !attr_done[dev]) {
    for (auto kern : {block_product_kernel<true, true>, block_product_kernel<true, false>,
                      block_product_kernel<false, true>, block_product_kernel<false, false>}) {
      const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES);
      if (e != cudaSuccess) return e;
    }
    if (dev < 64) attr_done[dev] = true;
  }
  if (!cut.pair) {
    const unsigned grid = (unsigned)std::min<int64_t>(cut.tiles * cut.ranges, std::max(sms, 1));
    return launch_pdl(swiglu ? block_product_kernel<true, false> : block_product_kernel<false, false>, dim3(grid),
                      dim3(NUM_THREADS), SMEM_BYTES, st, a);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * (unsigned)std::min<int64_t>(cut.tiles, std::max(sms / 2, 1)));
  cfg.blockDim = dim3(NUM_THREADS);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kUsePdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, swiglu ? block_product_kernel<true, true> : block_product_kernel<false, true>, a);
}

moe_status check_product(int n_groups, int n_cols, int k, int max_rows) {
  if (n_groups < 1) return fail(MOE_ERR_INVALID_ARG, "n_groups=%d < 1", n_groups);
  if (n_groups > kMaxGroups) return fail(MOE_ERR_UNSUPPORTED, "n_groups=%d > %d", n_groups, kMaxGroups);
  if (n_cols < 1) return fail(MOE_ERR_INVALID_ARG, "n_cols=%d < 1", n_cols);
  if (k < 16 || k % 16) return fail(MOE_ERR_INVALID_ARG, "k=%d must be a positive multiple of 16", k);
  if (max_rows < 0) return fail(MOE_ERR_INVALID_ARG, "max_rows=%d < 0", max_rows);
  // a group's rows are rounded up to whole tiles in 32 bits
  if (max_rows > 0x7FFFFFFF - (2 * BM - 1)) return fail(MOE_ERR_UNSUPPORTED, "max_rows=%d above 2^31 - %d", max_rows, 2 * BM);
  if (n_cols > 1 << 20 || k > 1 << 20) return fail(MOE_ERR_UNSUPPORTED, "n_cols=%d k=%d above 2^20", n_cols, k);
  if ((int64_t)n_groups * n_cols > 0x7FFFFFFF) return fail(MOE_ERR_UNSUPPORTED, "n_groups * n_cols above 2^31");
  // units are counted in 32 bits: row tiles x column tiles (of at least 128 columns)
  if (((int64_t)max_rows / BM + n_groups) * blocks_of(n_cols) > 0x3FFFFFFF)
    return fail(MOE_ERR_UNSUPPORTED, "max_rows=%d with n_cols=%d: too many tiles", max_rows, n_cols);
  return MOE_OK;
}

}  // namespace

void launch_bounded_wait_selftest(uint64_t limit_ns, int* err, cudaStream_t st) {
  bounded_wait_selftest_kernel<<<1, 32, 0, st>>>(limit_ns, err);
}

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
  return launch_status(e, "block product");
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
  return launch_status(e, "block experts");
}
