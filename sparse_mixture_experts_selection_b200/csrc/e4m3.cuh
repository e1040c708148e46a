// e4m3 quantization with power-of-two scales: the scale of a maximum and the
// packing of codes, shared by the row, tile and block quantizers.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace moe {

// e with 2^e the smallest power of two such that amax <= 448 * 2^e, i.e. with
// amax = M * 2^E (1 <= M < 2): e = E - 8 + [M > 1.75]; at least -126 (a normal
// fp32 scale, below which subnormal amax fall); 0 for amax == 0.
__device__ __forceinline__ int e4m3_scale_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax) & 0x7FFFFFFFu;
  // a mantissa above that of 1.75 (0x600000) carries into the exponent
  const int e = (int)((b + 0x1FFFFFu) >> 23) - (127 + 8);
  return b == 0 ? 0 : max(e, -126);
}

// 2^e, exact, for -126 <= e <= 127
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// Four codes, the first in the low byte: nearest, ties to even, saturating at 448.
__device__ __forceinline__ uint32_t e4m3_pack4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return (lo & 0xFFFFu) | (hi << 16);
}

}  // namespace moe
