// e4m3 quantization with power-of-two scales: the scale of a maximum and the
// packing of codes, shared by the row, tile and block quantizers.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace moe {

// e with 2^e the smallest power of two such that amax <= 448 * 2^e, i.e. with
// amax = M * 2^E (1 <= M < 2): e = E - 8 + [M > 1.75]; at least -126 (a normal
// fp32 scale); 0 for amax == 0.
__device__ __forceinline__ int e4m3_scale_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax) & 0x7FFFFFFFu;
  if (b == 0) return 0;
  int E;
  uint32_t mant;
  if ((b >> 23) == 0) {                        // subnormal amax
    const int p = 31 - __clz(b);
    E = p - 149;
    mant = (b << (23 - p)) & 0x7FFFFFu;
  } else {
    E = (int)(b >> 23) - 127;
    mant = b & 0x7FFFFFu;
  }
  const int e = E - 8 + (mant > 0x600000u ? 1 : 0);
  return e < -126 ? -126 : e;
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
