// Element conversions shared by the quantisers (weights and K/V cache).
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

namespace petit {

__device__ __forceinline__ void bf16x8_to_f32(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// Nearest E2M1 code of y, ties to the even-mantissa neighbour, saturating at
// 6; magnitude 0 always gives code 0 (no negative zero).  The grid is
// {0, .5, 1, 1.5, 2, 3, 4, 6} ("FP4 GEMM on Rubin/Blackwell with CUTLASS",
// section 2.1); the thresholds are the midpoints, with '>' where the lower
// neighbour is even and '>=' where the upper one is.
__device__ __forceinline__ uint32_t e2m1_nearest(float y) {
  const float a = fabsf(y);
  const uint32_t i = (a > 0.25f) + (a >= 0.75f) + (a > 1.25f) + (a >= 1.75f) + (a > 2.5f) +
                     (a >= 3.5f) + (a > 5.0f);
  return i | ((y < 0.0f && i != 0u) ? 8u : 0u);
}

// FP32 -> E4M3FN, round to nearest even, saturating to +-448 (hardware cvt;
// both halves get the same value so the byte order does not matter).
__device__ __forceinline__ uint32_t f32_to_e4m3(float t) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %1;" : "=h"(r) : "f"(t));
  return r & 0xFFu;
}

__device__ __forceinline__ float e4m3_to_f32(uint32_t b) {
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(b | (b << 8))));
  return __half2float(__ushort_as_half(static_cast<unsigned short>(h2 & 0xFFFFu)));
}

}  // namespace petit
