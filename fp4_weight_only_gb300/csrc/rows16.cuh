// Eight 16-bit elements and eight E4M3 elements at a time, to and from FP32.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace petit {

template <bool BF16>
__device__ __forceinline__ float2 unpack16(uint32_t w) {
  if constexpr (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// Two values rounded to nearest even, x in the low half.
template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float x, float y) {
  uint32_t w;
  if constexpr (BF16)
    *reinterpret_cast<__nv_bfloat162*>(&w) = __floats2bfloat162_rn(x, y);
  else
    *reinterpret_cast<__half2*>(&w) = __floats2half2_rn(x, y);
  return w;
}

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack16<BF16>(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack16<BF16>(x[0], x[1]), pack16<BF16>(x[2], x[3]), pack16<BF16>(x[4], x[5]),
                    pack16<BF16>(x[6], x[7]));
}

// E4M3 codes of x / scale: nearest even, at most 448, NaN stays NaN.
__device__ __forceinline__ uint2 e4m3x8(const float (&x)[8], float scale) {
  uint32_t r[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float* y = x + 4 * i;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r[i])
        : "f"(y[0] / scale), "f"(y[1] / scale), "f"(y[2] / scale), "f"(y[3] / scale));
  }
  return make_uint2(r[0], r[1]);
}

}  // namespace petit
