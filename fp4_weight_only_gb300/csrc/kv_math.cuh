// Small conversions and products of the K/V attention kernels.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ptx.cuh"

namespace petit {

__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two FP32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(r)
      : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)),
        "l"(reinterpret_cast<const uint64_t&>(c)));
  return reinterpret_cast<const float2&>(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(r)
      : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)));
  return reinterpret_cast<const float2&>(r);
}

// Adds the two FP16 of w to two FP32 sums, without a conversion between.
__device__ __forceinline__ void add_f16x2(float2& sum, uint32_t w) {
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tadd.rn.f32.f16 %0, a, %0;\n\tadd.rn.f32.f16 %1, b, %1;\n\t}"
      : "+f"(sum.x), "+f"(sum.y)
      : "r"(w));
}

// FP16x2 of 2^(lo + 9) and 2^(hi + 9), for lo, hi <= 3: through FP32's exponent
// field, whose conversion makes subnormals and zero of what is below FP16.
__device__ __forceinline__ uint32_t f16x2_power(int lo, int hi) {
  return pack_f16(__uint_as_float(static_cast<uint32_t>(max(lo + 136, 0)) << 23),
                  __uint_as_float(static_cast<uint32_t>(max(hi + 136, 0)) << 23));
}

// FP16 bits of 2^n, n <= 15: subnormal below 2^-14, zero below 2^-24.
__device__ __forceinline__ uint32_t f16_power(int n) {
  return n >= -14 ? static_cast<uint32_t>(n + 15) << 10 : 0x400u >> min(-14 - n, 31);
}

// Two 16-bit elements of a query row in FP32.
__device__ __forceinline__ float2 unpack2(uint32_t w, bool bf16) {
  if (bf16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// The same, rounded, for an output row.
__device__ __forceinline__ uint32_t pack2(float x, float y, bool bf16) {
  uint32_t w;
  if (bf16)
    *reinterpret_cast<__nv_bfloat162*>(&w) = __floats2bfloat162_rn(x, y);
  else
    *reinterpret_cast<__half2*>(&w) = __floats2half2_rn(x, y);
  return w;
}

// The power of two that brings a row's largest magnitude to 2^12..2^13 (at
// most 2^127), as an exponent: the row is then exact in FP16 but for elements
// 2^26 below its largest, which lose bits, and products with values up to
// 6 * 2^12 and their sums stay far inside FP32.
__device__ __forceinline__ int row_shift(float amax) {
  const int e = static_cast<int>(__float_as_uint(amax) >> 23);
  return amax == 0.0f ? 0 : min(139 - e, 127);
}

// The softmax's weights are FP16: 2^(x - m + kWeightLift) with m the running
// maximum in log2 units, which moves when a score passes it by kWeightRoom, so
// a weight is at most 2^15.  They have 11 bits down to 2^-21 of the row's
// largest, and what lies below is a multiple of 2^-31 of it: a long context's
// many small weights beside one large one still add up.  (Without the lift all
// below 2^-25 were lost.)
constexpr float kWeightLift = 7.0f, kWeightRoom = 8.0f;

// Natural logarithm of a row's sum of e^x, of its maximum and sum of weights.
__device__ __forceinline__ float lse_of(float m, float l) {
  return l == 0.0f ? -INFINITY : (m - kWeightLift + log2f(l)) * 0.69314718055994531f;
}

// Weight of a partial result with maximum m and sum l when results meet at
// maximum M (no key: none; a NaN sum stays one).
__device__ __forceinline__ float weight_of(float m, float l, float M) {
  return m == -INFINITY ? (l == 0.0f ? 0.0f : 1.0f) : ex2(m - M);
}

// Waits for a phase of an mbarrier with the whole warp.  The loop is kept
// short, because a kernel of many roles lives or dies by its instruction
// cache: time and the abort flag are looked at every 1024 tries only.  A wait
// that lasts `timeout_ns` raises the flag; with the flag up waits return
// without their phase, so that every role still walks on to its end.
__device__ __forceinline__ void wait_phase(uint64_t* bar, uint32_t parity, uint64_t timeout_ns, int* abort) {
  const uint32_t b = smem_u32(bar);
  uint64_t since = 0;
  for (uint32_t tries = 1; !mbar_try_wait(b, parity & 1); ++tries) {
    if ((tries & 1023u) == 0) {
      const uint64_t now = global_timer_ns();
      if (since == 0) since = now;
      if (now - since > timeout_ns) *reinterpret_cast<volatile int*>(abort) = 1;
      if (*reinterpret_cast<volatile int*>(abort)) break;
    }
  }
  __syncwarp();
}

}  // namespace petit
