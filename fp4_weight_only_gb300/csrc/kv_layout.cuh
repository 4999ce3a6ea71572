// Memory order of the 4-bit K/V cache, shared by the kernels that write and
// read it (the order itself is part of the C ABI, petit.h).
#pragma once

#include <cstdint>

#include "fp4_layout.cuh"

namespace petit {

constexpr int kKvGroup = 16;   // tokens per storage group

// One head's group of 16 tokens: K codes, K scales, V codes, V scales.
template <int D, int FMT>
struct KvGroup {
  static constexpr int kBlock = FmtTraits<FMT>::kBlock;   // elements per scale
  static constexpr int kRow = D / 2;                      // code bytes of a token
  static constexpr int kScales = D / kBlock;              // scale bytes of a token
  static constexpr int kKCodes = 0;
  static constexpr int kKScales = kKvGroup * kRow;
  static constexpr int kVCodes = kKScales + kKvGroup * kScales;
  static constexpr int kVScales = kVCodes + kKvGroup * kRow;
  static constexpr int kBytes = kVScales + kKvGroup * kScales;
  static_assert(kBytes % 16 == 0 && kVCodes % 16 == 0, "bulk copies and vector loads");
};

// Largest E8M0 code written to the cache: 6 * 2^(252 - 127) is a finite BF16
// number, so no cached value is infinite.
constexpr int kKvMaxE8m0 = 252;

// FP16x2 of the two E2M1 codes of byte I of w (low nibble in the low half).
// One conversion instruction for two codes; on GB300 it runs at the rate of
// the integer pipe and picks the byte itself, so the natural nibble order
// costs 4 instructions for 8 codes (shifts and masks take 9 with the codes
// rearranged offline, 16 without).
template <int I>
__device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t w) {
  static_assert(I >= 0 && I < 4, "byte of a word");
  uint32_t r;
  if constexpr (I == 0)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}"
        : "=r"(r) : "r"(w));
  else if constexpr (I == 1)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}"
        : "=r"(r) : "r"(w));
  else if constexpr (I == 2)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}"
        : "=r"(r) : "r"(w));
  else
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, d;\n\t}"
        : "=r"(r) : "r"(w));
  return r;
}

// FP16x2 of two E4M3 bytes (low byte in the low half); exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t b2) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(b2)));
  return r;
}

__device__ __forceinline__ float e8m0_to_f32(uint32_t c) {
  // code 0 stands for 2^-127, an FP32 subnormal
  return __uint_as_float(c ? c << 23 : 0x00400000u);
}

}  // namespace petit
