// The 4-bit K/V cache: quantising rows as they are written, and reading them
// back.  Both are one pass over the rows with nothing kept on chip, and what
// bounds them is memory: 8 heads of 128, 131071 tokens read in 113 us
// (6.1 TB/s), 8192 written and read back in 19.1 us (4.5 TB/s, two launches).
// Below some thousand tokens they are a launch: 1501 tokens read in 2.9 us, one
// written and read back in 3.8.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fp4_quant.cuh"
#include "internal.h"
#include "kv.h"
#include "kv_layout.cuh"

namespace petit {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void f16x8_to_f32(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

// Where token `slot`'s group of head h begins; nullptr when there is none
// (negative: skipped; past the cache: recorded).
__device__ __forceinline__ uint8_t* group_of(const KvCacheArgs& c, int64_t slot, int h, int group_bytes,
                                             uint32_t* status) {
  if (slot < 0) return nullptr;
  const int64_t page = slot >> c.page_shift;
  if (page >= c.num_pages) {
    if (status) atomicOr(status, kStatusBounds);
    return nullptr;
  }
  const int in_page = static_cast<int>(slot) & ((1 << c.page_shift) - 1);
  const int groups = 1 << (c.page_shift - 4);
  return c.data + page * c.page_stride +
         (static_cast<int64_t>(h) * groups + in_page / kKvGroup) * group_bytes;
}

// The largest magnitude among 16-bit elements, as their bits; NaN if one is.
template <bool BF16, int N>
__device__ __forceinline__ float amax_of(const uint4 (&v)[N]) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t a = w[j] & 0x7FFF7FFFu;
      if constexpr (BF16)
        asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(top) : "r"(a));
      else
        asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(top) : "r"(a));
    }
  }
  if constexpr (BF16) {
    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(top) : "r"(top >> 16));
    return __uint_as_float(top << 16);
  } else {
    asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(top) : "r"(top >> 16));
    return __half2float(__ushort_as_half(static_cast<unsigned short>(top & 0xFFFFu)));
  }
}

// E2M1 codes of eight finite values (nearest, ties to the even code, at most
// 6), the first in the low nibble; negative zeros as the hardware makes them.
__device__ __forceinline__ uint32_t e2m1x8(const float (&y)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return r;
}

// Negative zeros to zeros: a code without magnitude bits loses its sign.
__device__ __forceinline__ uint32_t no_negative_zeros(uint32_t w) {
  const uint32_t m = w & 0x77777777u;
  const uint32_t some = (m | m >> 1 | m >> 2) & 0x11111111u;
  return m | (w & some << 3);
}

// One block's codes and scale byte, by the weight quantiser's definition: FP32
// steps with IEEE rounding, code = nearest(x / d).  The quotient is taken as a
// product with 1 / d where that decides every code: it is within 2^-22 of the
// quotient, so where values 2^-20 above and below it have the same codes, the
// quotient has them too.  The rest (about one block in 10^4) is divided.
template <int FMT, bool BF16, int B>
__device__ __forceinline__ uint32_t quantize_block(const uint4 (&v)[B / 8], float g, uint32_t (&q)[B / 8]) {
  auto unpack = [&](int i, float(&x)[8]) {
    if constexpr (BF16)
      bf16x8_to_f32(v[i], x);
    else
      f16x8_to_f32(v[i], x);
  };
  float amax = amax_of<BF16>(v);
  const bool finite = amax < INFINITY;   // (not NaN either)
  if (!finite) {   // the definition's maximum leaves NaN out
    amax = 0.0f;
#pragma unroll 1
    for (int i = 0; i < B / 8; ++i) {
      float x[8];
      unpack(i, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(x[j]));
    }
  }
  if constexpr (FMT == kMXFP4) {
    const float y = fmaxf(amax, 1e-8f) / 6.0f;
    const uint32_t bits = __float_as_uint(y);
    const int ef = static_cast<int>(bits >> 23);
    const int e = (bits & 0x7FFFFFu) ? ef - 126 : ef - 127;  // exact ceil(log2 y)
    const uint32_t sc = min(e + 127, kKvMaxE8m0);
    const float inv = __uint_as_float((254u - sc) << 23);    // 2^(127 - sc), exact
#pragma unroll
    for (int i = 0; i < B / 8; ++i) {
      float x[8];
      unpack(i, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = finite || x[j] == x[j] ? x[j] * inv : 0.0f;   // (exact)
      q[i] = no_negative_zeros(e2m1x8(x));
    }
    return sc;
  } else {
    uint32_t sc = f32_to_e4m3(fmaxf(amax, 1e-8f) / (6.0f * g));
    if (sc == 0u) sc = 1u;
    const float d = e4m3_to_f32(sc) * g;
    const float inv = 1.0f / d;
    bool sure = finite && fabsf(inv) < 1e30f && fabsf(d) < 1e30f;
#pragma unroll
    for (int i = 0; i < B / 8; ++i) {
      float x[8], hi[8];
      unpack(i, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float y = x[j] * inv;
        hi[j] = y * (1.0f + 0x1p-20f);
        x[j] = y * (1.0f - 0x1p-20f);
      }
      q[i] = e2m1x8(x);
      sure = sure && q[i] == e2m1x8(hi);
      q[i] = no_negative_zeros(q[i]);
    }
    if (!sure) {
#pragma unroll 1
      for (int i = 0; i < B / 8; ++i) {
        float x[8];
        unpack(i, x);
        uint32_t w = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) w |= e2m1_nearest(x[j] / d) << (4 * j);
        q[i] = w;
      }
    }
    return sc;
  }
}

// A thread quantises a block (16 or 32 elements) of K and the same of V.  A row
// is the D elements of one (token, head); rows run over heads, then tokens, so
// consecutive threads read consecutive memory.
template <int D, int FMT, bool BF16>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(KvCacheArgs c, KvRows k, KvRows v,
                                                             const int64_t* __restrict__ slots,
                                                             uint32_t rows, uint32_t* status) {
  using G = KvGroup<D, FMT>;
  constexpr int B = G::kBlock;
  const uint32_t row = blockIdx.x * (kThreads / G::kScales) + threadIdx.x / G::kScales;
  const int blk = threadIdx.x % G::kScales;
  if (row >= rows) return;
  const uint32_t token = row / c.heads;
  const int h = row - token * c.heads;
  const int64_t slot = slots[token];
  uint4 x[2][B / 8];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const KvRows& r = s ? v : k;
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(r.data) + token * r.token_stride +
                                                      h * r.head_stride + blk * B);
#pragma unroll
    for (int i = 0; i < B / 8; ++i) x[s][i] = src[i];
  }
  uint8_t* grp = group_of(c, slot, h, G::kBytes, status);
  if (!grp) return;
  const int t = static_cast<int>(slot) & (kKvGroup - 1);
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const float g = FMT == kNVFP4 && c.scales ? c.scales[s * c.heads + h] : 1.0f;
    uint32_t q[B / 8];
    const uint32_t sc = quantize_block<FMT, BF16, B>(x[s], g, q);
    uint8_t* codes = grp + (s ? G::kVCodes : G::kKCodes) + t * G::kRow + blk * (B / 2);
    if constexpr (B == 16)
      *reinterpret_cast<uint2*>(codes) = make_uint2(q[0], q[1]);
    else
      *reinterpret_cast<uint4*>(codes) = make_uint4(q[0], q[1], q[2], q[3]);
    grp[(s ? G::kVScales : G::kKScales) + t * G::kScales + blk] = static_cast<uint8_t>(sc);
  }
}

// A thread decodes 8 codes (4 bytes in, 16 out) of K and of V, for kReadRows
// rows a pass apart: their loads are in flight together.
// (131071 tokens: 113 us with 2 and with 4, 135 with 1; 1501 tokens: 2.9, 3.1, 2.7.)
constexpr int kReadRows = 2;

template <int D, int FMT, bool BF16>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(KvCacheArgs c, const int64_t* __restrict__ slots,
                                                           KvRows k, KvRows v, uint32_t rows,
                                                           uint32_t* status) {
  using G = KvGroup<D, FMT>;
  constexpr int kPer = D / 8;                // threads of a row
  constexpr int kStep = kThreads / kPer;     // rows of a block's pass
  const uint32_t row0 = blockIdx.x * (kStep * kReadRows) + threadIdx.x / kPer;
  const int part = threadIdx.x % kPer;
  uint32_t w[kReadRows][2], sb[kReadRows][2];
  const uint8_t* grp[kReadRows];
  uint32_t token[kReadRows], head[kReadRows];
  int64_t slot[kReadRows];
#pragma unroll
  for (int i = 0; i < kReadRows; ++i) {
    const uint32_t row = row0 + i * kStep;
    token[i] = row / c.heads;
    head[i] = row - token[i] * c.heads;
    slot[i] = row < rows ? slots[token[i]] : -1;
  }
#pragma unroll
  for (int i = 0; i < kReadRows; ++i) {
    grp[i] = group_of(c, slot[i], head[i], G::kBytes, status);
    const int t = static_cast<int>(slot[i]) & (kKvGroup - 1);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      w[i][s] = sb[i][s] = 0;
      if (grp[i]) {
        w[i][s] = *reinterpret_cast<const uint32_t*>(grp[i] + (s ? G::kVCodes : G::kKCodes) + t * G::kRow + part * 4);
        sb[i][s] = grp[i][(s ? G::kVScales : G::kKScales) + t * G::kScales + part * 8 / G::kBlock];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kReadRows; ++i) {
    if (row0 + i * kStep >= rows) return;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const uint32_t p[4] = {e2m1x2_to_f16x2<0>(w[i][s]), e2m1x2_to_f16x2<1>(w[i][s]), e2m1x2_to_f16x2<2>(w[i][s]),
                             e2m1x2_to_f16x2<3>(w[i][s])};
      const float sc = FMT == kNVFP4 ? e4m3_to_f32(sb[i][s]) : e8m0_to_f32(sb[i][s]);
      const float g = FMT == kNVFP4 && c.scales ? c.scales[s * c.heads + head[i]] : 1.0f;
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&p[j]));
        // code * scale is exact in FP32; g rounds once, the output once more
        const float a = f.x * sc * g, b = f.y * sc * g;
        if constexpr (BF16)
          *reinterpret_cast<__nv_bfloat162*>(&o[j]) = __floats2bfloat162_rn(a, b);
        else
          *reinterpret_cast<__half2*>(&o[j]) = __floats2half2_rn(a, b);
      }
      const KvRows& r = s ? v : k;
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(r.data) + token[i] * r.token_stride + head[i] * r.head_stride +
                                part * 8) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

template <int D, int FMT, bool BF16>
cudaError_t append_as(const KvCacheArgs& c, const KvRows& k, const KvRows& v, const int64_t* slots, uint32_t rows,
                      uint32_t* status, cudaStream_t stream) {
  constexpr uint32_t per = kThreads / KvGroup<D, FMT>::kScales;
  kv_append_kernel<D, FMT, BF16><<<(rows + per - 1) / per, kThreads, 0, stream>>>(c, k, v, slots, rows, status);
  return cudaGetLastError();
}

template <int D, int FMT, bool BF16>
cudaError_t read_as(const KvCacheArgs& c, const int64_t* slots, const KvRows& k, const KvRows& v, uint32_t rows,
                    uint32_t* status, cudaStream_t stream) {
  constexpr uint32_t per = kThreads / (D / 8) * kReadRows;
  kv_read_kernel<D, FMT, BF16><<<(rows + per - 1) / per, kThreads, 0, stream>>>(c, slots, k, v, rows, status);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append(const KvCacheArgs& c, const KvRows& k, const KvRows& v, bool bf16, const int64_t* slots,
                             int64_t num_tokens, uint32_t* status, cudaStream_t stream) {
  const uint32_t rows = static_cast<uint32_t>(num_tokens * c.heads);
  return kv_dispatch(c.head_dim, c.fmt, bf16, [&](auto d, auto f, auto b) {
    return append_as<d, f, b>(c, k, v, slots, rows, status, stream);
  });
}

cudaError_t launch_kv_read(const KvCacheArgs& c, const int64_t* slots, int64_t num_tokens, const KvRows& k,
                           const KvRows& v, bool bf16, uint32_t* status, cudaStream_t stream) {
  const uint32_t rows = static_cast<uint32_t>(num_tokens * c.heads);
  return kv_dispatch(c.head_dim, c.fmt, bf16, [&](auto d, auto f, auto b) {
    return read_as<d, f, b>(c, slots, k, v, rows, status, stream);
  });
}

}  // namespace petit
