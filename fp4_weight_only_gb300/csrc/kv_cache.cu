// The 4-bit K/V cache: quantising rows as they are written, and reading them
// back.  Both are one pass over the rows with nothing kept on chip.
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

// A thread quantises one block (16 or 32 elements, 32 or 64 bytes in).  A row
// is the D elements of one (token, K or V, head): rows run over heads, then
// K/V, then tokens, so consecutive threads read consecutive memory.
template <int D, int FMT, bool BF16>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(KvCacheArgs c, KvRows k, KvRows v,
                                                             const int64_t* __restrict__ slots,
                                                             uint32_t rows, uint32_t* status) {
  using G = KvGroup<D, FMT>;
  constexpr int B = G::kBlock;
  const uint32_t row = blockIdx.x * (kThreads / G::kScales) + threadIdx.x / G::kScales;
  const int blk = threadIdx.x % G::kScales;
  if (row >= rows) return;
  const uint32_t th = row / c.heads;
  const int h = row - th * c.heads;
  const bool is_v = th & 1;
  const uint32_t token = th >> 1;
  const int64_t slot = slots[token];
  uint8_t* grp = group_of(c, slot, h, G::kBytes, status);
  if (!grp) return;
  const KvRows& r = is_v ? v : k;
  const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(r.data) + token * r.token_stride +
                                                    h * r.head_stride + blk * B);
  float x[B];
#pragma unroll
  for (int i = 0; i < B / 8; ++i) {
    float (&xi)[8] = *reinterpret_cast<float(*)[8]>(&x[8 * i]);
    if constexpr (BF16)
      bf16x8_to_f32(src[i], xi);
    else
      f16x8_to_f32(src[i], xi);
  }
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < B; ++i) amax = fmaxf(amax, fabsf(x[i]));
  uint32_t sc;
  uint32_t q[B / 8] = {};
  if constexpr (FMT == kNVFP4) {
    // FP32 steps with IEEE rounding, those of the weight quantiser
    const float g = c.scales ? c.scales[is_v * c.heads + h] : 1.0f;
    sc = f32_to_e4m3(fmaxf(amax, 1e-8f) / (6.0f * g));
    if (sc == 0u) sc = 1u;
    const float d = e4m3_to_f32(sc) * g;
#pragma unroll
    for (int i = 0; i < B; ++i) q[i >> 3] |= e2m1_nearest(x[i] / d) << (4 * (i & 7));
  } else {
    const float y = fmaxf(amax, 1e-8f) / 6.0f;
    const uint32_t bits = __float_as_uint(y);
    const int ef = static_cast<int>(bits >> 23);
    const int e = (bits & 0x7FFFFFu) ? ef - 126 : ef - 127;  // exact ceil(log2 y)
    sc = min(e + 127, kKvMaxE8m0);
    const float inv = __uint_as_float((254u - sc) << 23);    // 2^(127 - sc), exact
#pragma unroll
    for (int i = 0; i < B; ++i) q[i >> 3] |= e2m1_nearest(x[i] * inv) << (4 * (i & 7));
  }
  const int t = static_cast<int>(slot) & (kKvGroup - 1);
  uint8_t* codes = grp + (is_v ? G::kVCodes : G::kKCodes) + t * G::kRow + blk * (B / 2);
  if constexpr (B == 16)
    *reinterpret_cast<uint2*>(codes) = make_uint2(q[0], q[1]);
  else
    *reinterpret_cast<uint4*>(codes) = make_uint4(q[0], q[1], q[2], q[3]);
  grp[(is_v ? G::kVScales : G::kKScales) + t * G::kScales + blk] = static_cast<uint8_t>(sc);
}

// A thread decodes 8 codes (4 bytes in, 16 out).
template <int D, int FMT, bool BF16>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(KvCacheArgs c, const int64_t* __restrict__ slots,
                                                           KvRows k, KvRows v, uint32_t rows,
                                                           uint32_t* status) {
  using G = KvGroup<D, FMT>;
  constexpr int kPer = D / 8;   // threads of a row
  const uint32_t row = blockIdx.x * (kThreads / kPer) + threadIdx.x / kPer;
  const int part = threadIdx.x % kPer;
  if (row >= rows) return;
  const uint32_t th = row / c.heads;
  const int h = row - th * c.heads;
  const bool is_v = th & 1;
  const uint32_t token = th >> 1;
  const int64_t slot = slots[token];
  const uint8_t* grp = group_of(c, slot, h, G::kBytes, status);
  uint32_t w = 0;
  float s = 0.0f, g = 1.0f;
  if (grp) {
    const int t = static_cast<int>(slot) & (kKvGroup - 1);
    w = *reinterpret_cast<const uint32_t*>(grp + (is_v ? G::kVCodes : G::kKCodes) + t * G::kRow + part * 4);
    const uint32_t sb = grp[(is_v ? G::kVScales : G::kKScales) + t * G::kScales + part * 8 / G::kBlock];
    s = FMT == kNVFP4 ? e4m3_to_f32(sb) : e8m0_to_f32(sb);
    if (FMT == kNVFP4 && c.scales) g = c.scales[is_v * c.heads + h];
  }
  const uint32_t p[4] = {e2m1x2_to_f16x2<0>(w), e2m1x2_to_f16x2<1>(w), e2m1x2_to_f16x2<2>(w),
                         e2m1x2_to_f16x2<3>(w)};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&p[i]));
    // code * scale is exact in FP32; g rounds once, the output once more
    const float a = f.x * s * g, b = f.y * s * g;
    if constexpr (BF16)
      *reinterpret_cast<__nv_bfloat162*>(&o[i]) = __floats2bfloat162_rn(a, b);
    else
      *reinterpret_cast<__half2*>(&o[i]) = __floats2half2_rn(a, b);
  }
  const KvRows& r = is_v ? v : k;
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(r.data) + token * r.token_stride + h * r.head_stride +
                            part * 8) = make_uint4(o[0], o[1], o[2], o[3]);
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
  constexpr uint32_t per = kThreads / (D / 8);
  kv_read_kernel<D, FMT, BF16><<<(rows + per - 1) / per, kThreads, 0, stream>>>(c, slots, k, v, rows, status);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append(const KvCacheArgs& c, const KvRows& k, const KvRows& v, bool bf16, const int64_t* slots,
                             int64_t num_tokens, uint32_t* status, cudaStream_t stream) {
  const uint32_t rows = static_cast<uint32_t>(num_tokens * 2 * c.heads);
  return kv_dispatch(c.head_dim, c.fmt, bf16, [&](auto d, auto f, auto b) {
    return append_as<d, f, b>(c, k, v, slots, rows, status, stream);
  });
}

cudaError_t launch_kv_read(const KvCacheArgs& c, const int64_t* slots, int64_t num_tokens, const KvRows& k,
                           const KvRows& v, bool bf16, uint32_t* status, cudaStream_t stream) {
  const uint32_t rows = static_cast<uint32_t>(num_tokens * 2 * c.heads);
  return kv_dispatch(c.head_dim, c.fmt, bf16, [&](auto d, auto f, auto b) {
    return read_as<d, f, b>(c, slots, k, v, rows, status, stream);
  });
}

}  // namespace petit
