// Root-mean-square norm of rows with the residual's addition, in 16 bits or in
// E4M3 with scales:
//   s = x + r,  r' = round(s),  y = s * (mean(s^2) + eps)^(-1/2) * w
// in FP32 from the loads on: s is not rounded before the norm.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "layer.h"
#include "ptx.cuh"
#include "rows16.cuh"

namespace petit {
namespace {

constexpr int kWarp = 32;

template <int TPR, typename F>
__device__ __forceinline__ float row_reduce(float v, float* shared, F&& f) {
#pragma unroll
  for (int o = kWarp / 2; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  if constexpr (TPR > kWarp) {
    constexpr int kWarps = TPR / kWarp;
    const int lane = threadIdx.x & (kWarp - 1);
    if (lane == 0) shared[threadIdx.x / kWarp] = v;
    __syncthreads();
    v = shared[lane & (kWarps - 1)];
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  }
  return v;
}

// TPR threads a row (a block holds one row, or as many as warps where a row is
// a warp's), VPT vectors of 8 elements a thread.
template <int TPR, int VPT, bool BF16, bool E4M3>
__global__ void __launch_bounds__(TPR > kWarp ? TPR : 4 * kWarp) norm_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float part[2][TPR / kWarp];
  const int64_t row = TPR > kWarp ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * 4 + threadIdx.x / kWarp;
  const int t = TPR > kWarp ? threadIdx.x : threadIdx.x & (kWarp - 1);
  grid_dependency_wait();
  // (only now: what a kernel before this one wrote is in memory before the next one may begin)
  grid_launch_dependents();
  if (row >= a.rows) return;
  const int vectors = a.dim / 8;
  float s[VPT][8];
  float squares = 0.0f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * TPR + t;
    uint4 x = make_uint4(0, 0, 0, 0), r = x;
    if (v < vectors) {
      x = *reinterpret_cast<const uint4*>(a.x + row * a.x_stride + v * 8);
      if (a.residual) r = *reinterpret_cast<const uint4*>(a.residual + row * a.residual_stride + v * 8);
    }
    unpack8<BF16>(x, s[i]);
    if (a.residual) {
      float f[8];
      unpack8<BF16>(r, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[i][j] += f[j];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) squares += s[i][j] * s[i][j];
  }
  squares = row_reduce<TPR>(squares, part[0], [](float p, float q) { return p + q; });
  const float norm = rsqrtf(squares / static_cast<float>(a.dim) + a.eps);
  float top = 0.0f;   // of the row (fmaxf leaves NaN out)
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * TPR + t;
    if (v < vectors && a.sum)
      *reinterpret_cast<uint4*>(a.sum + row * a.sum_stride + v * 8) = pack8<BF16>(s[i]);
    if (v < vectors) {
      float w[8];
      if (!a.weight) {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = 1.0f;
      } else if (a.weight_f32) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.weight) + v * 8);
        const float4 lo = p[0], hi = p[1];
        w[0] = lo.x, w[1] = lo.y, w[2] = lo.z, w[3] = lo.w, w[4] = hi.x, w[5] = hi.y, w[6] = hi.z, w[7] = hi.w;
      } else {
        unpack8<BF16>(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.weight) + v * 8), w);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) s[i][j] = s[i][j] * norm * w[j];
    }
    if constexpr (!E4M3) {
      if (v < vectors)
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + row * a.out_stride + v * 8) = pack8<BF16>(s[i]);
    } else if (a.group != a.dim) {
      // a scale's elements lie in group / 8 neighbouring lanes
      float m = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(s[i][j]));
      for (int o = a.group / 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      const float scale = fmaxf(m, 1e-8f) / 448.0f;
      if (v < vectors) {
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.out) + row * a.out_stride + v * 8) = e4m3x8(s[i], scale);
        if (v % (a.group / 8) == 0) a.scales[row * a.scale_stride + v / (a.group / 8)] = scale;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(s[i][j]));
    }
  }
  if constexpr (E4M3) {
    if (a.group == a.dim) {
      top = row_reduce<TPR>(top, part[1], [](float p, float q) { return fmaxf(p, q); });
      const float scale = fmaxf(top, 1e-8f) / 448.0f;
      if (t == 0) a.scales[row * a.scale_stride] = scale;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = i * TPR + t;
        if (v < vectors)
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.out) + row * a.out_stride + v * 8) = e4m3x8(s[i], scale);
      }
    }
  }
}

template <int TPR, int VPT, bool BF16, bool E4M3>
cudaError_t launch(const NormArgs& a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(TPR > kWarp ? a.rows : (a.rows + 3) / 4));
  cfg.blockDim = dim3(TPR > kWarp ? TPR : 4 * kWarp);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_kernel<TPR, VPT, BF16, E4M3>, a);
}

template <int TPR, int VPT>
cudaError_t launch_as(const NormArgs& a, bool bf16, cudaStream_t s) {
  if (a.scales) return bf16 ? launch<TPR, VPT, true, true>(a, s) : launch<TPR, VPT, false, true>(a, s);
  return bf16 ? launch<TPR, VPT, true, false>(a, s) : launch<TPR, VPT, false, false>(a, s);
}

}  // namespace

cudaError_t launch_rms_norm(const NormArgs& a, bool bf16, cudaStream_t stream) {
  const int vectors = a.dim / 8;
  if (vectors <= 32) return launch_as<32, 1>(a, bf16, stream);
  if (vectors <= 128) return launch_as<32, 4>(a, bf16, stream);
  if (vectors <= 1024) return launch_as<256, 4>(a, bf16, stream);
  if (vectors <= 4096) return launch_as<1024, 4>(a, bf16, stream);
  return cudaErrorInvalidValue;
}

}  // namespace petit
