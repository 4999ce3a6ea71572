// Rotary positions of query and key heads.  Pair i of a head, (a, b), turns by
// the angle p * f_i of its token's position p:
//   a' = m (a cos - b sin),   b' = m (b cos + a sin)
// with a pair's elements side by side (interleaved) or rot_dim / 2 apart.
//
// Angles.  f_i is held in 2^-64 turns, so that p * f_i modulo a turn is the low
// half of an integer product, exact for any position (a position times a
// frequency in FP32 is 2^-4 radians off at 2^20).  Its upper 32 bits, a signed
// part of a turn, are the angle in -pi..pi that the hardware's sine and cosine
// take (2^-20.9 off at most: a sixteenth of FP16's rounding of the result, 2^-11
// of its size).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "layer.h"
#include "ptx.cuh"
#include "rows16.cuh"

namespace petit {
namespace {

constexpr int kThreads = 256;

template <int V>
struct Vec;
template <> struct Vec<8> { using T = uint4; };
template <> struct Vec<4> { using T = uint2; };
template <> struct Vec<2> { using T = uint32_t; };
template <> struct Vec<1> { using T = uint16_t; };

template <int V, bool BF16>
__device__ __forceinline__ void load(const uint16_t* p, float* x) {
  const typename Vec<V>::T v = *reinterpret_cast<const typename Vec<V>::T*>(p);
  if constexpr (V == 1) {
    x[0] = unpack16<BF16>(v).x;
  } else {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const float2 f = unpack16<BF16>(w[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

template <int V, bool BF16>
__device__ __forceinline__ void store(uint16_t* p, const float* x) {
  typename Vec<V>::T v;
  if constexpr (V == 1) {
    v = static_cast<uint16_t>(pack16<BF16>(x[0], 0.0f));
  } else {
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) w[i] = pack16<BF16>(x[2 * i], x[2 * i + 1]);
  }
  *reinterpret_cast<typename Vec<V>::T*>(p) = v;
}

// A thread turns V pairs (two vectors) of HPT heads of a token, `groups` heads
// apart; threads past the pairs copy the head's other elements.
template <int V, int HPT, bool INTER, bool BF16>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryArgs a, uint32_t units,
                                                          uint32_t groups) {
  const uint64_t index = static_cast<uint64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const uint32_t row = static_cast<uint32_t>(index / units);   // (below 2^32: checked by the host)
  const uint32_t u = static_cast<uint32_t>(index - static_cast<uint64_t>(row) * units);
  const int64_t token = row / groups;
  const int group = static_cast<int>(row - static_cast<uint32_t>(token) * groups);
  grid_dependency_wait();
  // (only now: what a kernel before this one wrote is in memory before the next one may begin)
  grid_launch_dependents();
  if (token >= a.tokens) return;
  const int turning = a.rot_dim / (2 * V);
  const bool rotate = static_cast<int>(u) < turning;
  // the two vectors' places in a head
  const int half = a.rot_dim / 2;
  int at0, at1;
  if (rotate) {
    at0 = INTER ? u * 2 * V : u * V;
    at1 = INTER ? at0 + V : at0 + half;
  } else {
    at0 = a.rot_dim + (u - turning) * 2 * V;
    at1 = at0 + V;
  }
  const bool second = at1 < a.head_dim;
  float x[HPT][2 * V];
  const uint16_t* src[HPT];
  uint16_t* dst[HPT];
#pragma unroll
  for (int i = 0; i < HPT; ++i) {
    const int h = group + i * static_cast<int>(groups);
    const bool is_q = h < a.q_heads;
    const int hh = is_q ? h : h - a.q_heads;
    const KvRows& in = is_q ? a.q : a.k;
    const KvRows& out = is_q ? a.q_out : a.k_out;
    src[i] = static_cast<const uint16_t*>(in.data) + token * in.token_stride + hh * in.head_stride;
    dst[i] = static_cast<uint16_t*>(out.data) + token * out.token_stride + hh * out.head_stride;
    if (h < a.heads) {
      load<V, BF16>(src[i] + at0, x[i]);
      if (second) load<V, BF16>(src[i] + at1, x[i] + V);
    }
  }
  float c[V], s[V];
  if (rotate) {
    const uint64_t p = a.positions_32 ? static_cast<uint64_t>(static_cast<int64_t>(static_cast<const int32_t*>(a.positions)[token]))
                                      : static_cast<uint64_t>(static_cast<const int64_t*>(a.positions)[token]);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int32_t part = static_cast<int32_t>((p * a.turns[u * V + j]) >> 32);
      const float angle = static_cast<float>(part) * 1.46291807926715968e-9f;   // 2 pi / 2^32
      c[j] = a.magnitude * __cosf(angle);
      s[j] = a.magnitude * __sinf(angle);
    }
  }
#pragma unroll
  for (int i = 0; i < HPT; ++i) {
    if (group + i * static_cast<int>(groups) >= a.heads) break;
    if (rotate) {
      float y[2 * V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int ia = INTER ? 2 * j : j, ib = INTER ? 2 * j + 1 : j + V;
        y[ia] = x[i][ia] * c[j] - x[i][ib] * s[j];
        y[ib] = x[i][ib] * c[j] + x[i][ia] * s[j];
      }
      store<V, BF16>(dst[i] + at0, y);
      store<V, BF16>(dst[i] + at1, y + V);
    } else {
      store<V, BF16>(dst[i] + at0, x[i]);
      if (second) store<V, BF16>(dst[i] + at1, x[i] + V);
    }
  }
}

template <int V, int HPT, bool INTER, bool BF16>
cudaError_t launch(const RotaryArgs& a, cudaStream_t stream) {
  const uint32_t rest = a.copy_rest ? (a.head_dim - a.rot_dim + 2 * V - 1) / (2 * V) : 0;
  const uint32_t units = a.rot_dim / (2 * V) + rest;
  const uint32_t groups = (a.heads + HPT - 1) / HPT;
  const uint64_t work = static_cast<uint64_t>(a.tokens) * groups * units;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((work + kThreads - 1) / kThreads));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rotary_kernel<V, HPT, INTER, BF16>, a, units, groups);
}

template <int V>
cudaError_t launch_as(const RotaryArgs& a, bool interleaved, bool bf16, cudaStream_t s) {
  if (interleaved) return bf16 ? launch<V, 2, true, true>(a, s) : launch<V, 2, true, false>(a, s);
  return bf16 ? launch<V, 2, false, true>(a, s) : launch<V, 2, false, false>(a, s);
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, bool interleaved, bool bf16, cudaStream_t stream) {
  // the widest vector that a pair's two elements allow (rows begin at 16-byte
  // boundaries, and so does every vector that divides rot_dim / 2)
  const int half = a.rot_dim / 2;
  if (half % 8 == 0) return launch_as<8>(a, interleaved, bf16, stream);
  if (half % 4 == 0) return launch_as<4>(a, interleaved, bf16, stream);
  if (half % 2 == 0) return launch_as<2>(a, interleaved, bf16, stream);
  return launch_as<1>(a, interleaved, bf16, stream);
}

}  // namespace petit
