// Launch interface of the operators around a decoder layer's products
// (norm.cu, rotary.cu) for the C ABI (abi_layer.cu).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "kv.h"

namespace petit {

struct NormArgs {
  const uint16_t* x;
  const uint16_t* residual;   // or null
  const void* weight;         // 16-bit elements or FP32, or null
  uint16_t* sum;              // or null
  void* out;                  // 16-bit elements, or E4M3 where scales is set
  float* scales;
  int64_t rows;
  int64_t x_stride, residual_stride, sum_stride, out_stride, scale_stride;   // elements
  int32_t dim;
  int32_t group_shift;        // a scale holds 2^group_shift vectors of 8 elements; 0: a row
  float eps;
  bool weight_f32;
};

cudaError_t launch_rms_norm(const NormArgs& a, bool bf16, cudaStream_t stream);

struct RotaryArgs {
  KvRows q, k, q_out, k_out;
  const uint64_t* turns;      // [rot_dim / 2], 2^-64 turns a position
  const void* positions;
  int64_t tokens;
  int32_t q_heads, heads;     // heads: q's and k's
  int32_t head_dim, rot_dim;
  float magnitude;
  bool positions_32;
  bool copy_rest;             // elements past rot_dim go to other rows
};

cudaError_t launch_rotary(const RotaryArgs& a, bool interleaved, bool bf16, cudaStream_t stream);

}  // namespace petit
