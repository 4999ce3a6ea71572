// Launch interface of the 4-bit K/V cache between the C ABI (abi_kv.cu) and
// the kernels (kv_cache.cu, kv_attn.cu).
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>
#include <type_traits>

#include "fp4_layout.cuh"

namespace petit {

struct KvCacheArgs {
  uint8_t* data;
  const float* scales;   // [2][heads] or null
  int64_t num_pages;
  int64_t page_stride;   // bytes
  int page_shift;        // log2 of the tokens a page
  uint32_t heads;
  int head_dim;
  int fmt;
};

struct KvRows {
  void* data;            // 16-bit elements
  int64_t token_stride;  // elements
  int64_t head_stride;
};

struct KvAttnArgs {
  KvCacheArgs cache;
  KvRows q, out;
  float* lse;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* q_offsets;   // null: max_q rows for every sequence
  int64_t table_stride;
  int64_t max_pages;
  int64_t total_q;
  int64_t max_q;
  int batch;
  int group;                  // query heads per K/V head
  float scale_log2;           // softmax scale * log2(e)
  bool causal;
  bool bf16;
  int64_t window;             // 0: none
  uint8_t* workspace;
  uint64_t timeout_ns;
  int device;
};

// Calls f with head_dim, format and type as integral constants.
template <typename F>
cudaError_t kv_dispatch(int head_dim, int fmt, bool bf16, F&& f) {
  auto by_type = [&](auto d, auto m) {
    return bf16 ? f(d, m, std::true_type{}) : f(d, m, std::false_type{});
  };
  auto by_fmt = [&](auto d) {
    return fmt == kNVFP4 ? by_type(d, std::integral_constant<int, kNVFP4>{})
                         : by_type(d, std::integral_constant<int, kMXFP4>{});
  };
  return head_dim == 128 ? by_fmt(std::integral_constant<int, 128>{})
                         : by_fmt(std::integral_constant<int, 64>{});
}

cudaError_t launch_kv_append(const KvCacheArgs& c, const KvRows& k, const KvRows& v, bool bf16, const int64_t* slots,
                             int64_t num_tokens, uint32_t* status, cudaStream_t stream);
cudaError_t launch_kv_read(const KvCacheArgs& c, const int64_t* slots, int64_t num_tokens, const KvRows& k,
                           const KvRows& v, bool bf16, uint32_t* status, cudaStream_t stream);

// Workspace of the attention kernels on a device with num_sms SMs: the
// header and counters of a GEMM's workspace, then partial results.
size_t kv_attention_workspace(int head_dim, int num_sms);
// Allows a kernel its dynamic shared memory, once per device.
template <auto KERNEL>
cudaError_t kv_allow_smem(int device, size_t bytes) {
  static std::atomic<bool> done[64];
  if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
  if (!done[device].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(bytes));
    if (e != cudaSuccess) return e;
    done[device].store(true, std::memory_order_release);
  }
  return cudaSuccess;
}

// The kernel for many query rows (kv_prompt.cu), for groups of at most
// kKvPromptGroup query heads, and its share of the workspace.
constexpr int kKvPromptGroup = 128;
constexpr int kKvPromptCtas = 160;
size_t kv_prompt_partials(int head_dim, int num_sms);
cudaError_t launch_kv_prompt(const KvAttnArgs& a, int num_sms, cudaStream_t stream);
cudaError_t launch_kv_attention(const KvAttnArgs& a, int num_sms, cudaStream_t stream);

}  // namespace petit
