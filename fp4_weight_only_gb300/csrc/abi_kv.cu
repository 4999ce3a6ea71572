// C ABI of the 4-bit K/V cache: argument validation and kernel dispatch.
// Validation always comes first and never touches the GPU, so a rejected
// call enqueues nothing.
#include <cmath>

#include "../../include/petit.h"
#include "internal.h"
#include "kv.h"
#include "kv_layout.cuh"

namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 24;
constexpr int64_t kMaxBatch = int64_t(1) << 20;
constexpr int64_t kMaxHeads = 1024;
constexpr uint64_t kTimeoutNs = 2000000000ull;   // no legitimate wait lasts 2 s

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

petit_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? PETIT_OK : PETIT_ERR_CUDA; }

// Bytes of a head's 16-token group, 0 for a geometry without kernels.
int group_bytes(int32_t head_dim, int fmt) {
  if (fmt == PETIT_FMT_NVFP4)
    return head_dim == 128 ? petit::KvGroup<128, petit::kNVFP4>::kBytes
           : head_dim == 64 ? petit::KvGroup<64, petit::kNVFP4>::kBytes : 0;
  if (fmt == PETIT_FMT_MXFP4)
    return head_dim == 128 ? petit::KvGroup<128, petit::kMXFP4>::kBytes
           : head_dim == 64 ? petit::KvGroup<64, petit::kMXFP4>::kBytes : 0;
  return 0;
}

petit_status_t check_cache(const petit_kv_cache_t* c, petit::KvCacheArgs* out) {
  if (!c || !c->data || c->num_pages < 1) return PETIT_ERR_INVALID_ARG;
  if (c->fmt != PETIT_FMT_NVFP4 && c->fmt != PETIT_FMT_MXFP4) return PETIT_ERR_INVALID_ARG;
  if (c->fmt == PETIT_FMT_MXFP4 && c->scales) return PETIT_ERR_INVALID_ARG;
  const size_t page = petit_kv_page_bytes(c->page_size, c->num_kv_heads, c->head_dim, c->fmt);
  if (page == 0 || c->num_pages > (int64_t(1) << 31)) return PETIT_ERR_UNSUPPORTED_SHAPE;
  if (c->page_stride < static_cast<int64_t>(page)) return PETIT_ERR_INVALID_ARG;
  if (c->page_stride > (int64_t(1) << 40)) return PETIT_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(c->data, 16) || c->page_stride % 16 || !aligned(c->scales, 4)) return PETIT_ERR_MISALIGNED;
  int shift = 4;
  while ((1 << shift) < c->page_size) ++shift;
  *out = {static_cast<uint8_t*>(c->data), c->scales, c->num_pages, c->page_stride, shift,
          static_cast<uint32_t>(c->num_kv_heads), c->head_dim,
          c->fmt == PETIT_FMT_NVFP4 ? petit::kNVFP4 : petit::kMXFP4};
  return PETIT_OK;
}

petit_status_t check_rows(const petit_rows_t* r, petit::KvRows* out) {
  if (!r || !r->data) return PETIT_ERR_INVALID_ARG;
  if (!aligned(r->data, 16) || r->token_stride % 8 || r->head_stride % 8) return PETIT_ERR_MISALIGNED;
  *out = {r->data, r->token_stride, r->head_stride};
  return PETIT_OK;
}

// The two copies share everything but the direction.
petit_status_t copy_common(bool append, const petit_kv_cache_t* cache, const petit_rows_t* k, const petit_rows_t* v,
                           int dtype, const int64_t* slots, int64_t n, void* ws, size_t ws_bytes,
                           petit_stream_t stream) {
  petit::KvCacheArgs c;
  petit::KvRows kr, vr;
  if (petit_status_t st = check_cache(cache, &c)) return st;
  if (n < 0 || (dtype != PETIT_BF16 && dtype != PETIT_F16)) return PETIT_ERR_INVALID_ARG;
  if (n > kMaxTokens || n * 2 * c.heads >= (int64_t(1) << 31)) return PETIT_ERR_UNSUPPORTED_SHAPE;
  if (ws && ws_bytes < petit::kWsHeaderBytes) return PETIT_ERR_WORKSPACE;
  if (!aligned(ws, 16)) return PETIT_ERR_MISALIGNED;
  if (n == 0) return PETIT_OK;
  if (petit_status_t st = check_rows(k, &kr)) return st;
  if (petit_status_t st = check_rows(v, &vr)) return st;
  if (!slots) return PETIT_ERR_INVALID_ARG;
  if (!aligned(slots, 8)) return PETIT_ERR_MISALIGNED;
  int sms = 0;
  if (int st = petit::usable_device(&sms)) return static_cast<petit_status_t>(st);
  uint32_t* status = static_cast<uint32_t*>(ws);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool bf16 = dtype == PETIT_BF16;
  return from_cuda(append ? petit::launch_kv_append(c, kr, vr, bf16, slots, n, status, s)
                          : petit::launch_kv_read(c, slots, n, kr, vr, bf16, status, s));
}

}  // namespace

extern "C" {

size_t petit_kv_page_bytes(int32_t page_size, int32_t num_kv_heads, int32_t head_dim, int fmt) {
  if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1)) || num_kv_heads < 1 ||
      num_kv_heads > kMaxHeads)
    return 0;
  return static_cast<size_t>(num_kv_heads) * (page_size / petit::kKvGroup) * group_bytes(head_dim, fmt);
}

petit_status_t petit_kv_append(const petit_kv_cache_t* cache, const petit_rows_t* k, const petit_rows_t* v, int dtype,
                               const int64_t* slots, int64_t num_tokens, void* workspace, size_t workspace_bytes,
                               petit_stream_t stream) {
  return copy_common(true, cache, k, v, dtype, slots, num_tokens, workspace, workspace_bytes, stream);
}

petit_status_t petit_kv_read(const petit_kv_cache_t* cache, const int64_t* slots, int64_t num_tokens,
                             const petit_rows_t* k_out, const petit_rows_t* v_out, int dtype, void* workspace,
                             size_t workspace_bytes, petit_stream_t stream) {
  return copy_common(false, cache, k_out, v_out, dtype, slots, num_tokens, workspace, workspace_bytes, stream);
}

size_t petit_kv_attention_workspace_bytes(int32_t num_kv_heads, int32_t head_dim, int fmt) {
  if (petit_kv_page_bytes(16, num_kv_heads, head_dim, fmt) == 0) return 0;
  int sms = 0;
  if (petit::usable_device(&sms)) return 0;
  return petit::kv_attention_workspace(head_dim, sms);
}

petit_status_t petit_kv_attention(const petit_kv_cache_t* cache, const petit_kv_attention_t* args, void* workspace,
                                  size_t workspace_bytes, petit_stream_t stream) {
  petit::KvAttnArgs a{};
  if (petit_status_t st = check_cache(cache, &a.cache)) return st;
  if (!args || args->batch < 0 || args->total_q < 0 || args->max_q < 0 || args->max_pages < 0 || args->window < 0 ||
      args->num_q_heads < 1 || (args->causal != 0 && args->causal != 1) ||
      (args->dtype != PETIT_BF16 && args->dtype != PETIT_F16) || !std::isfinite(args->scale))
    return PETIT_ERR_INVALID_ARG;
  if (args->window > 0 && !args->causal) return PETIT_ERR_INVALID_ARG;
  if (args->num_q_heads % cache->num_kv_heads) return PETIT_ERR_INVALID_ARG;
  const int64_t group = args->num_q_heads / cache->num_kv_heads;
  if (args->batch > kMaxBatch || args->total_q > kMaxTokens || args->max_q > kMaxTokens || group > kMaxHeads ||
      args->total_q * args->num_q_heads >= (int64_t(1) << 31) - 64 ||
      args->max_pages > (int64_t(1) << 30) / cache->page_size)
    return PETIT_ERR_UNSUPPORTED_SHAPE;
  if (!args->q_offsets && args->total_q != args->batch * args->max_q) return PETIT_ERR_INVALID_ARG;
  if (args->table_stride < args->max_pages) return PETIT_ERR_INVALID_ARG;
  if (args->batch == 0 || args->total_q == 0) return PETIT_OK;
  if (petit_status_t st = check_rows(&args->q, &a.q)) return st;
  if (petit_status_t st = check_rows(&args->out, &a.out)) return st;
  if (!args->seq_lens || (!args->block_table && args->max_pages > 0)) return PETIT_ERR_INVALID_ARG;
  if (!aligned(args->lse, 4) || !aligned(args->block_table, 4) || !aligned(args->seq_lens, 4) ||
      !aligned(args->q_offsets, 4))
    return PETIT_ERR_MISALIGNED;
  if (!workspace) return PETIT_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return PETIT_ERR_MISALIGNED;
  int sms = 0;
  if (int st = petit::usable_device(&sms, &a.device)) return static_cast<petit_status_t>(st);
  if (workspace_bytes < petit::kv_attention_workspace(cache->head_dim, sms)) return PETIT_ERR_WORKSPACE;
  a.lse = args->lse;
  a.block_table = args->block_table;
  a.seq_lens = args->seq_lens;
  a.q_offsets = args->q_offsets;
  a.table_stride = args->table_stride;
  a.max_pages = args->max_pages;
  a.total_q = args->total_q;
  a.max_q = args->max_q;
  a.batch = static_cast<int>(args->batch);
  a.group = static_cast<int>(group);
  a.scale_log2 = args->scale * 1.4426950408889634f;
  a.causal = args->causal != 0;
  a.bf16 = args->dtype == PETIT_BF16;
  // a window that reaches past any context is none
  a.window = args->window >= (int64_t(1) << 31) ? 0 : args->window;
  a.workspace = static_cast<uint8_t*>(workspace);
  a.timeout_ns = kTimeoutNs;
  return from_cuda(petit::launch_kv_attention(a, sms, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
