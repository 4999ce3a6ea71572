// Attention over the 4-bit K/V cache for few query rows a sequence (serving:
// one token, or a few drafted ones).
//
// For a K/V head's rows q_r (query tokens x heads of the group) and keys j
//     x_rj = scale * q_r . k_j,   o_r = sum_j 2^(x'_rj - m_r) v_j / sum_j 2^(x'_rj - m_r)
// with x' = x log2(e) and m_r a running maximum: one pass over the cache.
// What bounds it is reading the cache (D + 2 D / B bytes a token and head);
// the work per byte is the conversion of the codes, so both products are laid
// out to use each converted code once for all rows: keys (then head
// dimensions) are the 16 rows of mma.m16n8k16 and 8 query rows its columns,
//     S^T[16 keys, 8] = K[16, D] Q^T[D, 8],   O^T[D, 8] += V^T[D, 16] P^T[16, 8],
// and a group of 8 query heads wastes nothing.
//
// Layouts.  A lane of the MMA is (g, t) = (lane / 4, lane % 4).
//  - K: the contraction may run over D in any order, so lane t takes D/4
//    consecutive elements of a key (its own scales, one vector load) and Q is
//    loaded in the same order.
//  - V: lane g takes D/8 consecutive dimensions, for the four keys of the
//    lane's four contraction slots; the nibbles of two keys are interleaved
//    before the conversion, so that one conversion gives a pair over keys.
//  - Row r of a 16-key MMA is key kv_key_of_row(r): with consecutive keys in
//    lanes t, V's loads touch alternate halves of the banks.
//  - P moves from S^T's accumulator layout to the B operand with two 8x8
//    transposes (movmatrix), with no shared memory.
// Both products are FP16: codes times NVFP4 scales are exact in FP16, q is
// brought into FP16's range by a power of two per row (exact but for elements
// 2^26 below the row's largest), and p is rounded to 11 bits, which adds less
// than the rounding of a 16-bit output.  MXFP4 scales exceed FP16's range:
// K's are taken relative to the token's largest and V's relative to the
// largest seen in the dimension block, and the difference is applied in FP32
// (exact for scales up to 2^32 below that largest).
//
// Work split.  The keys of every (sequence, K/V head, block of 8 NB rows) are
// cut into tiles of 32; the tiles of the whole call, numbered in that order,
// are cut into equal ranges, one a CTA, so that ragged lengths balance without
// the host knowing them.  A CTA's producer warp fetches tiles with bulk copies
// into a ring; eight consumer warps take them in turn, each with its own
// running maximum, and meet when the CTA leaves an item.  Items cut between
// CTAs leave FP32 partials, and the last CTA to arrive adds them in CTA order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "kv.h"
#include "kv_layout.cuh"
#include "kv_math.cuh"
#include "ptx.cuh"

namespace petit {
namespace {

constexpr int kTile = 32;                    // keys of a tile
constexpr int kWarps = 8;                    // consumer warps
constexpr int kConsumers = kWarps * 32;
constexpr int kThreads = kConsumers + 32;
constexpr int kStages = 2 * kWarps;          // ring depth: a warp owns two stages
constexpr int kMaxCtas_ = 608;               // partial slots are sized for this

__device__ __forceinline__ int kv_key_of_row(int r) {   // r in 0..7; + 8 for the upper rows
  const int i = r >> 1;
  return (r & 1) ? (i ^ 1) + 4 : i;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ void consumers_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kConsumers) : "memory");
}

// ------------------------------------------------------------ work split
// What the kernels need of one sequence.
struct Seq {
  int len;      // keys
  int nq;       // query rows
  int q0;       // first query row
  int lo;       // first key of tile 0
  int tiles;    // tiles of an item, at least 1 so that empty rows are written
  int64_t blocks;   // row blocks
};

__device__ __forceinline__ Seq load_seq(const KvAttnArgs& a, int b, int rows_per_block, uint32_t* status) {
  Seq s;
  const int64_t cap = a.max_pages << a.cache.page_shift;
  s.len = a.seq_lens[b];
  bool bad = s.len < 0 || s.len > cap;
  s.len = s.len < 0 ? 0 : static_cast<int>(s.len < cap ? s.len : cap);
  if (a.q_offsets) {
    const int q0 = a.q_offsets[b], q1 = a.q_offsets[b + 1];
    const bool ok = q0 >= 0 && q1 >= q0 && q1 <= a.total_q;
    bad = bad || !ok;
    s.q0 = ok ? q0 : 0;
    s.nq = ok ? q1 - q0 : 0;
  } else {
    s.q0 = static_cast<int>(b * a.max_q);
    s.nq = static_cast<int>(a.max_q);
  }
  if (bad) atomicOr(status, kStatusBounds);
  s.lo = 0;
  if (a.window > 0) {
    const int64_t first = static_cast<int64_t>(s.len) - s.nq - a.window + 1;
    s.lo = first > 0 ? static_cast<int>(first) & ~(kTile - 1) : 0;
  }
  s.tiles = s.len > s.lo ? (s.len - s.lo + kTile - 1) / kTile : 1;
  s.blocks = (static_cast<int64_t>(s.nq) * a.group + rows_per_block - 1) / rows_per_block;
  return s;
}

__device__ __forceinline__ int64_t seq_tiles(const KvAttnArgs& a, const Seq& s) {
  return s.blocks * a.cache.heads * s.tiles;
}

// A CTA's range of tiles and where it begins.
struct Range {
  int64_t total;   // tiles of the whole call
  int64_t begin, end;
  int ctas;        // CTAs with a range
  int b;           // sequence of `begin`
  int64_t rem;     // tiles of it before `begin`
};

__device__ __forceinline__ int64_t range_begin(int64_t total, int ctas, int64_t c) { return total * c / ctas; }

// The CTA whose range holds tile x.
__device__ __forceinline__ int cta_of_tile(int64_t total, int ctas, int64_t x) {
  return static_cast<int>(((x + 1) * ctas + total - 1) / total) - 1;
}

// Every thread of the CTA calls this; `sh` holds kThreads / 32 + 4 values.
// A CTA gets at least kWarps tiles, one a warp: below that, more CTAs only
// add partials.
__device__ Range find_range(const KvAttnArgs& a, int rows_per_block, int64_t* sh, uint32_t* status) {
  constexpr int kW = kThreads / 32;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  Range r{};
  int64_t sum = 0;
  for (int b = tid; b < a.batch; b += kThreads) sum += seq_tiles(a, load_seq(a, b, rows_per_block, status));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if (lane == 0) sh[warp] = sum;
  __syncthreads();
  for (int w = 0; w < kW; ++w) r.total += sh[w];
  __syncthreads();
  const int64_t most = (r.total + kWarps - 1) / kWarps;
  r.ctas = most < gridDim.x ? static_cast<int>(most) : static_cast<int>(gridDim.x);
  if (static_cast<int>(blockIdx.x) >= r.ctas) {
    r.begin = r.end = 0;
    return r;
  }
  r.begin = range_begin(r.total, r.ctas, blockIdx.x);
  r.end = range_begin(r.total, r.ctas, blockIdx.x + 1);
  // find `begin`: prefix sums over sequences, a block of them at a time
  int64_t base = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
    const int b = b0 + tid;
    const int64_t mine = b < a.batch ? seq_tiles(a, load_seq(a, b, rows_per_block, status)) : 0;
    int64_t pre = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xFFFFFFFFu, pre, o);
      if (lane >= o) pre += v;
    }
    if (lane == 31) sh[warp] = pre;
    __syncthreads();
    int64_t before = base, all = 0;
    for (int w = 0; w < kW; ++w) {
      if (w < warp) before += sh[w];
      all += sh[w];
    }
    before += pre - mine;
    if (mine > 0 && before <= r.begin && r.begin < before + mine) {
      sh[kW] = b;
      sh[kW + 1] = r.begin - before;
    }
    base += all;
    __syncthreads();
    if (base > r.begin) break;
  }
  r.b = static_cast<int>(sh[kW]);
  r.rem = sh[kW + 1];
  return r;
}

// Walks the items of a range.  All threads of the CTA step it alike.
struct Walk {
  int64_t pos, end;
  int b;
  int64_t rem;
  Seq s;
  int h;           // K/V head
  int64_t block;   // row block
  int ta, tb;      // tiles of the item in this range

  __device__ __forceinline__ Walk(const KvAttnArgs& a, const Range& r, int rows_per_block, uint32_t* status)
      : pos(r.begin), end(r.end), b(r.b), rem(r.rem) {
    if (pos < end) {
      s = load_seq(a, b, rows_per_block, status);
      place();
    }
  }
  __device__ __forceinline__ bool done() const { return pos >= end; }
  __device__ __forceinline__ void place() {
    const int64_t item = rem / s.tiles;
    ta = static_cast<int>(rem - item * s.tiles);
    const int64_t left = end - pos;
    tb = left < s.tiles - ta ? ta + static_cast<int>(left) : s.tiles;
    h = static_cast<int>(item / s.blocks);
    block = item - static_cast<int64_t>(h) * s.blocks;
  }
  __device__ __forceinline__ void next(const KvAttnArgs& a, int rows_per_block, uint32_t* status) {
    pos += tb - ta;
    rem += tb - ta;
    if (pos >= end) return;
    if (rem == seq_tiles(a, s)) {
      rem = 0;
      do {
        s = load_seq(a, ++b, rows_per_block, status);
      } while (s.blocks == 0 && b + 1 < a.batch);
    }
    place();
  }
};

// ------------------------------------------------------------ the kernel
template <int N>
__device__ __forceinline__ void zero(uint32_t (&w)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) w[i] = 0;
}

// One 16-dimension step of O^T += V^T P^T: byte I of the interleaved words
// holds dimensions 2 i and 2 i + 1 of the lane's part for its four keys.
template <int I, int NB, int K>
__device__ __forceinline__ void pv_step(float (&o)[NB][K][4], const uint32_t (&p)[NB][2], int i, uint32_t lo01,
                                        uint32_t hi01, uint32_t lo23, uint32_t hi23, uint32_t s01, uint32_t s23) {
  const uint32_t a0 = mul2(e2m1x2_to_f16x2<I>(lo01), s01), a1 = mul2(e2m1x2_to_f16x2<I>(hi01), s01);
  const uint32_t a2 = mul2(e2m1x2_to_f16x2<I>(lo23), s23), a3 = mul2(e2m1x2_to_f16x2<I>(hi23), s23);
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) mma_f16(o[nb][i], a0, a1, a2, a3, p[nb][0], p[nb][1]);
}

template <int E>
__device__ __forceinline__ void load_row(const float* p, float (&v)[E]) {
  if constexpr (E == 4) {
    const float4 x = __ldcg(reinterpret_cast<const float4*>(p));
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
  } else {
    const float2 x = __ldcg(reinterpret_cast<const float2*>(p));
    v[0] = x.x, v[1] = x.y;
  }
}

// Row `row` of (sequence, K/V head) to the output: lane's D / 32 dimensions.
template <int D>
__device__ __forceinline__ void store_row(const KvAttnArgs& a, const Seq& s, int64_t row, int h, int lane, float M,
                                          float L, const float (&acc)[D / 32], float gv) {
  const int64_t tok = s.q0 + row / a.group;
  const int64_t head = static_cast<int64_t>(h) * a.group + row % a.group;
  const float inv = L == 0.0f ? 0.0f : gv / L;   // no key: zeros
  uint32_t w[D / 64];
#pragma unroll
  for (int i = 0; i < D / 64; ++i) w[i] = pack2(acc[2 * i] * inv, acc[2 * i + 1] * inv, a.bf16);
  uint16_t* dst = static_cast<uint16_t*>(a.out.data) + tok * a.out.token_stride + head * a.out.head_stride +
                  lane * (D / 32);
  if constexpr (D == 128)
    *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  else
    *reinterpret_cast<uint32_t*>(dst) = w[0];
  if (a.lse && lane == 0)
    a.lse[tok * (static_cast<int64_t>(a.cache.heads) * a.group) + head] =
        L == 0.0f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
}

template <int D, int FMT, int NB>
struct Smem {
  using G = KvGroup<D, FMT>;
  static constexpr int kStage = (kTile / kKvGroup) * G::kBytes;
  static constexpr int kORow = D + 4;   // padded row of the merge buffer
  alignas(128) uint8_t ring[kStages][kStage];
  float o[kWarps][8][kORow];
  float m[kWarps][8], l[kWarps][8];
  uint2 q[NB][D / 16][32];              // B operands
  uint64_t full[kStages], empty[kStages];
  int valid[kStages];                   // bit u: group u of the stage holds keys
  int64_t scan[kThreads / 32 + 2];
  int abort;
  int last;
};

template <int NB>
struct Partials {   // FP32, per CTA two slots (begins inside an item: 0, begins it: 1)
  static __host__ __device__ constexpr size_t floats(int D) { return static_cast<size_t>(NB) * 8 * (D + 2); }
};

template <int D, int FMT, int NB>
__global__ void __launch_bounds__(kThreads, NB == 1 ? 2 : 1) kv_attn_kernel(const __grid_constant__ KvAttnArgs a) {
  using S = Smem<D, FMT, NB>;
  using G = KvGroup<D, FMT>;
  constexpr int kRows = 8 * NB;
  constexpr int kK = D / 16;            // MMAs along D of the first product, row tiles of the second
  extern __shared__ __align__(128) uint8_t raw[];
  S& sm = *reinterpret_cast<S*>(raw);
  uint32_t* status = reinterpret_cast<uint32_t*>(a.workspace);
  uint32_t* counters = reinterpret_cast<uint32_t*>(a.workspace + kWsHeaderBytes);
  float* partials = reinterpret_cast<float*>(a.workspace + kWsHeaderBytes + kWsCountersBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&sm.full[i]), 1);
      mbar_init(smem_u32(&sm.empty[i]), 1);
    }
    sm.abort = 0;
    mbar_fence_init();
  }
  const Range range = find_range(a, kRows, sm.scan, status);   // (synchronises the CTA)
  if (range.begin >= range.end) return;
  const int64_t head_stride = static_cast<int64_t>(G::kBytes) << (a.cache.page_shift - 4);

  if (warp == kWarps) {
    // ------------------------------------------------------- producer
    const uint64_t policy = l2_policy_evict_first();
    uint32_t n = 0;   // tiles issued
    for (Walk w(a, range, kRows, status); !w.done(); w.next(a, kRows, status)) {
      const int32_t* table = a.block_table + w.b * a.table_stride;
      for (int t0 = w.ta; t0 < w.tb; t0 += 32) {
        // each lane finds the pages of one tile
        const int key0 = w.s.lo + (t0 + lane) * kTile;
        const uint8_t* src[2] = {nullptr, nullptr};
        int valid = 0;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int key = key0 + u * kKvGroup;
          if (t0 + lane < w.tb && key < w.s.len) {
            const int64_t page = table[key >> a.cache.page_shift];
            if (page >= 0 && page < a.cache.num_pages) {
              const int group = (key & ((1 << a.cache.page_shift) - 1)) / kKvGroup;
              src[u] = a.cache.data + page * a.cache.page_stride + w.h * head_stride + group * G::kBytes;
              valid |= 1 << u;
            } else {
              atomicOr(status, kStatusBounds);
            }
          }
        }
        const int count = min(32, w.tb - t0);
        for (int i = 0; i < count; ++i, ++n) {
          const int stage = n % kStages;
          if (n >= kStages && !mbar_wait_bounded(smem_u32(&sm.empty[stage]), (n / kStages - 1) & 1, a.timeout_ns,
                                                 &sm.abort))
            sm.abort = 1;
          __syncwarp();
          if (lane == i) {
            const uint32_t bar = smem_u32(&sm.full[stage]);
            sm.valid[stage] = valid;
            mbar_arrive_expect_tx(bar, (valid & 1 ? G::kBytes : 0) + (valid & 2 ? G::kBytes : 0));
            const uint32_t dst = smem_u32(sm.ring[stage]);
            if (valid == 3 && src[1] == src[0] + G::kBytes) {
              bulk_g2s(dst, src[0], 2 * G::kBytes, bar, policy);
            } else {
              if (valid & 1) bulk_g2s(dst, src[0], G::kBytes, bar, policy);
              if (valid & 2) bulk_g2s(dst + G::kBytes, src[1], G::kBytes, bar, policy);
            }
          }
          __syncwarp();
        }
      }
    }
    // no copy may be in flight when the CTA ends, also after an abort
    for (uint32_t i = n > kStages ? n - kStages : 0; i < n; ++i)
      mbar_wait_bounded(smem_u32(&sm.full[i % kStages]), (i / kStages) & 1, a.timeout_ns, nullptr);
    if (lane == 0 && sm.abort) atomicOr(status, kStatusTimeout);
    return;
  }

  // --------------------------------------------------------- consumers
  const int g = lane >> 2, t = lane & 3;
  const int key_a = kv_key_of_row(g);                  // K: this lane's keys are key_a and key_a + 8
  const int key_x = t, key_y = (t ^ 1) + 4;            // V: these and + 8
  constexpr int kKBytes = D / 8;                       // code bytes of a lane's part of a key
  constexpr int kKWords = kKBytes / 4;
  constexpr int kVBytes = D / 16;
  constexpr int kVWords = kVBytes / 4;
  const int k_scale = t * (D / 4) / G::kBlock;         // first scale of the lane's part
  const int v_scale = g * (D / 8) / G::kBlock;
  uint32_t n = 0;   // tiles of this CTA before the item

  for (Walk w(a, range, kRows, status); !w.done(); w.next(a, kRows, status)) {
    const Seq& s = w.s;
    const int rows = static_cast<int>(min(static_cast<int64_t>(kRows),
                                          static_cast<int64_t>(s.nq) * a.group - w.block * kRows));
    const int64_t row0 = w.block * kRows;
    const float gk = a.cache.scales ? a.cache.scales[w.h] : 1.0f;

    // Q: warp nb brings 8 rows to FP16; fq[nb][c] takes the scores of row
    // 8 nb + 2 t + c to log2 units
    if (warp < NB) {
      const int nb = warp;
      const int row = nb * 8 + g;
      float x[D / 4];
#pragma unroll
      for (int i = 0; i < D / 4; ++i) x[i] = 0.0f;
      if (row < rows) {
        const int64_t r = row0 + row;
        const int64_t tok = s.q0 + r / a.group;
        const int64_t head = w.h * a.group + r % a.group;
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q.data) +
                                                          tok * a.q.token_stride + head * a.q.head_stride +
                                                          t * (D / 4));
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const uint4 v = src[i];
          const uint32_t wd[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 f = unpack2(wd[j], a.bf16);
            x[8 * i + 2 * j] = f.x;
            x[8 * i + 2 * j + 1] = f.y;
          }
        }
      }
      float amax = 0.0f;
#pragma unroll
      for (int i = 0; i < D / 4; ++i) amax = fmaxf(amax, fabsf(x[i]));
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
      const int shift = row_shift(amax);
      const float up = ldexpf(1.0f, shift);
#pragma unroll
      for (int kk = 0; kk < kK; ++kk)
        sm.q[nb][kk][lane] = make_uint2(pack_f16(x[4 * kk] * up, x[4 * kk + 1] * up),
                                        pack_f16(x[4 * kk + 2] * up, x[4 * kk + 3] * up));
      if (t == 0) sm.m[nb][g] = ldexpf(a.scale_log2 * gk, -shift);
    }
    consumers_sync();
    float fq[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      fq[nb][0] = sm.m[nb][2 * t];
      fq[nb][1] = sm.m[nb][2 * t + 1];
    }
    uint2 qf[NB == 1 ? kK : 1];
    if constexpr (NB == 1) {
#pragma unroll
      for (int kk = 0; kk < kK; ++kk) qf[kk] = sm.q[0][kk][lane];
    }

    float o[NB][kK][4];
    float m[NB][2], l[NB][2];
    int vref = -1024;   // MXFP4: exponent code V is held relative to
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      m[nb][0] = m[nb][1] = -INFINITY;
      l[nb][0] = l[nb][1] = 0.0f;
#pragma unroll
      for (int i = 0; i < kK; ++i) o[nb][i][0] = o[nb][i][1] = o[nb][i][2] = o[nb][i][3] = 0.0f;
    }

    // tiles whose CTA-wide number is warp modulo kWarps
    const int count = w.tb - w.ta;
    for (int i = (warp - static_cast<int>(n % kWarps) + kWarps) % kWarps; i < count; i += kWarps) {
      const uint32_t num = n + i;
      const int stage = num % kStages;
      if (!mbar_wait_bounded(smem_u32(&sm.full[stage]), (num / kStages) & 1, a.timeout_ns, &sm.abort)) sm.abort = 1;
      __syncwarp();
      const uint8_t* base = sm.ring[stage];
      const int key0 = s.lo + (w.ta + i) * kTile;
      const int valid = sm.valid[stage];
      // the tile needs masks: it passes the keys every row sees, begins before
      // the first row's window ends, or lacks a page
      const bool masked = valid != 3 || key0 + kTile > (a.causal ? s.len - s.nq + 1 : s.len) ||
                          (a.window > 0 && key0 <= s.len - 1 - a.window);

      // ---- S^T = K Q^T for both groups
      float sc[2][NB][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint8_t* grp = base + u * G::kBytes;
        uint32_t wa[kKWords], wb[kKWords];
        {
          const uint8_t* pa = grp + G::kKCodes + key_a * G::kRow + t * kKBytes;
          const uint8_t* pb = pa + 8 * G::kRow;
          if constexpr (kKWords == 4) {
            const uint4 va = *reinterpret_cast<const uint4*>(pa), vb = *reinterpret_cast<const uint4*>(pb);
            wa[0] = va.x, wa[1] = va.y, wa[2] = va.z, wa[3] = va.w;
            wb[0] = vb.x, wb[1] = vb.y, wb[2] = vb.z, wb[3] = vb.w;
          } else {
            const uint2 va = *reinterpret_cast<const uint2*>(pa), vb = *reinterpret_cast<const uint2*>(pb);
            wa[0] = va.x, wa[1] = va.y;
            wb[0] = vb.x, wb[1] = vb.y;
          }
        }
        // FP16x2 scales of the lane's words
        uint32_t sa[kKWords], sb[kKWords];
        float ka = 1.0f, kb = 1.0f;   // MXFP4: what the token's scores still need
        const uint8_t* psa = grp + G::kKScales + key_a * G::kScales;
        const uint8_t* psb = psa + 8 * G::kScales;
        if constexpr (FMT == kNVFP4) {
          if constexpr (D == 128) {   // two scales, 16 elements each
            const uint32_t ha = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(psa + k_scale));
            const uint32_t hb = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(psb + k_scale));
            sa[0] = sa[1] = __byte_perm(ha, 0, 0x1010);
            sa[2] = sa[3] = __byte_perm(ha, 0, 0x3232);
            sb[0] = sb[1] = __byte_perm(hb, 0, 0x1010);
            sb[2] = sb[3] = __byte_perm(hb, 0, 0x3232);
          } else {
            sa[0] = sa[1] = e4m3x2_to_f16x2(psa[k_scale] * 0x0101u);
            sb[0] = sb[1] = e4m3x2_to_f16x2(psb[k_scale] * 0x0101u);
          }
        } else {
          int ca, cb, ma, mb;
          if constexpr (D == 128) {
            const uchar4 va = *reinterpret_cast<const uchar4*>(psa), vb = *reinterpret_cast<const uchar4*>(psb);
            ma = max(max(va.x, va.y), max(va.z, va.w));
            mb = max(max(vb.x, vb.y), max(vb.z, vb.w));
          } else {
            const uchar2 va = *reinterpret_cast<const uchar2*>(psa), vb = *reinterpret_cast<const uchar2*>(psb);
            ma = max(va.x, va.y);
            mb = max(vb.x, vb.y);
          }
          ca = psa[k_scale];
          cb = psb[k_scale];
          const uint32_t pa = f16_power(ca - ma + 12) * 0x10001u, pb = f16_power(cb - mb + 12) * 0x10001u;
#pragma unroll
          for (int j = 0; j < kKWords; ++j) sa[j] = pa, sb[j] = pb;
          // 2^(largest - 127 - 12)
          ka = e8m0_to_f32(ma) * 0.000244140625f;
          kb = e8m0_to_f32(mb) * 0.000244140625f;
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) sc[u][nb][0] = sc[u][nb][1] = sc[u][nb][2] = sc[u][nb][3] = 0.0f;
#pragma unroll
        for (int j = 0; j < kKWords; ++j) {
          const uint32_t a00 = mul2(e2m1x2_to_f16x2<0>(wa[j]), sa[j]), a01 = mul2(e2m1x2_to_f16x2<0>(wb[j]), sb[j]);
          const uint32_t a02 = mul2(e2m1x2_to_f16x2<1>(wa[j]), sa[j]), a03 = mul2(e2m1x2_to_f16x2<1>(wb[j]), sb[j]);
          const uint32_t a10 = mul2(e2m1x2_to_f16x2<2>(wa[j]), sa[j]), a11 = mul2(e2m1x2_to_f16x2<2>(wb[j]), sb[j]);
          const uint32_t a12 = mul2(e2m1x2_to_f16x2<3>(wa[j]), sa[j]), a13 = mul2(e2m1x2_to_f16x2<3>(wb[j]), sb[j]);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            uint2 b0, b1;
            if constexpr (NB == 1) {
              b0 = qf[2 * j];
              b1 = qf[2 * j + 1];
            } else {
              b0 = sm.q[nb][2 * j][lane];
              b1 = sm.q[nb][2 * j + 1][lane];
            }
            mma_f16(sc[u][nb], a00, a01, a02, a03, b0.x, b0.y);
            mma_f16(sc[u][nb], a10, a11, a12, a13, b1.x, b1.y);
          }
        }
        // to log2 units
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          sc[u][nb][0] *= FMT == kMXFP4 ? fq[nb][0] * ka : fq[nb][0];
          sc[u][nb][1] *= FMT == kMXFP4 ? fq[nb][1] * ka : fq[nb][1];
          sc[u][nb][2] *= FMT == kMXFP4 ? fq[nb][0] * kb : fq[nb][0];
          sc[u][nb][3] *= FMT == kMXFP4 ? fq[nb][1] * kb : fq[nb][1];
        }
      }
      if (masked) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int64_t row = row0 + nb * 8 + 2 * t + c;
            const int64_t p = a.causal ? s.len - s.nq + row / a.group : s.len - 1;
            const int64_t first = a.window > 0 ? p - a.window + 1 : 0;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int ja = key0 + u * kKvGroup + key_a, jb = ja + 8;
              const bool here = (valid >> u) & 1;
              if (!here || ja >= s.len || ja > p || ja < first) sc[u][nb][c] = -INFINITY;
              if (!here || jb >= s.len || jb > p || jb < first) sc[u][nb][2 + c] = -INFINITY;
            }
          }
        }
      }

      // ---- softmax: the reference maximum moves only when a score passes it
      // by 2^8, so most tiles need no exchange between lanes (p <= 2^8 fits FP16)
      uint32_t pb[2][NB][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float h0 = fmaxf(fmaxf(sc[0][nb][0], sc[0][nb][2]), fmaxf(sc[1][nb][0], sc[1][nb][2]));
        float h1 = fmaxf(fmaxf(sc[0][nb][1], sc[0][nb][3]), fmaxf(sc[1][nb][1], sc[1][nb][3]));
        if (__any_sync(0xFFFFFFFFu, h0 > m[nb][0] + 8.0f || h1 > m[nb][1] + 8.0f)) {
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) {
            h0 = fmaxf(h0, __shfl_xor_sync(0xFFFFFFFFu, h0, off));
            h1 = fmaxf(h1, __shfl_xor_sync(0xFFFFFFFFu, h1, off));
          }
          h0 = fmaxf(h0, m[nb][0]);
          h1 = fmaxf(h1, m[nb][1]);
          const float f0 = h0 == m[nb][0] ? 1.0f : ex2(m[nb][0] - h0);
          const float f1 = h1 == m[nb][1] ? 1.0f : ex2(m[nb][1] - h1);
          m[nb][0] = h0;
          m[nb][1] = h1;
          l[nb][0] *= f0;
          l[nb][1] *= f1;
#pragma unroll
          for (int i2 = 0; i2 < kK; ++i2) {
            o[nb][i2][0] *= f0;
            o[nb][i2][1] *= f1;
            o[nb][i2][2] *= f0;
            o[nb][i2][3] *= f1;
          }
        }
        // a row with no key yet: its scores are all -inf and p = 0
        const float m0 = m[nb][0] == -INFINITY ? 0.0f : m[nb][0];
        const float m1 = m[nb][1] == -INFINITY ? 0.0f : m[nb][1];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float p0 = ex2(sc[u][nb][0] - m0), p1 = ex2(sc[u][nb][1] - m1);
          const float p2 = ex2(sc[u][nb][2] - m0), p3 = ex2(sc[u][nb][3] - m1);
          l[nb][0] += p0 + p2;
          l[nb][1] += p1 + p3;
          pb[u][nb][0] = transpose8x8(pack_f16(p0, p1));
          pb[u][nb][1] = transpose8x8(pack_f16(p2, p3));
        }
      }

      // ---- O^T += V^T P^T
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint8_t* grp = base + u * G::kBytes;
        const uint8_t* pv = grp + G::kVCodes + g * kVBytes;
        uint32_t wx[kVWords], wy[kVWords], wz[kVWords], ww[kVWords];
        if constexpr (kVWords == 2) {
          const uint2 vx = *reinterpret_cast<const uint2*>(pv + key_x * G::kRow);
          const uint2 vy = *reinterpret_cast<const uint2*>(pv + key_y * G::kRow);
          const uint2 vz = *reinterpret_cast<const uint2*>(pv + (key_x + 8) * G::kRow);
          const uint2 vw = *reinterpret_cast<const uint2*>(pv + (key_y + 8) * G::kRow);
          wx[0] = vx.x, wx[1] = vx.y, wy[0] = vy.x, wy[1] = vy.y;
          wz[0] = vz.x, wz[1] = vz.y, ww[0] = vw.x, ww[1] = vw.y;
        } else {
          wx[0] = *reinterpret_cast<const uint32_t*>(pv + key_x * G::kRow);
          wy[0] = *reinterpret_cast<const uint32_t*>(pv + key_y * G::kRow);
          wz[0] = *reinterpret_cast<const uint32_t*>(pv + (key_x + 8) * G::kRow);
          ww[0] = *reinterpret_cast<const uint32_t*>(pv + (key_y + 8) * G::kRow);
        }
        const uint8_t* ps = grp + G::kVScales + v_scale;
        uint32_t c[4] = {ps[key_x * G::kScales], ps[key_y * G::kScales], ps[(key_x + 8) * G::kScales],
                         ps[(key_y + 8) * G::kScales]};
        if (masked) {
          // past the end the page may hold anything, NaN scales among it, and
          // 0 * NaN would reach the sums: such keys count as zeros
          const int j = key0 + u * kKvGroup;
          const bool here = (valid >> u) & 1;
          if (!here || j + key_x >= s.len) c[0] = 0, zero(wx);
          if (!here || j + key_y >= s.len) c[1] = 0, zero(wy);
          if (!here || j + key_x + 8 >= s.len) c[2] = 0, zero(wz);
          if (!here || j + key_y + 8 >= s.len) c[3] = 0, zero(ww);
        }
        uint32_t s01, s23;
        if constexpr (FMT == kNVFP4) {
          s01 = e4m3x2_to_f16x2(c[0] | c[1] << 8);
          s23 = e4m3x2_to_f16x2(c[2] | c[3] << 8);
        } else {
          int top = max(max(c[0], c[1]), max(c[2], c[3]));
          if (__any_sync(0xFFFFFFFFu, top > vref + 3)) {
            // the lanes of a dimension block share their reference
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            top = max(top, vref);
            const float f = top == vref ? 1.0f : ex2(static_cast<float>(vref - top));
            vref = top;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int i2 = 0; i2 < kK; ++i2) {
                o[nb][i2][0] *= f;
                o[nb][i2][1] *= f;
                o[nb][i2][2] *= f;
                o[nb][i2][3] *= f;
              }
          }
          const int r = 9 - vref;
          s01 = f16_power(static_cast<int>(c[0]) + r) | f16_power(static_cast<int>(c[1]) + r) << 16;
          s23 = f16_power(static_cast<int>(c[2]) + r) | f16_power(static_cast<int>(c[3]) + r) << 16;
        }
#pragma unroll
        for (int j = 0; j < kVWords; ++j) {
          // low nibbles of two keys side by side, then high nibbles
          const uint32_t lo01 = (wx[j] & 0x0F0F0F0Fu) | ((wy[j] << 4) & 0xF0F0F0F0u);
          const uint32_t hi01 = ((wx[j] >> 4) & 0x0F0F0F0Fu) | (wy[j] & 0xF0F0F0F0u);
          const uint32_t lo23 = (wz[j] & 0x0F0F0F0Fu) | ((ww[j] << 4) & 0xF0F0F0F0u);
          const uint32_t hi23 = ((wz[j] >> 4) & 0x0F0F0F0Fu) | (ww[j] & 0xF0F0F0F0u);
          pv_step<0>(o, pb[u], 4 * j + 0, lo01, hi01, lo23, hi23, s01, s23);
          pv_step<1>(o, pb[u], 4 * j + 1, lo01, hi01, lo23, hi23, s01, s23);
          pv_step<2>(o, pb[u], 4 * j + 2, lo01, hi01, lo23, hi23, s01, s23);
          pv_step<3>(o, pb[u], 4 * j + 3, lo01, hi01, lo23, hi23, s01, s23);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.empty[stage]));
    }
    n += count;

    // ---- the eight warps' results meet: warp r merges row r
    const float gv = a.cache.scales ? a.cache.scales[a.cache.heads + w.h] : 1.0f;
    const float vscale = FMT == kMXFP4 ? ldexpf(1.0f, max(vref, 0) - 127 - 9) : 1.0f;
    const bool whole = w.ta == 0 && w.tb == s.tiles;
    const int64_t item0 = w.pos - w.ta;   // the item's first tile in the call
    float* slot = partials + (2 * static_cast<size_t>(blockIdx.x) + (w.ta == 0 ? 1 : 0)) * Partials<NB>::floats(D);
    constexpr int kE = D / 32;            // dimensions of a lane in the merged rows
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      consumers_sync();   // the buffer is free (also: fq has been read)
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        l[nb][0] += __shfl_xor_sync(0xFFFFFFFFu, l[nb][0], off);
        l[nb][1] += __shfl_xor_sync(0xFFFFFFFFu, l[nb][1], off);
      }
      if (g == 0) {
        sm.m[warp][2 * t] = m[nb][0];
        sm.m[warp][2 * t + 1] = m[nb][1];
        sm.l[warp][2 * t] = l[nb][0];
        sm.l[warp][2 * t + 1] = l[nb][1];
      }
#pragma unroll
      for (int i = 0; i < kK; i += 2) {
        float* d0 = &sm.o[warp][2 * t][g * (D / 8) + 2 * i];
        float* d1 = &sm.o[warp][2 * t + 1][g * (D / 8) + 2 * i];
        *reinterpret_cast<float4*>(d0) = make_float4(o[nb][i][0] * vscale, o[nb][i][2] * vscale,
                                                     o[nb][i + 1][0] * vscale, o[nb][i + 1][2] * vscale);
        *reinterpret_cast<float4*>(d1) = make_float4(o[nb][i][1] * vscale, o[nb][i][3] * vscale,
                                                     o[nb][i + 1][1] * vscale, o[nb][i + 1][3] * vscale);
      }
      consumers_sync();
      float M = -INFINITY, L = 0.0f, acc[kE] = {};
#pragma unroll
      for (int v = 0; v < kWarps; ++v) M = fmaxf(M, sm.m[v][warp]);
#pragma unroll
      for (int v = 0; v < kWarps; ++v) {
        const float mv = sm.m[v][warp];
        const float f = mv == -INFINITY ? (sm.l[v][warp] == 0.0f ? 0.0f : 1.0f) : ex2(mv - M);
        L += f * sm.l[v][warp];
#pragma unroll
        for (int i = 0; i < kE; ++i) acc[i] += f * sm.o[v][warp][lane * kE + i];
      }
      const int row = nb * 8 + warp;
      if (whole) {
        if (row < rows) store_row<D>(a, s, row0 + row, w.h, lane, M, L, acc, gv);
      } else {
        float* pr = slot + static_cast<size_t>(row) * D + lane * kE;
#pragma unroll
        for (int i = 0; i < kE; ++i) pr[i] = acc[i];
        if (lane == 0) {
          slot[kRows * D + row] = M;
          slot[kRows * D + kRows + row] = L;
        }
      }
    }
    if (!whole) {
      const int c0 = cta_of_tile(range.total, range.ctas, item0);
      const int c1 = cta_of_tile(range.total, range.ctas, item0 + s.tiles - 1);
      consumers_sync();
      if (tid == 0) sm.last = atomic_add_acq_rel_gpu(&counters[c0], 1u) == static_cast<uint32_t>(c1 - c0);
      consumers_sync();
      if (sm.last) {
        if (tid == 0) counters[c0] = 0;   // every CTA of the item has arrived
        for (int row = warp; row < rows; row += kWarps) {
          const size_t ml = static_cast<size_t>(kRows) * D + row;
          float M = -INFINITY, L = 0.0f, acc[kE] = {};
          for (int c = c0 + lane; c <= c1; c += 32)
            M = fmaxf(M, __ldcg(partials + (2 * static_cast<size_t>(c) + (c == c0)) * Partials<NB>::floats(D) + ml));
#pragma unroll
          for (int off = 1; off < 32; off <<= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, off));
#pragma unroll 8
          for (int c = c0; c <= c1; ++c) {
            const float* p = partials + (2 * static_cast<size_t>(c) + (c == c0)) * Partials<NB>::floats(D);
            const float mc = __ldcg(p + ml), lc = __ldcg(p + ml + kRows);
            const float f = mc == -INFINITY ? (lc == 0.0f ? 0.0f : 1.0f) : ex2(mc - M);
            L += f * lc;
            float v[kE];
            load_row<kE>(p + static_cast<size_t>(row) * D + lane * kE, v);
#pragma unroll
            for (int i = 0; i < kE; ++i) acc[i] += f * v[i];
          }
          store_row<D>(a, s, row0 + row, w.h, lane, M, L, acc, gv);
        }
      }
    }
    consumers_sync();   // sm.q, sm.m and sm.last may be written again
  }
  if (tid == 0 && sm.abort) atomicOr(status, kStatusTimeout);
}

template <int D, int FMT, int NB>
cudaError_t launch_as(const KvAttnArgs& a, int num_sms, cudaStream_t stream) {
  auto* kernel = kv_attn_kernel<D, FMT, NB>;
  constexpr size_t kSmem = sizeof(Smem<D, FMT, NB>);
  if (cudaError_t e = kv_allow_smem<kv_attn_kernel<D, FMT, NB>>(a.device, kSmem)) return e;
  int grid = num_sms * (NB == 1 ? 2 : 1);
  if (grid > kMaxCtas_) grid = kMaxCtas_;
  kernel<<<grid, kThreads, kSmem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

size_t kv_attention_workspace(int head_dim, int num_sms) {
  const int ctas = 2 * num_sms < kMaxCtas_ ? 2 * num_sms : kMaxCtas_;
  const size_t own = sizeof(float) * 2 * ctas * Partials<4>::floats(head_dim);
  const size_t prompt = kv_prompt_partials(head_dim, num_sms);
  return kWsHeaderBytes + kWsCountersBytes + (own > prompt ? own : prompt);
}

cudaError_t launch_kv_attention(const KvAttnArgs& a, int num_sms, cudaStream_t stream) {
  const int64_t rows = a.max_q * a.group;
  if (rows > 16 && a.group <= kKvPromptGroup) return launch_kv_prompt(a, num_sms, stream);
  return kv_dispatch(a.cache.head_dim, a.cache.fmt, true, [&](auto d, auto f, auto) {
    if (rows <= 8) return launch_as<d, f, 1>(a, num_sms, stream);
    if (rows <= 16) return launch_as<d, f, 2>(a, num_sms, stream);
    return launch_as<d, f, 4>(a, num_sms, stream);
  });
}

}  // namespace petit
