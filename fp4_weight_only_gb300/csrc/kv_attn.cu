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
// into a ring; six consumer warps take them in turn, each with its own
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
#ifndef KVW
#define KVW 4
#define KVC 3
#define KVS 3
#endif
constexpr int kWarps = KVW;                    // consumer warps
constexpr int kConsumers = kWarps * 32;
constexpr int kThreads = kConsumers + 32;
constexpr int kMostCtas = 480;               // partial slots are sized for this
// What beginning and ending an item costs, in tiles: an item's first tile
// weighs 1 + kItemCost in the split, so that short contexts, whose items are
// mostly this, get no longer ranges than others.
#ifndef KIC
#define KIC 8
#endif
constexpr int kItemCost = KIC;
// The least a CTA gets: more than an item's cost, so that every CTA with units
// of an item has a tile of it, and about a tile a warp.
constexpr int kMinUnits = kWarps + kItemCost;

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
  int blocks;   // row blocks
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
  s.blocks = (s.nq * a.group + rows_per_block - 1) / rows_per_block;
  return s;
}

__device__ __forceinline__ int64_t seq_cost(const KvAttnArgs& a, const Seq& s) {
  return static_cast<int64_t>(s.blocks) * a.cache.heads * (s.tiles + kItemCost);
}

// A CTA's range and where it begins, in units of tiles: tile 0 of an item
// stands at the item's beginning, tile t > 0 kItemCost + t after it.
struct Range {
  int64_t total;   // of the whole call
  int64_t begin, end;
  int ctas;        // CTAs with a range
  int b;           // sequence of `begin`
  int64_t rem;     // units of it before `begin`
};

__device__ __forceinline__ int64_t range_begin(int64_t total, int ctas, int64_t c) { return total * c / ctas; }

// The CTA whose range holds unit x.
__device__ __forceinline__ int cta_of(int64_t total, int ctas, int64_t x) {
  return static_cast<int>(((x + 1) * ctas + total - 1) / total) - 1;
}

// Every thread of the CTA calls this; `sh` holds kThreads / 32 + 2 values.
__device__ Range find_range(const KvAttnArgs& a, int rows_per_block, int64_t* sh, uint32_t* status) {
  constexpr int kW = kThreads / 32;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  Range r{};
  int64_t sum = 0;
  for (int b = tid; b < a.batch; b += kThreads) sum += seq_cost(a, load_seq(a, b, rows_per_block, status));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if (lane == 0) sh[warp] = sum;
  __syncthreads();
  for (int w = 0; w < kW; ++w) r.total += sh[w];
  __syncthreads();
  const int64_t most = r.total > kMinUnits ? r.total / kMinUnits : r.total > 0;
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
    const int64_t mine = b < a.batch ? seq_cost(a, load_seq(a, b, rows_per_block, status)) : 0;
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

// Walks the items of a range; every role steps one of its own.  Positions are
// relative to the range's beginning (a range of 2^31 tiles would take an hour).
template <int N>
struct Walk {
  int span;        // the range's units
  int at;          // the item's first unit
  int b;
  int item;        // of the sequence: heads, and row blocks inside them
  Seq s;
  int h;           // K/V head
  int row0;        // first row of the block
  int rows;        // its rows
  int ta, tb;      // tiles of the item in this range

  __device__ __forceinline__ Walk(const KvAttnArgs& a, const Range& r, uint32_t* status)
      : span(static_cast<int>(r.end - r.begin)), b(r.b) {
    s = load_seq(a, b, N, status);
    const int64_t i = r.rem / (s.tiles + kItemCost);
    const int in = static_cast<int>(r.rem - i * (s.tiles + kItemCost));
    item = static_cast<int>(i);
    at = -in;
    // the first tile at or past the beginning
    ta = in == 0 ? 0 : in <= kItemCost ? 1 : in - kItemCost;
    if (ta < s.tiles)
      place(a);
    else   // the range begins between an item's only tile and the next item
      next_item(a, status);
  }
  __device__ __forceinline__ bool done() const { return at >= span; }
  __device__ __forceinline__ void place(const KvAttnArgs& a) {
    const int below = span - at - kItemCost;   // tiles below the range's end
    tb = below >= s.tiles ? s.tiles : below > ta ? below : ta + 1;
    h = item / s.blocks;
    row0 = (item - h * s.blocks) * N;
    rows = min(N, s.nq * a.group - row0);
  }
  __device__ __forceinline__ void next_item(const KvAttnArgs& a, uint32_t* status) {
    at += s.tiles + kItemCost;
    if (done()) return;
    if (++item == s.blocks * static_cast<int>(a.cache.heads)) {
      item = 0;
      do {
        s = load_seq(a, ++b, N, status);
      } while (s.blocks == 0 && b + 1 < a.batch);
    }
    ta = 0;
    place(a);
  }
  __device__ __forceinline__ void next(const KvAttnArgs& a, uint32_t* status) {
    if (tb < s.tiles)
      at = span;
    else
      next_item(a, status);
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

// Weight of a partial result with maximum m and sum l when results meet at
// maximum M (no key: none; a NaN sum stays one).
__device__ __forceinline__ float weight_of(float m, float l, float M) {
  return m == -INFINITY ? (l == 0.0f ? 0.0f : 1.0f) : ex2(m - M);
}

template <int E>
__device__ __forceinline__ void load_row(const float* p, float (&v)[E]) {
  if constexpr (E == 4) {
    const float4 x = *reinterpret_cast<const float4*>(p);
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
  } else {
    const float2 x = *reinterpret_cast<const float2*>(p);
    v[0] = x.x, v[1] = x.y;
  }
}

// Partials pass through L2: they were written by other SMs.
template <int E>
__device__ __forceinline__ void load_part(const float* p, float (&v)[E]) {
  if constexpr (E == 4) {
    const float4 x = __ldcg(reinterpret_cast<const float4*>(p));
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
  } else {
    const float2 x = __ldcg(reinterpret_cast<const float2*>(p));
    v[0] = x.x, v[1] = x.y;
  }
}

template <int E>
__device__ __forceinline__ void store_part(float* p, const float (&v)[E]) {
  if constexpr (E == 4)
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  else
    *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
}

// Row `row` of (sequence, K/V head) to the output: lane's D / 32 dimensions.
template <int D>
__device__ __forceinline__ void store_row(const KvAttnArgs& a, const Seq& s, int row, int h, int lane, float M,
                                          float L, const float (&acc)[D / 32], float gv) {
  const int64_t tok = s.q0 + row / a.group;
  const int64_t head = h * a.group + row % a.group;
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
  // CTAs an SM, and stages a warp: as many as registers and shared memory give
  static constexpr int kCtas = NB == 1 ? KVC : 2;
  static constexpr int kSlots = NB == 1 ? KVS : 2;
  static constexpr int kStages = kSlots * kWarps;
  // a warp's eight rows of results fit the stage it used last
  static constexpr int kORow = D + 4;
  static_assert(8 * kORow * 4 <= kStage, "results in a stage");
  alignas(128) uint8_t ring[kStages][kStage];
  static constexpr int kQueries = NB == 1 ? 4 : 2;   // items whose queries are on chip
  static constexpr int kList = 64;          // tiles listed ahead
  static_assert(kStages <= 32, "a lane a stage");
  alignas(16) uint16_t raw[kQueries][8 * NB][D];   // queries as they come
  const uint8_t* list[kList][2];            // where the groups of coming tiles lie
  uint4 q[NB][D / 32][32];                  // B operands, a lane's of two MMAs together
  float fq[8 * NB];                         // takes a row's scores to log2 units
  float m[kWarps][8], l[kWarps][8];
  uint64_t full[kStages], empty[kStages], qfull[kQueries], qfree[kQueries];
  int valid[kStages];                       // bit u: group u of the stage holds keys
  int held[kWarps];                         // the stage that holds a warp's results, or -1
  int64_t scan[kThreads / 32 + 2];
  int abort;
  int last;
};

// FP32, per CTA two slots (an item it begins inside of: 0, one it begins: 1).
template <int NB>
__host__ __device__ constexpr size_t partial_floats(int D) { return static_cast<size_t>(NB) * 8 * (D + 2); }

template <int D, int FMT, int NB>
__global__ void __launch_bounds__(kThreads, Smem<D, FMT, NB>::kCtas) kv_attn_kernel(const __grid_constant__ KvAttnArgs a) {
  using S = Smem<D, FMT, NB>;
  using G = KvGroup<D, FMT>;
  constexpr int kRows = 8 * NB;
  constexpr int kK = D / 16;            // MMAs along D of the first product, row tiles of the second
  extern __shared__ __align__(128) uint8_t raw_smem[];
  S& sm = *reinterpret_cast<S*>(raw_smem);
  uint32_t* status = reinterpret_cast<uint32_t*>(a.workspace);
  uint32_t* counters = reinterpret_cast<uint32_t*>(a.workspace + kWsHeaderBytes);
  float* partials = reinterpret_cast<float*>(a.workspace + kWsHeaderBytes + kWsCountersBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto wait = [&](uint64_t* bar, uint32_t phase) { wait_phase(bar, phase, a.timeout_ns, &sm.abort); };

  if (tid == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(smem_u32(&sm.full[i]), 1);
      mbar_init(smem_u32(&sm.empty[i]), 1);
    }
    for (int i = 0; i < S::kQueries; ++i) {
      mbar_init(smem_u32(&sm.qfull[i]), 1);
      mbar_init(smem_u32(&sm.qfree[i]), 1);
    }
    sm.abort = 0;
    mbar_fence_init();
  }
  const Range range = find_range(a, kRows, sm.scan, status);   // (synchronises the CTA)
  if (range.begin >= range.end) return;
  Walk<kRows> w(a, range, status);
  uint32_t items = 0;   // items before this one

  if (warp == kWarps) {
    // ------------------------------------------------------- producer
    // Issuing a copy takes a warp about 470 cycles on GB300 whatever the size,
    // and some 60 more for each further lane that issues with it.  So lane i
    // feeds stage i (tiles i, i + kStages, ...) and all lanes whose stage is
    // free issue together; where the tiles lie comes from a list in shared
    // memory that the warp writes ahead, 32 tiles at a time.
    const int64_t head_stride = static_cast<int64_t>(G::kBytes) << (a.cache.page_shift - 4);
    const uint64_t policy = l2_policy_evict_first();
    uint32_t listed = 0;              // tiles in the list so far
    int t0 = w.done() ? 0 : w.ta;     // next tile of the item to list
    bool begun = false;               // its queries are on their way
    uint32_t num = lane;              // this lane's next tile
    const bool feeds = lane < S::kStages;
    uint64_t idle = 0;
    bool all = w.done();              // everything is listed
    while (true) {
      if (!all && listed + 32 <= __reduce_min_sync(0xFFFFFFFFu, feeds ? num : ~0u) + S::kList) {
        const int buf = items % S::kQueries;
        if (!begun &&
            __all_sync(0xFFFFFFFFu, items < S::kQueries ||
                                        mbar_test_wait(smem_u32(&sm.qfree[buf]), (items / S::kQueries - 1) & 1))) {
          if (lane == 0) mbar_arrive_expect_tx(smem_u32(&sm.qfull[buf]), w.rows * D * 2);
          __syncwarp();
          if (lane < w.rows) {
            const int r = w.row0 + lane;
            const uint16_t* src = static_cast<const uint16_t*>(a.q.data) +
                                  static_cast<int64_t>(w.s.q0 + r / a.group) * a.q.token_stride +
                                  static_cast<int64_t>(w.h * a.group + r % a.group) * a.q.head_stride;
            bulk_g2s(smem_u32(sm.raw[buf][lane]), src, D * 2, smem_u32(&sm.qfull[buf]), l2_policy_evict_normal());
          }
          begun = true;
        }
        if (begun) {
          // each lane finds the pages of one tile
          const int32_t* table = a.block_table + w.b * a.table_stride;
          const int key0 = w.s.lo + (t0 + lane) * kTile;
          const uint8_t* src[2] = {nullptr, nullptr};
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int key = key0 + u * kKvGroup;
            if (t0 + lane < w.tb && key < w.s.len) {
              const int64_t page = table[key >> a.cache.page_shift];
              if (page >= 0 && page < a.cache.num_pages)
                src[u] = a.cache.data + page * a.cache.page_stride + w.h * head_stride +
                         ((key & ((1 << a.cache.page_shift) - 1)) / kKvGroup) * G::kBytes;
              else
                atomicOr(status, kStatusBounds);
            }
          }
          const int count = min(32, w.tb - t0);
          if (lane < count) {
            sm.list[(listed + lane) % S::kList][0] = src[0];
            sm.list[(listed + lane) % S::kList][1] = src[1];
          }
          __syncwarp();
          listed += count;
          t0 += count;
          if (t0 == w.tb) {
            w.next(a, status);
            ++items;
            begun = false;
            all = w.done();
            t0 = w.ta;
          }
        }
      }
      const uint32_t round = num / S::kStages;
      const bool go = feeds && num < listed &&
                      (round == 0 || mbar_test_wait(smem_u32(&sm.empty[lane]), (round - 1) & 1));
      if (go) {
        const uint8_t* src0 = sm.list[num % S::kList][0];
        const uint8_t* src1 = sm.list[num % S::kList][1];
        const uint32_t bar = smem_u32(&sm.full[lane]), dst = smem_u32(sm.ring[lane]);
        sm.valid[lane] = (src0 ? 1 : 0) | (src1 ? 2 : 0);
        mbar_arrive_expect_tx(bar, (src0 ? G::kBytes : 0) + (src1 ? G::kBytes : 0));
        if (src0 && src1 == src0 + G::kBytes) {
          bulk_g2s(dst, src0, 2 * G::kBytes, bar, policy);
        } else {
          if (src0) bulk_g2s(dst, src0, G::kBytes, bar, policy);
          if (src1) bulk_g2s(dst + G::kBytes, src1, G::kBytes, bar, policy);
        }
        num += S::kStages;
      }
      if (all && !__any_sync(0xFFFFFFFFu, feeds && num < listed)) break;
      if (__any_sync(0xFFFFFFFFu, go)) {
        idle = 0;
      } else {
        // (nothing was free: leave the issue slots to the others for a moment)
        const uint64_t now = global_timer_ns();
        if (idle == 0) idle = now;
        if (now - idle > a.timeout_ns) *reinterpret_cast<volatile int*>(&sm.abort) = 1;
        if (__any_sync(0xFFFFFFFFu, *reinterpret_cast<volatile int*>(&sm.abort) != 0)) break;
        __nanosleep(20);
      }
    }
    // no copy may be in flight when the CTA ends, also after an abort
    __syncwarp();
    if (feeds && num >= S::kStages)
      mbar_wait_bounded(smem_u32(&sm.full[lane]), (num / S::kStages - 1) & 1, a.timeout_ns, nullptr);
    items += begun;
    for (uint32_t i = items > S::kQueries ? items - S::kQueries : 0; i < items; ++i)
      mbar_wait_bounded(smem_u32(&sm.qfull[i % S::kQueries]), (i / S::kQueries) & 1, a.timeout_ns, nullptr);
    __syncwarp();
    if (lane == 0 && sm.abort) atomicOr(status, kStatusTimeout);
    return;
  }

  // --------------------------------------------------------- consumers
  const int g = lane >> 2, t = lane & 3;
  const int key_a = kv_key_of_row(g);                  // K: this lane's keys are key_a and key_a + 8
  const int key_x = t, key_y = (t ^ 1) + 4;            // V: these and + 8
  constexpr int kKWords = D / 32;                      // code words of a lane's part of a key
  constexpr int kVWords = D / 64;
  // byte offsets of the lane's parts in a group
  const int k_codes = G::kKCodes + key_a * G::kRow + t * (D / 8);
  const int k_scales = G::kKScales + key_a * G::kScales + t * (D / 4) / G::kBlock;
  const int v_codes = G::kVCodes + g * (D / 16);
  const int v_scales = G::kVScales + g * (D / 8) / G::kBlock;
  int next_warp = 0;             // the warp that takes the CTA's next tile
  int slot = 0;                  // of this warp's stages
  uint32_t phase = 0;

#pragma unroll 1
  for (; !w.done(); w.next(a, status), ++items) {
    const Seq& s = w.s;
    // ---- Q: warp nb brings eight rows to FP16 B operands (lane (g, t): row g,
    // D / 4 elements from t's on); fq takes a row's scores to log2 units
    wait(&sm.qfull[items % S::kQueries], items / S::kQueries);
    if (warp < NB) {
      const int row = warp * 8 + g;
      const uint4* src = reinterpret_cast<const uint4*>(&sm.raw[items % S::kQueries][row][t * (D / 4)]);
      uint4 x[D / 32];
      float amax = 0.0f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        x[i] = row < w.rows ? src[i] : make_uint4(0, 0, 0, 0);
        const uint32_t wd[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = unpack2(wd[j], a.bf16);
          amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
      const int shift = row_shift(amax);
      const float up = ldexpf(1.0f, shift);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint32_t wd[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        uint32_t o2[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = unpack2(wd[j], a.bf16);
          o2[j] = pack_f16(f.x * up, f.y * up);
        }
        sm.q[warp][i][lane] = make_uint4(o2[0], o2[1], o2[2], o2[3]);
      }
      if (t == 0) sm.fq[row] = ldexpf(a.scale_log2 * (a.cache.scales ? a.cache.scales[w.h] : 1.0f), -shift);
    }
    consumers_sync();
    if (tid == 0) mbar_arrive(smem_u32(&sm.qfree[items % S::kQueries]));
    float fq[NB][2];   // of rows 8 nb + 2 t and + 1
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      fq[nb][0] = sm.fq[nb * 8 + 2 * t];
      fq[nb][1] = sm.fq[nb * 8 + 2 * t + 1];
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

    // S^T = K Q^T of a tile (two groups of 16 keys), in log2 units
    auto scores = [&](const uint8_t* base, float (&sc)[2][NB][4]) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        // [e]: key key_a + 8 e of group u
        uint32_t wk[2][kKWords], sk[2][FMT == kNVFP4 && D == 128 ? 2 : 1];
        float fk[2];   // MXFP4: what the token's scores still need
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint8_t* p = base + u * G::kBytes + 8 * e * G::kRow + k_codes;
          if constexpr (kKWords == 4) {
            const uint4 v = *reinterpret_cast<const uint4*>(p);
            wk[e][0] = v.x, wk[e][1] = v.y, wk[e][2] = v.z, wk[e][3] = v.w;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(p);
            wk[e][0] = v.x, wk[e][1] = v.y;
          }
          const uint8_t* ps = base + u * G::kBytes + 8 * e * G::kScales + k_scales;
          if constexpr (FMT == kMXFP4) {
            // a key's scales lie in the lanes t of its g
            const int c = *ps;
            int top = max(c, __shfl_xor_sync(0xFFFFFFFFu, c, 1));
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            sk[e][0] = f16_power(c - top + 12) * 0x10001u;
            fk[e] = e8m0_to_f32(top) * 0.000244140625f;   // 2^(largest - 127 - 12)
          } else if constexpr (D == 128) {   // two scales, 16 elements each
            const uint32_t h = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(ps));
            sk[e][0] = __byte_perm(h, 0, 0x1010);
            sk[e][1] = __byte_perm(h, 0, 0x3232);
          } else {
            sk[e][0] = e4m3x2_to_f16x2(*ps * 0x0101u);
          }
        }
        // two chains of products, for their latency
        float c0[NB][4] = {}, c1[NB][4] = {};
#pragma unroll
        for (int j = 0; j < kKWords; ++j) {
          const uint32_t wa = wk[0][j], wb = wk[1][j];
          const uint32_t sa = sk[0][FMT == kNVFP4 && D == 128 ? j / 2 : 0];
          const uint32_t sb = sk[1][FMT == kNVFP4 && D == 128 ? j / 2 : 0];
          const uint32_t a00 = mul2(e2m1x2_to_f16x2<0>(wa), sa), a01 = mul2(e2m1x2_to_f16x2<0>(wb), sb);
          const uint32_t a02 = mul2(e2m1x2_to_f16x2<1>(wa), sa), a03 = mul2(e2m1x2_to_f16x2<1>(wb), sb);
          const uint32_t a10 = mul2(e2m1x2_to_f16x2<2>(wa), sa), a11 = mul2(e2m1x2_to_f16x2<2>(wb), sb);
          const uint32_t a12 = mul2(e2m1x2_to_f16x2<3>(wa), sa), a13 = mul2(e2m1x2_to_f16x2<3>(wb), sb);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            const uint4 b = sm.q[nb][j][lane];
            mma_f16(c0[nb], a00, a01, a02, a03, b.x, b.y);
            mma_f16(c1[nb], a10, a11, a12, a13, b.z, b.w);
          }
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sc[u][nb][e] = (c0[nb][e] + c1[nb][e]) * (FMT == kMXFP4 ? fq[nb][e & 1] * fk[e >> 1] : fq[nb][e & 1]);
      }
    };

    // tile `i`'s softmax weights and its part of O; base: its codes
    auto weigh = [&](const uint8_t* base, int i, int valid, float (&sc)[2][NB][4]) {
      const int key0 = s.lo + (w.ta + i) * kTile;
      // the tile needs masks: it passes the keys every row sees, begins before
      // the last row's window, or lacks a page
      const bool masked = valid != 3 || key0 + kTile > (a.causal ? s.len - s.nq + 1 : s.len) ||
                          (a.window > 0 && key0 <= s.len - 1 - a.window);
      if (masked) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const bool here = (valid >> u) & 1;
          const int j0 = key0 + u * kKvGroup;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int p = a.causal ? s.len - s.nq + (w.row0 + nb * 8 + 2 * t + c) / a.group : s.len - 1;
              const int64_t first = a.window > 0 ? p - a.window + 1 : 0;
              const int ja = j0 + key_a, jb = ja + 8;
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
        uint32_t wv[4][kVWords], cv[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = (e & 1 ? key_y : key_x) + (e & 2 ? 8 : 0);
          const uint8_t* pv = base + u * G::kBytes + v_codes + key * G::kRow;
          if constexpr (kVWords == 2) {
            const uint2 v = *reinterpret_cast<const uint2*>(pv);
            wv[e][0] = v.x, wv[e][1] = v.y;
          } else {
            wv[e][0] = *reinterpret_cast<const uint32_t*>(pv);
          }
          cv[e] = base[u * G::kBytes + v_scales + key * G::kScales];
        }
        if (masked) {
          // past the end the page may hold anything, NaN scales among it, and
          // 0 * NaN would reach the sums: such keys count as zeros
          const bool here = (valid >> u) & 1;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!here || key0 + u * kKvGroup + (e & 1 ? key_y : key_x) + (e & 2 ? 8 : 0) >= s.len) cv[e] = 0, zero(wv[e]);
        }
        uint32_t s01, s23;
        if constexpr (FMT == kNVFP4) {
          s01 = e4m3x2_to_f16x2(cv[0] | cv[1] << 8);
          s23 = e4m3x2_to_f16x2(cv[2] | cv[3] << 8);
        } else {
          int top = max(max(static_cast<int>(cv[0]), static_cast<int>(cv[1])), max(static_cast<int>(cv[2]), static_cast<int>(cv[3])));
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
          s01 = f16_power(static_cast<int>(cv[0]) + r) | f16_power(static_cast<int>(cv[1]) + r) << 16;
          s23 = f16_power(static_cast<int>(cv[2]) + r) | f16_power(static_cast<int>(cv[3]) + r) << 16;
        }
#pragma unroll
        for (int j = 0; j < kVWords; ++j) {
          // low nibbles of two keys side by side, then high nibbles
          const uint32_t x = wv[0][j], y = wv[1][j], z = wv[2][j], v = wv[3][j];
          const uint32_t lo01 = (x & 0x0F0F0F0Fu) | ((y << 4) & 0xF0F0F0F0u);
          const uint32_t hi01 = ((x >> 4) & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u);
          const uint32_t lo23 = (z & 0x0F0F0F0Fu) | ((v << 4) & 0xF0F0F0F0u);
          const uint32_t hi23 = ((z >> 4) & 0x0F0F0F0Fu) | (v & 0xF0F0F0F0u);
          pv_step<0>(o, pb[u], 4 * j + 0, lo01, hi01, lo23, hi23, s01, s23);
          pv_step<1>(o, pb[u], 4 * j + 1, lo01, hi01, lo23, hi23, s01, s23);
          pv_step<2>(o, pb[u], 4 * j + 2, lo01, hi01, lo23, hi23, s01, s23);
          pv_step<3>(o, pb[u], 4 * j + 3, lo01, hi01, lo23, hi23, s01, s23);
        }
      }
    };

    // ---- the warp's tiles of the item: every kWarps-th
    const int count = w.tb - w.ta;
    int i = warp - next_warp;
    if (i < 0) i += kWarps;
    next_warp = (next_warp + count) % kWarps;
    int stage = -1;   // the last one stays held: the results go there
#pragma unroll 1
    for (; i < count; i += kWarps) {
      if (stage >= 0) {
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.empty[stage]));
      }
      stage = slot * kWarps + warp;
      wait(&sm.full[stage], phase);
      if (++slot == S::kSlots) {
        slot = 0;
        phase ^= 1u;
      }
      float sc[2][NB][4];
      scores(sm.ring[stage], sc);
      weigh(sm.ring[stage], i, sm.valid[stage], sc);
    }
    __syncwarp();

    // ---- the warps' results meet: each puts its eight rows (unscaled O,
    // maximum, sum) into its last stage, a warp then adds a row of all warps
    const float gv = a.cache.scales ? a.cache.scales[a.cache.heads + w.h] : 1.0f;
    const float vscale = FMT == kMXFP4 ? ldexpf(1.0f, max(vref, 0) - 127 - 9) : 1.0f;
    const bool whole = count == s.tiles;
    constexpr size_t kPart = partial_floats<NB>(D);
    constexpr int kE = D / 32;            // dimensions of a lane in a merged row
    float* mine = partials + (2 * static_cast<size_t>(blockIdx.x) + (w.ta == 0 ? 1 : 0)) * kPart;
    auto results = [&](int v) { return reinterpret_cast<float(*)[S::kORow]>(sm.ring[v]); };   // [8]
    if (lane == 0) sm.held[warp] = stage;
    auto merge = [&](int nb, bool out) {
#pragma unroll 1
      for (int r8 = warp; r8 < 8; r8 += kWarps) {
        float M = -INFINITY, L = 0.0f, acc[kE] = {};
        for (int v = 0; v < kWarps; ++v)
          if (sm.held[v] >= 0) M = fmaxf(M, sm.m[v][r8]);
        for (int v = 0; v < kWarps; ++v) {
          if (sm.held[v] < 0) continue;
          const float f = weight_of(sm.m[v][r8], sm.l[v][r8], M);
          float x[kE];
          load_row<kE>(&results(sm.held[v])[r8][lane * kE], x);
          L += f * sm.l[v][r8];
#pragma unroll
          for (int e = 0; e < kE; ++e) acc[e] += f * x[e];
        }
        const int row = nb * 8 + r8;
        if (out) {
          if (row < w.rows) store_row<D>(a, s, w.row0 + row, w.h, lane, M, L, acc, gv);
        } else {
          store_part<kE>(mine + row * D + lane * kE, acc);
          if (lane == 0) {
            mine[kRows * D + row] = M;
            mine[kRows * D + kRows + row] = L;
          }
        }
      }
    };
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      if (nb > 0) consumers_sync();   // the stages and sums are free
      if (stage >= 0) {
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
        float* d0 = &results(stage)[2 * t][g * (D / 8)];
        float* d1 = &results(stage)[2 * t + 1][g * (D / 8)];
#pragma unroll
        for (int i2 = 0; i2 < kK; i2 += 2) {
          *reinterpret_cast<float4*>(d0 + 2 * i2) = make_float4(o[nb][i2][0] * vscale, o[nb][i2][2] * vscale,
                                                                o[nb][i2 + 1][0] * vscale, o[nb][i2 + 1][2] * vscale);
          *reinterpret_cast<float4*>(d1 + 2 * i2) = make_float4(o[nb][i2][1] * vscale, o[nb][i2][3] * vscale,
                                                                o[nb][i2 + 1][1] * vscale, o[nb][i2 + 1][3] * vscale);
        }
      }
      consumers_sync();
      merge(nb, whole);
    }
    if (!whole) {
      const int64_t item0 = range.begin + w.at;
      const int c0 = cta_of(range.total, range.ctas, item0);
      const int c1 = cta_of(range.total, range.ctas, item0 + (s.tiles > 1 ? s.tiles - 1 + kItemCost : 0));
      consumers_sync();
      if (tid == 0) sm.last = atomic_add_acq_rel_gpu(&counters[c0], 1u) == static_cast<uint32_t>(c1 - c0);
      consumers_sync();
      if (sm.last) {
        if (tid == 0) counters[c0] = 0;   // every CTA of the item has arrived
        // the warps that hold a stage add the partials of every so-manieth CTA,
        // eight rows at a time; then their sums meet as above
        int before = 0, holders = 0;
        for (int v = 0; v < kWarps; ++v) {
          before += v < warp && sm.held[v] >= 0;
          holders += sm.held[v] >= 0;
        }
#pragma unroll 1
        for (int nb = 0; nb < NB; ++nb) {
          consumers_sync();   // the stages are free
          if (stage >= 0) {
#pragma unroll 1
            for (int r0 = 0; r0 < 8; r0 += 4) {
              float M[4], L[4], acc[4][kE];
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                M[r] = -INFINITY;
                L[r] = 0.0f;
#pragma unroll
                for (int e = 0; e < kE; ++e) acc[r][e] = 0.0f;
              }
#pragma unroll 1
              for (int c = c0 + before; c <= c1; c += holders) {
                const float* p = partials + (2 * static_cast<size_t>(c) + (c == c0)) * kPart;
                const int row = nb * 8 + r0;
                const float4 mc = __ldcg(reinterpret_cast<const float4*>(p + kRows * D + row));
                const float4 lc = __ldcg(reinterpret_cast<const float4*>(p + kRows * D + kRows + row));
                float x[4][kE];
#pragma unroll
                for (int r = 0; r < 4; ++r) load_part<kE>(p + (row + r) * D + lane * kE, x[r]);
                const float m4[4] = {mc.x, mc.y, mc.z, mc.w}, l4[4] = {lc.x, lc.y, lc.z, lc.w};
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                  const float top = fmaxf(M[r], m4[r]);
                  const float f0 = weight_of(M[r], L[r], top), f1 = weight_of(m4[r], l4[r], top);
                  M[r] = top;
                  L[r] = L[r] * f0 + l4[r] * f1;
#pragma unroll
                  for (int e = 0; e < kE; ++e) acc[r][e] = acc[r][e] * f0 + x[r][e] * f1;
                }
              }
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                store_part<kE>(&results(stage)[r0 + r][lane * kE], acc[r]);
                if (lane == 0) {
                  sm.m[warp][r0 + r] = M[r];
                  sm.l[warp][r0 + r] = L[r];
                }
              }
            }
          }
          consumers_sync();
          merge(nb, true);
        }
      }
    }
    fence_async_shared();   // (results in the stages, before the next copies into them)
    consumers_sync();       // stages, sums, queries and sm.last may be written again
    if (stage >= 0 && lane == 0) mbar_arrive(smem_u32(&sm.empty[stage]));
  }
  if (tid == 0 && sm.abort) atomicOr(status, kStatusTimeout);
}

template <int D, int FMT, int NB>
cudaError_t launch_as(const KvAttnArgs& a, int num_sms, cudaStream_t stream) {
  using S = Smem<D, FMT, NB>;
  static_assert(S::kCtas * (sizeof(S) + 1024) <= 228 * 1024, "shared memory");
  if (cudaError_t e = kv_allow_smem<kv_attn_kernel<D, FMT, NB>>(a.device, sizeof(S))) return e;
  const int grid = S::kCtas * num_sms < kMostCtas ? S::kCtas * num_sms : kMostCtas;
  kv_attn_kernel<D, FMT, NB><<<grid, kThreads, sizeof(S), stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

size_t kv_attention_workspace(int head_dim, int num_sms) {
  const size_t ctas = 3 * num_sms < kMostCtas ? 3 * num_sms : kMostCtas;
  const size_t own = sizeof(float) * 2 * ctas * partial_floats<2>(head_dim);
  const size_t prompt = kv_prompt_partials(head_dim, num_sms);
  return kWsHeaderBytes + kWsCountersBytes + (own > prompt ? own : prompt);
}

cudaError_t launch_kv_attention(const KvAttnArgs& a, int num_sms, cudaStream_t stream) {
  const int64_t rows = a.max_q * a.group;
  if (rows > 16 && a.group <= kKvPromptGroup) return launch_kv_prompt(a, num_sms, stream);
  return kv_dispatch(a.cache.head_dim, a.cache.fmt, true, [&](auto d, auto f, auto) {
    if (rows <= 8) return launch_as<d, f, 1>(a, num_sms, stream);
    return launch_as<d, f, 2>(a, num_sms, stream);
  });
}

}  // namespace petit
