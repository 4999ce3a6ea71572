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
// 2^26 below the row's largest), and p is rounded to FP16 (kv_math.cuh): 2^-11
// of a weight at most, an eighth of what a BF16 output's rounding may be and as
// much as an FP16 output's.  (FP32 weights would need a second and a third
// product each.)  Sums are of the rounded weights, so that what rounding does
// to all alike cancels.  MXFP4 scales exceed FP16's range: they are taken
// relative to the largest that the warp has met in the item, for K and for V,
// and that is applied in FP32 (exact for scales up to 2^32 below it).
//
// Work split.  The keys of every (sequence, K/V head, block of 8 NB rows) are
// cut into tiles; the tiles of the whole call, numbered in that order, are cut
// into equal ranges, one a CTA, so that ragged lengths balance without the host
// knowing them.  A CTA's producer warp fetches tiles with bulk copies into a
// ring; four consumer warps take them in turn, each with its own running
// maximum, and meet when the CTA leaves an item.  Items cut between CTAs leave
// FP32 partials, and the last CTA to arrive adds them in CTA order.
//
// Measured, 8 K/V heads of 128: one sequence of 1000 tokens 9 us (launch,
// range, one tile a warp and the join), of 131071 39 us (3.8 TB/s: 24 us of
// streaming at the 6.2 TB/s that reads alone reach, the rest is the first
// copies' latency and the join); 64 ragged sequences up to 8192 in NVFP4 71 us
// (4.3 TB/s), in MXFP4 80; 160 up to 16000 in MXFP4 with 4 query heads a K/V
// head 321 us (4.4 TB/s).  What holds the last two is latency at 15 warps an
// SM: some 350 warp instructions for 16 keys of a head (71 of them conversions
// and 170 FP16 scale products and byte selection), issued in 55 % of the cycles,
// with waits for their own results as the first stall and no unit near its rate
// (ALU 47 %, tensor cores 23 %, DRAM 53 %).
#include <cfloat>
#include <climits>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "kv.h"
#include "kv_layout.cuh"
#include "kv_math.cuh"
#include "ptx.cuh"

namespace petit {
namespace {

constexpr int kWarps = 4;                    // consumer warps
constexpr int kConsumers = kWarps * 32;
constexpr int kThreads = kConsumers + 32;
constexpr int kMostCtas = 480;               // partial slots are sized for this
constexpr int kGroupCounters = kMostCtas;    // counters[kGroupCounters + ..]: arrivals of groups of partials
// Partials joined in one step; more in groups of about their square root: one
// sequence of 131071 tokens over 8 heads (57 partials each) takes 39 us, 42 in
// one step, and over one head (456) 21 us, 54 in one step.
constexpr int kJoinFlat = 16;

// Keys of a tile: 4.5 KB of codes and scales in either head dimension.
template <int D>
constexpr int kTileOf = D == 64 ? 64 : 32;

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
  int first;    // first key that a query of the sequence sees: those before it,
                // outside every window, may be gone (no page, any bytes)
  int lo;       // first key of tile 0
  int tiles;    // tiles of an item, at least 1 so that empty rows are written
  int blocks;   // row blocks
};

template <int TILE, int ROWS>
__device__ __forceinline__ Seq load_seq(const KvAttnArgs& a, int b, uint32_t* status) {
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
  s.first = 0;
  if (a.window > 0) {
    const int64_t first = static_cast<int64_t>(s.len) - s.nq - a.window + 1;
    s.first = first > 0 ? static_cast<int>(first) : 0;
  }
  s.lo = s.first & ~(TILE - 1);
  s.tiles = s.len > s.lo ? (s.len - s.lo + TILE - 1) / TILE : 1;
  s.blocks = (s.nq * a.group + ROWS - 1) / ROWS;
  return s;
}

// A CTA's range and where it begins.  Ranges are counted in units of tiles, and
// an item weighs its tiles and `cost` more, for what beginning and ending one
// takes: tile 0 stands at the item's beginning, tile t > 0 cost + t after it.
struct Range {
  int64_t total;   // units of the whole call
  int64_t begin, end;
  int64_t rem;     // units of sequence b before `begin`
  int cost;
  int ctas;        // CTAs with a range
  int b;           // sequence of `begin`
};

// The first unit of CTA c's range.
__device__ __forceinline__ int64_t range_begin(int64_t total, int ctas, int c) {
  if (total < (1 << 21)) return static_cast<uint32_t>(total) * c / ctas;   // (c < 2^10; 64-bit division is slow)
  return total * c / ctas;
}

// The CTA whose range holds unit x.
__device__ __forceinline__ int cta_of(int64_t total, int ctas, int64_t x) {
  return static_cast<int>(((x + 1) * ctas + total - 1) / total) - 1;
}

// An item's cost.  With more items than CTAs to run them, ranges of equal tiles
// would give a CTA of many short items a multiple of the others' time (16 tiles
// was the best of 0 to 40 for 512 ragged items: 71 us, 94 at 0).  With few long
// items it only makes ranges longer than need be; with few short ones it keeps
// them whole.
__device__ __forceinline__ int item_cost(int64_t tiles, int64_t items) {
  return 2 * items > gridDim.x ? 16 : tiles >= 16 * items ? 0 : 4;
}

// Every thread of the CTA calls this (and it synchronises them); `sh` holds
// 2 kThreads / 32 + 2 values.
template <int TILE, int ROWS>
__device__ Range find_range(const KvAttnArgs& a, int64_t* sh, uint32_t* status) {
  constexpr int kW = kThreads / 32;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto measure = [&](int b, int64_t& tiles, int64_t& items) {
    tiles = items = 0;
    if (b >= a.batch) return;
    const Seq s = load_seq<TILE, ROWS>(a, b, status);
    items = static_cast<int64_t>(s.blocks) * a.cache.heads;
    tiles = items * s.tiles;
  };
  int64_t tiles = 0, items = 0, my_tiles, my_items;
  if (a.batch == 1) {
    measure(0, tiles, items);
    my_tiles = tid == 0 ? tiles : 0;
    my_items = tid == 0 ? items : 0;
    __syncthreads();
  } else {
    measure(tid, my_tiles, my_items);
    int64_t t = my_tiles, n = my_items;
    for (int b = tid + kThreads; b < a.batch; b += kThreads) {
      int64_t x, y;
      measure(b, x, y);
      t += x;
      n += y;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
      n += __shfl_xor_sync(0xFFFFFFFFu, n, o);
    }
    if (lane == 0) {
      sh[2 * warp] = t;
      sh[2 * warp + 1] = n;
    }
    __syncthreads();
    for (int w = 0; w < kW; ++w) {
      tiles += sh[2 * w];
      items += sh[2 * w + 1];
    }
  }
  Range r{};
  r.cost = item_cost(tiles, items);
  r.total = tiles + r.cost * items;
  // at least a tile a warp, and more than an item's cost, so that every CTA
  // with units of an item has a tile of it
  const int least = kWarps + r.cost;
  r.ctas = r.total >= static_cast<int64_t>(gridDim.x) * least ? static_cast<int>(gridDim.x)
           : r.total >= least                                 ? static_cast<int>(r.total) / least
                                                              : r.total > 0;
  if (static_cast<int>(blockIdx.x) >= r.ctas) return r;
  r.begin = range_begin(r.total, r.ctas, blockIdx.x);
  r.end = range_begin(r.total, r.ctas, blockIdx.x + 1);
  if (a.batch == 1) {
    r.rem = r.begin;
    return r;
  }
  // find `begin`: prefix sums over sequences, a block of them at a time
  int64_t base = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
    const int b = b0 + tid;
    if (b0 > 0) measure(b, my_tiles, my_items);
    const int64_t mine = my_tiles + r.cost * my_items;
    int64_t pre = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xFFFFFFFFu, pre, o);
      if (lane >= o) pre += v;
    }
    __syncthreads();   // (what sh held has been read)
    if (lane == 31) sh[warp] = pre;
    __syncthreads();
    int64_t before = base, all = 0;
    for (int w = 0; w < kW; ++w) {
      if (w < warp) before += sh[w];
      all += sh[w];
    }
    before += pre - mine;
    if (mine > 0 && before <= r.begin && r.begin < before + mine) {
      sh[2 * kW] = b;
      sh[2 * kW + 1] = r.begin - before;
    }
    base += all;
    if (base > r.begin) break;
  }
  __syncthreads();
  r.b = static_cast<int>(sh[2 * kW]);
  r.rem = sh[2 * kW + 1];
  return r;
}

// Walks the items of a range; every role steps one of its own.  Positions are
// relative to the range's beginning (a range of 2^31 tiles would take an hour).
template <int TILE, int ROWS>
struct Walk {
  int span;        // the range's units
  int cost;
  int at;          // the item's first unit
  int b;
  int item;        // of the sequence: heads, and row blocks inside them
  Seq s;
  int h;           // K/V head
  int row0;        // first row of the block
  int rows;        // its rows
  int ta, tb;      // tiles of the item in this range

  __device__ __forceinline__ Walk(const KvAttnArgs& a, const Range& r, uint32_t* status)
      : span(static_cast<int>(r.end - r.begin)), cost(r.cost), b(r.b) {
    s = load_seq<TILE, ROWS>(a, b, status);
    const int64_t i = r.rem < INT_MAX ? static_cast<int>(r.rem) / (s.tiles + cost) : r.rem / (s.tiles + cost);
    const int in = static_cast<int>(r.rem - i * (s.tiles + cost));
    item = static_cast<int>(i);
    at = -in;
    // the first tile at or past the beginning
    ta = in == 0 ? 0 : in <= cost ? 1 : in - cost;
    if (ta < s.tiles)
      place(a);
    else   // the range begins between an item's only tile and the next item
      next_item(a, status);
  }
  __device__ __forceinline__ bool done() const { return at >= span; }
  __device__ __forceinline__ void place(const KvAttnArgs& a) {
    const int below = span - at - cost;   // tiles below the range's end
    tb = below >= s.tiles ? s.tiles : below > ta ? below : ta + 1;
    h = item / s.blocks;
    row0 = (item - h * s.blocks) * ROWS;
    rows = min(ROWS, s.nq * a.group - row0);
  }
  __device__ __forceinline__ void next_item(const KvAttnArgs& a, uint32_t* status) {
    at += s.tiles + cost;
    if (done()) return;
    if (++item == s.blocks * static_cast<int>(a.cache.heads)) {
      item = 0;
      do {
        s = load_seq<TILE, ROWS>(a, ++b, status);
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
__device__ __forceinline__ void store_row(const KvAttnArgs& a, int q0, int row, int h, int lane, float M,
                                          float L, const float (&acc)[D / 32], float gv) {
  const int64_t tok = q0 + row / a.group;
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
    a.lse[tok * (static_cast<int64_t>(a.cache.heads) * a.group) + head] = lse_of(M, L);
}

template <int D, int FMT, int NB>
struct Smem {
  using G = KvGroup<D, FMT>;
  static constexpr int kTile = kTileOf<D>;
  static constexpr int kGroups = kTile / kKvGroup;   // of a tile
  static constexpr int kStage = kGroups * G::kBytes;
  // CTAs an SM, and stages a warp: as many as registers and shared memory give
  static constexpr int kCtas = NB == 1 ? 3 : 2;
  static constexpr int kSlots = 3;
  static constexpr int kStages = kSlots * kWarps;
  // a warp's eight rows of results fit the stage it used last
  static constexpr int kORow = D + 4;
  static_assert(8 * kORow * 4 <= kStage, "results in a stage");
  alignas(128) uint8_t ring[kStages][kStage];
  static constexpr int kQueries = NB == 1 ? 4 : 2;   // items whose queries are on chip
  static constexpr int kList = 64;          // tiles listed ahead
  static_assert(kStages <= 32, "a lane a stage");
  alignas(16) uint16_t raw[kQueries][8 * NB][D];   // queries as they come
  const uint8_t* list[kList][kGroups];      // where the groups of coming tiles lie
  uint4 q[NB][D / 32][32];                  // B operands, a lane's of two MMAs together
  float fq[8 * NB];                         // takes a row's scores to log2 units
  float m[kWarps][8], l[kWarps][8];
  uint64_t full[kStages], empty[kStages], qfull[kQueries], qfree[kQueries];
  int valid[kStages];                       // bit u: group u of the stage holds keys
  int held[kWarps];                         // the stage that holds a warp's results, or -1
  int64_t scan[2 * kThreads / 32 + 2];
  Range range;
  int abort;
  int last;
};

// FP32, per CTA two slots (an item it begins inside of: 0, one it begins: 1).
template <int NB>
__host__ __device__ constexpr size_t partial_floats(int D) { return static_cast<size_t>(NB) * 8 * (D + 2); }

// The end of an item that CTAs share: its partial rows are written; the last
// CTA to arrive joins them.
template <int D, int FMT, int NB>
__device__ __forceinline__ void finish_split(const KvAttnArgs& a, Smem<D, FMT, NB>& sm, int q0, int tiles, int at, int h,
                                             int row0, int rows) {
  constexpr int kRows = 8 * NB, kE = D / 32;
  constexpr size_t kPart = partial_floats<NB>(D);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t* counters = reinterpret_cast<uint32_t*>(a.workspace + kWsHeaderBytes);
  float* partials = reinterpret_cast<float*>(a.workspace + kWsHeaderBytes + kWsCountersBytes);
  const float gv = a.cache.scales ? a.cache.scales[a.cache.heads + h] : 1.0f;
  const int64_t item0 = sm.range.begin + at;
  const int c0 = cta_of(sm.range.total, sm.range.ctas, item0);
  const int c1 = cta_of(sm.range.total, sm.range.ctas, item0 + (tiles > 1 ? tiles - 1 + sm.range.cost : 0));
  const int parts = c1 - c0 + 1;   // contributor k of the item is CTA c0 + k
  auto last_of = [&](uint32_t* counter, int of) {   // are this CTA's sums the last of `of`?
    consumers_sync();
    if (tid == 0) {
      const bool last = atomic_add_acq_rel_gpu(counter, 1u) == static_cast<uint32_t>(of - 1);
      if (last) *counter = 0;   // everyone has arrived
      sm.last = last;
    }
    consumers_sync();
    return sm.last != 0;
  };
  // Joins contributors from, from + step, ... below `to` (at most 32), into the
  // output or the first one's place.  A warp joins whole rows, a contributor's
  // maximum and sum to a lane.
  auto join = [&](int from, int to, int step, bool out) {
    const int n = (to - from + step - 1) / step;
    auto part = [&](int i) {
      const int k = from + min(i, n - 1) * step;
      return partials + (2 * static_cast<size_t>(c0 + k) + (k == 0)) * kPart;
    };
#pragma unroll 1
    for (int first_row = warp; first_row < rows; first_row += 2 * kWarps) {   // two rows at a time
      constexpr int kBatch = 4;   // contributors on their way together
      float m[2], l[2], f[2], x[2][kBatch][kE], y[2][kE] = {};
      auto row_of = [&](int i) { return min(first_row + i * kWarps, rows - 1); };
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        m[i] = __ldcg(part(lane) + kRows * D + row_of(i));
        l[i] = __ldcg(part(lane) + kRows * D + kRows + row_of(i));
      }
#pragma unroll
      for (int e = 0; e < kBatch; ++e)
#pragma unroll
        for (int i = 0; i < 2; ++i) load_part<kE>(part(e) + row_of(i) * D + lane * kE, x[i][e]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float own = m[i];
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) m[i] = fmaxf(m[i], __shfl_xor_sync(0xFFFFFFFFu, m[i], off));
        f[i] = lane < n ? weight_of(own, l[i], m[i]) : 0.0f;
        l[i] = lane < n ? f[i] * l[i] : 0.0f;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], off);
      }
#pragma unroll 1
      for (int j = 0; j < n; j += kBatch) {
#pragma unroll
        for (int e = 0; e < kBatch; ++e)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float fe = __shfl_sync(0xFFFFFFFFu, f[i], j + e);   // (past n: the weight is 0, the row another's)
#pragma unroll
            for (int k = 0; k < kE; ++k) y[i][k] += fe * x[i][e][k];
          }
        if (j + kBatch < n) {
#pragma unroll
          for (int e = 0; e < kBatch; ++e)
#pragma unroll
            for (int i = 0; i < 2; ++i) load_part<kE>(part(j + kBatch + e) + row_of(i) * D + lane * kE, x[i][e]);
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = first_row + i * kWarps;
        if (row >= rows) continue;
        if (out) {
          store_row<D>(a, q0, row0 + row, h, lane, m[i], l[i], y[i], gv);
        } else {
          float* place = part(0);
          store_part<kE>(place + row * D + lane * kE, y[i]);
          if (lane == 0) {
            place[kRows * D + row] = m[i];
            place[kRows * D + kRows + row] = l[i];
          }
        }
      }
    }
  };
  if (parts <= kJoinFlat) {
    if (last_of(&counters[c0], parts)) join(0, parts, 1, true);
  } else {
    // groups of about the square root, each joined by its last arriver
    int per = 5;
    while (per * per < parts) ++per;
    const int k = static_cast<int>(blockIdx.x) - c0;
    const int first = k / per * per, groups = (parts + per - 1) / per;
    const int size = min(per, parts - first);
    // (a group of one is joined as it is, so that the leader of any later
    // group than the first begins no other item: its counter is this item's)
    if (size == 1 || last_of(&counters[kGroupCounters + c0 + first], size)) {
      if (size > 1) join(first, first + size, 1, false);
      if (last_of(&counters[c0], groups)) join(0, parts, per, true);
    }
  }
}

template <int D, int FMT, int NB>
__global__ void __launch_bounds__(kThreads, Smem<D, FMT, NB>::kCtas) kv_attn_kernel(const __grid_constant__ KvAttnArgs a) {
  using S = Smem<D, FMT, NB>;
  using G = KvGroup<D, FMT>;
  constexpr int kRows = 8 * NB;
  constexpr int kTile = S::kTile, kU = S::kGroups;
  constexpr int kK = D / 16;            // MMAs along D of the first product, row tiles of the second
  extern __shared__ __align__(128) uint8_t raw_smem[];
  S& sm = *reinterpret_cast<S*>(raw_smem);
  uint32_t* status = reinterpret_cast<uint32_t*>(a.workspace);
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
  const Range range = find_range<kTile, kRows>(a, sm.scan, status);
  if (range.begin >= range.end) return;
  if (tid == 0) sm.range = range;   // (for items that CTAs share)
  Walk<kTile, kRows> w(a, range, status);
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
          const uint8_t* src[kU];
#pragma unroll
          for (int u = 0; u < kU; ++u) {
            const int key = key0 + u * kKvGroup;
            src[u] = nullptr;
            if (t0 + lane < w.tb && key < w.s.len && key + kKvGroup > w.s.first) {
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
#pragma unroll
            for (int u = 0; u < kU; ++u) sm.list[(listed + lane) % S::kList][u] = src[u];
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
        const uint32_t bar = smem_u32(&sm.full[lane]), dst = smem_u32(sm.ring[lane]);
        const uint8_t* src[kU];
        int valid = 0;
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          src[u] = sm.list[num % S::kList][u];
          valid |= (src[u] != nullptr) << u;
        }
        sm.valid[lane] = valid;
        mbar_arrive_expect_tx(bar, __popc(valid) * G::kBytes);
        // groups that follow one another in memory go with one copy (each is
        // compared with the one before it: the last may lie kU - 1 groups after
        // the first and those between them anywhere)
        bool run = true;
#pragma unroll
        for (int u = 0; u < kU; ++u) run = run && src[u] && src[u] == src[0] + u * G::kBytes;
#pragma unroll
        for (int u = 0; u < kU; u += 2) {
          if (kU == 4 && u == 0 && run) {
            bulk_g2s(dst, src[0], kU * G::kBytes, bar, policy);
            break;
          }
          if (src[u] && src[u + 1] == src[u] + G::kBytes) {
            bulk_g2s(dst + u * G::kBytes, src[u], 2 * G::kBytes, bar, policy);
          } else {
            if (src[u]) bulk_g2s(dst + u * G::kBytes, src[u], G::kBytes, bar, policy);
            if (src[u + 1]) bulk_g2s(dst + (u + 1) * G::kBytes, src[u + 1], G::kBytes, bar, policy);
          }
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
      // (the scale's sign goes with Q, so that the factors are not negative)
      const float factor = a.scale_log2 * (a.cache.scales ? a.cache.scales[w.h] : 1.0f);
      const float up = copysignf(ldexpf(1.0f, shift), factor);
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
      // (nor zero, so that a masked score stays -inf)
      const float f = ldexpf(fabsf(factor), -shift);
      if (t == 0) sm.fq[row] = f < FLT_MIN ? FLT_MIN : f;
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
    // reference maxima in log2 units (ref: 0 while there is none), what a score
    // has to pass to move one, and the sums (in [0] and [1])
    float m[NB][2], ref[NB][2], pass[NB][2], l[NB][4];
    // MXFP4: exponent codes K and V are held relative to, and the rows' factors
    // for scores of such K
    int kref = 0, vref = 0;
    float fk[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      m[nb][0] = m[nb][1] = pass[nb][0] = pass[nb][1] = -INFINITY;
      fk[nb][0] = fk[nb][1] = FLT_MIN;
      ref[nb][0] = ref[nb][1] = 0.0f;
      l[nb][0] = l[nb][1] = l[nb][2] = l[nb][3] = 0.0f;
#pragma unroll
      for (int i = 0; i < kK; ++i) o[nb][i][0] = o[nb][i][1] = o[nb][i][2] = o[nb][i][3] = 0.0f;
    }

    // S^T = K Q^T of a tile (groups of 16 keys), short of the rows' factors
    auto scores = [&](const uint8_t* base, float (&sc)[kU][NB][4]) {
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        // [e]: key key_a + 8 e of group u
        uint32_t wk[2][kKWords], sk[2][FMT == kNVFP4 && D == 128 ? 2 : 1];
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
            sk[e][0] = f16x2_power(*ps - kref, *ps - kref);
          } else if constexpr (D == 128) {   // two scales, 16 elements each
            const uint32_t h = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(ps));
            sk[e][0] = __byte_perm(h, 0, 0x1010);
            sk[e][1] = __byte_perm(h, 0, 0x3232);
          } else {
            sk[e][0] = e4m3x2_to_f16x2(*ps * 0x0101u);
          }
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) sc[u][nb][0] = sc[u][nb][1] = sc[u][nb][2] = sc[u][nb][3] = 0.0f;
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
            mma_f16(sc[u][nb], a00, a01, a02, a03, b.x, b.y);
            mma_f16(sc[u][nb], a10, a11, a12, a13, b.z, b.w);
          }
        }
      }
    };

    // tile `i`'s softmax weights and its part of O; base: its codes
    auto weigh = [&](const uint8_t* base, int i, int valid, float (&sc)[kU][NB][4]) {
      const int key0 = s.lo + (w.ta + i) * kTile;
      // the tile needs masks: it passes the keys every row sees, begins before
      // the last row's window, or lacks a page
      const bool masked = valid != (1 << kU) - 1 || key0 + kTile > (a.causal ? s.len - s.nq + 1 : s.len) ||
                          (a.window > 0 && key0 <= s.len - 1 - a.window);
      if (masked) {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
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

      float(&fac)[NB][2] = FMT == kMXFP4 ? fk : fq;
      // ---- softmax: the reference maximum moves only when a score passes it
      // by 2^kWeightRoom, so most tiles need no exchange between lanes
      uint32_t pb[kU][NB][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float h0 = fmaxf(sc[0][nb][0], sc[0][nb][2]), h1 = fmaxf(sc[0][nb][1], sc[0][nb][3]);
#pragma unroll
        for (int u = 1; u < kU; ++u) {
          h0 = fmaxf(h0, fmaxf(sc[u][nb][0], sc[u][nb][2]));
          h1 = fmaxf(h1, fmaxf(sc[u][nb][1], sc[u][nb][3]));
        }
        if (__any_sync(0xFFFFFFFFu, h0 > pass[nb][0] || h1 > pass[nb][1])) {
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) {
            h0 = fmaxf(h0, __shfl_xor_sync(0xFFFFFFFFu, h0, off));
            h1 = fmaxf(h1, __shfl_xor_sync(0xFFFFFFFFu, h1, off));
          }
          const float h[2] = {h0, h1};
          float f[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float top = fmaxf(h[c] * fac[nb][c], m[nb][c]);
            f[c] = top == m[nb][c] ? 1.0f : ex2(m[nb][c] - top);
            m[nb][c] = top;
            // (a row with no key yet: its scores are all -inf, and p = 0)
            ref[nb][c] = top == -INFINITY ? 0.0f : top - kWeightLift;
            pass[nb][c] = (top + kWeightRoom) / fac[nb][c];
            l[nb][c] *= f[c];
          }
#pragma unroll
          for (int i2 = 0; i2 < kK; ++i2) {
            o[nb][i2][0] *= f[0];
            o[nb][i2][1] *= f[1];
            o[nb][i2][2] *= f[0];
            o[nb][i2][3] *= f[1];
          }
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const float p0 = ex2(fmaf(sc[u][nb][0], fac[nb][0], -ref[nb][0]));
          const float p1 = ex2(fmaf(sc[u][nb][1], fac[nb][1], -ref[nb][1]));
          const float p2 = ex2(fmaf(sc[u][nb][2], fac[nb][0], -ref[nb][0]));
          const float p3 = ex2(fmaf(sc[u][nb][3], fac[nb][1], -ref[nb][1]));
          pb[u][nb][0] = transpose8x8(pack_f16(p0, p1));
          pb[u][nb][1] = transpose8x8(pack_f16(p2, p3));
          // the sums: a product with ones
          mma_f16(l[nb], 0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u, pb[u][nb][0], pb[u][nb][1]);
        }
      }

      // ---- O^T += V^T P^T
#pragma unroll
      for (int u = 0; u < kU; ++u) {
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
          // past the end and before the window the page may hold anything, NaN
          // scales among it, and 0 * NaN would reach the sums: such keys' scales
          // count as zeros
          const bool here = (valid >> u) & 1;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = key0 + u * kKvGroup + (e & 1 ? key_y : key_x) + (e & 2 ? 8 : 0);
            if (!here || key >= s.len || key < s.first) cv[e] = 0;
          }
        }
        uint32_t s01, s23;
        if constexpr (FMT == kNVFP4) {
          s01 = e4m3x2_to_f16x2(cv[0] | cv[1] << 8);
          s23 = e4m3x2_to_f16x2(cv[2] | cv[3] << 8);
        } else {
          s01 = f16x2_power(static_cast<int>(cv[0]) - vref, static_cast<int>(cv[1]) - vref);
          s23 = f16x2_power(static_cast<int>(cv[2]) - vref, static_cast<int>(cv[3]) - vref);
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

    // MXFP4: raises the references where a scale of the tile passes one by more
    // than 2^3, up to which 6 times a scale stays inside FP16 (relative to a
    // reference, scales are 2^9 and down to 2^-23 of it exact)
    auto refer = [&](const uint8_t* base, int i, int valid) {
      const int key0 = s.lo + (w.ta + i) * kTile;
      int tk = 0, tv = 0;
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const uint8_t* grp = base + u * G::kBytes;
        // the group's 16 tokens' scales, kScales bytes each for K and for V: a
        // lane looks at the bytes of token lane / 2
        const int tok = lane >> 1;
        const int key = key0 + u * kKvGroup + tok;
        const bool here = ((valid >> u) & 1) && key < s.len && key >= s.first;
        constexpr int kB = G::kScales / 2;   // 1 or 2
        const uint8_t* pk = grp + G::kKScales + tok * G::kScales + (lane & 1) * kB;
        const uint8_t* pv = grp + G::kVScales + tok * G::kScales + (lane & 1) * kB;
        if (here) {
#pragma unroll
          for (int e = 0; e < kB; ++e) {
            tk = max(tk, static_cast<int>(pk[e]));
            tv = max(tv, static_cast<int>(pv[e]));
          }
        }
      }
      if (__any_sync(0xFFFFFFFFu, tk > kref + 3 || tv > vref + 3)) {
        tk = max(kref, static_cast<int>(__reduce_max_sync(0xFFFFFFFFu, tk)));
        tv = max(vref, static_cast<int>(__reduce_max_sync(0xFFFFFFFFu, tv)));
        const float f = tv == vref ? 1.0f : ex2(static_cast<float>(vref - tv));
        kref = tk;
        vref = tv;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float x = fq[nb][c] * ldexpf(1.0f, kref - 136);
            fk[nb][c] = x < FLT_MIN ? FLT_MIN : x;
            pass[nb][c] = (m[nb][c] + kWeightRoom) / fk[nb][c];
          }
#pragma unroll
          for (int i2 = 0; i2 < kK; ++i2) {
            o[nb][i2][0] *= f;
            o[nb][i2][1] *= f;
            o[nb][i2][2] *= f;
            o[nb][i2][3] *= f;
          }
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
      if constexpr (FMT == kMXFP4) refer(sm.ring[stage], i, sm.valid[stage]);
      float sc[kU][NB][4];
      scores(sm.ring[stage], sc);
      weigh(sm.ring[stage], i, sm.valid[stage], sc);
    }
    __syncwarp();

    // ---- the warps' results meet: each puts its eight rows (unscaled O,
    // maximum, sum) into its last stage, a warp then adds a row of all warps
    const float gv = a.cache.scales ? a.cache.scales[a.cache.heads + w.h] : 1.0f;
    const float vscale = FMT == kMXFP4 ? ldexpf(1.0f, vref - 136) : 1.0f;
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
          if (row < w.rows) store_row<D>(a, s.q0, w.row0 + row, w.h, lane, M, L, acc, gv);
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
    if (!whole) finish_split<D, FMT, NB>(a, sm, s.q0, s.tiles, w.at, w.h, w.row0, w.rows);
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
  // By the rows of a K/V head in a sequence, on average: this kernel's work grows
  // with the rows of all sequences, the tensor-memory kernel's is a 128-row
  // tile's for each sequence whatever its rows are.  Us here / there, NVFP4,
  // group 8, ragged contexts of up to 4096 tokens, 8 K/V heads:
  //   rows of every sequence       32        40        48        64
  //    8 sequences, heads of 64   30 / 34   30 / 34   31 / 34   35 / 34
  //    8 sequences, of 128        36 / 45   35 / 46   36 / 46   44 / 46
  //   24 sequences, heads of 64   41 / 46   51 / 46   52 / 46   62 / 46
  //   24 sequences, of 128        55 / 65   74 / 66   75 / 66   95 / 67
  //   64 to 8192 tokens, of 128  211 / 256 308 / 258 309 / 258 406 / 258
  //   and ragged, on average       27        34        40
  //   24 sequences, heads of 64   40 / 45   40 / 46
  //   24 sequences, of 128        51 / 62   57 / 62
  //   64 sequences, of 128                           154 / 142
  // (MXFP4 alike: 24 of 48 rows 59 / 54 and 85 / 82.)  One prompt piece of 200
  // tokens among 63 single ones (33 rows on average) 68 / 120 and 98 / 161.
  // With fewer (sequence, head) pairs than SMs contexts are cut, and the limit
  // is higher; two contexts of 60000 are the exception (74 / 68 at 40 rows).  The
  // longest sequence counts too, lest a long prompt in a batch that is padded
  // with empty sequences come here.
  // Up to 8 rows the one-column instance: three CTAs of it fit an SM, two of
  // the other.  64 ragged contexts up to 8192 take 70 us, 102 with two columns,
  // one of 131071 39 and 52.  Groups beyond 128 heads have no tile of whole
  // tokens in the other kernel.
  const int64_t rows = a.max_q * a.group;
  const int64_t limit = static_cast<int64_t>(a.batch) * a.cache.heads <= num_sms ? 48 : 36;
  const bool few = a.total_q * a.group <= limit * a.batch && rows <= 2048;
  if (!few && a.group <= kKvPromptGroup) return launch_kv_prompt(a, num_sms, stream);
  return kv_dispatch(a.cache.head_dim, a.cache.fmt, true, [&](auto d, auto f, auto) {
    if (rows <= 8) return launch_as<d, f, 1>(a, num_sms, stream);
    return launch_as<d, f, 2>(a, num_sms, stream);
  });
}

}  // namespace petit
