// Attention over the 4-bit K/V cache for many query rows a sequence (prompts
// and long drafts), on the 5th-generation tensor cores.
//
// The rows of a K/V head (query tokens x heads of the group, token by token)
// are cut into items of up to two 128-row MMA tiles; an item meets its keys
// 128 at a time:
//     S_q = Q_q K^T (shared x shared memory -> tensor memory),
//     P_q = 2^(S_q f - m) (registers, back into S_q's columns as FP16),
//     O_q += P_q V (tensor x shared memory -> tensor memory),  q = 0, 1.
// With both formats in FP16 the products are those of kv_attn.cu; what bounds
// the kernel is the two MMAs (4 D FLOP a row and key) next to the 128 x 128
// exponentials and the conversion of a 128-key tile of K and V, which two row
// tiles share.  Warps by role, each with its own barriers:
//   0-3, 4-7   softmax of row tile 0 and 1: a thread holds a row, so maximum
//              and sum need no exchange; while one tile's scores are in the
//              registers the tensor cores work on the other tile
//   8-11       V: a thread converts 8 tokens by D / 8 dimensions and writes
//              them transposed (contraction along the tokens)
//   12-13      K: a thread converts two tokens' rows (codes -> FP16, swizzled)
//   14         issues the MMAs
// Codes go from global memory to registers a tile ahead; the converted tiles
// are double-buffered.  Tensor memory: O_0, O_1, S_0, S_1 (all 512 columns at
// D = 128).
//
// The key tiles of all items are cut into equal ranges as in kv_attn.cu; an
// item cut between CTAs leaves FP32 partials that the last arriver adds.
//
// Measured: 4096 new tokens behind 12288, 64 query heads of 128 over 8 NVFP4
// heads, 1.43 ms, 1.34 PFLOP/s (70 % of a cuBLAS product's rate; MXFP4 1.63 ms,
// FP16 outputs 1.49): a softmax warpgroup's pass over 128 x 128 scores is the
// longest stage, the tensor pipe is busy 52 % of the time.  Five ragged pieces of
// 3 to 1100 tokens with a window of 1024, heads of 64, MXFP4, FP16, 65 us:
// an item's beginning and end (8 to 10 k cycles) next to 13 tiles.
#include <cfloat>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "kv.h"
#include "kv_layout.cuh"
#include "kv_math.cuh"
#include "ptx.cuh"

namespace petit {
namespace {

constexpr int kKeys = 128;        // keys of a tile
constexpr int kRowTile = 128;     // rows of an MMA tile
constexpr int kRows = 2 * kRowTile;
constexpr int kVWarp = 8, kKWarp = 12, kMmaWarp = 14;
constexpr int kThreads = 32 * 16;   // (warp 15 has no work)
// The split counts units: an item's tiles, and its cost.
//  - Many items (more than half the CTAs): beginning and ending one costs some
//    9 k cycles beside 2 to 4 k a tile, so it counts kItemCost tiles, and a CTA
//    gets kMinUnits at least: more than the cost, so that every CTA with units
//    of an item has a tile of it.  (24 drafts: 51 us, 79 without a cost.)
//  - Few items: each is cut into equal pieces of kFewTiles tiles or more, none
//    of which begins a second item; short ones into pairs of tiles.  64 query
//    heads over 8: 8 tokens at 2000 take 20.5 us (as above: 26.5), 100 at 6000
//    37.9 (40.2), 200 of a new prompt 22 (31), 64 of two sequences at 4000 53
//    (49).
constexpr int kItemCost = 4, kMinUnits = 8, kFewTiles = 4;
constexpr int kRing = 4;          // per-tile facts: written at most two tiles ahead of their last reader

// ------------------------------------------------------------ work split
struct Seq {
  int len, nq, q0;
  int tokens;     // query tokens of an item (whole tokens)
  int row_tiles;  // items along the rows, per head
};

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
  s.tokens = kRows / a.group;
  s.row_tiles = (s.nq + s.tokens - 1) / s.tokens;
  return s;
}

struct Keys {
  int lo;      // first key of tile 0, a multiple of kKeys
  int tiles;   // at least 1, so that rows without keys are written
};

// First key that a row of the item sees: those before it, outside every window,
// may be gone (no page, any bytes).
__device__ __forceinline__ int first_key(const KvAttnArgs& a, const Seq& s, int rt) {
  // (len and nq are below 2^31, a window 1..2^31 - 1 in 32 bits)
  const int last = s.len - s.nq + rt * s.tokens + 1;   // keys that the first row sees without a window
  const int window = static_cast<int>(a.window);
  return a.window > 0 && last > window ? last - window : 0;
}

__device__ __forceinline__ Keys item_keys(const KvAttnArgs& a, const Seq& s, int rt) {
  const int t0 = rt * s.tokens, t1 = min(s.nq, t0 + s.tokens) - 1;
  const int64_t hi = a.causal ? static_cast<int64_t>(s.len) - s.nq + t1 : s.len - 1;
  Keys k;
  k.lo = first_key(a, s, rt) & ~(kKeys - 1);
  k.tiles = hi >= k.lo ? static_cast<int>(hi - k.lo) / kKeys + 1 : 1;
  return k;
}

// Tiles and items: of a sequence (every lane of the warp calls this), or more.
struct Work {
  int64_t tiles, items;
};
__device__ __forceinline__ Work seq_work(const KvAttnArgs& a, int b, uint32_t* status) {
  const Seq s = load_seq(a, b, status);
  int64_t sum = 0;
  for (int rt = threadIdx.x & 31; rt < s.row_tiles; rt += 32) sum += item_keys(a, s, rt).tiles;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  return {sum * a.cache.heads, static_cast<int64_t>(s.row_tiles) * a.cache.heads};
}

__device__ __forceinline__ int64_t range_begin(int64_t total, int ctas, int64_t c) { return total * c / ctas; }
// The CTA whose range holds unit x.
__device__ __forceinline__ int cta_of(int64_t total, int ctas, int64_t x) {
  return static_cast<int>(((x + 1) * ctas + total - 1) / total) - 1;
}

// Walks the items of a CTA's range of units, in the order sequence, row tile,
// head.  An item's tile 0 stands at its beginning, tile t > 0 cost + t after
// it.  Positions are relative to the range's beginning.
struct Walk {
  int64_t total, begin;   // units of the call; the range's first
  int ctas;
  int cost;               // of an item
  int span;               // the range's units
  int at;                 // the item's first unit
  int b, rt, h;
  Seq s;
  Keys k;
  int ta, tb;             // tiles of the item in this range

  __device__ __forceinline__ bool done() const { return at >= span; }
  __device__ __forceinline__ void cut() {
    const int below = span - at - cost;   // tiles below the range's end
    tb = below >= k.tiles ? k.tiles : below > ta ? below : ta + 1;
  }
  __device__ __forceinline__ void next_item(const KvAttnArgs& a, uint32_t* status) {
    at += k.tiles + cost;
    if (done()) return;
    if (++h == static_cast<int>(a.cache.heads)) {
      h = 0;
      if (++rt == s.row_tiles) {
        rt = 0;
        do {
          s = load_seq(a, ++b, status);
        } while (s.row_tiles == 0 && b + 1 < a.batch);
      }
      k = item_keys(a, s, rt);
    }
    ta = 0;
    cut();
  }
  __device__ __forceinline__ void next(const KvAttnArgs& a, uint32_t* status) {
    if (tb < k.tiles)
      at = span;
    else
      next_item(a, status);
  }
};

constexpr int kSeqChunk = 64;

// Every thread of the CTA calls this; sh holds kSeqChunk values.
__device__ Walk find_range(const KvAttnArgs& a, Work* sh, uint32_t* status) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kW = kThreads / 32;
  auto chunk = [&](int b0) {   // the work of the sequences b0.. into sh; returns their sum
    __syncthreads();
    for (int i = warp; i < kSeqChunk; i += kW) {
      const Work t = b0 + i < a.batch ? seq_work(a, b0 + i, status) : Work{0, 0};
      if (lane == 0) sh[i] = t;
    }
    __syncthreads();
    Work sum = {sh[lane].tiles + sh[lane + 32].tiles, sh[lane].items + sh[lane + 32].items};
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      sum.tiles += __shfl_xor_sync(0xFFFFFFFFu, sum.tiles, o);
      sum.items += __shfl_xor_sync(0xFFFFFFFFu, sum.items, o);
    }
    return sum;
  };
  Walk w{};
  Work all = {0, 0};
  for (int b0 = 0; b0 < a.batch; b0 += kSeqChunk) {
    const Work sum = chunk(b0);
    all.tiles += sum.tiles;
    all.items += sum.items;
  }
  const int grid = static_cast<int>(gridDim.x);
  auto units = [&](const Work& x) { return x.tiles + w.cost * x.items; };
  if (2 * all.items <= grid) {
    const int items = static_cast<int>(all.items);
    const int64_t pieces = items == 0 ? 0 : all.tiles / (items * kFewTiles);
    w.cost = 0;
    w.total = units(all);
    w.ctas = pieces >= 2 ? items * static_cast<int>(pieces < grid / items ? pieces : grid / items)
                         : static_cast<int>((all.tiles + 1) / 2 < grid ? (all.tiles + 1) / 2 : grid);
  } else {
    w.cost = kItemCost;
    w.total = units(all);
    w.ctas = w.total >= static_cast<int64_t>(grid) * kMinUnits ? grid : max(static_cast<int>(w.total) / kMinUnits, 1);
  }
  if (static_cast<int>(blockIdx.x) >= w.ctas) return w;   // (an empty range: done)
  w.begin = range_begin(w.total, w.ctas, blockIdx.x);
  w.span = static_cast<int>(range_begin(w.total, w.ctas, blockIdx.x + 1) - w.begin);
  int64_t before = 0;
  int b0 = 0;
  for (;; b0 += kSeqChunk) {
    const int64_t sum = a.batch > kSeqChunk ? units(chunk(b0)) : w.total;
    if (before + sum > w.begin) break;
    before += sum;
  }
  w.b = b0;
  while (before + units(sh[w.b - b0]) <= w.begin) before += units(sh[w.b++ - b0]);
  w.s = load_seq(a, w.b, status);
  // the row tile: prefix sums of 32 at a time
  for (int rt0 = 0;; rt0 += 32) {
    const int64_t mine =
        rt0 + lane < w.s.row_tiles ? static_cast<int64_t>(item_keys(a, w.s, rt0 + lane).tiles + w.cost) * a.cache.heads
                                   : 0;
    int64_t pre = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xFFFFFFFFu, pre, o);
      if (lane >= o) pre += v;
    }
    const unsigned over = __ballot_sync(0xFFFFFFFFu, before + pre > w.begin);
    if (over) {
      const int l = __ffs(over) - 1;
      w.rt = rt0 + l;
      before += __shfl_sync(0xFFFFFFFFu, pre - mine, l);
      break;
    }
    before += __shfl_sync(0xFFFFFFFFu, pre, 31);
  }
  w.k = item_keys(a, w.s, w.rt);
  const int item = w.k.tiles + w.cost;
  w.h = static_cast<int>((w.begin - before) / item);
  const int in = static_cast<int>(w.begin - before - static_cast<int64_t>(w.h) * item);
  w.at = -in;
  w.ta = in == 0 ? 0 : in <= w.cost ? 1 : in - w.cost;   // the first tile at or past the beginning
  if (w.ta < w.k.tiles)
    w.cut();
  else   // the range begins between an item's only tile and the next item
    w.next_item(a, status);
  return w;
}

// ------------------------------------------------------------ the kernel
template <int D>
struct Smem {
  alignas(1024) uint8_t q[2][D / 64][kRowTile * 128];   // 64 dimensions a slab, 128-byte swizzle
  uint8_t k[2][D / 64][kKeys * 128];
  uint8_t v[2][kKeys / 64][D * 128];                    // 64 tokens a slab
  uint64_t qfull[2], sfull[2], pfull[2], ofull[2], kfull[2], kfree[2], vfull[2], vfree[2], fin;
  Work scan[kSeqChunk];
  float kfac[kRing][4];       // MXFP4: factor of the scores of 32 keys
  float m1[kRowTile], l1[kRowTile];   // what the second half of an item's keys leaves
  uint32_t valid[kRing][4];   // of 32 keys: bit 0, 1: the 16-key group's page is in the cache
  int vtop;                   // MXFP4: largest V scale of the tile
  float vscale[kRing];        // MXFP4: what O needs if the item ends with this tile
  uint32_t tmem;
  int abort;
  int last;
};

template <int D>
__host__ __device__ constexpr size_t partial_floats() { return static_cast<size_t>(kRows) * (D + 2); }

template <int D, int FMT, bool BF16>
__global__ void __launch_bounds__(kThreads, 1) kv_prompt_kernel(const __grid_constant__ KvAttnArgs a) {
  using S = Smem<D>;
  using G = KvGroup<D, FMT>;
  constexpr uint32_t kO = 0, kS = 2 * D;                 // tensor-memory columns
  constexpr uint32_t kColumns = 512;                     // (384 used at D = 64: sizes are powers of two)
  constexpr uint32_t kIdescS = idesc_f16_f32(kRowTile, kKeys), kIdescO = idesc_f16_f32(kRowTile, D);
  extern __shared__ __align__(1024) uint8_t raw[];
  S& sm = *reinterpret_cast<S*>(raw);
  uint32_t* status = reinterpret_cast<uint32_t*>(a.workspace);
  uint32_t* counters = reinterpret_cast<uint32_t*>(a.workspace + kWsHeaderBytes);
  float* partials = reinterpret_cast<float*>(a.workspace + kWsHeaderBytes + kWsCountersBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto wait = [&](uint64_t* bar, uint32_t phase) { wait_phase(bar, phase, a.timeout_ns, &sm.abort); };

  if (tid == 0) {
    sm.abort = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sm.qfull[i]), 4);
      mbar_init(smem_u32(&sm.sfull[i]), 1);
      mbar_init(smem_u32(&sm.pfull[i]), 4);
      mbar_init(smem_u32(&sm.ofull[i]), 1);
      mbar_init(smem_u32(&sm.kfull[i]), 2);
      mbar_init(smem_u32(&sm.kfree[i]), 1);
      mbar_init(smem_u32(&sm.vfull[i]), 4);
      mbar_init(smem_u32(&sm.vfree[i]), 1);
    }
    mbar_init(smem_u32(&sm.fin), 1);
    mbar_fence_init();
  }
  Walk w = find_range(a, sm.scan, status);   // (synchronises the CTA)
  if (w.done()) return;
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&sm.tmem), kColumns);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  const int64_t head_stride = static_cast<int64_t>(G::kBytes) << (a.cache.page_shift - 4);
  // 16-token group of `key` in sequence w.b, or null (also where all of it lies
  // before the first key that is seen)
  auto group_of = [&](int key, int first) -> const uint8_t* {
    if (key >= w.s.len || (key | (kKvGroup - 1)) < first) return nullptr;
    const int64_t page = a.block_table[w.b * a.table_stride + (key >> a.cache.page_shift)];
    if (page < 0 || page >= a.cache.num_pages) {
      atomicOr(status, kStatusBounds);
      return nullptr;
    }
    return a.cache.data + page * a.cache.page_stride + w.h * head_stride +
           ((key & ((1 << a.cache.page_shift) - 1)) / kKvGroup) * G::kBytes;
  };
  uint32_t n = 0;   // tiles before the item in this CTA

  if (warp == kMmaWarp) {
    // ---------------------------------------------------------- MMA issue
    uint32_t items[2] = {0, 0}, ptiles[2] = {0, 0};
    auto scores = [&](int q, uint32_t num) {
      if (elect_one()) {
        const uint32_t qa = smem_u32(sm.q[q]), ka = smem_u32(sm.k[num & 1]);
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
          mma_ss_f16(tmem + kS + q * kKeys,
                     smem_desc_kmajor_sw128(qa + (j >> 2) * (kRowTile * 128)) + (j & 3) * 2,
                     smem_desc_kmajor_sw128(ka + (j >> 2) * (kKeys * 128)) + (j & 3) * 2, kIdescS, j > 0);
        mma_commit(smem_u32(&sm.sfull[q]));
      }
      __syncwarp();
    };
    auto commit = [&](uint64_t* bar) {
      if (elect_one()) mma_commit(smem_u32(bar));
      __syncwarp();
    };
    for (; !w.done(); w.next(a, status)) {
      const int tiles = w.tb - w.ta;
      const int rows = min(w.s.tokens, w.s.nq - w.rt * w.s.tokens) * a.group;
      // tile `num` for row tile (or half) q; `first`: it begins O_q, `last`: it ends it
      auto weigh = [&](int q, uint32_t num, bool first, bool last) {
        if (elect_one()) {
          const uint32_t va = smem_u32(sm.v[num & 1]);
#pragma unroll
          for (int j = 0; j < kKeys / 16; ++j)
            mma_ts_f16(tmem + kO + q * D, tmem + kS + q * kKeys + j * 8,
                       smem_desc_kmajor_sw128(va + (j >> 2) * (D * 128)) + (j & 3) * 2, kIdescO, !first || j > 0);
          if (last) mma_commit(smem_u32(&sm.ofull[q]));
        }
        __syncwarp();
      };
      auto await_p = [&](int q) { wait(&sm.pfull[q], ptiles[q]++ & 1); };
      auto await_k = [&](uint32_t num) { wait(&sm.kfull[num & 1], (num >> 1) & 1); };
      auto await_v = [&](uint32_t num) { wait(&sm.vfull[num & 1], (num >> 1) & 1); };
      if (rows > kRowTile) {
        // two row tiles, each of which meets every key tile
        await_k(n);
        for (int q = 0; q < 2; ++q) {
          wait(&sm.qfull[q], items[q]++ & 1);
          tc_fence_after();
          scores(q, n);
        }
        commit(&sm.kfree[n & 1]);
        for (int i = 0; i < tiles; ++i) {
          const uint32_t num = n + i;
          for (int q = 0; q < 2; ++q) {
            await_p(q);
            if (q == 0) await_v(num);
            tc_fence_after();
            weigh(q, num, i == 0, i + 1 == tiles);
            if (i + 1 < tiles) {
              if (q == 0) {
                await_k(num + 1);
                tc_fence_after();
              }
              scores(q, num + 1);
            }
          }
          commit(&sm.vfree[num & 1]);
          if (i + 1 < tiles) commit(&sm.kfree[(num + 1) & 1]);
        }
      } else {
        // one row tile: its even and its odd key tiles as two chains
        auto begin = [&](int q, uint32_t num) {
          await_k(num);
          tc_fence_after();
          scores(q, num);
          commit(&sm.kfree[num & 1]);
        };
        for (int q = 0; q < min(2, tiles); ++q) {
          wait(&sm.qfull[q], items[q]++ & 1);
          begin(q, n + q);
        }
        for (int i = 0; i < tiles; ++i) {
          const uint32_t num = n + i;
          await_p(i & 1);
          await_v(num);
          tc_fence_after();
          weigh(i & 1, num, i < 2, i + 2 >= tiles);
          commit(&sm.vfree[num & 1]);
          if (i + 2 < tiles) begin(i & 1, num + 2);
        }
      }
      n += tiles;
    }
    commit(&sm.fin);
    mbar_wait_bounded(smem_u32(&sm.fin), 0, a.timeout_ns, nullptr);
  } else if (warp > kMmaWarp) {
    // (no work)
  } else if (warp >= kVWarp && warp < kKWarp) {
    // ------------------------------------------------------------------ V
    constexpr int kD = D / 8;          // dimensions of a thread
    constexpr int kW = kD / 8;         // code words of a token
    const int vw = warp - kVWarp;
    const int slab = vw & 1, kg = lane & 7;
    const int d0 = (vw >> 1) * (D / 2) + (lane >> 3) * kD;
    const int key_in = slab * 64 + kg * 8;
    uint32_t wd[8][kW];
    uint32_t sc[8];
    auto load = [&](int tile) {
      const int key = w.k.lo + tile * kKeys + key_in;
      const int first = first_key(a, w.s, w.rt);
      const uint8_t* grp = group_of(key, first);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int t = (kg & 1) * 8 + i;
#pragma unroll
        for (int j = 0; j < kW; ++j) wd[i][j] = 0;
        sc[i] = 0;
        if (grp) {
          const uint8_t* p = grp + G::kVCodes + t * G::kRow + d0 / 2;
          if constexpr (kW == 2) {
            const uint2 v = *reinterpret_cast<const uint2*>(p);
            wd[i][0] = v.x;
            wd[i][1] = v.y;
          } else {
            wd[i][0] = *reinterpret_cast<const uint32_t*>(p);
          }
          sc[i] = grp[G::kVScales + t * G::kScales + d0 / G::kBlock];
        }
      }
      // a token past the end or before the window may hold anything, and 0 times
      // a NaN scale would reach the sums: its scale counts as zero
      if (key < first || key + 8 > w.s.len) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (key + i < first || key + i >= w.s.len) sc[i] = 0;
      }
    };
    if (!w.done()) load(w.ta);
    while (!w.done()) {
      const int tiles = w.tb - w.ta;
      int vref = 0;
      for (int i = 0; i < tiles; ++i) {
        const uint32_t num = n + i;
        if (num >= 2) wait(&sm.vfree[num & 1], ((num >> 1) - 1) & 1);
        uint32_t s2[4];
        if constexpr (FMT == kNVFP4) {
#pragma unroll
          for (int p = 0; p < 4; ++p) s2[p] = e4m3x2_to_f16x2(sc[2 * p] | sc[2 * p + 1] << 8);
        } else {
          // the scales are taken relative to the largest so far in the item
          uint32_t top = 0;
#pragma unroll
          for (int p = 0; p < 8; ++p) top = max(top, sc[p]);
          top = __reduce_max_sync(0xFFFFFFFFu, top);
          if (warp == kVWarp && lane == 0) sm.vtop = 0;
          asm volatile("bar.sync 2, 128;" ::: "memory");
          if (lane == 0) atomicMax(&sm.vtop, static_cast<int>(top));
          asm volatile("bar.sync 2, 128;" ::: "memory");
          const int t = max(vref, sm.vtop);
          asm volatile("bar.sync 2, 128;" ::: "memory");
          if (warp == kVWarp && lane == 0) {
            sm.vscale[num % kRing] = ldexpf(1.0f, t - 127 - 12);
          }
          vref = t;
#pragma unroll
          for (int p = 0; p < 4; ++p)
            s2[p] = f16_power(static_cast<int>(sc[2 * p]) - vref + 12) |
                    f16_power(static_cast<int>(sc[2 * p + 1]) - vref + 12) << 16;
        }
        uint8_t* dst = sm.v[num & 1][slab];
        auto put = [&](int d, uint32_t x0, uint32_t x1, uint32_t x2, uint32_t x3) {
          *reinterpret_cast<uint4*>(dst + d * 128 + ((kg ^ (d & 7)) << 4)) = make_uint4(x0, x1, x2, x3);
        };
#pragma unroll
        for (int j = 0; j < kW; ++j) {
          uint32_t lo[4], hi[4];   // dimension pairs of two tokens side by side
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            const uint32_t x = wd[2 * p][j], y = wd[2 * p + 1][j];
            lo[p] = (x & 0x0F0F0F0Fu) | ((y << 4) & 0xF0F0F0F0u);
            hi[p] = ((x >> 4) & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u);
          }
          const int d = d0 + 8 * j;
          put(d + 0, mul2(e2m1x2_to_f16x2<0>(lo[0]), s2[0]), mul2(e2m1x2_to_f16x2<0>(lo[1]), s2[1]),
              mul2(e2m1x2_to_f16x2<0>(lo[2]), s2[2]), mul2(e2m1x2_to_f16x2<0>(lo[3]), s2[3]));
          put(d + 1, mul2(e2m1x2_to_f16x2<0>(hi[0]), s2[0]), mul2(e2m1x2_to_f16x2<0>(hi[1]), s2[1]),
              mul2(e2m1x2_to_f16x2<0>(hi[2]), s2[2]), mul2(e2m1x2_to_f16x2<0>(hi[3]), s2[3]));
          put(d + 2, mul2(e2m1x2_to_f16x2<1>(lo[0]), s2[0]), mul2(e2m1x2_to_f16x2<1>(lo[1]), s2[1]),
              mul2(e2m1x2_to_f16x2<1>(lo[2]), s2[2]), mul2(e2m1x2_to_f16x2<1>(lo[3]), s2[3]));
          put(d + 3, mul2(e2m1x2_to_f16x2<1>(hi[0]), s2[0]), mul2(e2m1x2_to_f16x2<1>(hi[1]), s2[1]),
              mul2(e2m1x2_to_f16x2<1>(hi[2]), s2[2]), mul2(e2m1x2_to_f16x2<1>(hi[3]), s2[3]));
          put(d + 4, mul2(e2m1x2_to_f16x2<2>(lo[0]), s2[0]), mul2(e2m1x2_to_f16x2<2>(lo[1]), s2[1]),
              mul2(e2m1x2_to_f16x2<2>(lo[2]), s2[2]), mul2(e2m1x2_to_f16x2<2>(lo[3]), s2[3]));
          put(d + 5, mul2(e2m1x2_to_f16x2<2>(hi[0]), s2[0]), mul2(e2m1x2_to_f16x2<2>(hi[1]), s2[1]),
              mul2(e2m1x2_to_f16x2<2>(hi[2]), s2[2]), mul2(e2m1x2_to_f16x2<2>(hi[3]), s2[3]));
          put(d + 6, mul2(e2m1x2_to_f16x2<3>(lo[0]), s2[0]), mul2(e2m1x2_to_f16x2<3>(lo[1]), s2[1]),
              mul2(e2m1x2_to_f16x2<3>(lo[2]), s2[2]), mul2(e2m1x2_to_f16x2<3>(lo[3]), s2[3]));
          put(d + 7, mul2(e2m1x2_to_f16x2<3>(hi[0]), s2[0]), mul2(e2m1x2_to_f16x2<3>(hi[1]), s2[1]),
              mul2(e2m1x2_to_f16x2<3>(hi[2]), s2[2]), mul2(e2m1x2_to_f16x2<3>(hi[3]), s2[3]));
        }
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.vfull[num & 1]));
        if (i + 1 < tiles) load(w.ta + i + 1);
      }
      n += tiles;
      w.next(a, status);
      if (!w.done()) load(w.ta);
    }
  } else if (warp >= kKWarp) {
    // ------------------------------------------------------------------ K
    constexpr int kW = D / 8;          // code words of a token
    constexpr int kS = (G::kScales + 3) / 4;
    const int kw = warp - kKWarp;
    uint32_t wd[2][kW], sc[2][kS];     // tokens kw 32 + lane and 64 + that
    bool have[2] = {false, false};
    auto load = [&](int tile) {
      const int first = first_key(a, w.s, w.rt);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int key = w.k.lo + tile * kKeys + x * 64 + kw * 32 + lane;
        const uint8_t* grp = group_of(key, first);
        have[x] = grp != nullptr && key >= first;
#pragma unroll
        for (int j = 0; j < kW; ++j) wd[x][j] = 0;
#pragma unroll
        for (int j = 0; j < kS; ++j) sc[x][j] = 0;
        if (have[x]) {
          const int t = key % kKvGroup;
          const uint4* p = reinterpret_cast<const uint4*>(grp + G::kKCodes + t * G::kRow);
#pragma unroll
          for (int j = 0; j < kW / 4; ++j) {
            const uint4 v = p[j];
            wd[x][4 * j] = v.x, wd[x][4 * j + 1] = v.y, wd[x][4 * j + 2] = v.z, wd[x][4 * j + 3] = v.w;
          }
          const uint8_t* ps = grp + G::kKScales + t * G::kScales;
          if constexpr (G::kScales == 8) {
            const uint2 v = *reinterpret_cast<const uint2*>(ps);
            sc[x][0] = v.x, sc[x][1] = v.y;
          } else if constexpr (G::kScales == 4) {
            sc[x][0] = *reinterpret_cast<const uint32_t*>(ps);
          } else {
            sc[x][0] = *reinterpret_cast<const uint16_t*>(ps);
          }
        }
      }
    };
    if (!w.done()) load(w.ta);
    while (!w.done()) {
      const int tiles = w.tb - w.ta;
      for (int i = 0; i < tiles; ++i) {
        const uint32_t num = n + i;
        if (num >= 2) wait(&sm.kfree[num & 1], ((num >> 1) - 1) & 1);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int key_in = x * 64 + kw * 32 + lane, part = 2 * x + kw;
          const unsigned held = __ballot_sync(0xFFFFFFFFu, have[x]);
          int top = 0;
          if constexpr (FMT == kMXFP4) {
#pragma unroll
            for (int p = 0; p < G::kScales; ++p) top = max(top, static_cast<int>((sc[x][0] >> (8 * p)) & 0xFFu));
            top = static_cast<int>(__reduce_max_sync(0xFFFFFFFFu, static_cast<uint32_t>(top)));
          }
          if (lane == 0) {
            sm.valid[num % kRing][part] = (held & 0xFFFFu ? 1u : 0u) | (held >> 16 ? 2u : 0u);
            if constexpr (FMT == kMXFP4) sm.kfac[num % kRing][part] = e8m0_to_f32(top) * 0.000244140625f;
          }
          uint8_t* dst = &sm.k[num & 1][0][key_in * 128];
          uint32_t s2 = 0;
#pragma unroll
          for (int j = 0; j < kW; ++j) {
            if (j % (G::kBlock / 8) == 0) {   // this word begins a block
              const int blk = j / (G::kBlock / 8);
              const uint32_t b = (sc[x][blk / 4] >> (8 * (blk % 4))) & 0xFFu;
              if constexpr (FMT == kNVFP4)
                s2 = e4m3x2_to_f16x2(b * 0x0101u);
              else
                s2 = f16_power(static_cast<int>(b) - top + 12) * 0x10001u;
            }
            *reinterpret_cast<uint4*>(dst + (j >> 3) * (kKeys * 128) + (((j & 7) ^ (key_in & 7)) << 4)) =
                make_uint4(mul2(e2m1x2_to_f16x2<0>(wd[x][j]), s2), mul2(e2m1x2_to_f16x2<1>(wd[x][j]), s2),
                           mul2(e2m1x2_to_f16x2<2>(wd[x][j]), s2), mul2(e2m1x2_to_f16x2<3>(wd[x][j]), s2));
          }
        }
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.kfull[num & 1]));
        if (i + 1 < tiles) load(w.ta + i + 1);
      }
      n += tiles;
      w.next(a, status);
      if (!w.done()) load(w.ta);
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int q = warp >> 2;
    const int row_in = (warp & 3) * 32 + lane;            // row of the MMA tile = tensor-memory lane
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_tmem = tmem + lanes + kS + q * kKeys, o_tmem = tmem + lanes + kO + q * D;
    uint32_t my_items = 0, my_tiles = 0;
    for (; !w.done(); w.next(a, status)) {
      const int tiles = w.tb - w.ta;
      const int tok0 = w.rt * w.s.tokens;
      const int rows = min(w.s.tokens, w.s.nq - tok0) * a.group;
      const bool whole = tiles == w.k.tiles;
      // one row tile: both groups take it, the second its odd key tiles
      const bool one = rows <= kRowTile;
      const bool works = q == 0 || !one || tiles > 1, puts = q == 0 || !one;
      const int tile_row = one ? 0 : q * kRowTile;
      const int row = tile_row + row_in;
      const bool mine = row < rows;
      const int tok = tok0 + min(row, rows - 1) / a.group;   // (a row past the last masks like it)
      const int64_t head = static_cast<int64_t>(w.h) * a.group + (mine ? row % a.group : 0);
      const float gv = a.cache.scales ? a.cache.scales[a.cache.heads + w.h] : 1.0f;
      float m = -INFINITY, l = 0.0f;
      float vs = 1.0f;
      if (works) {
        // ---- the row to FP16, swizzled; the sign of the scale goes with it
        float f;
        {
          const float gk = a.cache.scales ? a.cache.scales[w.h] : 1.0f;
          // the warp copies its 32 rows with whole rows in an access (a thread's
          // own row at a time would touch 32 lines in each), then a thread takes
          // its own
          constexpr int kPer = D / 8;   // 16-byte parts of a row
          const uint64_t own = mine ? reinterpret_cast<uint64_t>(static_cast<const uint16_t*>(a.q.data) +
                                                                 (w.s.q0 + static_cast<int64_t>(tok)) * a.q.token_stride +
                                                                 head * a.q.head_stride)
                                    : 0;
          const int part = lane % kPer;
#pragma unroll 4
          for (int j = 0; j < kPer; ++j) {
            const int from = j * (32 / kPer) + lane / kPer, r = (warp & 3) * 32 + from;
            const uint64_t src = __shfl_sync(0xFFFFFFFFu, own, from);
            cp_async16(smem_u32(&sm.q[q][part >> 3][r * 128 + (((part & 7) ^ (r & 7)) << 4)]),
                       src ? reinterpret_cast<const uint8_t*>(src) + 16 * part : a.q.data, src ? 16 : 0);
          }
          cp_async_wait_all();
          __syncwarp();
          // (the row stays in registers for the second pass, at some 400 bytes of
          // spills an item at D = 128: read again from shared memory it takes 92,
          // and the 4096-token piece 1.455 ms in place of 1.436)
          uint4 x[D / 8];
#pragma unroll
          for (int j = 0; j < D / 8; ++j)
            x[j] = *reinterpret_cast<const uint4*>(&sm.q[q][j >> 3][row_in * 128 + (((j & 7) ^ (row_in & 7)) << 4)]);
          float amax = 0.0f;
#pragma unroll
          for (int j = 0; j < D / 8; ++j) {
            const uint32_t wd[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 v = unpack2(wd[e], BF16);
              amax = fmaxf(amax, fmaxf(fabsf(v.x), fabsf(v.y)));
            }
          }
          const int shift = row_shift(amax);
          const float factor = a.scale_log2 * gk;
          const float up = copysignf(ldexpf(1.0f, shift), factor);
          f = ldexpf(fabsf(factor), -shift);
#pragma unroll
          for (int j = 0; j < D / 8; ++j) {
            const uint32_t wd[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 v = unpack2(wd[e], BF16);
              o[e] = pack_f16(v.x * up, v.y * up);
            }
            *reinterpret_cast<uint4*>(&sm.q[q][j >> 3][row_in * 128 + (((j & 7) ^ (row_in & 7)) << 4)]) =
                make_uint4(o[0], o[1], o[2], o[3]);
          }
          fence_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sm.qfull[q]));
        }
        // keys this row sees, and those every row of the tile sees
        const int hi = a.causal ? w.s.len - w.s.nq + tok : w.s.len - 1;
        const int64_t first = a.window > 0 ? static_cast<int64_t>(hi) - a.window + 1 : 0;
        const int lo = first > 0 ? static_cast<int>(first) : 0;
        const int tok_a = tok0 + tile_row / a.group, tok_b = tok0 + (min(rows, tile_row + kRowTile) - 1) / a.group;
        const int all_hi = a.causal ? w.s.len - w.s.nq + tok_a : w.s.len - 1;
        const int64_t all_lo = a.window > 0 ? static_cast<int64_t>(w.s.len) - w.s.nq + tok_b - a.window + 1 : 0;

        // (the products of the tiles before are in O when a tile's scores have come)
        auto scale_o = [&](float r) {
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            uint32_t o[16];
            tmem_ld_x16(o_tmem + 16 * c, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * r);
            tmem_st_x16(o_tmem + 16 * c, o);
          }
        };
        const int first_tile = one ? q : 0;
#pragma unroll 1
        for (int i = first_tile; i < tiles; i += one ? 2 : 1) {
          const uint32_t num = n + i;
          const int key0 = w.k.lo + (w.ta + i) * kKeys;
          wait(&sm.sfull[q], my_tiles++ & 1);
          tc_fence_after();
          uint32_t valid = 0;
#pragma unroll
          for (int c = 0; c < 4; ++c) valid |= sm.valid[num % kRing][c] << (2 * c);
          const bool masked = valid != 0xFFu || key0 + kKeys - 1 > all_hi || key0 < all_lo;
          // factor of 32 keys' scores; not zero, so that a masked score stays
          // -inf (2^-126 of a score is nothing)
          auto factor_of = [&](int c) {
            const float fc = FMT == kMXFP4 ? f * sm.kfac[num % kRing][c] : f;
            return fc < FLT_MIN ? FLT_MIN : fc;
          };
          auto mask = [&](int c, float(&x)[32]) {
            const int from = lo - key0 - 32 * c, to = hi - key0 - 32 * c;
            // keys from..to of the 32, and of the groups that are there
            uint32_t keep = to < 0 ? 0u : to >= 31 ? ~0u : (2u << to) - 1u;
            keep &= from <= 0 ? ~0u : from > 31 ? 0u : ~0u << from;
            if (!((valid >> (2 * c)) & 1)) keep &= 0xFFFF0000u;
            if (!((valid >> (2 * c + 1)) & 1)) keep &= 0x0000FFFFu;
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((keep >> e) & 1)) x[e] = -INFINITY;
          };
          // ---- one pass: a chunk's scores become weights of the reference
          // maximum as it stands, which moves only when passed by 2^kWeightRoom;
          // then O, and the tile's weights so far, are scaled: by a power of two
          // (the reference is a whole number), so that a weight that has been
          // rounded to FP16 is rounded again below its range only
          float2 sum = make_float2(0.0f, 0.0f);
          auto weigh = [&](int c, float(&xa)[32], float(&xb)[32]) {   // 64 keys
            if (masked) {
              mask(c, xa);
              mask(c + 1, xb);
            }
            const float fa = factor_of(c), fb = factor_of(c + 1);
            float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, u[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int e = 0; e < 32; ++e) t[e & 3] = fmaxf(t[e & 3], xa[e]), u[e & 3] = fmaxf(u[e & 3], xb[e]);
            const float top = fmaxf(fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) * fa,
                                    fmaxf(fmaxf(u[0], u[1]), fmaxf(u[2], u[3])) * fb);
            while (__any_sync(0xFFFFFFFFu, top > m + kWeightRoom)) {
              // (weights and O that this tile has stored are loaded again)
              tmem_wait_st();
              float r = 1.0f;
              if (top > m + kWeightRoom) {
                // 2^-24, FP16's least number, at a time (2^-64 leaves nothing, so
                // that this takes three times at most)
                const float up = top - m < 64.0f ? fminf(ceilf(top), m + 24.0f) : ceilf(top);
                r = ex2(m - up);
                m = up;
                l *= r;
                sum.x *= r;
                sum.y *= r;
              }
              if (i > first_tile) scale_o(r);
              const __half2 rh = __float2half2_rn(r);
#pragma unroll 1
              for (int c2 = 0; c2 < c; ++c2) {
                uint32_t p[16];
                tmem_ld_x16(s_tmem + 16 * c2, p);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) p[e] = mul2(p[e], reinterpret_cast<const uint32_t&>(rh));
                tmem_st_x16(s_tmem + 16 * c2, p);
              }
            }
            const float ref = m == -INFINITY ? 0.0f : kWeightLift - m;
            const float2 ref2 = make_float2(ref, ref);
            auto put = [&](int at, float(&x)[32], float fc) {
              const float2 fc2 = make_float2(fc, fc);
              uint32_t p[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float2 y = fma2(make_float2(x[2 * e], x[2 * e + 1]), fc2, ref2);
                const float2 pe = make_float2(ex2(y.x), ex2(y.y));
                p[e] = pack_f16(pe.x, pe.y);
                // FP16 outputs: the sum is of the rounded weights, so that what
                // rounding does to the keys with most of a row's weight cancels:
                // errors are 1.3 times an exact product's, 1.4 to 1.5 with the
                // sum of the unrounded, which BF16's own rounding hides (8 bits)
                // and which takes 1.42 ms in place of 1.49 (4096-token piece)
                if constexpr (BF16)
                  sum = add2(sum, pe);
                else
                  add_f16x2(sum, p[e]);
              }
              tmem_st_x16(s_tmem + 16 * at, p);
            };
            put(c, xa, fa);
            put(c + 1, xb, fb);
          };
          // (the loop stays rolled: this kernel's roles share an instruction cache.
          // 64 keys at a time, 4096-token piece: 1.43 ms, 32 keys 1.54, 16 keys
          // 1.98; a vote, a wait and a store's latency a chunk)
#pragma unroll 1
          for (int c = 0; c < 4; c += 2) {
            uint32_t ra[32], rb[32];
            tmem_ld_x32(s_tmem + 32 * c, ra);
            tmem_ld_x32(s_tmem + 32 * c + 32, rb);
            tmem_wait_ld();
            weigh(c, reinterpret_cast<float(&)[32]>(ra), reinterpret_cast<float(&)[32]>(rb));
          }
          l += sum.x + sum.y;
          // MXFP4: V is held relative to a reference that has risen since this
          // chain's last tile, perhaps (looked at last, when V has long come)
          if constexpr (FMT == kMXFP4) {
            wait(&sm.vfull[num & 1], (num >> 1) & 1);
            const float now = sm.vscale[num % kRing];
            if (i > first_tile && now != vs) {
              tmem_wait_st();   // (the tile may have scaled O already)
              scale_o(vs / now);   // (powers of two)
            }
            vs = now;
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sm.pfull[q]));
        }
        wait(&sm.ofull[q], my_items++ & 1);
        tc_fence_after();
      }
      n += tiles;
      // ---- the halves of one row tile's keys meet, where the queries were
      // (every product with them is done when both groups have seen ofull)
      float4* other = reinterpret_cast<float4*>(&sm.q[0][0][0]);   // [D / 4][128 rows]
      float w0 = vs, w1 = 0.0f;
      const bool meet = one && tiles > 1;
      if (meet) {
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (q == 1) {
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            uint32_t r[16];
            tmem_ld_x16(o_tmem + 16 * c, r);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 4; ++e)
              other[(4 * c + e) * kRowTile + row_in] =
                  make_float4(__uint_as_float(r[4 * e]) * vs, __uint_as_float(r[4 * e + 1]) * vs,
                              __uint_as_float(r[4 * e + 2]) * vs, __uint_as_float(r[4 * e + 3]) * vs);
          }
          tc_fence_before();
          sm.m1[row_in] = m;
          sm.l1[row_in] = l;
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (q == 0) {
          const float m1 = sm.m1[row_in], l1 = sm.l1[row_in], M = fmaxf(m, m1);
          const float f0 = weight_of(m, l, M);
          w1 = weight_of(m1, l1, M);
          w0 *= f0;
          l = l * f0 + l1 * w1;
          m = M;
        }
      }
      // ---- O of the row: the output, or a partial
      const int64_t out_row = w.s.q0 + static_cast<int64_t>(tok);
      auto store_out = [&](int c, const float(&x)[16], float inv, int64_t place) {   // 16 dimensions from 16 c on
        uint16_t* dst = static_cast<uint16_t*>(a.out.data) + place + 16 * c;
#pragma unroll
        for (int e = 0; e < 2; ++e)
          reinterpret_cast<uint4*>(dst)[e] =
              make_uint4(pack2(x[8 * e] * inv, x[8 * e + 1] * inv, BF16), pack2(x[8 * e + 2] * inv, x[8 * e + 3] * inv, BF16),
                         pack2(x[8 * e + 4] * inv, x[8 * e + 5] * inv, BF16),
                         pack2(x[8 * e + 6] * inv, x[8 * e + 7] * inv, BF16));
      };
      auto store_lse = [&](float M, float L) {
        if (a.lse) a.lse[out_row * (static_cast<int64_t>(a.cache.heads) * a.group) + head] = lse_of(M, L);
      };
      float* slot = partials + (2 * static_cast<size_t>(blockIdx.x) + (w.ta == 0 ? 1 : 0)) * partial_floats<D>();
      if (puts) {
        const float inv = l == 0.0f ? 0.0f : gv / l;   // no key: zeros
#pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
          uint32_t r[16];
          float x[16];
          tmem_ld_x16(o_tmem + 16 * c, r);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = __uint_as_float(r[e]) * w0;
          if (meet) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float4 y = other[(4 * c + e) * kRowTile + row_in];
              x[4 * e] += w1 * y.x, x[4 * e + 1] += w1 * y.y, x[4 * e + 2] += w1 * y.z, x[4 * e + 3] += w1 * y.w;
            }
          }
          if (whole) {
            if (mine) store_out(c, x, inv, out_row * a.out.token_stride + head * a.out.head_stride);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              reinterpret_cast<float4*>(slot)[(4 * c + e) * kRows + row] =
                  make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
          }
        }
        if (whole) {
          if (mine) store_lse(m, l);
        } else {
          slot[kRows * D + row] = m;
          slot[kRows * D + kRows + row] = l;
        }
        tc_fence_before();
      }
      if (!whole) {
        const int64_t item0 = w.begin + w.at;
        const int c0 = cta_of(w.total, w.ctas, item0);
        const int c1 = cta_of(w.total, w.ctas, item0 + (w.k.tiles > 1 ? w.k.tiles - 1 + w.cost : 0));
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (tid == 0) sm.last = atomic_add_acq_rel_gpu(&counters[c0], 1u) == static_cast<uint32_t>(c1 - c0);
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (sm.last) {
          if (tid == 0) counters[c0] = 0;   // every CTA of the item has arrived
          // The item's parts, weighed by their maxima.  First a thread takes a
          // row's maxima and sums; the weights' exponents stay where the queries
          // were, as many as fit there.  Then all threads take 16 dimensions of a
          // row at a time, two parts of them in flight.  (Short code: it comes
          // cold into the instruction cache.)
          constexpr int kKept = sizeof(sm.q) / (kRows * sizeof(float)) - 4, kAt = 4;
          float* kept = reinterpret_cast<float*>(&sm.q[0][0][0]);      // [kKept][kRows], then maxima, factors, places
          float* const top = kept + kKept * kRows;
          int64_t* const place = reinterpret_cast<int64_t*>(top + 2 * kRows);
          const int parts = c1 - c0 + 1;
          auto part = [&](int c) {
            return partials + (2 * static_cast<size_t>(c0 + c) + (c == 0)) * partial_floats<D>();
          };
          if (tid < rows) {
            float M = -INFINITY, L = 0.0f;
#pragma unroll 1
            for (int c = 0; c < parts; c += kAt) {
              float pm[kAt], pl[kAt];
#pragma unroll
              for (int e = 0; e < kAt; ++e) {
                const float* from = part(min(c + e, parts - 1)) + kRows * D + tid;
                pm[e] = __ldcg(from);
                pl[e] = __ldcg(from + kRows);
              }
#pragma unroll
              for (int e = 0; e < kAt; ++e) {
                if (c + e >= parts) break;
                const float to = fmaxf(M, pm[e]);
                L = L * weight_of(M, L, to) + pl[e] * weight_of(pm[e], pl[e], to);
                M = to;
                if (c + e < kKept) kept[(c + e) * kRows + tid] = pm[e];
              }
            }
            top[tid] = M;
            top[kRows + tid] = L == 0.0f ? 0.0f : gv / L;   // (NaN: the whole row)
            const int64_t token = w.s.q0 + static_cast<int64_t>(tok0 + tid / a.group);
            const int64_t to_head = static_cast<int64_t>(w.h) * a.group + tid % a.group;
            place[tid] = token * a.out.token_stride + to_head * a.out.head_stride;
            if (a.lse)
              a.lse[token * (static_cast<int64_t>(a.cache.heads) * a.group) + to_head] = lse_of(M, L);
          }
          asm volatile("bar.sync 1, 256;" ::: "memory");
          const int elements = rows * (D / 16);
#pragma unroll 1
          for (int e = tid; e < elements; e += 256) {
            const int d16 = e / rows, r = e - d16 * rows;
            const float M = top[r];
            float x[16] = {};
#pragma unroll 1
            for (int c = 0; c < parts; c += 2) {
              float4 v[2][4];
#pragma unroll
              for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  v[p][k] = __ldcg(reinterpret_cast<const float4*>(part(min(c + p, parts - 1))) + (4 * d16 + k) * kRows + r);
#pragma unroll
              for (int p = 0; p < 2; ++p) {
                if (c + p >= parts) break;
                const float fe =
                    weight_of(c + p < kKept ? kept[(c + p) * kRows + r] : __ldcg(part(c + p) + kRows * D + r), 0.0f, M);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  x[4 * k] += fe * v[p][k].x, x[4 * k + 1] += fe * v[p][k].y;
                  x[4 * k + 2] += fe * v[p][k].z, x[4 * k + 3] += fe * v[p][k].w;
                }
              }
            }
            store_out(d16, x, top[kRows + r], place[r]);
          }
        }
      }
      // sm.last, and queries where the halves met, may be written again
      if (!whole || meet) asm volatile("bar.sync 1, 256;" ::: "memory");
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) {
    tmem_dealloc(tmem, kColumns);
    if (lane == 0 && sm.abort) atomicOr(status, kStatusTimeout);
  }
}

template <int D, int FMT, bool BF16>
cudaError_t launch_as(const KvAttnArgs& a, int num_sms, cudaStream_t stream) {
  // more than half of an SM's shared memory, whatever D is: one CTA an SM, and
  // none of a GEMM's CTAs beside it (both allocate all of tensor memory)
  constexpr size_t kSmem = sizeof(Smem<D>) > 120 * 1024 ? sizeof(Smem<D>) : 120 * 1024;
  if (cudaError_t e = kv_allow_smem<kv_prompt_kernel<D, FMT, BF16>>(a.device, kSmem)) return e;
  kv_prompt_kernel<D, FMT, BF16><<<num_sms < kKvPromptCtas ? num_sms : kKvPromptCtas, kThreads, kSmem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

size_t kv_prompt_partials(int head_dim, int num_sms) {
  const size_t ctas = num_sms < kKvPromptCtas ? num_sms : kKvPromptCtas;
  return sizeof(float) * 2 * ctas * (head_dim == 128 ? partial_floats<128>() : partial_floats<64>());
}

cudaError_t launch_kv_prompt(const KvAttnArgs& a, int num_sms, cudaStream_t stream) {
  return kv_dispatch(a.cache.head_dim, a.cache.fmt, a.bf16,
                     [&](auto d, auto f, auto b) { return launch_as<d, f, b>(a, num_sms, stream); });
}

}  // namespace petit
