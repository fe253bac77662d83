// head_gemm.cu -- the three products of the head on the fifth-generation tensor cores:
//
//   logits     z = hidden . weight^T      rows x columns, inner dimension dim
//   d_hidden   g . weight                 rows x dim, inner dimension the piece's columns
//   d_weight   g^T . hidden               columns x dim, inner dimension the live rows
//
// The last two are one launch: they read the same gradient, neither needs the other, and the tiles of
// one fill the SMs that the last tiles of the other leave idle.
//
// A pair of CTAs, one per SM, walks 256 x 256 tiles of the result; each holds 128 rows of it. A
// producer thread in each brings its half of both operands, 64 elements of the inner dimension at a
// time, into a ring of shared memory stages (tensor map loads, 128-byte swizzle); one thread of the
// pair issues the products (M = 256), whose accumulators alternate between two halves of tensor
// memory; eight warps turn one half into its result while the other fills. Operands are
// read as they lie: where the outer dimension is the contiguous one (weight in d_hidden, both in
// d_weight) the descriptors say so, and nothing is transposed in memory.
//
// Why pairs: a single CTA's 128 x 256 tile reads 48 KiB for 512 cycles of products, and the path from
// L2 into an SM carries 64 bytes a cycle: the tensor pipe was 69-71% busy at 18 TB/s of such
// reads. A pair shares the second operand, 32 KiB for the same products, and keeps it 80% busy. Up
// to 128 rows one CTA works alone (CTAS = 1): half of a pair's product would be padding rows (8 rows,
// 1024 x 32768: 17 us a call alone, 30 us in pairs).
//
// The accumulator puts a row of the tile into one lane, so the softmax statistics of a row are
// one thread's registers: no shuffles.
#include <limits.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "device.cuh"
#include "head.h"
#include "launch.cuh"
#include "maps.h"
#include "program.h"
#include "tc.cuh"

namespace relay {
namespace {

// Bit 1: a wait ran out, the call's outputs are unspecified.
__device__ unsigned g_head_fault;

constexpr int kBM = 128, kBN = 256;  // rows of one CTA, columns of the product
// What depends on the number of CTAs that make one product and on the parts of its operands. A step is 64
// elements of the inner dimension; of fp32 operands 32, with all three parts of both in one stage: every
// part is used two or three times, and bringing it once halves what the path from L2 carries.
template <int PLANES, int CTAS>
struct Shape {
  static constexpr int kM = CTAS * kBM;       // rows of the product
  static constexpr int kShare = kBN / CTAS;   // columns (B's rows) one CTA brings
  static constexpr int kK = PLANES == 3 ? 32 : 64;
  static constexpr int kLoad = PLANES == 3 ? 3 : 1;  // parts in a stage
  static constexpr int kAPart = kBM * kK * 2, kBPart = kShare * kK * 2;
  static constexpr int kABytes = kLoad * kAPart, kStageBytes = kABytes + kLoad * kBPart;
  static constexpr int kStages = PLANES == 3 ? (CTAS == 2 ? 4 : 2) : CTAS == 2 ? 6 : 4;
};
static_assert(2 * kBM == kHeadRowTile && kBN == kHeadTile, "tiles are what rows and columns are padded to");
constexpr int kRingBytes = 192 * 1024;
template <int PLANES, int CTAS>
constexpr bool kFits = Shape<PLANES, CTAS>::kStages * Shape<PLANES, CTAS>::kStageBytes <= kRingBytes &&
                       Shape<PLANES, CTAS>::kStageBytes % 1024 == 0;
static_assert(kFits<1, 1> && kFits<1, 2> && kFits<3, 1> && kFits<3, 2>, "stages fit the ring, on 1024-byte addresses");
constexpr int kFinishWarps = 8;                        // warps that turn accumulators into results
constexpr int kOutWarpBytes = 32 * 64 * 2;             // 32 rows x 64 columns of 16 bits, one per warp
constexpr int kOutBytes = kFinishWarps * kOutWarpBytes;
constexpr int kSmemBytes = 1024 + kRingBytes + kOutBytes;
// Three groups of four warps: one that loads and multiplies (two threads of it), two that
// finish. The finishing threads hold 128 accumulators each, so registers move to them: at launch
// every thread has kLaunchRegs, and 56 + 2 * 224 = 3 * 168. The launch checks that the kernel was
// given exactly that many.
constexpr int kGemmThreads = 128 + 32 * kFinishWarps;
constexpr int kLaunchRegs = 168, kFeedRegs = 56, kFinishRegs = 224;
static_assert(kFeedRegs + 2 * kFinishRegs == 3 * kLaunchRegs, "the groups' registers add up to the launch's");
constexpr int kMine = kBN / 2;                         // columns of a tile's row one thread finishes

enum Product { kStats, kStatsKeep, kGradient, kBack };

// Inner steps summed in tensor memory before the sum moves on into registers. The tensor
// cores cut what does not fit 24 bits at every product instead of rounding it, which drifts with
// the length of the chain: a product costs a sum of one sign about 1e-7 of it. At dim 4096 in one chain the loss was
// several times as far from its 64-bit value as an fp32 sum. A chain of 48 products leaves it 3.7e-7 off at
// 2047 x 2048 x 50001 (32 products: 2.6e-7 and 1% more time; 64: 5.5e-7 and 1% less; the plain fp32 form 4e-7). The
// gradients of a bf16 head move on every 256 products: over 8192 products of one sign (131072 tokens, or as many
// columns) their mean is then 0.6e-5 and 1.4e-5 low, where one chain was 8.0e-4 and 7.8e-4 low, half of what rounding to bf16
// does, and always towards 0. It takes 1% more time at 2047 x 2048 x 50001 (610 -> 616 us) and 3% at
// 8192 x 4096 x 131072 (18.5 -> 19.0 ms); 384 products: 2.5e-5, 0.5% faster.
template <int P, int PLANES>
constexpr int kChain = PLANES == 3 ? 4 : P == kBack ? 64 : 12;

struct GemmArgs {
  CUtensorMap a;                         // first operand: hidden (logits), gradient (d_hidden)
  CUtensorMap aw;                        // the gradient as d_weight's first operand
  CUtensorMap b[RELAY_HEAD_MAX_SHARDS];  // weight shards, or the packed weight
  CUtensorMap hid;                       // hidden as d_weight's second operand
  CUtensorMap c[RELAY_HEAD_MAX_SHARDS];  // results: gradient or codes (logits), d_weight
  CUtensorMap dh;                        // d_hidden's partial sums
  HeadGeom g;
  HeadWork w;
  HeadShards sh;
  int32_t extra;     // bytes a stage waits for that no load brings (test of the bounded waits)
  int32_t maps;      // which of the maps above are in use, in the order a, b, c, hid, dh, aw
  int32_t tile_lo, tile_hi;
  int32_t want_dh, want_dw;
  int32_t first;     // d_hidden: overwrite the partial sums
  int32_t whole;     // d_hidden: an uncut sum goes straight to its row (HeadWork.whole)
  int32_t out_map;   // d_weight: its rows can be stored through tensor maps
  int32_t group;     // logits: row tiles walked together before the next column tile
};

// This CTA's rows of one tile of the result, and the inner range behind it.
struct Item {
  int row0, col0;          // first row of this CTA's half and first column of the tile
  int tile, shard, v0;     // padded column tile, its shard, the shard's weight row it starts at
  int k_lo, k_hi;          // inner steps (d_hidden: column tiles)
  int split;
  bool weight;             // kBack: a tile of d_weight
};

// Which tiles a pair of CTAs takes, in order. Tiles of one cost go round the pairs. kBack has two
// kinds: d_hidden's long tiles go round first, and the pairs left out in the last round take as
// many of d_weight's as that round lasts before the rest goes round all.
struct Schedule {
  int cuts;                // head_cuts
  int pairs, mine;         // pairs of CTAs, and which this is
  int long_items, items;   // d_hidden's, all
  int late, lead, led;     // first pair without a last long tile; tiles each such pair takes ahead; their sum
  __device__ __forceinline__ int at(int slot) const {
    int i = mine + slot * pairs;
    if (i < long_items) return i;
    slot -= (long_items - mine + pairs - 1) / pairs * (mine < long_items);
    if (mine >= late) {
      if (slot < lead) {
        i = long_items + slot * (pairs - late) + mine - late;
        return i < long_items + led ? i : -1;
      }
      slot -= lead;
    }
    i = long_items + led + slot * pairs + mine;
    return i < items ? i : -1;
  }
};

template <int P, int CTAS>
__device__ __forceinline__ Schedule schedule(const GemmArgs& p, int live, int cuts) {
  constexpr int kM = CTAS * kBM;
  const int mt = (live + kM - 1) / kM, tiles = p.tile_hi - p.tile_lo;
  const int nd = (p.g.dim + kBN - 1) / kBN;
  Schedule s{};
  s.cuts = 1;
  s.pairs = gridDim.x / CTAS;
  s.mine = blockIdx.x / CTAS;
  if (P != kBack) {
    s.items = mt * tiles;
    return s;
  }
  const int short_items = p.want_dw ? tiles * (kHeadTile / kM) * nd : 0;
  if (p.want_dh) {
    s.cuts = cuts;
    s.long_items = mt * nd * s.cuts;
  }
  s.items = s.long_items + short_items;
  s.late = s.long_items % s.pairs;
  if (s.late > 0) {
    s.lead = min((int)(head_long_steps(tiles, s.cuts) / head_short_steps(live)), short_items / (s.pairs - s.late));
    s.led = s.lead * (s.pairs - s.late);
  }
  return s;
}

template <int P, int PLANES, int CTAS>
__device__ __forceinline__ Item item_at(const GemmArgs& p, const Schedule& sched, int live, int rank, int i) {
  constexpr int kM = CTAS * kBM, kPerTile = kHeadTile / kM, kK = Shape<PLANES, CTAS>::kK;
  const int mt = (live + kM - 1) / kM, tiles = p.tile_hi - p.tile_lo;
  const int nd = (p.g.dim + kBN - 1) / kBN;
  Item t{};
  if (P == kBack) {
    t.weight = i >= sched.long_items;
    if (t.weight) i -= sched.long_items;
    // the tiles of dim side by side: a piece of the gradient is read once
    t.col0 = i % nd * kBN;
    i /= nd;
    if (t.weight) {
      const int within = i % kPerTile * kM + rank * kBM;
      t.tile = p.tile_lo + i / kPerTile;
      t.shard = head_shard_of_tile(p.g, t.tile);
      t.v0 = (t.tile - p.g.tile0[t.shard]) * kHeadTile + within;
      t.row0 = (t.tile - p.tile_lo) * kHeadTile + within;
      t.k_hi = (live + kK - 1) / kK;
    } else {
      t.split = i % sched.cuts;
      t.row0 = i / sched.cuts * kM + rank * kBM;
      t.k_lo = p.tile_lo + (int)((int64_t)tiles * t.split / sched.cuts);
      t.k_hi = p.tile_lo + (int)((int64_t)tiles * (t.split + 1) / sched.cuts);
    }
  } else {
    const int per = p.group * tiles, band = i / per, in_band = i % per;
    const int width = min(p.group, mt - band * p.group);
    t.row0 = (band * p.group + in_band % width) * kM + rank * kBM;
    t.tile = p.tile_lo + in_band / width;
    t.shard = head_shard_of_tile(p.g, t.tile);
    t.v0 = (t.tile - p.g.tile0[t.shard]) * kHeadTile;
    t.col0 = (t.tile - p.tile_lo) * kHeadTile;
    t.k_hi = (p.g.dim + kK - 1) / kK;
  }
  return t;
}

// Inner steps of a tile, one call of f(step) each.
template <int P, int KK, class F>
__device__ __forceinline__ bool for_steps(const GemmArgs& p, const Item& t, F f) {
  if (P != kBack || t.weight) {
    for (int k = t.k_lo; k < t.k_hi; ++k)
      if (!f(k, 0, 0)) return false;
    return true;
  }
  for (int tile = t.k_lo; tile < t.k_hi; ++tile) {
    const int shard = head_shard_of_tile(p.g, tile), v0 = (tile - p.g.tile0[shard]) * kHeadTile;
    for (int k = 0; k < kHeadTile / KK; ++k) {
      if (v0 + k * KK >= p.g.rows[shard]) break;  // padding columns: their gradient is 0
      if (!f((tile - p.tile_lo) * (kHeadTile / KK) + k, shard, v0 + k * KK)) return false;
    }
  }
  return true;
}

// How many they are.
template <int P, int KK>
__device__ __forceinline__ int count_steps(const GemmArgs& p, const Item& t) {
  if (P != kBack || t.weight) return t.k_hi - t.k_lo;
  int steps = 0;
  for (int tile = t.k_lo; tile < t.k_hi;) {  // a shard at a time: only its last tile has fewer
    const int shard = head_shard_of_tile(p.g, tile), end = min(t.k_hi, p.g.tile0[shard + 1]);
    const int v0 = (tile - p.g.tile0[shard]) * kHeadTile, v1 = (end - p.g.tile0[shard]) * kHeadTile;
    steps += (min(v1, p.g.rows[shard]) - v0 + KK - 1) / KK;
    tile = end;
  }
  return steps;
}

// Products of parts that make up an fp32 product, small ones first: 2 0 0 1 1 0 with 0 2 1 0 1 0.
constexpr int kPairs = 6;
__device__ __forceinline__ int pair_a(int i) { return (0x200110 >> (4 * (5 - i))) & 15; }
__device__ __forceinline__ int pair_b(int i) { return (0x021010 >> (4 * (5 - i))) & 15; }
// Stages a step fills, one part of a two-part gradient (PLANES 2) after the other: both for d_weight, the
// first part alone for d_hidden, whose products are not hidden behind writes: 16 rows,
// 4096 x 131072 take 645 us with one part, 679 with two for d_weight, 865 with two for both.
template <int PLANES>
__device__ __forceinline__ int fills(const Item& t) { return PLANES == 2 && t.weight ? 2 : 1; }

// full: the stage barriers of the pair's first CTA; empty: this CTA's own.
template <int P, int PLANES, int CTAS>
__device__ void produce(const GemmArgs& p, const Schedule& sched, int live, int rank, uint32_t ring, uint32_t full, uint32_t empty,
                        volatile int* gave_up) {
  const uint32_t pair_full = pair_addr(full, 0);
  using S = Shape<PLANES, CTAS>;
  constexpr int kK = S::kK;
  const int share = rank * S::kShare;
  int stage = 0;
  uint32_t phase = 0;
  int64_t issued = 0;
  bool ok = true;
  for (int slot = 0, i; ok && (i = sched.at(slot)) >= 0; ++slot) {
    const Item t = item_at<P, PLANES, CTAS>(p, sched, live, rank, i);
    ok = for_steps<P, kK>(p, t, [&](int k, int k_shard, int k_v) {
      for (int fill = fills<PLANES>(t) - 1; fill >= 0; --fill) {  // the smaller part first
        if (!bar_wait(empty + 8 * stage, phase ^ 1, gave_up)) return false;
        const uint32_t bar = pair_full + 8 * stage;
        if (rank == 0) bar_expect(full + 8 * stage, CTAS * S::kStageBytes + p.extra);
        ++issued;
#pragma unroll
        for (int part = 0; part < S::kLoad; ++part) {
          const uint32_t sa = ring + stage * S::kStageBytes + part * S::kAPart;
          const uint32_t sb = ring + stage * S::kStageBytes + S::kABytes + part * S::kBPart;
          const int a_row = (part + fill) * p.g.mpad, b_row = part * p.g.mpad;          // planes of rows
          const int wrow = part * p.g.tile0[RELAY_HEAD_MAX_SHARDS] * kHeadTile;         // of the packed weight
          if (P == kBack && t.weight) {
            for (int j = 0; j < kBM / 64; ++j)
              map_load<CTAS>(sa + j * 128 * kK, &p.aw, t.row0 + 64 * j, a_row + k * kK, bar);
            for (int j = 0; j < S::kShare / 64; ++j)
              map_load<CTAS>(sb + j * 128 * kK, &p.hid, t.col0 + share + 64 * j, b_row + k * kK, bar);
          } else if (P == kBack) {
            map_load<CTAS>(sa, &p.a, k * kK, a_row + t.row0, bar);
            const bool packed = p.w.wpack != nullptr;
            const CUtensorMap* m = &p.b[packed ? 0 : k_shard];
            const int y = packed ? wrow + p.g.tile0[k_shard] * kHeadTile + k_v : k_v;
            for (int j = 0; j < S::kShare / 64; ++j) map_load<CTAS>(sb + j * 128 * kK, m, t.col0 + share + 64 * j, y, bar);
          } else {
            map_load<CTAS>(sa, &p.a, k * kK, a_row + t.row0, bar);
            if (p.w.wpack != nullptr)
              map_load<CTAS>(sb, &p.b[0], k * kK, wrow + t.tile * kHeadTile + share, bar);
            else
              map_load<CTAS>(sb, &p.b[t.shard], k * kK, t.v0 + share, bar);
          }
        }
        if (++stage == S::kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
      return true;
    });
  }
  if (ok) return;
  // giving up: no load may still be on its way into shared memory when the CTA leaves. The first CTA's
  // barriers count both CTAs' loads, and the pair leaves together; what they do not count (a stage
  // only one of the two asked for) lands in microseconds.
  const uint64_t start = global_ns();
  for (int back = 0; rank == 0 && back < S::kStages && back < issued; ++back) {
    if (--stage < 0) {
      stage = S::kStages - 1;
      phase ^= 1;
    }
    while (!bar_try(full + 8 * stage, phase) && global_ns() - start < kWaitNs) {
    }
  }
  const uint64_t drained = global_ns();
  while (global_ns() - drained < 10000000ull) {
  }
}

template <int P, int PLANES, int CTAS>
__device__ void multiply(const GemmArgs& p, const Schedule& sched, int live, uint32_t ring, uint32_t full, uint32_t empty,
                         uint32_t acc_full, uint32_t acc_empty, uint32_t drain, uint32_t tmem,
                         volatile int* gave_up) {
  using S = Shape<PLANES, CTAS>;
  constexpr bool kBOuter = P == kBack;
  int stage = 0, n = 0;
  uint32_t phase = 0;
  bool ok = true;
  for (int slot = 0, i; ok && (i = sched.at(slot)) >= 0; ++slot) {
    const Item t = item_at<P, PLANES, CTAS>(p, sched, live, 0, i);
    const bool a_outer = P == kBack && t.weight;
    const uint32_t desc = a_outer ? product_desc(S::kM, kBN, true, kBOuter) : product_desc(S::kM, kBN, false, kBOuter);
    int in_chain = 0;
    auto open = [&] {
      const bool free = bar_wait(acc_empty + 8 * (n & 1), ((n >> 1) & 1) ^ 1, gave_up);
      tc_fence_after();
      return free;
    };
    if (!(ok = open())) break;
    ok = for_steps<P, Shape<PLANES, CTAS>::kK>(p, t, [&](int, int, int) {
      if (in_chain == kChain<P, PLANES>) {
        tc_commit<CTAS>(acc_full + 8 * (n & 1));
        ++n;
        in_chain = 0;
        if (!open()) return false;
      }
      const uint32_t acc = tmem + (n & 1) * kBN;
      const int n_fills = fills<PLANES>(t);
      for (int fill = 0; fill < n_fills; ++fill) {
        if (!bar_wait(full + 8 * stage, phase, gave_up)) return false;
        tc_fence_after();
        const uint32_t sa = ring + stage * S::kStageBytes;
        const uint64_t da = operand_desc<S::kK>(sa, a_outer), db = operand_desc<S::kK>(sa + S::kABytes, kBOuter);
#pragma unroll
        for (int k = 0; k < S::kK / 16; ++k) {
          const uint64_t ka = da + k * operand_step(a_outer), kb = db + k * operand_step(kBOuter);
          const bool more = in_chain > 0 || fill > 0 || k > 0;
          if constexpr (PLANES == 3) {
#pragma unroll
            for (int pair = 0; pair < kPairs; ++pair)
              tc_product<CTAS>(acc, ka + pair_a(pair) * (S::kAPart >> 4), kb + pair_b(pair) * (S::kBPart >> 4), desc,
                               more || pair > 0);
          } else {
            tc_product<CTAS>(acc, ka, kb, desc, more);
          }
        }
        tc_commit<CTAS>(empty + 8 * stage);
        if (++stage == S::kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
      ++in_chain;
      return true;
    });
    if (ok) tc_commit<CTAS>(acc_full + 8 * (n++ & 1));
  }
  // giving up: products still running write the tensor memory that is about to be freed
  if (!ok) {
    tc_commit<CTAS>(drain);
    const uint64_t start = global_ns();
    while (!bar_try(drain, 0) && global_ns() - start < kWaitNs) {
    }
  }
}

// Two values rounded to bf16, packed; they keep what the rounding left.
__device__ __forceinline__ uint32_t take_part(float& a, float& b) {
  const uint32_t r = bf16x2_rn(a, b);
  a = __fsub_rn(a, __uint_as_float(r << 16));
  b = __fsub_rn(b, __uint_as_float(r & 0xffff0000u));
  return r;
}

// Stores 32 rows x 64 columns of 16-bit values through a warp's staging buffer.
struct Stager {
  uint32_t buf;
  // the store before may still be reading the buffer
  __device__ __forceinline__ void open() {
    if (threadIdx.x % 32 == 0) store_wait_read<0>();
    __syncwarp();
  }
  // eight of the row's columns (group 0..7)
  __device__ __forceinline__ void put(int group, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    const int row = threadIdx.x % 32;
    const uint32_t at = buf + row * 128 + ((group ^ (row & 7)) << 4);
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
  }
  __device__ __forceinline__ void close(const CUtensorMap* map, int x, int y, bool add = false) {
    fence_async_smem();
    __syncwarp();
    if (threadIdx.x % 32 == 0) {
      if (add) map_add(map, x, y, buf);
      else map_store(map, x, y, buf);
      store_commit();
    }
  }
};

// The thread's 128 values rounded to bf16, stored 64 columns at a time; v keeps the rest.
__device__ __forceinline__ void store_part(Stager& out, float (&v)[kMine], const CUtensorMap* map,
                                           int x, int y, int columns) {
#pragma unroll
  for (int c = 0; c < kMine; c += 64) {
    if (c >= columns) break;
    out.open();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = c + 8 * j;
      out.put(j, take_part(v[i], v[i + 1]), take_part(v[i + 2], v[i + 3]), take_part(v[i + 4], v[i + 5]),
              take_part(v[i + 6], v[i + 7]));
    }
    out.close(map, x + c, y);
  }
}

// The entries of one row, walked in ascending column order.
struct Entries {
  const int32_t* col;
  const float* q;
  float* z;
  int n, at, next;
  __device__ __forceinline__ void seek(const HeadWork& w, const HeadGeom& g, int row, int live, int first) {
    const int64_t r = row < live ? (int64_t)w.perm[row] * g.top : 0;
    col = w.ent_col + r;
    q = w.ent_q + r;
    z = w.ent_z + r;
    n = row < live ? g.top : 0;
    int lo = 0, hi = n;
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (col[mid] < first) lo = mid + 1;
      else hi = mid;
    }
    at = lo;
    next = at < n ? col[at] : INT_MAX;
  }
  __device__ __forceinline__ void step() { next = ++at < n ? col[at] : INT_MAX; }
};

// The thread's value of a column known only at run time. Written as selects that the compiler does
// not see through: it would put the 128 registers into memory to index them.
__device__ __forceinline__ float value_at(const float (&v)[kMine], int at) {
  float r = 0.0f;
#pragma unroll
  for (int j = 0; j < kMine; ++j)
    asm("{\n.reg .pred p;\nsetp.eq.s32 p, %1, %2;\nselp.f32 %0, %3, %0, p;\n}" : "+f"(r) : "r"(at), "r"(j), "f"(v[j]));
  return r;
}

// Steps of 2^-10 below the maximum, in log2 units, as the low 16 bits of the result's bits:
// kCodeZero (2^-64 of the maximum and less) stands for 0.
__device__ __forceinline__ uint32_t code_bits(float log2_below) {
  return __float_as_uint(fminf(fmaf(log2_below, -kCodeSteps, 8388608.0f), 8388608.0f + kCodeZero));
}

// (a - ref) * scale and (b - ref) * scale, each operation on both at once: 4096 x 256 x 50000 with gradients 503 us with
// one fused operation a value, which the ends of the range do not allow, 517 us with two, 512 us with pairs.
__device__ __forceinline__ float2 below(float a, float b, float ref, float scale) {
  float2 r;
  asm("{\n.reg .b64 v, m, s;\nmov.b64 v, {%2, %3};\nmov.b64 m, {%4, %4};\nmov.b64 s, {%5, %5};\n"
      "add.rn.f32x2 v, v, m;\nmul.rn.f32x2 v, v, s;\nmov.b64 {%0, %1}, v;\n}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a), "f"(b), "f"(-ref), "f"(scale));
  return r;
}

// v: the thread's row of the accumulator, columns [part * 128, part * 128 + 128) of the tile.
template <int P, int PLANES>
__device__ __forceinline__ void finish_logits(const GemmArgs& p, const Item& t, int live, float (&v)[kMine],
                                              int quarter, int part, const Entries& seeked, Stager& out) {
  const int row = t.row0 + quarter * 32 + threadIdx.x % 32;
  const int first = t.tile * kHeadTile + part * kMine;        // padded column of v[0]
  const int valid = p.g.rows[t.shard] - t.v0 - part * kMine;  // columns with a weight row; may be <= 0
  const float scale = head_log2_scale(p.g);
  const int x = t.col0 + part * kMine, y = t.row0 + quarter * 32;
  Entries e = seeked;
  if (P != kGradient) {
    while (e.next < first + kMine) {
      e.z[e.at] = value_at(v, e.next - first);
      e.step();
    }
    float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    if (valid < kMine) {
#pragma unroll
      for (int j = 0; j < kMine; ++j)
        if (j >= valid) v[j] = -INFINITY;
    }
#pragma unroll
    for (int j = 0; j < kMine; ++j) m[j & 3] = fmaxf(m[j & 3], v[j]);
    const float top = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
    // a row of nothing but -inf: exponentials relative to 0 are 0, not NaN
    const float ref = top > -INFINITY ? top : 0.0f;
    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (P == kStatsKeep && PLANES == 1) {
#pragma unroll
      for (int c = 0; c < kMine; c += 64) {
        out.open();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          uint32_t code[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int at = c + 8 * j + 2 * i;
            const float2 x = below(v[at], v[at + 1], ref, scale);
            sum[i] += exp2_approx(x.x) + exp2_approx(x.y);
            code[i] = __byte_perm(code_bits(x.x), code_bits(x.y), 0x5410);
          }
          out.put(j, code[0], code[1], code[2], code[3]);
        }
        out.close(&p.c[0], x + c, y);
      }
    } else {
#pragma unroll
      for (int j = 0; j < kMine; j += 2) {
        const float2 x = below(v[j], v[j + 1], ref, scale);
        v[j] = exp2_approx(x.x);
        v[j + 1] = exp2_approx(x.y);
        sum[j & 3] += v[j];
        sum[(j & 3) + 1] += v[j + 1];
      }
      if (P == kStatsKeep) {
#pragma unroll 1
        for (int i = 0; i < p.w.grad_planes; ++i) store_part(out, v, &p.c[0], x, i * p.g.mpad + y, kMine);
      }
    }
    p.w.part[(int64_t)(t.tile * 2 + part) * p.g.mpad + row] =
        make_float2(top, (sum[0] + sum[1]) + (sum[2] + sum[3]));
    return;
  }
  const float2 lse = row < live ? p.w.lse[row] : make_float2(0.0f, 0.0f);
  const float weight = row < live ? p.w.wrow[row] : 0.0f;
#pragma unroll
  for (int j = 0; j < kMine; ++j)
    v[j] = j < valid && row < live ? weight * exp2_approx(fmaf(v[j] - lse.x, scale, -lse.y)) : 0.0f;
  while (e.next < first + kMine) {
    const float d = weight * e.q[e.at];
    const int at = e.next - first;
#pragma unroll
    for (int j = 0; j < kMine; ++j) v[j] -= j == at ? d : 0.0f;
    e.step();
  }
#pragma unroll 1
  for (int i = 0; i < p.w.grad_planes; ++i) store_part(out, v, &p.c[0], x, i * p.g.mpad + y, kMine);
}

template <int PLANES>
__device__ __forceinline__ void finish_dhidden(const GemmArgs& p, const Item& t, int live, int cuts,
                                               float (&v)[kMine], int quarter, int part, Stager& out) {
  const int r0 = t.row0 + quarter * 32, row = r0 + threadIdx.x % 32, d0 = t.col0 + part * kMine;
  const int valid = p.g.dim - d0;
  if (valid <= 0 || r0 >= live) return;
  if (t.k_lo >= t.k_hi) {  // a cut without columns: nothing was multiplied
#pragma unroll
    for (int j = 0; j < kMine; ++j) v[j] = 0.0f;
  }
  if (!p.whole || cuts > 1) {
    // partial sums: whole lines through the staging buffer, added to where a piece came before (one
    // addition per element and launch: in a fixed order). Rows past the live ones go unread.
#pragma unroll
    for (int c = 0; c < kMine; c += 32) {
      if (c >= valid) break;
      out.open();
#pragma unroll
      for (int j = 0; j < 8; ++j)
        out.put(j, __float_as_uint(v[c + 4 * j]), __float_as_uint(v[c + 4 * j + 1]), __float_as_uint(v[c + 4 * j + 2]),
                __float_as_uint(v[c + 4 * j + 3]));
      out.close(&p.dh, d0 + c, t.split * p.g.mpad + r0, !p.first);
    }
    return;
  }
  if (row >= live) return;
  if (PLANES < 3) {
    uint16_t* to = static_cast<uint16_t*>(p.sh.dh) + p.w.perm[row] * p.sh.dh_ld + d0;
#pragma unroll
    for (int j = 0; j < kMine; j += 8) {
      if (j >= valid) break;
      if (j + 8 <= valid) {
        *reinterpret_cast<uint4*>(to + j) = TBF16::pack(v + j);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (j + i < valid) to[j + i] = (uint16_t)(bf16x2_rn(v[j + i], 0.0f) & 0xffffu);
      }
    }
    return;
  }
  // an uncut fp32 sum of the only piece is d_hidden's row itself
  float* to = static_cast<float*>(p.sh.dh) + p.w.perm[row] * p.sh.dh_ld + d0;
#pragma unroll
  for (int j = 0; j < kMine; j += 4) {
    if (j + 4 <= valid) {
      *reinterpret_cast<float4*>(to + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (j + i < valid) to[j + i] = v[j + i];
    }
  }
}

// The staging buffer's 32 rows (128 bytes of each) to columns no tensor map can store: row by row, with
// neighbouring lanes on neighbouring elements. Rare, and kept out of the unrolled path.
template <class T>
__device__ __noinline__ void copy_rows(uint32_t buf, T* to, int64_t ld, int rows, int columns) {
  __syncwarp();
  constexpr int kAtOnce = 8;  // rows whose elements are read before any is stored
  for (int e = threadIdx.x % 32; e < columns; e += 32)
    for (int r0 = 0; r0 < rows; r0 += kAtOnce) {
      uint32_t x[kAtOnce];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const int r = r0 + i;
        const uint32_t at = buf + r * 128 + (((e * (int)sizeof(T) / 16) ^ (r & 7)) << 4) + e * (int)sizeof(T) % 16;
        if constexpr (sizeof(T) == 2) {
          uint16_t h;
          asm volatile("ld.shared.b16 %0, [%1];" : "=h"(h) : "r"(at) : "memory");
          x[i] = h;
        } else {
          asm volatile("ld.shared.b32 %0, [%1];" : "=r"(x[i]) : "r"(at) : "memory");
        }
      }
      T* row = to + r0 * ld + e;
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i, row += ld) {
        if (r0 + i >= rows) break;
        if constexpr (sizeof(T) == 2) *row = (uint16_t)x[i];
        else *row = __uint_as_float(x[i]);
      }
    }
  __syncwarp();
}

template <int PLANES>
__device__ __forceinline__ void finish_dweight(const GemmArgs& p, const Item& t, float (&v)[kMine], int quarter,
                                               int part, Stager& out) {
  using T = std::conditional_t<PLANES == 3, float, uint16_t>;
  constexpr int kCols = 128 / (int)sizeof(T);
  const int r0 = t.v0 + quarter * 32, d0 = t.col0 + part * kMine;
  const int rows = p.g.rows[t.shard], valid = p.g.dim - d0;
  if (r0 >= rows || valid <= 0) return;
  if (t.k_hi == 0) {  // no live row: nothing was multiplied
#pragma unroll
    for (int j = 0; j < kMine; ++j) v[j] = 0.0f;
  }
  // 128 bytes of each of the warp's 32 rows at a time
#pragma unroll
  for (int c = 0; c < kMine; c += kCols) {
    if (c >= valid) break;
    out.open();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (PLANES < 3) {
        const int i = c + 8 * j;
        out.put(j, bf16x2_rn(v[i], v[i + 1]), bf16x2_rn(v[i + 2], v[i + 3]), bf16x2_rn(v[i + 4], v[i + 5]),
                bf16x2_rn(v[i + 6], v[i + 7]));
      } else {
        const int i = c + 4 * j;
        out.put(j, __float_as_uint(v[i]), __float_as_uint(v[i + 1]), __float_as_uint(v[i + 2]), __float_as_uint(v[i + 3]));
      }
    }
    // a store through the map writes 16 bytes at a time, also where the row ends inside them: the last columns of
    // such rows are stored by hand
    if (p.out_map && (valid - c >= kCols || (valid - c) * (int)sizeof(T) % 16 == 0))
      out.close(&p.c[t.shard], d0 + c, r0);
    else
      copy_rows<T>(out.buf, static_cast<T*>(p.sh.dw[t.shard]) + r0 * p.sh.dw_ld + d0 + c, p.sh.dw_ld, min(32, rows - r0),
                   min(kCols, valid - c));
  }
}

template <int P, int PLANES, int CTAS>
__global__ void __launch_bounds__(kGemmThreads, 1) head_product_kernel(const __grid_constant__ GemmArgs p) {
  constexpr int kStages = Shape<PLANES, CTAS>::kStages;
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t s_bar[2 * kStages + 5];
  __shared__ uint32_t s_tmem;
  __shared__ int s_gave_up;
  const int warp = threadIdx.x / 32, rank = (int)pair_rank();
  dep_launch();
  const uint32_t ring = (smem_addr(smem_raw) + 1023) & ~1023u, staging = ring + kRingBytes;
  const uint32_t full = smem_addr(s_bar), empty = full + 8 * kStages, acc_full = empty + 8 * kStages,
                 acc_empty = acc_full + 16, drain = acc_empty + 16;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      bar_init(full + 8 * i, 1);
      bar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(acc_full + 8 * i, 1);
      bar_init(acc_empty + 8 * i, CTAS * kFinishWarps);  // of all CTAs, at the first's
    }
    bar_init(drain, 1);
    s_gave_up = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 2 && threadIdx.x % 32 <= 2 * RELAY_HEAD_MAX_SHARDS + 3) {
    // the maps' descriptors, on their way before the first load asks for them (a map that is not
    // used holds zeros, and is not fetched)
    const int i = threadIdx.x % 32;
    const CUtensorMap* m = i == 0 ? &p.a : i <= RELAY_HEAD_MAX_SHARDS ? &p.b[i - 1]
                           : i <= 2 * RELAY_HEAD_MAX_SHARDS ? &p.c[i - 1 - RELAY_HEAD_MAX_SHARDS]
                           : i == 2 * RELAY_HEAD_MAX_SHARDS + 1 ? &p.hid : i == 2 * RELAY_HEAD_MAX_SHARDS + 2 ? &p.dh : &p.aw;
    if ((p.maps >> i) & 1) map_prefetch(m);
  }
  if (warp == 1) tmem_alloc<CTAS>(smem_addr(&s_tmem), 512);
  tc_fence_before();
  __syncthreads();
  if (CTAS == 2) pair_sync();  // the other CTA's barriers are ready
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  dep_wait();
  const int2 counted = *reinterpret_cast<const int2*>(p.w.n_live);
  const int live = counted.x;
  const Schedule sched = schedule<P, CTAS>(p, live, counted.y);  // a pair without a tile passes through
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFeedRegs));
    if (threadIdx.x == 0) produce<P, PLANES, CTAS>(p, sched, live, rank, ring, full, empty, &s_gave_up);
    if (threadIdx.x == 32 && rank == 0)
      multiply<P, PLANES, CTAS>(p, sched, live, ring, full, empty, acc_full, acc_empty, drain, tmem, &s_gave_up);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kFinishRegs));
    // warps 4 to 7 finish a tile's first 128 columns, 8 to 11 its last; a warp reads the quarter of
    // tensor memory's lanes that its number gives it
    const int quarter = warp % 4, part = warp / 4 - 1;
    Stager out{staging + (warp - 4) * kOutWarpBytes};
    int n = 0;
    bool ok = true;
    const uint32_t first_empty = pair_addr(acc_empty, 0);
    for (int slot = 0, i; ok && (i = sched.at(slot)) >= 0; ++slot) {
      const Item t = item_at<P, PLANES, CTAS>(p, sched, live, rank, i);
      Entries e;
      if (P <= kGradient)  // under the products
        e.seek(p.w, p.g, t.row0 + quarter * 32 + threadIdx.x % 32, live, t.tile * kHeadTile + part * kMine);
      const int steps = count_steps<P, Shape<PLANES, CTAS>::kK>(p, t);
      const int chains = max(1, (steps + kChain<P, PLANES> - 1) / kChain<P, PLANES>);
      float v[kMine];
      for (int c = 0; c < chains; ++c, ++n) {
        const int half = n & 1;
        if (!(ok = __all_sync(~0u, bar_wait(acc_full + 8 * half, (n >> 1) & 1, &s_gave_up)))) break;
        tc_fence_after();
        const uint32_t acc = tmem + half * kBN + part * kMine + ((uint32_t)(quarter * 32) << 16);
        if (c == 0) {
#pragma unroll
          for (int j = 0; j < kMine; j += 16) tmem_load16(acc + j, v + j);
        } else {
#pragma unroll
          for (int j = 0; j < kMine; j += 16) {
            float u[16];
            tmem_load16(acc + j, u);
#pragma unroll
            for (int k = 0; k < 16; ++k) v[j + k] = __fadd_rn(v[j + k], u[k]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (threadIdx.x % 32 == 0) bar_arrive_pair(first_empty + 8 * half);
      }
      if (!ok) break;
      if constexpr (P == kBack) {
        if (t.weight) finish_dweight<PLANES>(p, t, v, quarter, part, out);
        else finish_dhidden<PLANES>(p, t, live, sched.cuts, v, quarter, part, out);
      } else finish_logits<P, PLANES>(p, t, live, v, quarter, part, e, out);
    }
    if (threadIdx.x % 32 == 0) store_wait_all();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (CTAS == 2) pair_sync();  // neither CTA's memory is used by the other any more
  if (threadIdx.x == 0 && s_gave_up) atomicOr(&g_head_fault, 2u);
  if (warp == 1) {
    tc_fence_after();
    tmem_free<CTAS>(tmem, 512);
  }
}

// ------------------------------------------------------------------ host side --

thread_local int t_extra = 0;

// A matrix [rows][cols], row stride ld elements, read or written in boxes: bf16 by 64 columns or fp32 by 32
// (128 bytes, 128-byte swizzle), or bf16 by 32 (64 bytes, 64-byte swizzle).
enum BoxKind { kBf16By64, kF32By32, kBf16By32 };
bool matrix_map(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, int64_t ld, int box_rows,
                BoxKind kind = kBf16By64) {
  const EncodeFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)ld * (kind == kF32By32 ? 4 : 2)};
  const cuuint32_t box[2] = {kind == kBf16By64 ? 64u : 32u, (cuuint32_t)box_rows}, unit[2] = {1, 1};
  return fn(m, kind == kF32By32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
            const_cast<void*>(p), dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
            kind == kBf16By32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int P>
bool maps_for(GemmArgs* a, int dtype) {
  const HeadGeom& g = a->g;
  const HeadWork& w = a->w;
  const int planes = head_planes(dtype);
  const int64_t padded = (int64_t)g.tile0[RELAY_HEAD_MAX_SHARDS] * kHeadTile;
  const int step = planes == 3 ? Shape<3, 1>::kK : Shape<1, 1>::kK;
  const BoxKind inner = planes == 3 ? kBf16By32 : kBf16By64;  // boxes of one inner step
  bool ok = true;
  // the weight: boxes of a CTA's share of 256 rows by a step of dim (logits), or of a step of rows by 64 (d_hidden)
  constexpr int kB = 1, kC = kB + RELAY_HEAD_MAX_SHARDS, kHid = kC + RELAY_HEAD_MAX_SHARDS, kDh = kHid + 1, kAw = kDh + 1;
  a->maps = 1;
  auto weight = [&](int box_rows, BoxKind kind) {
    if (w.wpack != nullptr) {
      a->maps |= 1 << kB;
      ok &= matrix_map(&a->b[0], w.wpack, planes * padded, g.dim, w.dim_pad, box_rows, kind);
    } else {
      for (int s = 0; s < g.A; ++s)
        if (g.rows[s] > 0) {
          a->maps |= 1 << (kB + s);
          ok &= matrix_map(&a->b[s], a->sh.w[s], g.rows[s], g.dim, a->sh.w_ld, box_rows, kind);
        }
    }
  };
  const int64_t hid_rows = (int64_t)planes * g.mpad, grad_rows = (int64_t)w.grad_planes * g.mpad;
  if (P == kBack) {
    ok &= matrix_map(&a->a, w.grad, grad_rows, w.grad_ld, w.grad_ld, kBM, inner);
    if (a->want_dh) {
      weight(step, kBf16By64);
      a->maps |= 1 << kDh;
      ok &= matrix_map(&a->dh, w.dh, (int64_t)w.splits * g.mpad, g.dim, w.dh_ld, 32, kF32By32);
    }
    if (a->want_dw) {
      a->maps |= 1 << kHid | 1 << kAw;
      ok &= matrix_map(&a->hid, w.hid, hid_rows, g.dim, w.dim_pad, step);
      ok &= matrix_map(&a->aw, w.grad, grad_rows, w.grad_ld, w.grad_ld, step);
      a->out_map = 1;
      for (int s = 0; s < g.A; ++s)
        if (g.rows[s] > 0)
          a->out_map &= reinterpret_cast<uintptr_t>(a->sh.dw[s]) % 16 == 0 && a->sh.dw_ld * esize_of(dtype) % 16 == 0;
      if (a->out_map)
        for (int s = 0; s < g.A; ++s)
          if (g.rows[s] > 0) {
            a->maps |= 1 << (kC + s);
            ok &= matrix_map(&a->c[s], a->sh.dw[s], g.rows[s], g.dim, a->sh.dw_ld, 32, planes == 3 ? kF32By32 : kBf16By64);
          }
    }
  } else {
    ok &= matrix_map(&a->a, w.hid, hid_rows, g.dim, w.dim_pad, kBM, inner);
    weight(kBN / g.ctas, inner);
    if (P != kStats) {
      a->maps |= 1 << kC;
      ok &= matrix_map(&a->c[0], w.grad, grad_rows, w.grad_ld, w.grad_ld, 32);
    }
  }
  return ok;
}

template <int P, int PLANES, int CTAS>
cudaError_t launch(const GemmArgs& a, int64_t items, cudaStream_t s) {
  static thread_local int ready_device = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  auto* kernel = head_product_kernel<P, PLANES, CTAS>;
  if (ready_device != dev) {
    cudaFuncAttributes attr;
    e = cudaFuncGetAttributes(&attr, kernel);
    if (e != cudaSuccess) return e;
    if (attr.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;  // the split would wait forever
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    ready_device = dev;
  }
  const int blocks = (int)std::min<int64_t>(CTAS * items, a.g.sms / CTAS * CTAS);
  return launch_chained_clusters(kernel, CTAS, blocks, kGemmThreads, kSmemBytes, s, a);
}

template <int P>
cudaError_t run(const HeadGeom& g, const HeadWork& w, const HeadShards& sh, int dtype, int lo, int hi, bool first,
                bool dh, bool dw, cudaStream_t s) {
  GemmArgs a{};
  a.g = g;
  a.w = w;
  a.sh = sh;
  a.tile_lo = lo;
  a.tile_hi = hi;
  a.first = first;
  a.whole = w.whole;
  a.extra = t_extra;
  a.want_dh = dh;
  a.want_dw = dw;
  // row tiles whose packed hidden rows take 64 MiB, half of L2
  const int rows = kBM * g.ctas;
  const int64_t mt = (g.tokens + rows - 1) / rows, tiles = hi - lo, nd = (g.dim + kBN - 1) / kBN;
  a.group = (int)std::max<int64_t>(1, std::min<int64_t>(mt, (64ll << 20) / ((int64_t)rows * w.dim_pad * 2 * head_planes(dtype))));
  if (!maps_for<P>(&a, dtype)) return cudaErrorInvalidValue;
  const int64_t items = P == kBack ? (dh ? mt * nd * w.splits : 0) + (dw ? tiles * (kHeadTile / rows) * nd : 0) : mt * tiles;
  if (items > INT_MAX) return cudaErrorInvalidValue;  // 2^31 tiles of 128 x 256
  if constexpr (P == kBack) {
    if (dtype == RELAY_BF16) return g.ctas == 1 ? launch<P, 2, 1>(a, items, s) : launch<P, 1, 2>(a, items, s);
    return g.ctas == 1 ? launch<P, kHeadPlanesF32, 1>(a, items, s) : launch<P, kHeadPlanesF32, 2>(a, items, s);
  }
  if constexpr (P != kBack) {
    if (g.ctas == 1)
      return dtype == RELAY_BF16 ? launch<P, 1, 1>(a, items, s) : launch<P, kHeadPlanesF32, 1>(a, items, s);
    return dtype == RELAY_BF16 ? launch<P, 1, 2>(a, items, s) : launch<P, kHeadPlanesF32, 2>(a, items, s);
  }
}

}  // namespace

cudaError_t head_logits(const HeadGeom& g, const HeadWork& w, const HeadShards& sh, int dtype, int tile_lo,
                        int tile_hi, HeadLogits mode, cudaStream_t s) {
  switch (mode) {
    case kHeadStats: return run<kStats>(g, w, sh, dtype, tile_lo, tile_hi, false, false, false, s);
    case kHeadStatsKeep: return run<kStatsKeep>(g, w, sh, dtype, tile_lo, tile_hi, false, false, false, s);
    default: return run<kGradient>(g, w, sh, dtype, tile_lo, tile_hi, false, false, false, s);
  }
}

cudaError_t head_back(const HeadGeom& g, const HeadWork& w, const HeadShards& sh, int dtype, int tile_lo, int tile_hi,
                      bool first, bool dh, bool dw, cudaStream_t s) {
  return run<kBack>(g, w, sh, dtype, tile_lo, tile_hi, first, dh, dw, s);
}

void head_test_extra(int bytes) { t_extra = bytes; }

cudaError_t head_read_fault(unsigned* fault) {
  cudaError_t e = cudaMemcpyFromSymbol(fault, g_head_fault, sizeof *fault);
  if (e != cudaSuccess || *fault == 0) return e;
  const unsigned zero = 0;
  return cudaMemcpyToSymbol(g_head_fault, &zero, sizeof zero);
}

}  // namespace relay
