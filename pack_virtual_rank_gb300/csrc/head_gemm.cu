// head_gemm.cu -- the three products of the head on the fifth-generation tensor cores:
//
//   logits     z = hidden . weight^T      rows x columns, inner dimension dim
//   d_hidden   g . weight                 rows x dim, inner dimension the piece's columns
//   d_weight   g^T . hidden               columns x dim, inner dimension the live rows
//
// One CTA per SM walks 128 x 256 tiles of the result. A producer thread brings 64 elements of the
// inner dimension at a time into a ring of shared memory stages (tensor map loads, 128-byte
// swizzle); one thread issues the products, whose accumulators alternate between two halves of
// tensor memory; four warps turn one half into its result while the other fills. Operands are
// read as they lie: where the outer dimension is the contiguous one (weight in d_hidden, both in
// d_weight) the descriptors say so, and nothing is transposed in memory.
//
// The accumulator puts a row of the tile into one lane, so the softmax statistics of a row are
// one thread's registers: no shuffles.
#include <limits.h>
#include <math.h>

#include <algorithm>

#include "device.cuh"
#include "head.h"
#include "program.h"
#include "tc.cuh"

namespace relay {
namespace {

// Bit 1: a wait ran out, the call's outputs are unspecified.
__device__ unsigned g_head_fault;

constexpr int kBM = 128, kBN = 256, kBK = 64;
constexpr int kStages = 4;
constexpr int kABytes = kBM * kBK * 2, kBBytes = kBN * kBK * 2, kStageBytes = kABytes + kBBytes;
constexpr int kOutWarpBytes = 32 * 64 * 2;             // 32 rows x 64 columns of bf16
constexpr int kOutBytes = 4 * 2 * kOutWarpBytes;       // four warps, two buffers each
constexpr int kSmemBytes = 1024 + kStages * kStageBytes + kOutBytes;
constexpr int kGemmThreads = 192;
constexpr float kLog2e = 1.4426950408889634f;

enum Product { kStats, kStatsKeep, kGradient, kDHidden, kDWeight };

struct GemmArgs {
  CUtensorMap a;
  CUtensorMap b[RELAY_HEAD_MAX_SHARDS];
  CUtensorMap c[RELAY_HEAD_MAX_SHARDS];
  HeadGeom g;
  HeadWork w;
  HeadShards sh;
  int32_t tile_lo, tile_hi;
  int32_t first;     // d_hidden: overwrite the partial sums
  int32_t out_map;   // d_weight: its rows can be stored through tensor maps
  int32_t group;     // logits: row tiles walked together before the next column tile
};

// One tile of the result and the inner range behind it.
struct Item {
  int row0, col0;          // first row and column of the tile
  int tile, shard, v0;     // padded column tile, its shard, first row of the shard's weight
  int k_lo, k_hi;          // inner steps of 64 (d_hidden: column tiles)
  int split;
};

template <int P>
__device__ __forceinline__ int item_count(const GemmArgs& p, int live) {
  const int mt = (live + kBM - 1) / kBM, tiles = p.tile_hi - p.tile_lo;
  const int nd = (p.g.dim + kBN - 1) / kBN;
  if (P == kDHidden) return mt * nd * p.w.splits;
  if (P == kDWeight) return tiles * 2 * nd;
  return mt * tiles;
}

template <int P>
__device__ __forceinline__ Item item_at(const GemmArgs& p, int live, int i) {
  const int mt = (live + kBM - 1) / kBM, tiles = p.tile_hi - p.tile_lo;
  const int nd = (p.g.dim + kBN - 1) / kBN;
  Item t{};
  if (P == kDHidden) {
    // every column tile of a row tile runs side by side: the gradient's rows are read once
    t.col0 = i % nd * kBN;
    i /= nd;
    t.split = i % p.w.splits;
    t.row0 = i / p.w.splits * kBM;
    t.k_lo = p.tile_lo + (int)((int64_t)tiles * t.split / p.w.splits);
    t.k_hi = p.tile_lo + (int)((int64_t)tiles * (t.split + 1) / p.w.splits);
  } else if (P == kDWeight) {
    t.col0 = i % nd * kBN;
    i /= nd;
    t.tile = p.tile_lo + i / 2;
    t.shard = head_shard_of_tile(p.g, t.tile);
    t.v0 = (t.tile - p.g.tile0[t.shard]) * kHeadTile + i % 2 * kBM;
    t.row0 = (t.tile - p.tile_lo) * kHeadTile + i % 2 * kBM;
    t.k_hi = t.v0 < p.g.rows[t.shard] ? (live + kBK - 1) / kBK : 0;
  } else {
    const int per = p.group * tiles, band = i / per, in_band = i % per;
    const int width = min(p.group, mt - band * p.group);
    t.row0 = (band * p.group + in_band % width) * kBM;
    t.tile = p.tile_lo + in_band / width;
    t.shard = head_shard_of_tile(p.g, t.tile);
    t.v0 = (t.tile - p.g.tile0[t.shard]) * kHeadTile;
    t.col0 = (t.tile - p.tile_lo) * kHeadTile;
    t.k_hi = (p.g.dim + kBK - 1) / kBK;
  }
  return t;
}

// Inner steps of a tile, one call of f(step) each.
template <int P, class F>
__device__ __forceinline__ bool for_steps(const GemmArgs& p, const Item& t, F f) {
  if constexpr (P != kDHidden) {
    for (int k = t.k_lo; k < t.k_hi; ++k)
      if (!f(k, 0, 0)) return false;
    return true;
  } else {
  for (int tile = t.k_lo; tile < t.k_hi; ++tile) {
    const int shard = head_shard_of_tile(p.g, tile), v0 = (tile - p.g.tile0[shard]) * kHeadTile;
    for (int k = 0; k < kHeadTile / kBK; ++k) {
      if (v0 + k * kBK >= p.g.rows[shard]) break;  // padding columns: their gradient is 0
      if (!f((tile - p.tile_lo) * (kHeadTile / kBK) + k, shard, v0 + k * kBK)) return false;
    }
  }
  return true;
  }
}

// Pairs of parts whose products make up an fp32 product.
template <int PLANES>
constexpr int kPairs = PLANES == 1 ? 1 : 6;
__device__ __forceinline__ int pair_a(int i) { return (0x200110 >> (4 * (5 - i))) & 15; }  // 2 0 0 1 1 0
__device__ __forceinline__ int pair_b(int i) { return (0x021010 >> (4 * (5 - i))) & 15; }  // 0 2 1 0 1 0

template <int P, int PLANES>
__device__ void produce(const GemmArgs& p, int live, uint32_t ring, uint32_t full, uint32_t empty,
                        volatile int* gave_up) {
  int stage = 0;
  uint32_t phase = 0;
  int64_t issued = 0;
  const int items = item_count<P>(p, live);
  bool ok = true;
  for (int i = blockIdx.x; ok && i < items; i += gridDim.x) {
    const Item t = item_at<P>(p, live, i);
    ok = for_steps<P>(p, t, [&](int k, int k_shard, int k_v) {
      for (int pair = 0; pair < kPairs<PLANES>; ++pair) {
        const int pa = PLANES == 1 ? 0 : pair_a(pair), pb = PLANES == 1 ? 0 : pair_b(pair);
        if (!bar_wait(empty + 8 * stage, phase ^ 1, gave_up)) return false;
        const uint32_t bar = full + 8 * stage, sa = ring + stage * kStageBytes, sb = sa + kABytes;
        bar_expect(bar, kStageBytes);
        ++issued;
        const int wrow = pb * p.g.tile0[RELAY_HEAD_MAX_SHARDS] * kHeadTile;  // plane of a packed weight
        if (P == kDHidden) {
          map_load(sa, &p.a, k * kBK, pa * p.g.mpad + t.row0, bar);
          const bool packed = p.w.wpack != nullptr;
          const CUtensorMap* m = &p.b[packed ? 0 : k_shard];
          const int y = packed ? wrow + p.g.tile0[k_shard] * kHeadTile + k_v : k_v;
          for (int j = 0; j < kBN / 64; ++j) map_load(sb + j * 8192, m, t.col0 + 64 * j, y, bar);
        } else if (P == kDWeight) {
          for (int j = 0; j < kBM / 64; ++j)
            map_load(sa + j * 8192, &p.a, t.row0 + 64 * j, pa * p.g.mpad + k * kBK, bar);
          for (int j = 0; j < kBN / 64; ++j)
            map_load(sb + j * 8192, &p.b[0], t.col0 + 64 * j, pb * p.g.mpad + k * kBK, bar);
        } else {
          map_load(sa, &p.a, k * kBK, pa * p.g.mpad + t.row0, bar);
          if (p.w.wpack != nullptr)
            map_load(sb, &p.b[0], k * kBK, wrow + t.tile * kHeadTile, bar);
          else
            map_load(sb, &p.b[t.shard], k * kBK, t.v0, bar);
        }
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
      return true;
    });
  }
  if (ok) return;
  // giving up: no load may still be on its way into shared memory when the CTA leaves
  const uint64_t start = global_ns();
  for (int back = 0; back < kStages && back < issued; ++back) {
    if (--stage < 0) {
      stage = kStages - 1;
      phase ^= 1;
    }
    while (!bar_try(full + 8 * stage, phase) && global_ns() - start < kWaitNs) {
    }
  }
}

template <int P, int PLANES>
__device__ void multiply(const GemmArgs& p, int live, uint32_t ring, uint32_t full, uint32_t empty,
                         uint32_t acc_full, uint32_t acc_empty, uint32_t drain, uint32_t tmem,
                         volatile int* gave_up) {
  constexpr bool kAOuter = P == kDWeight, kBOuter = P == kDWeight || P == kDHidden;
  constexpr uint32_t kDesc = product_desc(kBM, kBN, kAOuter, kBOuter);
  int stage = 0, n = 0;
  uint32_t phase = 0;
  const int items = item_count<P>(p, live);
  bool ok = true;
  for (int i = blockIdx.x; ok && i < items; i += gridDim.x, ++n) {
    const Item t = item_at<P>(p, live, i);
    const int half = n & 1;
    if (!(ok = bar_wait(acc_empty + 8 * half, ((n >> 1) & 1) ^ 1, gave_up))) break;
    tc_fence_after();
    const uint32_t acc = tmem + half * kBN;
    bool started = false;
    ok = for_steps<P>(p, t, [&](int, int, int) {
      for (int pair = 0; pair < kPairs<PLANES>; ++pair) {
        if (!bar_wait(full + 8 * stage, phase, gave_up)) return false;
        tc_fence_after();
        const uint32_t sa = ring + stage * kStageBytes;
        const uint64_t da = operand_desc(sa, kAOuter), db = operand_desc(sa + kABytes, kBOuter);
#pragma unroll
        for (int k = 0; k < kBK / 16; ++k) {
          tc_product(acc, da + k * operand_step(kAOuter), db + k * operand_step(kBOuter), kDesc, started);
          started = true;
        }
        tc_commit(empty + 8 * stage);
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
      return true;
    });
    if (ok) tc_commit(acc_full + 8 * half);
  }
  // giving up: products still running write the tensor memory that is about to be freed
  if (!ok) {
    tc_commit(drain);
    const uint64_t start = global_ns();
    while (!bar_try(drain, 0) && global_ns() - start < kWaitNs) {
    }
  }
}

// Splits v into PLANES bf16 parts; returns part `part` of each of two values, packed.
__device__ __forceinline__ uint32_t part_pair(float a, float b, int part) {
  uint32_t r = bf16x2_rn(a, b);
  for (int i = 0; i < part; ++i) {
    a = __fsub_rn(a, __uint_as_float(r << 16));
    b = __fsub_rn(b, __uint_as_float(r & 0xffff0000u));
    r = bf16x2_rn(a, b);
  }
  return r;
}

// Stores 32 rows x 64 columns of bf16 through a warp's two staging buffers.
struct Stager {
  uint32_t base;
  int n = 0;
  // the buffer may still be read by the store before last
  __device__ __forceinline__ uint32_t open() {
    if (threadIdx.x % 32 == 0) store_wait_read<1>();
    __syncwarp();
    return base + (n++ & 1) * kOutWarpBytes;
  }
  // 32 of the row's 64 columns (half 0 or 1)
  static __device__ __forceinline__ void put(uint32_t buf, int half, const float (&v)[32], int part) {
    const int row = threadIdx.x % 32;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t at = buf + row * 128 + (((half * 4 + j) ^ (row & 7)) << 4);
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(part_pair(v[8 * j], v[8 * j + 1], part)),
                   "r"(part_pair(v[8 * j + 2], v[8 * j + 3], part)), "r"(part_pair(v[8 * j + 4], v[8 * j + 5], part)),
                   "r"(part_pair(v[8 * j + 6], v[8 * j + 7], part))
                   : "memory");
    }
  }
  __device__ __forceinline__ void close(uint32_t buf, const CUtensorMap* map, int x, int y) {
    fence_async_smem();
    __syncwarp();
    if (threadIdx.x % 32 == 0) {
      map_store(map, x, y, buf);
      store_commit();
    }
  }
};

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

template <int P, int PLANES>
__device__ __forceinline__ void finish_logits(const GemmArgs& p, const Item& t, int live, uint32_t acc,
                                              int quarter, Stager& out) {
  const int lane = threadIdx.x % 32, row = t.row0 + quarter * 32 + lane;
  const int first = t.tile * kHeadTile;                       // padded column of the tile
  const int valid = min(kHeadTile, p.g.rows[t.shard] - t.v0);
  const float scale = p.g.inv_tau * kLog2e;
  Entries e;
  e.seek(p.w, p.g, row, live, first);
  float v[32];
  float top = -INFINITY, sum = 0.0f;
  if (P == kStatsKeep) {
    // the exponentials are kept relative to the tile's maximum, which must be known first
    for (int c = 0; c < valid; c += 32) {
      tmem_load32(acc + c, v);
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (c + j < valid) top = fmaxf(top, v[j]);
    }
  }
  const float lse = P == kGradient && row < live ? p.w.lse[row] : 0.0f;
  const float weight = P == kGradient && row < live ? p.w.wrow[row] : 0.0f;
  uint32_t buf = 0;
  for (int c = 0; c < kHeadTile; c += 32) {
    if (P == kStats && c >= valid) break;
    tmem_load32(acc + c, v);
    if (P != kGradient && e.next < first + c + 32) {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        while (e.next == first + c + j) {
          e.z[e.at] = v[j] * p.g.inv_tau;
          e.step();
        }
    }
    if (P == kStats) {
      float m = top;
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        if (c + j >= valid) v[j] = -INFINITY;
        m = fmaxf(m, v[j]);
      }
      // a row of nothing but -inf so far: exponentials relative to 0 are 0, not NaN
      const float ref = m > -INFINITY ? m * scale : 0.0f;
      sum = top > -INFINITY || sum != sum ? sum * exp2_approx(fmaf(top, scale, -ref)) : 0.0f;
      top = m;
      float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < 32; ++j) part[j & 3] += exp2_approx(fmaf(v[j], scale, -ref));
      sum += (part[0] + part[1]) + (part[2] + part[3]);
      continue;
    }
    if (P == kStatsKeep) {
      const float ref = top > -INFINITY ? top * scale : 0.0f;
      float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        v[j] = c + j < valid ? exp2_approx(fmaf(v[j], scale, -ref)) : 0.0f;
        part[j & 3] += v[j];
      }
      sum += (part[0] + part[1]) + (part[2] + part[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        v[j] = c + j < valid && row < live ? weight * exp2_approx(fmaf(v[j], scale, -lse)) : 0.0f;
      if (e.next < first + c + 32) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          while (e.next == first + c + j) {
            v[j] = fmaf(-weight, e.q[e.at], v[j]);
            e.step();
          }
      }
    }
    // the warp's 32 rows, 64 columns to a store
    if (c % 64 == 0) buf = out.open();
    Stager::put(buf, c / 32 & 1, v, 0);
    if (c % 64 == 32) out.close(buf, &p.c[0], t.col0 + c - 32, t.row0 + quarter * 32);
    if (PLANES > 1) {
      // the other parts of these 32 columns, straight to memory
      const int64_t at = (int64_t)row * p.w.grad_ld + t.col0 + c;
#pragma unroll
      for (int part = 1; part < PLANES; ++part) {
        uint4* to = reinterpret_cast<uint4*>(p.w.grad + part * (int64_t)p.g.mpad * p.w.grad_ld + at);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          to[j] = make_uint4(part_pair(v[8 * j], v[8 * j + 1], part), part_pair(v[8 * j + 2], v[8 * j + 3], part),
                             part_pair(v[8 * j + 4], v[8 * j + 5], part), part_pair(v[8 * j + 6], v[8 * j + 7], part));
      }
    }
  }
  if (P != kGradient)
    p.w.part[(int64_t)t.tile * p.g.mpad + row] = make_float2(top > -INFINITY ? top * scale : -INFINITY, sum);
}

__device__ __forceinline__ void finish_dhidden(const GemmArgs& p, const Item& t, int live, uint32_t acc, int quarter) {
  const int row = t.row0 + quarter * 32 + threadIdx.x % 32;
  float* to = p.w.dh + ((int64_t)t.split * p.g.mpad + row) * p.g.dim + t.col0;
  const int valid = min(kBN, p.g.dim - t.col0);
  const bool vec = p.g.dim % 4 == 0;
  float v[32];
  for (int c = 0; c < valid; c += 32) {
    tmem_load32(acc + c, v);
    if (t.k_lo >= t.k_hi)  // a cut without columns: nothing was multiplied
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = 0.0f;
    if (row >= live) continue;
    if (vec) {
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        if (c + j >= valid) break;
        float4* at = reinterpret_cast<float4*>(to + c + j);
        float4 o = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
        if (!p.first) {
          const float4 b = *at;
          o = make_float4(b.x + o.x, b.y + o.y, b.z + o.z, b.w + o.w);
        }
        *at = o;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (c + j < valid) to[c + j] = p.first ? v[j] : to[c + j] + v[j];
    }
  }
}

template <int PLANES>
__device__ __forceinline__ void finish_dweight(const GemmArgs& p, const Item& t, uint32_t acc, int quarter, Stager& out) {
  const int r0 = t.v0 + quarter * 32, row = r0 + threadIdx.x % 32;
  const int rows = p.g.rows[t.shard], valid = min(kBN, p.g.dim - t.col0);
  if (r0 >= rows) return;
  float v[32];
  for (int c = 0; c < valid; c += 64) {
    uint32_t buf = 0;
    if (PLANES == 1 && p.out_map) buf = out.open();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      tmem_load32(acc + c + 32 * h, v);
      if (t.k_hi == 0)  // no live row: nothing was multiplied
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = 0.0f;
      if (PLANES == 1 && p.out_map) {
        Stager::put(buf, h, v, 0);
        continue;
      }
      if (row >= rows) continue;
      const int64_t at = (int64_t)row * p.sh.dw_ld + t.col0 + c + 32 * h;
      if (PLANES == 1) {
        uint16_t* to = static_cast<uint16_t*>(p.sh.dw[t.shard]) + at;
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (c + 32 * h + j < valid) to[j] = (uint16_t)(bf16x2_rn(v[j], 0.0f) & 0xffffu);
      } else {
        float* to = static_cast<float*>(p.sh.dw[t.shard]) + at;
        if (p.out_map && c + 32 * h + 32 <= valid) {
#pragma unroll
          for (int j = 0; j < 32; j += 4)
            *reinterpret_cast<float4*>(to + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (c + 32 * h + j < valid) to[j] = v[j];
        }
      }
    }
    if (PLANES == 1 && p.out_map) out.close(buf, &p.c[t.shard], t.col0 + c, r0);
  }
}

template <int P, int PLANES>
__global__ void __launch_bounds__(kGemmThreads, 1) head_product_kernel(const __grid_constant__ GemmArgs p) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t s_bar[2 * kStages + 5];
  __shared__ uint32_t s_tmem;
  __shared__ int s_gave_up;
  const int live = *p.w.n_live, warp = threadIdx.x / 32;
  const int items = item_count<P>(p, live);
  if ((int)blockIdx.x >= items) return;
  const uint32_t ring = (smem_addr(smem_raw) + 1023) & ~1023u, staging = ring + kStages * kStageBytes;
  const uint32_t full = smem_addr(s_bar), empty = full + 8 * kStages, acc_full = empty + 8 * kStages,
                 acc_empty = acc_full + 16, drain = acc_empty + 16;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      bar_init(full + 8 * i, 1);
      bar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(acc_full + 8 * i, 1);
      bar_init(acc_empty + 8 * i, 4);
    }
    bar_init(drain, 1);
    s_gave_up = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 1) tmem_alloc(smem_addr(&s_tmem), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  if (warp == 0) {
    if (threadIdx.x == 0) produce<P, PLANES>(p, live, ring, full, empty, &s_gave_up);
  } else if (warp == 1) {
    if (threadIdx.x == 32)
      multiply<P, PLANES>(p, live, ring, full, empty, acc_full, acc_empty, drain, tmem, &s_gave_up);
  } else {
    const int quarter = warp % 4;
    Stager out{staging + quarter * 2 * kOutWarpBytes};
    int n = 0;
    for (int i = blockIdx.x; i < items; i += gridDim.x, ++n) {
      const Item t = item_at<P>(p, live, i);
      const int half = n & 1;
      if (!__all_sync(~0u, bar_wait(acc_full + 8 * half, (n >> 1) & 1, &s_gave_up))) break;
      tc_fence_after();
      const uint32_t acc = tmem + half * kBN + ((uint32_t)(quarter * 32) << 16);
      if (P == kDHidden) finish_dhidden(p, t, live, acc, quarter);
      else if (P == kDWeight) finish_dweight<PLANES>(p, t, acc, quarter, out);
      else finish_logits<P, PLANES>(p, t, live, acc, quarter, out);
      tc_fence_before();
      __syncwarp();
      if (threadIdx.x % 32 == 0) bar_arrive(acc_empty + 8 * half);
    }
    if (threadIdx.x % 32 == 0) store_wait_all();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && s_gave_up) atomicOr(&g_head_fault, 2u);
  if (warp == 1) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
}

// ------------------------------------------------------------------ host side --

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return static_cast<EncodeFn>(nullptr);
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

// A bf16 matrix [rows][cols] (row stride ld elements) read or written in boxes of 64 columns.
bool matrix_map(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, int64_t ld, int box_rows) {
  const EncodeFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, unit[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p), dims, strides, box, unit,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int P>
bool maps_for(GemmArgs* a, int dtype) {
  const HeadGeom& g = a->g;
  const HeadWork& w = a->w;
  const int planes = head_planes(dtype);
  const int64_t padded = (int64_t)g.tile0[RELAY_HEAD_MAX_SHARDS] * kHeadTile;
  bool ok = true;
  // the weight: boxes of 256 rows by 64 of dim (logits), or of 64 rows by 64 (d_hidden)
  auto weight = [&](int box_rows) {
    if (w.wpack != nullptr) {
      ok &= matrix_map(&a->b[0], w.wpack, planes * padded, g.dim, w.dim_pad, box_rows);
    } else {
      for (int s = 0; s < g.A; ++s)
        if (g.rows[s] > 0) ok &= matrix_map(&a->b[s], a->sh.w[s], g.rows[s], g.dim, a->sh.w_ld, box_rows);
    }
  };
  const int64_t grad_rows = (int64_t)planes * g.mpad;
  if (P == kDHidden) {
    ok &= matrix_map(&a->a, w.grad, grad_rows, w.grad_ld, w.grad_ld, kBM);
    weight(kBK);
  } else if (P == kDWeight) {
    ok &= matrix_map(&a->a, w.grad, grad_rows, w.grad_ld, w.grad_ld, kBK);
    ok &= matrix_map(&a->b[0], w.hid, grad_rows, g.dim, w.dim_pad, kBK);
    a->out_map = 1;
    for (int s = 0; s < g.A; ++s)
      if (g.rows[s] > 0)
        a->out_map &= reinterpret_cast<uintptr_t>(a->sh.dw[s]) % 16 == 0 && a->sh.dw_ld * esize_of(dtype) % 16 == 0;
    if (planes == 1 && a->out_map)
      for (int s = 0; s < g.A; ++s)
        if (g.rows[s] > 0) ok &= matrix_map(&a->c[s], a->sh.dw[s], g.rows[s], g.dim, a->sh.dw_ld, 32);
  } else {
    ok &= matrix_map(&a->a, w.hid, grad_rows, g.dim, w.dim_pad, kBM);
    weight(kBN);
    if (P != kStats) ok &= matrix_map(&a->c[0], w.grad, grad_rows, w.grad_ld, w.grad_ld, 32);
  }
  return ok;
}

template <int P, int PLANES>
cudaError_t launch(const GemmArgs& a, int64_t items, cudaStream_t s) {
  static thread_local int ready_device = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (ready_device != dev) {
    e = cudaFuncSetAttribute(head_product_kernel<P, PLANES>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    ready_device = dev;
  }
  const int blocks = (int)std::min<int64_t>(items, sm_count());
  head_product_kernel<P, PLANES><<<blocks, kGemmThreads, kSmemBytes, s>>>(a);
  return cudaGetLastError();
}

template <int P>
cudaError_t run(const HeadGeom& g, const HeadWork& w, const HeadShards& sh, int dtype, int lo, int hi, bool first,
                cudaStream_t s) {
  GemmArgs a{};
  a.g = g;
  a.w = w;
  a.sh = sh;
  a.tile_lo = lo;
  a.tile_hi = hi;
  a.first = first;
  // row tiles whose packed hidden rows take 64 MiB, half of L2
  const int64_t mt = g.mpad / kBM, tiles = hi - lo, nd = (g.dim + kBN - 1) / kBN;
  a.group = (int)std::max<int64_t>(1, std::min<int64_t>(mt, (64ll << 20) / ((int64_t)kBM * w.dim_pad * 2 * head_planes(dtype))));
  if (!maps_for<P>(&a, dtype)) return cudaErrorInvalidValue;
  const int64_t items = P == kDHidden ? mt * nd * w.splits : P == kDWeight ? tiles * 2 * nd : mt * tiles;
  if (items > INT_MAX) return cudaErrorInvalidValue;
  return dtype == RELAY_BF16 ? launch<P, 1>(a, items, s) : launch<P, kHeadPlanesF32>(a, items, s);
}

}  // namespace

cudaError_t head_logits(const HeadGeom& g, const HeadWork& w, const HeadShards& sh, int dtype, int tile_lo,
                        int tile_hi, HeadLogits mode, cudaStream_t s) {
  switch (mode) {
    case kHeadStats: return run<kStats>(g, w, sh, dtype, tile_lo, tile_hi, false, s);
    case kHeadStatsKeep: return run<kStatsKeep>(g, w, sh, dtype, tile_lo, tile_hi, false, s);
    default: return run<kGradient>(g, w, sh, dtype, tile_lo, tile_hi, false, s);
  }
}

cudaError_t head_dhidden(const HeadGeom& g, const HeadWork& w, const HeadShards& sh, int dtype, int tile_lo,
                         int tile_hi, bool first, cudaStream_t s) {
  return run<kDHidden>(g, w, sh, dtype, tile_lo, tile_hi, first, s);
}

cudaError_t head_dweight(const HeadGeom& g, const HeadWork& w, const HeadShards& sh, int dtype, int tile_lo,
                         int tile_hi, cudaStream_t s) {
  return run<kDWeight>(g, w, sh, dtype, tile_lo, tile_hi, false, s);
}

int head_splits(const HeadGeom& g, int tiles) {
  const int64_t items = (int64_t)(g.mpad / kBM) * ((g.dim + kBN - 1) / kBN);
  if (items == 0) return 1;
  // as many cuts as one round of the GPU's SMs takes, at least one column tile each
  return (int)std::max<int64_t>(1, std::min<int64_t>(tiles, 152 / items));
}

cudaError_t head_read_fault(unsigned* fault) {
  cudaError_t e = cudaMemcpyFromSymbol(fault, g_head_fault, sizeof *fault);
  if (e != cudaSuccess || *fault == 0) return e;
  const unsigned zero = 0;
  return cudaMemcpyToSymbol(g_head_fault, &zero, sizeof zero);
}

}  // namespace relay
