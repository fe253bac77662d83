// head_rows.cu -- the per-row work around the head's products: the teacher's entries, the
// packing of the live rows, the joining of the tiles' softmax statistics with the loss, and the
// final d_hidden rows. All of it streams; none of it is a visible share of a call whose
// products are large, and for small calls what counts is the number of launches.
#include <limits.h>
#include <math.h>

#include "device.cuh"
#include "head.h"
#include "launch.cuh"

namespace relay {
namespace {

constexpr int kThreadsRows = 256;

__device__ __forceinline__ float load_as_f32(const float* p) { return *p; }
__device__ __forceinline__ float load_as_f32(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
__device__ __forceinline__ void store_from_f32(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_from_f32(uint16_t* p, float v) {
  *p = (uint16_t)(bf16x2_rn(v, 0.0f) & 0xffffu);
}

// Padded column of a vocabulary id, or INT32_MAX when the id is outside the vocabulary.
__device__ __forceinline__ int column_of(const HeadGeom& g, int id) {
  if (id < 0 || id >= g.vocab) return INT_MAX;
  int a = 0;
  while (a + 1 < g.A && id >= g.base[a + 1]) ++a;
  return g.tile0[a] * kHeadTile + (id - g.base[a]);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// The three bf16 parts of an fp32 value; an infinity or NaN is its first part alone. Every part multiplies parts of
// the other operand (six of the nine products), so what one product says about infinities the others must not
// contradict: a logit that is -inf has to come out as -inf, not as NaN.
//
// `below`: each part is the largest bf16 value below what is left, so that all parts have the value's sign and none
// is 0 (for a value of 2^-95 at least, whose third part bf16 still holds). Their sum is the value exactly. Hidden is
// always split so: its parts times an infinite weight, or parts of products that leave fp32's range, are infinite with one
// sign, and a hidden value of 0 times an infinite weight is NaN as it should be. A weight is split so
// from 512 on. Smaller ones are rounded: the second part of a weight below 512 is at most 1 and brings no product out of
// range by itself, and rounded parts keep what the three left-out products amount to at 1.5e-7 of a product (both operands
// split below: 4e-7, and always towards 0).
template <bool HIDDEN>
__device__ __forceinline__ void parts_of(float v, uint16_t (&o)[3]) {
  const uint32_t u = __float_as_uint(v), size = u & 0x7fffffffu;
  if (size >= 0x7f800000u) {
    o[0] = (uint16_t)((v != v ? u | 0x00400000u : u) >> 16);
    o[1] = o[2] = 0;
    return;
  }
  const bool below = HIDDEN || size >= 0x44000000u;  // 512
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const uint32_t bits = __float_as_uint(v);
    uint32_t r = bf16x2_rn(v, 0.0f) << 16;
    if (i < 2 && below) r = (bits & 0x7fffffffu) == 0 ? bits : (bits - 1) & 0xffff0000u;
    o[i] = (uint16_t)(r >> 16);
    v = __fsub_rn(v, __uint_as_float(r));
  }
}

// A warp copies one row to its packed place: bf16 as it is, fp32 in three parts, `plane` elements
// apart. Columns from dim to pad, and all of them when from is NULL, are 0. vec: 16-byte loads.
template <bool HIDDEN>
__device__ __forceinline__ void pack_row(uint16_t* to, int64_t, const uint16_t* from, int dim, int pad, bool vec) {
  const int lane = threadIdx.x % 32;
  if (from != nullptr && !vec) {
    // rows off the 16-byte grid: each output vector out of the two aligned blocks that hold it (a block
    // is read only where it holds bytes of the row)
    const uintptr_t at = reinterpret_cast<uintptr_t>(from);
    const unsigned shift = at & 15u;
    const unsigned char* base = reinterpret_cast<const unsigned char*>(at - shift);
    const int bytes = dim * 2 + (int)shift;
    for (int v = lane; v < pad / 8; v += 32) {
      const uint4 lo = v * 16 < bytes ? ld_once(base + v * 16) : make_uint4(0, 0, 0, 0);
      const uint4 hi = shift != 0 && v * 16 + 16 < bytes ? ld_once(base + v * 16 + 16) : make_uint4(0, 0, 0, 0);
      uint4 x = shift_pair(lo, hi, shift);
      if (v * 8 + 8 > dim) {  // past the row: 0
        uint16_t e[8];
        memcpy(e, &x, 16);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (v * 8 + i >= dim) e[i] = 0;
        memcpy(&x, e, 16);
      }
      reinterpret_cast<uint4*>(to)[v] = x;
    }
    return;
  }
  const int vecs = from == nullptr ? pad / 8 : dim / 8;
  for (int v0 = lane; v0 < vecs; v0 += 4 * 32) {
    uint4 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[i] = from != nullptr && v0 + 32 * i < vecs ? ld_once(from + (v0 + 32 * i) * 8) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (v0 + 32 * i < vecs) reinterpret_cast<uint4*>(to)[v0 + 32 * i] = x[i];
  }
  for (int d = vecs * 8 + lane; d < pad; d += 32) to[d] = d < dim ? from[d] : (uint16_t)0;
}
template <bool HIDDEN>
__device__ __forceinline__ void pack_row(uint16_t* to, int64_t plane, const float* from, int dim, int pad, bool vec) {
  const int lane = threadIdx.x % 32;
  for (int d0 = lane * 8; d0 < pad; d0 += 8 * 32) {  // pad is a multiple of 8
    float x[8];
    if (from != nullptr && vec && d0 + 8 <= dim) {
      TF32::unpack(ld_once(from + d0), x);
      TF32::unpack(ld_once(from + d0 + 4), x + 4);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = from != nullptr && d0 + i < dim ? from[d0 + i] : 0.0f;
    }
    uint16_t o[8][3];
#pragma unroll
    for (int i = 0; i < 8; ++i) parts_of<HIDDEN>(x[i], o[i]);
#pragma unroll
    for (int k = 0; k < 3; ++k)
      *reinterpret_cast<uint4*>(to + k * plane + d0) =
          make_uint4(o[0][k] | (uint32_t)o[1][k] << 16, o[2][k] | (uint32_t)o[3][k] << 16,
                     o[4][k] | (uint32_t)o[5][k] << 16, o[6][k] | (uint32_t)o[7][k] << 16);
  }
}
template <class T>
__device__ __forceinline__ void zero_row(T* to, int n) {
  for (int d = threadIdx.x % 32; d < n; d += 32) store_from_f32(to + d, 0.0f);
}

// The padded weight: one warp per padded row.
template <class T>
__global__ void __launch_bounds__(kThreadsRows)
    pack_weight_kernel(const HeadGeom g, const HeadWork w, const HeadShards sh, int vec) {
  dep_launch();
  dep_wait();
  const int rows = g.tile0[RELAY_HEAD_MAX_SHARDS] * kHeadTile;
  const int row = blockIdx.x * (kThreadsRows / 32) + threadIdx.x / 32;  // rows: a multiple of 256
  const int a = head_shard_of_tile(g, row / kHeadTile), v = row - g.tile0[a] * kHeadTile;
  const T* from = v < g.rows[a] ? static_cast<const T*>(sh.w[a]) + v * sh.w_ld : nullptr;
  pack_row<false>(w.wpack + (int64_t)row * w.dim_pad, (int64_t)rows * w.dim_pad, from, g.dim, w.dim_pad, vec);
}

// One warp per row: the entries' columns in ascending order (by counting, each lane holds up to
// four), and the teacher's probabilities beside them. An id given twice keeps two entries. Returns whether
// the row takes part.
template <class T>
__device__ __forceinline__ bool teacher_row(const HeadGeom& g, const HeadWork& w, const T* logits, const int32_t* index,
                                            int row) {
  constexpr int kPer = RELAY_HEAD_MAX_TOP / 32;
  const int lane = threadIdx.x % 32;
  const int64_t at = (int64_t)row * g.top;
  int col[kPer], rank[kPer];
  float s[kPer];
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane + 32 * i;
    col[i] = e < g.top ? column_of(g, index[at + e]) : INT_MAX;
    // an absent entry's logit is not looked at
    s[i] = col[i] != INT_MAX ? load_as_f32(logits + at + e) : -INFINITY;
    top = fmaxf(top, s[i]);
    rank[i] = 0;
  }
  top = warp_max(top);
  bool nan = false;
#pragma unroll
  for (int i = 0; i < kPer; ++i) nan |= s[i] != s[i];
  nan = __any_sync(~0u, nan);
  const bool live = nan || top > -INFINITY;
  float sum = 0.0f, q[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    // the maximum first, then the temperature: the type's lowest value over a temperature below 1
    // would be -inf
    q[i] = live && col[i] != INT_MAX ? expf((s[i] - top) * g.inv_tau) : 0.0f;
    sum += q[i];
  }
  sum = warp_sum(sum);
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    if (32 * j >= g.top) break;
    for (int l = 0; l < 32; ++l) {
      const int other = __shfl_sync(~0u, col[j], l), e = l + 32 * j;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        rank[i] += other < col[i] || (other == col[i] && e < lane + 32 * i);
    }
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (lane + 32 * i >= g.top) continue;
    w.ent_col[at + rank[i]] = col[i];
    w.ent_q[at + rank[i]] = live ? q[i] / sum : 0.0f;
  }
  return live;
}
template <class T>
__global__ void __launch_bounds__(kThreadsRows) teacher_kernel(const HeadGeom g, const HeadWork w,
                                                               const T* logits, const int32_t* index) {
  dep_launch();
  dep_wait();
  const int row = blockIdx.x * (kThreadsRows / 32) + threadIdx.x / 32;
  if (row >= g.tokens) return;
  const bool live = teacher_row(g, w, logits, index, row);
  if (threadIdx.x % 32 == 0) w.live[row] = live;
}

// Where a row's flag comes from: its target; teacher_kernel; or, in a small batch of few entries, its entries,
// which every block then reads itself: a launch less.
enum RowSource { kFromTarget, kFromFlag, kFromEntries };
constexpr int kEntriesTop = 16, kEntriesTokens = 512;

template <RowSource SOURCE, class TT>
__device__ __forceinline__ bool row_live(const HeadGeom& g, const HeadWork& w, const int32_t* index, const TT* teacher,
                                         int row) {
  if (SOURCE == kFromFlag) return w.live[row] != 0;
  if (SOURCE == kFromEntries) {
    bool live = false;
#pragma unroll
    for (int k = 0; k < kEntriesTop; ++k) {
      if (k >= g.top) break;
      const int id = index[row * g.top + k];
      const float t = load_as_f32(teacher + row * g.top + k);
      live |= id >= 0 && id < g.vocab && !(t == -INFINITY);  // a NaN is an entry
    }
    return live;
  }
  const int t = index[row];
  return t >= 0 && t < g.vocab;
}

// A block owns `per` consecutive rows. It counts the live rows before them itself (a read of
// every row's flag, from L2: no second launch, no order between blocks; 8 us at 2047 rows, 161 us at 131072,
// which counts only beside products of few columns), then a warp per row
// copies the live ones to their packed places and zeroes the places the others leave free
// behind the last live row, as far as products read them. Ignored rows get loss 0 and d_hidden 0.
template <class T, RowSource SOURCE, class TT>
__global__ void __launch_bounds__(kThreadsRows)
    pack_kernel(const HeadGeom g, const HeadWork w, const T* hidden, int64_t ld, const int32_t* index,
                const TT* teacher, const float* row_weight, float* loss, T* dh, int64_t dh_ld, int per, int vec) {
  constexpr int kWarps = kThreadsRows / 32;
  __shared__ int s_before, s_total, s_warp[kWarps], s_place[kThreadsRows];
  dep_launch();
  dep_wait();
  const int lo = blockIdx.x * per, hi = min(lo + per, g.tokens), lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  if (threadIdx.x == 0) s_before = s_total = 0;
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll 4
  for (int r = threadIdx.x; r < g.tokens; r += kThreadsRows) {
    const int live = row_live<SOURCE>(g, w, index, teacher, r);
    total += live;
    before += r < lo ? live : 0;
  }
  before = __reduce_add_sync(~0u, before);
  total = __reduce_add_sync(~0u, total);
  if (lane == 0) {
    atomicAdd(&s_before, before);  // integers: any order gives the same sum
    atomicAdd(&s_total, total);
  }
  __syncthreads();
  total = s_total;
  int packed = s_before;  // live rows before row `base`
  const int row_tile = head_row_tile(g), read_end = (total + row_tile - 1) / row_tile * row_tile;
  if (blockIdx.x == 0 && warp == 0) {
    const int cuts = head_cuts(g, w, total);
    if (lane == 0) {
      w.n_live[0] = total;
      w.n_live[1] = cuts;
    }
  }
  const int64_t plane = (int64_t)g.mpad * w.dim_pad;
  for (int base = lo; base < hi; base += kThreadsRows) {
    const int mine = base + threadIdx.x;
    const bool live = mine < hi && row_live<SOURCE>(g, w, index, teacher, mine);
    const unsigned votes = __ballot_sync(~0u, live);
    if (lane == 0) s_warp[warp] = __popc(votes);
    __syncthreads();
    int ahead = packed + __popc(votes & ((1u << lane) - 1));
    for (int i = 0; i < warp; ++i) ahead += s_warp[i];
    for (int i = 0; i < kWarps; ++i) packed += s_warp[i];
    if (mine < hi) {
      const int place = live ? ahead : total + (mine - ahead);
      s_place[threadIdx.x] = live ? place : ~place;
      w.perm[place] = mine;
      w.wrow[place] = live ? (row_weight ? row_weight[mine] : 1.0f) * g.tau : 0.0f;
      if (!live) loss[mine] = 0.0f;
      if (SOURCE == kFromTarget && live) {
        w.ent_col[mine] = column_of(g, index[mine]);
        w.ent_q[mine] = 1.0f;
      }
    }
    __syncthreads();
    for (int i = warp; base + i < hi && i < kThreadsRows; i += kWarps) {
      const int r = base + i, place = s_place[i];
      if (SOURCE == kFromEntries) teacher_row(g, w, teacher, index, r);
      if (place >= 0) {
        pack_row<true>(w.hid + (int64_t)place * w.dim_pad, plane, hidden + r * ld, g.dim, w.dim_pad, vec);
      } else {
        if (dh != nullptr) zero_row(dh + r * dh_ld, g.dim);
        if (~place < read_end)
          pack_row<true>(w.hid + (int64_t)~place * w.dim_pad, plane, static_cast<const T*>(nullptr), g.dim, w.dim_pad, vec);
      }
    }
    __syncthreads();
  }
  // places past the last row of the batch
  for (int place = g.tokens + blockIdx.x * kWarps + warp; place < g.mpad; place += gridDim.x * kWarps) {
    if (lane == 0) {
      w.perm[place] = 0;
      w.wrow[place] = 0.0f;
    }
    if (place < read_end)
      pack_row<true>(w.hid + (int64_t)place * w.dim_pad, plane, static_cast<const T*>(nullptr), g.dim, w.dim_pad, vec);
  }
}

// Joins the (max, sum) of a row's columns into its log-sum-exp and writes its loss. A block takes
// 32 rows: lanes are rows (the statistics of the same columns are contiguous over rows), warps
// stride over the columns and join in shared memory, in a fixed order. Then a warp per row sums
// its entries.
constexpr int kCombineWarps = 32;
__device__ __forceinline__ void join(float& m, float& s, float pm, float ps, float scale) {
  const float top = fmaxf(m, pm);
  // -inf - -inf: a side that holds nothing yet adds nothing
  s = (m > -INFINITY || s != s ? s * exp2f((m - top) * scale) : 0.0f) +
      (pm > -INFINITY || ps != ps ? ps * exp2f((pm - top) * scale) : 0.0f);
  m = top;
}
// Joins the lanes' shares; every lane gets the row's largest logit and the log2 of its sum.
__device__ __forceinline__ float2 join_warp(float m, float s, float scale) {
  const int lane = threadIdx.x % 32;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float pm = __shfl_xor_sync(~0u, m, o), ps = __shfl_xor_sync(~0u, s, o);
    // both sides of a pair join in the same order: the lower lane's share first
    float am = lane & o ? pm : m, as = lane & o ? ps : s;
    join(am, as, lane & o ? m : pm, lane & o ? s : ps, scale);
    m = am;
    s = as;
  }
  return make_float2(m, log2f(s));
}
// The loss of a packed row, by one warp.
template <bool DISTILL>
__device__ __forceinline__ void row_loss(const HeadGeom& g, const HeadWork& w, int row, float2 lse, float* loss) {
  const int lane = threadIdx.x % 32, r = w.perm[row];
  const float log_sum = lse.y * 0.6931471805599453f;
  const int64_t at = (int64_t)r * g.top;
  if (!DISTILL) {
    if (lane == 0) loss[r] = (lse.x - w.ent_z[at]) + log_sum;
    return;
  }
  float sum = 0.0f;
  for (int k = lane; k < g.top; k += 32) {
    const float q = w.ent_q[at + k];
    if (w.ent_col[at + k] != INT_MAX && q != 0.0f)  // 0 log 0 = 0
      sum += q * (logf(q) + ((lse.x - w.ent_z[at + k]) * g.inv_tau + log_sum));
  }
  sum = warp_sum(sum);
  if (lane == 0) loss[r] = g.tau * g.tau * sum;
}
template <bool DISTILL>
__global__ void __launch_bounds__(32 * kCombineWarps) combine_kernel(const HeadGeom g, const HeadWork w, float* loss) {
  __shared__ float s_max[kCombineWarps][33], s_sum[kCombineWarps][33];
  dep_launch();
  dep_wait();
  const int live = *w.n_live, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int row = blockIdx.x * 32 + lane, parts = g.tile0[RELAY_HEAD_MAX_SHARDS] * (kHeadTile / kHeadStatTile);
  if ((int)blockIdx.x * 32 >= live) return;
  const float scale = head_log2_scale(g);
  float m = -INFINITY, s = 0.0f;
  if (row < live)
    for (int t = warp; t < parts; t += 4 * kCombineWarps) {
      float2 p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        p[i] = t + i * kCombineWarps < parts ? w.part[(int64_t)(t + i * kCombineWarps) * g.mpad + row]
                                             : make_float2(-INFINITY, 0.0f);
#pragma unroll
      for (int i = 0; i < 4; ++i) join(m, s, p[i].x, p[i].y, scale);
    }
  s_max[warp][lane] = m;
  s_sum[warp][lane] = s;
  __syncthreads();
  // warp i takes row i: lanes are the warps' shares
  const int mine = blockIdx.x * 32 + warp;
  if (mine >= live) return;
  const float2 lse = join_warp(s_max[lane][warp], s_sum[lane][warp], scale);
  if (lane == 0) w.lse[mine] = lse;
  row_loss<DISTILL>(g, w, mine, lse, loss);
}

// Kept exponentials to the gradient of the logits, in place: each is relative to the maximum of
// its columns, so the difference to the row's log-sum-exp makes it a probability. The
// entries' columns are computed from their fp32 logits instead: p - 1 of a confident row
// would otherwise be the rounding error of p. A block takes 8192 columns of a row (kScaleCols); rows after the
// live ones, as far as products read them, become 0.
constexpr int kScaleVecs = 4;  // 16-byte vectors in flight per thread and plane
constexpr int kScaleCols = kThreadsRows * 8 * kScaleVecs;
static_assert(RELAY_HEAD_MAX_TOP <= kThreadsRows && kScaleCols % (32 * kHeadStatTile) == 0, "an entry per thread; whole shares");
// JOIN 1 (cross entropy), 2 (distillation): the block has the whole row, and does combine_kernel's
// work for it first.
template <int PLANES, int JOIN>
__global__ void __launch_bounds__(kThreadsRows) scale_kernel(const HeadGeom g, const HeadWork w, float* loss) {
  __shared__ float2 s_lse;
  dep_launch();
  dep_wait();
  const int row = blockIdx.x, col0 = blockIdx.y * kScaleCols;
  const int cols = g.tile0[RELAY_HEAD_MAX_SHARDS] * kHeadTile;
  const int64_t plane = (int64_t)g.mpad * w.grad_ld;
  uint16_t* line = w.grad + (int64_t)row * w.grad_ld;
  // everything is asked for before anything is waited for: all of it lies inside the workspace,
  // whether the row is live or not
  uint4 in[kScaleVecs][PLANES];
  float ref[kScaleVecs];
#pragma unroll
  for (int k = 0; k < kScaleVecs; ++k) {
    const int col = col0 + (k * kThreadsRows + threadIdx.x) * 8;
    if (col >= cols) continue;
#pragma unroll
    for (int i = 0; i < PLANES; ++i) in[k][i] = ld_once(line + i * plane + col);
    ref[k] = w.part[(int64_t)(col / kHeadStatTile) * g.mpad + row].x;
  }
  constexpr int kShares = kScaleCols / kHeadStatTile / 32;  // statistics of a whole row, per lane
  float2 share[kShares];
  if (JOIN != 0 && threadIdx.x < 32) {
#pragma unroll
    for (int i = 0; i < kShares; ++i) {
      const int t = threadIdx.x + 32 * i;
      share[i] = t < cols / kHeadStatTile ? w.part[(int64_t)t * g.mpad + row] : make_float2(-INFINITY, 0.0f);
    }
  }
  const int live = *w.n_live, row_tile = head_row_tile(g);
  const int64_t at = (int64_t)w.perm[row] * g.top;
  const bool on = row < live;
  const float weight = w.wrow[row], scale = head_log2_scale(g);
  float2 lse = JOIN == 0 ? w.lse[row] : make_float2(0.0f, 0.0f);
  if (row >= (live + row_tile - 1) / row_tile * row_tile) return;
  // the thread's entry, if any: at most RELAY_HEAD_MAX_TOP of them
  const bool has = on && (int)threadIdx.x < g.top;
  const int ent_col = has ? w.ent_col[at + threadIdx.x] : INT_MAX;
  const float ent_z = has && ent_col != INT_MAX ? w.ent_z[at + threadIdx.x] : 0.0f;
  if (JOIN != 0 && on) {
    if (threadIdx.x < 32) {
      float m = -INFINITY, s = 0.0f;
#pragma unroll
      for (int i = 0; i < kShares; ++i) join(m, s, share[i].x, share[i].y, scale);
      const float2 all = join_warp(m, s, scale);
      if (threadIdx.x == 0) s_lse = all;
    }
    __syncthreads();
    lse = s_lse;
    if (threadIdx.x >= kThreadsRows - 32) row_loss<JOIN == 2>(g, w, row, lse, loss);
  }
#pragma unroll
  for (int k = 0; k < kScaleVecs; ++k) ref[k] = fmaf(ref[k] - lse.x, scale, -lse.y);
#pragma unroll
  for (int k = 0; k < kScaleVecs; ++k) {
    const int col = col0 + (k * kThreadsRows + threadIdx.x) * 8;
    if (col >= cols) continue;
    float v[8];
    if (!on) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0.0f;
    } else if (PLANES == 1) {
      const uint32_t word[4] = {in[k][0].x, in[k][0].y, in[k][0].z, in[k][0].w};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // the code as a float: 2^23 + code has it in its low bits
        const uint32_t code = j & 1 ? word[j / 2] >> 16 : word[j / 2] & 0xffffu;
        const float steps = __fsub_rn(__uint_as_float(0x4b000000u | code), 8388608.0f);
        const float p = weight * exp2_approx(fmaf(steps, -1.0f / kCodeSteps, ref[k]));
        v[j] = steps < kCodeZero || ref[k] != ref[k] ? p : 0.0f;
      }
    } else {
      const float f = weight * exp2f(ref[k]);
      float x[8], y[8];
      TBF16::unpack(in[k][0], v);
      TBF16::unpack(in[k][PLANES > 1 ? 1 : 0], x);
      TBF16::unpack(in[k][PLANES > 1 ? 2 : 0], y);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = __fadd_rn(__fadd_rn(y[j], x[j]), v[j]) * f;
    }
    for (int i = 0; i < w.grad_planes; ++i) {
      const uint4 out = TBF16::pack(v);
      *reinterpret_cast<uint4*>(line + i * plane + col) = out;
      if (i + 1 == w.grad_planes) break;
      float r[8];
      TBF16::unpack(out, r);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = __fsub_rn(v[j], r[j]);
    }
  }
  if (!on) return;
  __syncthreads();
  {
    const int k = threadIdx.x, c = ent_col;
    if (c < col0 || c >= col0 + kScaleCols || c >= cols || (k > 0 && w.ent_col[at + k - 1] == c)) return;
    float q = 0.0f;  // an id given several times: its first entry sums them
    for (int j = k; j < g.top && w.ent_col[at + j] == c; ++j) q += w.ent_q[at + j];
    float v = weight * (exp2f(fmaf(ent_z - lse.x, scale, -lse.y)) - q);
    for (int i = 0; i < w.grad_planes; ++i) {
      const uint32_t r = bf16x2_rn(v, 0.0f) & 0xffffu;
      line[i * plane + c] = (uint16_t)r;
      v = __fsub_rn(v, __uint_as_float(r << 16));
    }
  }
}

// Sums the cuts of d_hidden in order and puts each row where it belongs. Rows whose d_hidden the
// product wrote itself (one cut, one piece) need nothing.
template <class T>
__global__ void __launch_bounds__(kThreadsRows)
    write_dh_kernel(const HeadGeom g, const HeadWork w, T* dh, int64_t ld, int vec) {
  dep_launch();
  dep_wait();
  const int live = w.n_live[0], cuts = w.n_live[1];
  if (w.whole && cuts == 1) return;
  const int64_t cut = (int64_t)g.mpad * w.dh_ld;
  constexpr int kLanes = 4;
  const int64_t vecs = vec ? (int64_t)live * (g.dim / kLanes) : 0;
  const int64_t first = (int64_t)blockIdx.x * kThreadsRows + threadIdx.x, stride = (int64_t)gridDim.x * kThreadsRows;
  for (int64_t i = first; i < vecs; i += stride) {
    const int row = (int)(i / (g.dim / kLanes)), d = (int)(i % (g.dim / kLanes)) * kLanes;
    const float* from = w.dh + (int64_t)row * w.dh_ld + d;
    float4 sum = *reinterpret_cast<const float4*>(from);
#pragma unroll 8
    for (int c = 1; c < cuts; ++c) {
      const float4 x = *reinterpret_cast<const float4*>(from + c * cut);
      sum = make_float4(sum.x + x.x, sum.y + x.y, sum.z + x.z, sum.w + x.w);
    }
    T* to = dh + (int64_t)w.perm[row] * ld + d;
    if (sizeof(T) == 2)
      *reinterpret_cast<uint2*>(to) = make_uint2(bf16x2_rn(sum.x, sum.y), bf16x2_rn(sum.z, sum.w));
    else
      *reinterpret_cast<float4*>(to) = sum;
  }
  if (vec) return;
  for (int64_t i = first; i < (int64_t)live * g.dim; i += stride) {
    const int row = (int)(i / g.dim), d = (int)(i % g.dim);
    const float* from = w.dh + (int64_t)row * w.dh_ld + d;
    float sum = from[0];
#pragma unroll 4
    for (int c = 1; c < cuts; ++c) sum += from[c * cut];
    store_from_f32(dh + (int64_t)w.perm[row] * ld + d, sum);
  }
}

int ceil_div(int a, int b) { return (int)(((int64_t)a + b - 1) / b); }
int64_t esize(int dtype) { return dtype == RELAY_BF16 ? 2 : 4; }

}  // namespace

cudaError_t head_teacher(const HeadGeom& g, const HeadWork& w, const void* teacher, int teacher_dtype,
                         const int32_t* index, cudaStream_t s) {
  if (g.top <= kEntriesTop && g.tokens <= kEntriesTokens) return cudaSuccess;  // the packing does it
  const int blocks = ceil_div(g.tokens, kThreadsRows / 32);
  if (teacher_dtype == RELAY_BF16)
    return launch_chained(teacher_kernel<uint16_t>, blocks, kThreadsRows, 0, s, g, w,
                          static_cast<const uint16_t*>(teacher), index);
  return launch_chained(teacher_kernel<float>, blocks, kThreadsRows, 0, s, g, w, static_cast<const float*>(teacher),
                        index);
}

template <class T, class TT>
static cudaError_t pack_typed(const HeadGeom& g, const HeadWork& w, const void* hidden, int64_t ld,
                              const int32_t* index, const void* teacher, const float* row_weight, float* loss,
                              void* dh, int64_t dh_ld, cudaStream_t s) {
  // a warp per row; at most 2048 blocks read every row's flag
  constexpr int kWarps = kThreadsRows / 32;
  const int per = ceil_div(ceil_div(g.tokens, 2048), kWarps) * kWarps;
  // (a few more for a small batch: they zero the places past it)
  const int pad = ceil_div(head_row_tile(g), kWarps), blocks = ceil_div(g.tokens, per) > pad ? ceil_div(g.tokens, per) : pad;
  const int vec = reinterpret_cast<uintptr_t>(hidden) % 16 == 0 && ld * sizeof(T) % 16 == 0;
  auto* kernel = teacher == nullptr ? pack_kernel<T, kFromTarget, TT>
                 : g.top <= kEntriesTop && g.tokens <= kEntriesTokens ? pack_kernel<T, kFromEntries, TT>
                                                                      : pack_kernel<T, kFromFlag, TT>;
  return launch_chained(kernel, blocks, kThreadsRows, 0, s, g, w, static_cast<const T*>(hidden), ld, index,
                        static_cast<const TT*>(teacher), row_weight, loss, static_cast<T*>(dh), dh_ld, per, vec);
}

cudaError_t head_pack(const HeadGeom& g, const HeadWork& w, int dtype, const void* hidden, int64_t hidden_ld,
                      const int32_t* index, const void* teacher, int teacher_dtype, const float* row_weight,
                      float* loss, void* d_hidden, int64_t d_hidden_ld, cudaStream_t s) {
  if (dtype == RELAY_BF16)
    return teacher_dtype == RELAY_BF16
               ? pack_typed<uint16_t, uint16_t>(g, w, hidden, hidden_ld, index, teacher, row_weight, loss, d_hidden, d_hidden_ld, s)
               : pack_typed<uint16_t, float>(g, w, hidden, hidden_ld, index, teacher, row_weight, loss, d_hidden, d_hidden_ld, s);
  return teacher_dtype == RELAY_BF16
             ? pack_typed<float, uint16_t>(g, w, hidden, hidden_ld, index, teacher, row_weight, loss, d_hidden, d_hidden_ld, s)
             : pack_typed<float, float>(g, w, hidden, hidden_ld, index, teacher, row_weight, loss, d_hidden, d_hidden_ld, s);
}

cudaError_t head_pack_weight(const HeadGeom& g, const HeadWork& w, const HeadShards& sh, int dtype, cudaStream_t s) {
  const int blocks = g.tile0[RELAY_HEAD_MAX_SHARDS] * kHeadTile / (kThreadsRows / 32);
  int vec = sh.w_ld * esize(dtype) % 16 == 0;
  for (int a = 0; a < g.A; ++a)
    if (g.rows[a] > 0) vec &= reinterpret_cast<uintptr_t>(sh.w[a]) % 16 == 0;
  return launch_chained(dtype == RELAY_BF16 ? pack_weight_kernel<uint16_t> : pack_weight_kernel<float>, blocks,
                        kThreadsRows, 0, s, g, w, sh, vec);
}

cudaError_t head_combine(const HeadGeom& g, const HeadWork& w, bool distill, float* loss, cudaStream_t s) {
  return launch_chained(distill ? combine_kernel<true> : combine_kernel<false>, ceil_div(g.tokens, 32),
                        32 * kCombineWarps, 0, s, g, w, loss);
}

bool head_scale_fits(const HeadGeom& g) { return ceil_div(g.tile0[RELAY_HEAD_MAX_SHARDS] * kHeadTile, kScaleCols) <= 65535; }
bool head_scale_joins(const HeadGeom& g) { return g.tile0[RELAY_HEAD_MAX_SHARDS] * kHeadTile <= kScaleCols; }

template <int PLANES>
static cudaError_t scale_typed(const HeadGeom& g, const HeadWork& w, bool distill, float* loss, cudaStream_t s) {
  const dim3 grid(g.mpad, ceil_div(g.tile0[RELAY_HEAD_MAX_SHARDS] * kHeadTile, kScaleCols));  // a piece is bounded
  auto* kernel = !head_scale_joins(g) ? scale_kernel<PLANES, 0> : distill ? scale_kernel<PLANES, 2> : scale_kernel<PLANES, 1>;
  return launch_chained(kernel, grid, kThreadsRows, 0, s, g, w, loss);
}
cudaError_t head_scale(const HeadGeom& g, const HeadWork& w, int dtype, bool distill, float* loss, cudaStream_t s) {
  return dtype == RELAY_BF16 ? scale_typed<1>(g, w, distill, loss, s) : scale_typed<kHeadPlanesF32>(g, w, distill, loss, s);
}

cudaError_t head_write_dh(const HeadGeom& g, const HeadWork& w, int dtype, void* d_hidden,
                          int64_t d_hidden_ld, cudaStream_t s) {
  const int64_t work = (int64_t)g.tokens * ceil_div(g.dim, 4);
  const int blocks = (int)(work < 2432ll * kThreadsRows ? (work + kThreadsRows - 1) / kThreadsRows : 2432);  // 16 per SM
  const int vec = g.dim % 4 == 0 && d_hidden_ld % 4 == 0 &&
                  reinterpret_cast<uintptr_t>(d_hidden) % (4 * esize(dtype)) == 0;
  if (dtype == RELAY_BF16)
    return launch_chained(write_dh_kernel<uint16_t>, blocks, kThreadsRows, 0, s, g, w, static_cast<uint16_t*>(d_hidden),
                          d_hidden_ld, vec);
  return launch_chained(write_dh_kernel<float>, blocks, kThreadsRows, 0, s, g, w, static_cast<float*>(d_hidden),
                        d_hidden_ld, vec);
}

}  // namespace relay
