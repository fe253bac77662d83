// head_rows.cu -- the per-row work around the head's products: the teacher's entries, the
// packing of the live rows, the joining of the tiles' softmax statistics with the loss, and the
// final d_hidden rows. All of it streams; none of it is a visible share of a call whose
// products are large, and for small calls what counts is the number of launches.
#include <limits.h>
#include <math.h>

#include "device.cuh"
#include "head.h"

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

// The three bf16 parts of an fp32 value. A value that rounds to infinity is cut instead, and an
// infinity or NaN is its first part alone.
__device__ __forceinline__ void parts_of(float v, uint16_t (&o)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    uint32_t r = bf16x2_rn(v, 0.0f) << 16;
    if ((r & 0x7f800000u) == 0x7f800000u && v == v) r = __float_as_uint(v) & 0xffff0000u;
    o[i] = (uint16_t)(r >> 16);
    const float left = __fsub_rn(v, __uint_as_float(r));
    v = (r & 0x7f800000u) == 0x7f800000u ? 0.0f : left;
  }
}

// Copies one row to its packed place: bf16 as it is, fp32 in three parts, `plane` elements apart.
// Columns from dim to pad, and all of them when from is NULL, are 0.
__device__ __forceinline__ void pack_row(uint16_t* to, int64_t, const uint16_t* from, int dim, int pad, bool vec) {
  const int whole_vecs = from != nullptr && vec ? dim / 8 : 0;
  for (int v = threadIdx.x; v < whole_vecs; v += kThreadsRows)
    reinterpret_cast<uint4*>(to)[v] = ld_stream_v4(from + v * 8);
  for (int d = whole_vecs * 8 + threadIdx.x; d < pad; d += kThreadsRows)
    to[d] = from != nullptr && d < dim ? from[d] : (uint16_t)0;
}
__device__ __forceinline__ void pack_row(uint16_t* to, int64_t plane, const float* from, int dim, int pad, bool) {
  for (int d = threadIdx.x; d < pad; d += kThreadsRows) {
    uint16_t o[3] = {0, 0, 0};
    if (from != nullptr && d < dim) parts_of(from[d], o);
#pragma unroll
    for (int i = 0; i < 3; ++i) to[i * plane + d] = o[i];
  }
}

// The padded weight: one block per padded row.
template <class T>
__global__ void __launch_bounds__(kThreadsRows) pack_weight_kernel(const HeadGeom g, const HeadWork w, const HeadShards sh) {
  const int row = blockIdx.x, a = head_shard_of_tile(g, row / kHeadTile), v = row - g.tile0[a] * kHeadTile;
  const T* from = v < g.rows[a] ? static_cast<const T*>(sh.w[a]) + v * sh.w_ld : nullptr;
  pack_row(w.wpack + (int64_t)row * w.dim_pad, (int64_t)gridDim.x * w.dim_pad, from, g.dim, w.dim_pad, false);
}

// One warp per row: the entries' columns in ascending order (by counting, each lane holds up to
// four), and the teacher's probabilities beside them. An id given twice keeps two entries.
template <class T>
__global__ void __launch_bounds__(kThreadsRows) teacher_kernel(const HeadGeom g, const HeadWork w,
                                                               const T* logits, const int32_t* index) {
  constexpr int kPer = RELAY_HEAD_MAX_TOP / 32;
  const int row = blockIdx.x * (kThreadsRows / 32) + threadIdx.x / 32, lane = threadIdx.x % 32;
  if (row >= g.tokens) return;
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
  if (lane == 0) w.live[row] = live;
}

template <bool DISTILL>
__device__ __forceinline__ bool row_live(const HeadGeom& g, const HeadWork& w, const int32_t* targets, int row) {
  if (DISTILL) return w.live[row] != 0;
  const int t = targets[row];
  return t >= 0 && t < g.vocab;
}

// A block owns `per` consecutive rows. It counts the live rows before them itself (a read of
// every row's flag, from L2: no second launch, no order between blocks), then copies its live
// rows to their packed places and zeroes the places its other rows leave free behind the last
// live row, as far as products read them. Ignored rows get loss 0 and d_hidden 0 here.
template <class T, bool DISTILL>
__global__ void __launch_bounds__(kThreadsRows)
    pack_kernel(const HeadGeom g, const HeadWork w, const T* hidden, int64_t ld, const int32_t* targets,
                const float* row_weight, float* loss, T* dh, int64_t dh_ld, int per, int vec) {
  __shared__ int s_before, s_total;
  const int lo = blockIdx.x * per, hi = min(lo + per, g.tokens);
  if (threadIdx.x == 0) s_before = s_total = 0;
  __syncthreads();
  int before = 0, total = 0;
  for (int r = threadIdx.x; r < g.tokens; r += kThreadsRows) {
    const int live = row_live<DISTILL>(g, w, targets, r);
    total += live;
    before += r < lo ? live : 0;
  }
  before = __reduce_add_sync(~0u, before);
  total = __reduce_add_sync(~0u, total);
  if (threadIdx.x % 32 == 0) {
    atomicAdd(&s_before, before);  // integers: any order gives the same sum
    atomicAdd(&s_total, total);
  }
  __syncthreads();
  total = s_total;
  int packed = s_before;          // live rows before row r
  const int read_end = (total + kHeadRowTile - 1) / kHeadRowTile * kHeadRowTile;
  if (blockIdx.x == 0 && threadIdx.x == 0) *w.n_live = total;
  const int64_t plane = (int64_t)g.mpad * w.dim_pad;
  for (int r = lo; r < hi; ++r) {
    const bool live = row_live<DISTILL>(g, w, targets, r);
    const int place = live ? packed : total + (r - packed);
    packed += live;
    if (threadIdx.x == 0) {
      w.perm[place] = r;
      w.wrow[place] = live ? (row_weight ? row_weight[r] : 1.0f) * g.tau : 0.0f;
      if (!live) loss[r] = 0.0f;
      if (!DISTILL && live) {
        w.ent_col[r] = column_of(g, targets[r]);
        w.ent_q[r] = 1.0f;
      }
    }
    if (!live && dh != nullptr)
      for (int d = threadIdx.x; d < g.dim; d += kThreadsRows) store_from_f32(dh + r * dh_ld + d, 0.0f);
    if (!live && place >= read_end) continue;
    pack_row(w.hid + (int64_t)place * w.dim_pad, plane, live ? hidden + r * ld : nullptr, g.dim, w.dim_pad, vec);
  }
  // places past the last row of the batch
  if (blockIdx.x == gridDim.x - 1)
    for (int place = g.tokens; place < g.mpad; ++place) {
      if (threadIdx.x == 0) {
        w.perm[place] = 0;
        w.wrow[place] = 0.0f;
      }
      if (place < read_end)
        pack_row(w.hid + (int64_t)place * w.dim_pad, plane, static_cast<const T*>(nullptr), g.dim, w.dim_pad, false);
    }
}

// Joins the tiles' (max, sum) of a row into its log-sum-exp and writes its loss. A block takes
// 32 rows: lanes are rows (the statistics of a tile are contiguous over rows), warps stride over
// the tiles and join in shared memory, in a fixed order.
constexpr int kCombineWarps = 16;
template <bool DISTILL>
__global__ void __launch_bounds__(32 * kCombineWarps)
    combine_kernel(const HeadGeom g, const HeadWork w, float* loss) {
  __shared__ float s_max[kCombineWarps][32], s_sum[kCombineWarps][32];
  const int live = *w.n_live, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int row = blockIdx.x * 32 + lane, tiles = g.tile0[RELAY_HEAD_MAX_SHARDS] * (kHeadTile / kHeadStatTile);
  if ((int)blockIdx.x * 32 >= live) return;
  float m = -INFINITY, s = 0.0f;
  if (row < live)
    for (int t = warp; t < tiles; t += kCombineWarps) {
      const float2 p = w.part[(int64_t)t * g.mpad + row];
      const float top = fmaxf(m, p.x);
      // -inf - -inf: a side that holds nothing yet adds nothing
      s = (m > -INFINITY || s != s ? s * exp2f(m - top) : 0.0f) + (p.x > -INFINITY || p.y != p.y ? p.y * exp2f(p.x - top) : 0.0f);
      m = top;
    }
  s_max[warp][lane] = m;
  s_sum[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || row >= live) return;
  for (int i = 1; i < kCombineWarps; ++i) {
    const float pm = s_max[i][lane], ps = s_sum[i][lane], top = fmaxf(m, pm);
    s = (m > -INFINITY || s != s ? s * exp2f(m - top) : 0.0f) + (pm > -INFINITY || ps != ps ? ps * exp2f(pm - top) : 0.0f);
    m = top;
  }
  const float lse2 = m + log2f(s), lse = lse2 * 0.6931471805599453f;
  w.lse[row] = lse2;
  const int r = w.perm[row];
  const int64_t at = (int64_t)r * g.top;
  if (!DISTILL) {
    loss[r] = lse - w.ent_z[at];
  } else {
    float sum = 0.0f;
    for (int k = 0; k < g.top; ++k) {
      const float q = w.ent_q[at + k];
      if (w.ent_col[at + k] == INT_MAX) break;
      if (q != 0.0f) sum += q * (logf(q) - (w.ent_z[at + k] - lse));  // 0 log 0 = 0
    }
    loss[r] = g.tau * g.tau * sum;
  }
}

// Kept exponentials to the gradient of the logits, in place: each is relative to the maximum of
// its columns, so the difference to the row's log-sum-exp makes it a probability. The
// entries' columns are computed from their fp32 logits instead: p - 1 of a confident row
// would otherwise be the rounding error of p. A block takes 2048 columns of a row; rows after the
// live ones, as far as products read them, become 0.
constexpr int kScaleCols = kThreadsRows * 8;
template <int PLANES>
__global__ void __launch_bounds__(kThreadsRows) scale_kernel(const HeadGeom g, const HeadWork w) {
  const int live = *w.n_live, row = blockIdx.x;
  if (row >= (live + kHeadRowTile - 1) / kHeadRowTile * kHeadRowTile) return;
  const int col0 = blockIdx.y * kScaleCols, col = col0 + threadIdx.x * 8;
  const int cols = g.tile0[RELAY_HEAD_MAX_SHARDS] * kHeadTile;
  const int64_t plane = (int64_t)g.mpad * w.grad_ld;
  uint16_t* line = w.grad + (int64_t)row * w.grad_ld;
  const bool on = row < live;
  const float lse = on ? w.lse[row] : 0.0f, weight = on ? w.wrow[row] : 0.0f;
  if (col < cols) {
    const float ref = on ? w.part[(int64_t)(col / kHeadStatTile) * g.mpad + row].x - lse : 0.0f;
    uint4 in[PLANES], out[PLANES];
    float v[8];
#pragma unroll
    for (int i = 0; i < PLANES; ++i) in[i] = *reinterpret_cast<const uint4*>(line + i * plane + col);
    if (PLANES == 1) {
      const uint32_t word[4] = {in[0].x, in[0].y, in[0].z, in[0].w};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // the code as a float: 2^23 + code has it in its low bits
        const uint32_t code = j & 1 ? word[j / 2] >> 16 : word[j / 2] & 0xffffu;
        const float steps = __fsub_rn(__uint_as_float(0x4b000000u | code), 8388608.0f);
        const float p = exp2f(fmaf(steps, -1.0f / kCodeSteps, ref));
        v[j] = on && (steps < kCodeZero || ref != ref) ? weight * p : 0.0f;
      }
    } else {
      const float f = on ? weight * exp2f(ref) : 0.0f;
      float x[8], y[8];
      TBF16::unpack(in[0], v);
      TBF16::unpack(in[PLANES - 2], x);
      TBF16::unpack(in[PLANES - 1], y);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = on ? __fadd_rn(__fadd_rn(y[j], x[j]), v[j]) * f : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < PLANES; ++i) {
      out[i] = TBF16::pack(v);
      float r[8];
      TBF16::unpack(out[i], r);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = __fsub_rn(v[j], r[j]);
      *reinterpret_cast<uint4*>(line + i * plane + col) = out[i];
    }
  }
  if (!on) return;
  __syncthreads();
  const int64_t at = (int64_t)w.perm[row] * g.top;
  for (int k = threadIdx.x; k < g.top; k += kThreadsRows) {
    const int c = w.ent_col[at + k];
    if (c < col0 || c >= col0 + kScaleCols || c >= cols || (k > 0 && w.ent_col[at + k - 1] == c)) continue;
    float q = 0.0f;  // an id given several times: its first entry sums them
    for (int j = k; j < g.top && w.ent_col[at + j] == c; ++j) q += w.ent_q[at + j];
    float v = weight * (exp2f(fmaf(w.ent_z[at + k], 1.4426950408889634f, -lse)) - q);
#pragma unroll
    for (int i = 0; i < PLANES; ++i) {
      const uint32_t r = bf16x2_rn(v, 0.0f) & 0xffffu;
      line[i * plane + c] = (uint16_t)r;
      v = __fsub_rn(v, __uint_as_float(r << 16));
    }
  }
}

template <class T>
__global__ void __launch_bounds__(kThreadsRows)
    write_dh_kernel(const HeadGeom g, const HeadWork w, T* dh, int64_t ld) {
  const int live = *w.n_live;
  for (int row = blockIdx.x; row < live; row += gridDim.x) {
    T* to = dh + (int64_t)w.perm[row] * ld;
    const float* from = w.dh + (int64_t)row * g.dim;
    for (int d = threadIdx.x; d < g.dim; d += kThreadsRows) {
      float sum = from[d];
      for (int i = 1; i < w.splits; ++i) sum += from[(int64_t)i * g.mpad * g.dim + d];
      store_from_f32(to + d, sum);
    }
  }
}

int ceil_div(int a, int b) { return (a + b - 1) / b; }

}  // namespace

cudaError_t head_teacher(const HeadGeom& g, const HeadWork& w, const void* teacher, int teacher_dtype,
                         const int32_t* index, cudaStream_t s) {
  const int blocks = ceil_div(g.tokens, kThreadsRows / 32);
  if (teacher_dtype == RELAY_BF16)
    teacher_kernel<<<blocks, kThreadsRows, 0, s>>>(g, w, static_cast<const uint16_t*>(teacher), index);
  else
    teacher_kernel<<<blocks, kThreadsRows, 0, s>>>(g, w, static_cast<const float*>(teacher), index);
  return cudaGetLastError();
}

template <class T>
static cudaError_t pack_typed(const HeadGeom& g, const HeadWork& w, bool distill, const void* hidden,
                              int64_t ld, const int32_t* targets, const float* row_weight, float* loss,
                              void* dh, int64_t dh_ld, cudaStream_t s) {
  // at most 1024 blocks read every row's flag; a few rows each while the batch is small
  const int per = ceil_div(g.tokens, 1024) > 4 ? ceil_div(g.tokens, 1024) : 4;
  const int blocks = ceil_div(g.tokens, per);
  const int vec = reinterpret_cast<uintptr_t>(hidden) % 16 == 0 && ld * sizeof(T) % 16 == 0;
  const T* from = static_cast<const T*>(hidden);
  if (distill)
    pack_kernel<T, true><<<blocks, kThreadsRows, 0, s>>>(g, w, from, ld, targets, row_weight, loss,
                                                         static_cast<T*>(dh), dh_ld, per, vec);
  else
    pack_kernel<T, false><<<blocks, kThreadsRows, 0, s>>>(g, w, from, ld, targets, row_weight, loss,
                                                          static_cast<T*>(dh), dh_ld, per, vec);
  return cudaGetLastError();
}

cudaError_t head_pack(const HeadGeom& g, const HeadWork& w, int dtype, bool distill, const void* hidden,
                      int64_t hidden_ld, const int32_t* targets, const float* row_weight, float* loss,
                      void* d_hidden, int64_t d_hidden_ld, cudaStream_t s) {
  if (dtype == RELAY_BF16)
    return pack_typed<uint16_t>(g, w, distill, hidden, hidden_ld, targets, row_weight, loss, d_hidden, d_hidden_ld, s);
  return pack_typed<float>(g, w, distill, hidden, hidden_ld, targets, row_weight, loss, d_hidden, d_hidden_ld, s);
}

cudaError_t head_combine(const HeadGeom& g, const HeadWork& w, bool distill, float* loss, cudaStream_t s) {
  const int blocks = ceil_div(g.tokens, 32);
  if (distill)
    combine_kernel<true><<<blocks, 32 * kCombineWarps, 0, s>>>(g, w, loss);
  else
    combine_kernel<false><<<blocks, 32 * kCombineWarps, 0, s>>>(g, w, loss);
  return cudaGetLastError();
}

cudaError_t head_pack_weight(const HeadGeom& g, const HeadWork& w, const HeadShards& sh, int dtype, cudaStream_t s) {
  const int blocks = g.tile0[RELAY_HEAD_MAX_SHARDS] * kHeadTile;
  if (dtype == RELAY_BF16)
    pack_weight_kernel<uint16_t><<<blocks, kThreadsRows, 0, s>>>(g, w, sh);
  else
    pack_weight_kernel<float><<<blocks, kThreadsRows, 0, s>>>(g, w, sh);
  return cudaGetLastError();
}

cudaError_t head_scale(const HeadGeom& g, const HeadWork& w, int dtype, cudaStream_t s) {
  const int cols = g.tile0[RELAY_HEAD_MAX_SHARDS] * kHeadTile;
  const dim3 grid(g.mpad, ceil_div(cols, kScaleCols));  // few column blocks: a piece is bounded
  if (dtype == RELAY_BF16)
    scale_kernel<1><<<grid, kThreadsRows, 0, s>>>(g, w);
  else
    scale_kernel<kHeadPlanesF32><<<grid, kThreadsRows, 0, s>>>(g, w);
  return cudaGetLastError();
}

cudaError_t head_write_dh(const HeadGeom& g, const HeadWork& w, int dtype, void* d_hidden,
                          int64_t d_hidden_ld, cudaStream_t s) {
  const int blocks = g.tokens < 4096 ? g.tokens : 4096;
  if (dtype == RELAY_BF16)
    write_dh_kernel<<<blocks, kThreadsRows, 0, s>>>(g, w, static_cast<uint16_t*>(d_hidden), d_hidden_ld);
  else
    write_dh_kernel<<<blocks, kThreadsRows, 0, s>>>(g, w, static_cast<float*>(d_hidden), d_hidden_ld);
  return cudaGetLastError();
}

}  // namespace relay
