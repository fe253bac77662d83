// head_gemm.cu -- the three products of the head, on the FMA pipes: a 64 x 64 tile per block of
// 256 threads, 4 x 4 results each, the inner dimension 16 at a time through shared memory.
// Products and sums are fp32 for both types.
#include <limits.h>
#include <math.h>

#include "device.cuh"
#include "head.h"

namespace relay {
namespace {

constexpr int kT = 64, kK = 16;

__device__ __forceinline__ float as_f32(float v) { return v; }
__device__ __forceinline__ float as_f32(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t* p, float v) { *p = (uint16_t)(bf16x2_rn(v, 0.0f) & 0xffffu); }

// acc[i][j] = sum_k a(m0 + ty + 16 i, k) b(n0 + tx + 16 j, k); a and b return 0 out of range.
template <class LA, class LB>
__device__ __forceinline__ void tile_product(float (&acc)[4][4], LA a, LB b, int64_t K, int m0, int n0) {
  __shared__ float sa[kK][kT + 1], sb[kK][kT + 1];
  const int t = threadIdx.x, tx = t % 16, ty = t / 16;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
  for (int64_t k0 = 0; k0 < K; k0 += kK) {
    __syncthreads();
    for (int e = t; e < kK * kT; e += 256) {
      const int k = e % kK, r = e / kK;
      sa[k][r] = k0 + k < K ? a(m0 + r, k0 + k) : 0.0f;
      sb[k][r] = k0 + k < K ? b(n0 + r, k0 + k) : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kK; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[i][j] = fmaf(sa[k][ty + 16 * i], sb[k][tx + 16 * j], acc[i][j]);
  }
}

// Weight row of a padded column, or -1 for padding.
__device__ __forceinline__ int weight_row(const HeadGeom& g, int col, int* shard) {
  const int a = head_shard_of_tile(g, col / kHeadTile), v = col - g.tile0[a] * kHeadTile;
  *shard = a;
  return v < g.rows[a] ? v : -1;
}

template <class T>
__global__ void __launch_bounds__(256)
    logits_kernel(const HeadGeom g, const HeadWork w, const HeadShards sh, int col0, bool gradient) {
  const int live = *w.n_live, m0 = blockIdx.y * kT, n0 = col0 + blockIdx.x * kHeadTile;
  if (m0 >= (live + kHeadRowTile - 1) / kHeadRowTile * kHeadRowTile) return;
  __shared__ float s_max[kT][16], s_sum[kT][16];
  const T* hid = static_cast<const T*>(w.hid);
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  int shard;
  weight_row(g, n0, &shard);
  const T* wt = static_cast<const T*>(sh.w[shard]);
  const int v0 = n0 - g.tile0[shard] * kHeadTile, rows = g.rows[shard];
  float run_max[4], run_sum[4];
  for (int i = 0; i < 4; ++i) {
    run_max[i] = -INFINITY;
    run_sum[i] = 0.0f;
  }
  for (int n = 0; n < kHeadTile; n += kT) {
    float acc[4][4];
    tile_product(
        acc, [&](int m, int64_t k) { return as_f32(hid[(int64_t)m * w.dim_pad + k]); },
        [&](int v, int64_t k) { return v < rows ? as_f32(wt[v * sh.w_ld + k]) : 0.0f; }, g.dim, m0, v0 + n);
    for (int i = 0; i < 4; ++i) {
      const int row = m0 + ty + 16 * i;
      const int64_t at = (int64_t)(row < live ? w.perm[row] : 0) * g.top;
      for (int j = 0; j < 4; ++j) {
        const int col = n0 + n + tx + 16 * j;
        const bool in = row < live && v0 + n + tx + 16 * j < rows;
        const float z = acc[i][j] * g.inv_tau;
        float q = 0.0f;
        if (in)
          for (int k = 0; k < g.top; ++k)
            if (w.ent_col[at + k] == col) {
              q += w.ent_q[at + k];
              if (!gradient) w.ent_z[at + k] = z;
            }
        if (gradient) {
          const float p = in ? expf(z - w.lse[row]) : 0.0f;
          put(static_cast<T*>(w.grad) + row * w.grad_ld + (col - col0), in ? w.wrow[row] * (p - q) : 0.0f);
        } else if (in) {
          const float top = fmaxf(run_max[i], z);
          run_sum[i] = (run_max[i] > -INFINITY ? run_sum[i] * expf(run_max[i] - top) : 0.0f) +
                       (z != z ? z : z > -INFINITY ? expf(z - top) : 0.0f);
          run_max[i] = top;
        }
      }
    }
  }
  if (gradient) return;
  for (int i = 0; i < 4; ++i) {
    s_max[ty + 16 * i][tx] = run_max[i];
    s_sum[ty + 16 * i][tx] = run_sum[i];
  }
  __syncthreads();
  if (threadIdx.x < kT) {
    float top = -INFINITY, sum = 0.0f;
    for (int x = 0; x < 16; ++x) top = fmaxf(top, s_max[threadIdx.x][x]);
    for (int x = 0; x < 16; ++x) {
      const float m = s_max[threadIdx.x][x], s = s_sum[threadIdx.x][x];
      sum += s != s ? s : m > -INFINITY ? s * expf(m - top) : 0.0f;
    }
    w.part[(int64_t)(n0 / kHeadTile) * g.mpad + m0 + threadIdx.x] = make_float2(top, sum);
  }
}

template <class T>
__global__ void __launch_bounds__(256)
    dhidden_kernel(const HeadGeom g, const HeadWork w, const HeadShards sh, int col0, int cols, bool first) {
  const int live = *w.n_live, m0 = blockIdx.y * kT, n0 = blockIdx.x * kT;
  if (m0 >= live) return;
  const T* grad = static_cast<const T*>(w.grad);
  float acc[4][4];
  tile_product(
      acc, [&](int m, int64_t k) { return as_f32(grad[m * w.grad_ld + k]); },
      [&](int d, int64_t k) {
        int shard;
        const int v = weight_row(g, col0 + (int)k, &shard);
        return v >= 0 && d < g.dim ? as_f32(static_cast<const T*>(sh.w[shard])[v * sh.w_ld + d]) : 0.0f;
      },
      cols, m0, n0);
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + threadIdx.x / 16 + 16 * i, d = n0 + threadIdx.x % 16 + 16 * j;
      if (m >= live || d >= g.dim) continue;
      float* p = w.dh + (int64_t)m * g.dim + d;
      *p = first ? acc[i][j] : *p + acc[i][j];
    }
}

template <class T>
__global__ void __launch_bounds__(256)
    dweight_kernel(const HeadGeom g, const HeadWork w, const HeadShards sh, int col0) {
  const int live = *w.n_live, m0 = blockIdx.y * kT, n0 = blockIdx.x * kT;  // m: column of the piece
  const T* grad = static_cast<const T*>(w.grad);
  const T* hid = static_cast<const T*>(w.hid);
  float acc[4][4];
  tile_product(
      acc, [&](int c, int64_t k) { return as_f32(grad[k * w.grad_ld + c]); },
      [&](int d, int64_t k) { return d < g.dim ? as_f32(hid[k * w.dim_pad + d]) : 0.0f; }, live, m0, n0);
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int c = m0 + threadIdx.x / 16 + 16 * i, d = n0 + threadIdx.x % 16 + 16 * j;
      int shard;
      const int v = weight_row(g, col0 + c, &shard);
      if (v >= 0 && d < g.dim) put(static_cast<T*>(sh.dw[shard]) + v * sh.dw_ld + d, acc[i][j]);
    }
}

}  // namespace

cudaError_t head_logits(const HeadGeom& g, const HeadWork& w, const HeadShards& sh, int dtype,
                        int tile_lo, int tile_hi, bool gradient, cudaStream_t s) {
  const dim3 grid(tile_hi - tile_lo, g.mpad / kT);
  if (dtype == RELAY_BF16)
    logits_kernel<uint16_t><<<grid, 256, 0, s>>>(g, w, sh, tile_lo * kHeadTile, gradient);
  else
    logits_kernel<float><<<grid, 256, 0, s>>>(g, w, sh, tile_lo * kHeadTile, gradient);
  return cudaGetLastError();
}

cudaError_t head_dhidden(const HeadGeom& g, const HeadWork& w, const HeadShards& sh, int dtype,
                         int tile_lo, int tile_hi, bool first, cudaStream_t s) {
  const dim3 grid((g.dim + kT - 1) / kT, g.mpad / kT);
  const int cols = (tile_hi - tile_lo) * kHeadTile;
  if (dtype == RELAY_BF16)
    dhidden_kernel<uint16_t><<<grid, 256, 0, s>>>(g, w, sh, tile_lo * kHeadTile, cols, first);
  else
    dhidden_kernel<float><<<grid, 256, 0, s>>>(g, w, sh, tile_lo * kHeadTile, cols, first);
  return cudaGetLastError();
}

cudaError_t head_dweight(const HeadGeom& g, const HeadWork& w, const HeadShards& sh, int dtype,
                         int tile_lo, int tile_hi, cudaStream_t s) {
  const dim3 grid((g.dim + kT - 1) / kT, (tile_hi - tile_lo) * (kHeadTile / kT));
  if (dtype == RELAY_BF16)
    dweight_kernel<uint16_t><<<grid, 256, 0, s>>>(g, w, sh, tile_lo * kHeadTile);
  else
    dweight_kernel<float><<<grid, 256, 0, s>>>(g, w, sh, tile_lo * kHeadTile);
  return cudaGetLastError();
}

}  // namespace relay
