// head.h -- internal: the output projection with a sharded vocabulary (relay_linear_xent,
// relay_linear_distill): geometry, workspace and the launches behind the entry points.
//
// Vocabulary columns are numbered in a padded space: every shard starts at a multiple of
// kHeadTile columns, so that a tile of columns, of the logits' gradient or of a product's
// inner dimension lies in one shard. Padding columns have no weight row; their
// gradient is 0.
//
// Rows are compacted: the rows that take part ("live") are copied, in order, to the front of
// the workspace copy of hidden, and rows after them up to a multiple of kHeadRowTile hold 0.
// An ignored row is therefore never multiplied by anything (NaN * 0 is NaN), and costs
// nothing. How many rows are live is known on the device only: launches are sized for
// all of them and leave early.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "relay.h"

namespace relay {

constexpr int kHeadTile = 256;     // columns a shard is padded to
constexpr int kHeadRowTile = 256;  // rows the live rows are padded to
constexpr int kHeadStatTile = 128; // columns one (max, sum) of a row stands for

// The form in which the exponentials of a bf16 head are kept: how far a logit lies below the
// largest of its row's kHeadStatTile columns, in log2 units, in steps of 2^-10 and 16 bits. That is
// within 2^-11 ln 2 = 3.4e-4 of the exponential, a sixth of bf16's step, at the same width, so
// the gradient is as good as rounded once; bf16 exponentials would round it twice (1.7e-3 each,
// in the mean). 65535 stands for 0 (an exponential 2^-64 of the largest).
constexpr float kCodeSteps = 1024.0f;
constexpr float kCodeZero = 65535.0f;

struct HeadGeom {
  int32_t A, top;                           // shards; entries per row (1 for cross entropy)
  int32_t tokens, dim;
  int32_t tile0[RELAY_HEAD_MAX_SHARDS + 1]; // first padded tile of each shard, then the total
  int32_t rows[RELAY_HEAD_MAX_SHARDS];
  int32_t base[RELAY_HEAD_MAX_SHARDS];      // first vocabulary id of each shard
  int32_t vocab;
  int32_t mpad;                             // tokens rounded up to kHeadRowTile
  int32_t sms;
  int32_t ctas;                             // that make one product: 2, or 1 for few rows
  float tau, inv_tau;
};

#ifdef __CUDACC__
__host__ __device__ __forceinline__
#else
inline
#endif
int head_row_tile(const HeadGeom& g) { return kHeadRowTile / 2 * g.ctas; }  // rows of one product

#ifdef __CUDACC__
__host__ __device__ __forceinline__
#else
inline
#endif
int head_shard_of_tile(const HeadGeom& g, int tile) {
  int a = 0;
  while (a + 1 < g.A && tile >= g.tile0[a + 1]) ++a;
  return a;
}

// Matrices the products read are bf16. An fp32 value is held as three bf16 parts that sum to
// it (to 2^-26 of it at least), in three planes; a product of two such matrices is the sum of six
// products of parts. The three left out are at most 1.5e-7 of it (2^-22.7; see the packing for the split).
constexpr int kHeadPlanesF32 = 3;
inline int head_planes(int dtype) { return dtype == RELAY_F32 ? kHeadPlanesF32 : 1; }
// Parts the gradient of a logit is held in. One bf16 value is as exact as the bf16 results want where
// rounding errors average over many rows. Up to 128 rows they do not (a weight row's gradient may be
// one token's), and d_weight's products wait for its writes, so that a second part there costs little.
inline int head_grad_planes(int dtype, int ctas) { return dtype == RELAY_F32 ? kHeadPlanesF32 : ctas == 1 ? 2 : 1; }

#ifdef __CUDACC__
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
#endif

// Softmax statistics are kept as the largest logit itself and the sum of the exponentials below it, and a logit meets
// the largest before the temperature and log2 e: the type's lowest and largest values times log2 e leave
// fp32's range, their differences end at an exponential of 0. A row's log-sum-exp is not joined into
// one number either: next to a large logit the log of the sum would be lost.
#ifdef __CUDACC__
__device__ __forceinline__ float head_log2_scale(const HeadGeom& g) { return g.inv_tau * 1.4426950408889634f; }
#endif

// Everything a call works with on the device.
struct HeadWork {
  int32_t* n_live;    // [2]: live rows, cuts of the vocabulary for d_hidden
  int32_t* perm;      // [mpad] packed row -> row of hidden
  float* wrow;        // [mpad] row weight * tau (0 past the live rows)
  uint16_t* hid;      // [planes][mpad][dim_pad] packed hidden
  int32_t dim_pad;    // a multiple of 64
  uint16_t* wpack;    // [planes][tiles * kHeadTile][dim_pad] packed weight, or NULL: read in place
  uint8_t* live;      // [tokens]            (distill)
  int32_t* ent_col;   // [tokens][top] entries' padded columns, ascending; INT32_MAX: absent
  float* ent_q;       // [tokens][top]
  float* ent_z;       // [tokens][top] the entries' logits
  float2* part;       // [2 tiles][mpad] (largest logit, sum of exp((z - it) / tau)) of kHeadStatTile columns
  float2* lse;        // [mpad] the row's largest logit, and the log2 of its sum
  uint16_t* grad;     // [grad_planes][mpad][grad_ld] of one piece: codes or exponentials, then the gradient
  int32_t grad_planes;
  int64_t grad_ld;    // columns per row
  float* dh;          // [splits][mpad][dh_ld] fp32 partial sums of d_hidden
  int32_t dh_ld;      // dim rounded up to 4
  int32_t splits;     // most cuts of the vocabulary d_hidden may take
  int32_t tiles_per_piece;
  int32_t with_dw;    // d_weight's tiles run beside d_hidden's
  int32_t whole;      // one piece, and d_hidden's rows take 16-byte stores: uncut sums go straight there
};

// Cuts of the vocabulary for d_hidden, whose tiles alone are too few, or too long beside what else
// runs, to fill the GPU evenly. Costs are in inner steps of one tile (64 columns, about 0.27 us):
// the rounds of the GPU's products over d_hidden's tiles, or all the work spread evenly plus the
// longest tile at its end, whichever is more; plus writing and reading a cut's fp32 partial sums (8 bytes
// a value; a step's time moves about 1.8 MB). The live rows are known on the device only: the packing
// kernel leaves the number beside theirs.
#ifdef __CUDACC__
constexpr int kHeadOpenSteps = 4;  // steps a tile costs besides its own
__device__ __forceinline__ float head_long_steps(int tiles, int cuts) {  // a tile of d_hidden
  return (float)(((uint32_t)tiles * 4 + cuts - 1) / cuts + kHeadOpenSteps);
}
__device__ __forceinline__ float head_short_steps(int live) { return (float)((live + 63) / 64 + kHeadOpenSteps); }  // of d_weight
__device__ __forceinline__ int head_cuts(const HeadGeom& g, const HeadWork& w, int live) {
  // whole warps call it: a lane prices two numbers of cuts (there are at most 64)
  const int pairs = g.ctas == 1 ? g.sms : g.sms / 2, nd = (g.dim + kHeadTile - 1) / kHeadTile;
  const int rows = head_row_tile(g);
  const float items = (float)((live + rows - 1) / rows) * (float)nd;
  if (w.splits == 1 || items >= 4.0f * (float)pairs) return 1;
  const float move = 0.2f + (float)live * (float)g.dim * (1.0f / 225000.0f);
  const float dw_steps = w.with_dw ? head_short_steps(live) : 0.0f;
  const float dw_work = (float)w.tiles_per_piece * (float)(g.ctas == 1 ? 2 * nd : nd) * dw_steps;
  const float each = 1.0f / (float)pairs;
  float least = INFINITY;
  int best = 1;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int s = 1 + threadIdx.x % 32 + 32 * i;
    const float steps = head_long_steps(w.tiles_per_piece, s);
    const float rounds = ceilf(items * (float)s * each) * steps;
    const float spread = (items * (float)s * steps + dw_work) * each + (w.with_dw ? dw_steps : steps);
    const float cost = fmaxf(rounds, spread) + (s > 1 ? (float)s * move : 0.0f);
    if (s <= w.splits && cost < least) {
      least = cost;
      best = s;
    }
  }
  // positive floats order as integers do
  const uint32_t all = __reduce_min_sync(~0u, __float_as_uint(least));
  return (int)__reduce_min_sync(~0u, __float_as_uint(least) == all ? (uint32_t)best : ~0u);
}
#endif

struct HeadShards {
  const void* w[RELAY_HEAD_MAX_SHARDS];
  void* dw[RELAY_HEAD_MAX_SHARDS];
  int64_t w_ld, dw_ld;
  void* dh;  // d_hidden, for a product that writes it itself
  int64_t dh_ld;
};

// head_rows.cu
cudaError_t head_teacher(const HeadGeom& g, const HeadWork& w, const void* teacher, int teacher_dtype,
                         const int32_t* index, cudaStream_t s);
cudaError_t head_pack(const HeadGeom& g, const HeadWork& w, int dtype, const void* hidden, int64_t hidden_ld,
                      const int32_t* index, const void* teacher, int teacher_dtype, const float* row_weight,
                      float* loss, void* d_hidden, int64_t d_hidden_ld, cudaStream_t s);
cudaError_t head_pack_weight(const HeadGeom& g, const HeadWork& w, const HeadShards& sh, int dtype,
                             cudaStream_t s);
cudaError_t head_combine(const HeadGeom& g, const HeadWork& w, bool distill, float* loss,
                         cudaStream_t s);
// Kept exponentials to the gradient. Where a row is short (head_scale_joins) it does head_combine's work
// as well: one launch less.
bool head_scale_joins(const HeadGeom& g);
bool head_scale_fits(const HeadGeom& g);  // in one launch
cudaError_t head_scale(const HeadGeom& g, const HeadWork& w, int dtype, bool distill, float* loss, cudaStream_t s);
cudaError_t head_write_dh(const HeadGeom& g, const HeadWork& w, int dtype, void* d_hidden,
                          int64_t d_hidden_ld, cudaStream_t s);

// head_gemm.cu
enum HeadLogits { kHeadStats, kHeadStatsKeep, kHeadGradient };
cudaError_t head_logits(const HeadGeom& g, const HeadWork& w, const HeadShards& sh, int dtype,
                        int tile_lo, int tile_hi, HeadLogits mode, cudaStream_t s);
// d_hidden and d_weight of one piece, either or both. first: the first piece.
cudaError_t head_back(const HeadGeom& g, const HeadWork& w, const HeadShards& sh, int dtype, int tile_lo, int tile_hi,
                      bool first, bool dh, bool dw, cudaStream_t s);
// Makes the calling thread's next products wait for `bytes` more than their loads bring.
void head_test_extra(int bytes);
// Reads and clears the products' fault word.
cudaError_t head_read_fault(unsigned* fault);

}  // namespace relay
