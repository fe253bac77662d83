// router.cuh -- what the routers (router.cu, grouped_router.cu) share: a row's values in the registers of a few lanes,
// keys in the order of values, reductions over the lanes of a row, and the host's checks.
#pragma once

#include <math.h>

#include <algorithm>
#include <string>

#include "device.cuh"
#include "launch.cuh"
#include "program.h"
#include "spans.h"

namespace relay {

// Joins the blocks' partial counts and probability sums in a fixed order -- router.cu.
cudaError_t router_join(const int32_t* part_count, const float* part_prob, int blocks, int experts, int32_t* counts,
                        float* prob_sum, cudaStream_t stream);
// The gradient of softmax scores -- router.cu. The arguments have been checked.
struct SoftmaxBackward {
  const void* logits;
  void* d_logits;
  int64_t ld, d_ld, tokens;
  int dtype, experts, top, normalize;
  float scale;
  const int32_t* index;
  const float* d_gate;
  const float* d_prob;
};
cudaError_t router_softmax_backward(const SoftmaxBackward& b, cudaStream_t stream);

namespace {

constexpr int kRouterThreads = 256, kRouterWarps = kRouterThreads / 32;
constexpr uint32_t kKeyNegInf = 0x007fffffu;  // order_key(-inf)

__device__ __forceinline__ float ld1(const float* p) { return *p; }
__device__ __forceinline__ float ld1(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
__device__ __forceinline__ void st1(float* p, float v) { *p = v; }
__device__ __forceinline__ void st1(uint16_t* p, float v) { *p = (uint16_t)(bf16x2_rn(v, 0.0f) & 0xffffu); }

// Unsigned and in the order of the value; +0 and -0 equal; 0 is left for "none". A NaN's key is
// out of order.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(__fadd_rn(v, 0.0f));
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k >> 31) ? k & 0x7fffffffu : ~k);
}
// The upper 22 bits of the key, then the expert counted down.
constexpr uint32_t kExpertMask = RELAY_ROUTER_MAX_EXPERTS - 1;
static_assert(kExpertMask == 1023, "ten bits of a key name the expert");
__device__ __forceinline__ uint32_t unique_key(float v, int e) {
  return (order_key(v) & ~kExpertMask) | (kExpertMask - (uint32_t)e);
}
__device__ __forceinline__ int key_expert(uint32_t k) { return (int)(kExpertMask - (k & kExpertMask)); }
__device__ __forceinline__ float sum_warp(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}
// Over the L lanes of a row.
template <int L>
__device__ __forceinline__ float sum_row(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}
template <int L>
__device__ __forceinline__ uint32_t max_row(uint32_t v) {
  if constexpr (L == 32) {
    return __reduce_max_sync(~0u, v);
  } else {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(~0u, v, o));
    return v;
  }
}
// exp(x - m). The difference first: x and m may be the type's lowest value, which has no log2.
__device__ __forceinline__ float exp_below(float x, float m) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"((x - m) * 1.4426950408889634f));
  return y;
}

// A lane's N values of a row as they lie in memory, -inf past the last expert. bytes: what one
// load may take (16, 8, or one value), by the alignment of the rows.
template <class T, int N>
struct Lane {
  static constexpr int kWords = N * (int)sizeof(T) / 4, kPerWord = 4 / (int)sizeof(T);
  static constexpr uint32_t kNegInf = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;
  uint32_t word[kWords];
  __device__ __forceinline__ void load(const T* x, int e0, int experts, int bytes) {
    if (bytes == 16 && e0 + N <= experts) {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const uint4 u = *reinterpret_cast<const uint4*>(x + e0 + i * kPerWord);
        word[i] = u.x; word[i + 1] = u.y; word[i + 2] = u.z; word[i + 3] = u.w;
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < kWords; ++i) word[i] = kNegInf;
    if (bytes == 16) {
#pragma unroll
      for (int i = 0; i < kWords; i += 4)
        if (e0 + i * kPerWord < experts) {
          const uint4 u = *reinterpret_cast<const uint4*>(x + e0 + i * kPerWord);
          word[i] = u.x; word[i + 1] = u.y; word[i + 2] = u.z; word[i + 3] = u.w;
        }
    } else if (bytes == 8) {
#pragma unroll
      for (int i = 0; i < kWords; i += 2)
        if (e0 + i * kPerWord < experts) {
          const uint2 u = *reinterpret_cast<const uint2*>(x + e0 + i * kPerWord);
          word[i] = u.x; word[i + 1] = u.y;
        }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (e0 + i < experts) {
          if constexpr (sizeof(T) == 4) word[i] = __float_as_uint(x[e0 + i]);
          else word[i / 2] = i % 2 ? (word[i / 2] & 0xffffu) | (uint32_t)x[e0 + i] << 16 : (word[i / 2] & 0xffff0000u) | x[e0 + i];
        }
    }
  }
  __device__ __forceinline__ void values(float (&v)[N]) const {
#pragma unroll
    for (int i = 0; i < N; ++i)
      v[i] = sizeof(T) == 4 ? __uint_as_float(word[i])
                            : __uint_as_float(i % 2 ? word[i / kPerWord] & 0xffff0000u : word[i / kPerWord] << 16);
  }
  static __device__ __forceinline__ void store(T* x, const float (&v)[N], int e0, int experts, int bytes) {
    uint32_t w[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i)
      w[i] = sizeof(T) == 4 ? __float_as_uint(v[i]) : bf16x2_rn(v[i * kPerWord], v[i * kPerWord + kPerWord - 1]);
    if (bytes == 16) {
#pragma unroll
      for (int i = 0; i < kWords; i += 4)
        if (e0 + i * kPerWord < experts)
          *reinterpret_cast<uint4*>(x + e0 + i * kPerWord) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    } else if (bytes == 8) {
#pragma unroll
      for (int i = 0; i < kWords; i += 2)
        if (e0 + i * kPerWord < experts)
          *reinterpret_cast<uint2*>(x + e0 + i * kPerWord) = make_uint2(w[i], w[i + 1]);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (e0 + i < experts) st1(x + e0 + i, v[i]);
    }
  }
};

// Blocks of the forward pass, whose statistics are joined afterwards: at most four an SM of the
// GB300's 152 (also with another device current, so that the workspace is one size). Two rounds
// of one block are not worth a second launch.
int64_t forward_blocks(int64_t tokens, int rows) {
  if (tokens <= 2 * rows) return 1;
  return std::min<int64_t>((tokens + rows - 1) / rows, 4 * 152);
}

// Bytes one load of a lane's values may take: rows aligned to them, and made of whole ones.
int load_bytes(const void* p, int64_t ld, int64_t esize, int experts) {
  for (int bytes = 16; bytes > 4; bytes /= 2)
    if (reinterpret_cast<uintptr_t>(p) % bytes == 0 && ld * esize % bytes == 0 && experts * esize % bytes == 0)
      return bytes;
  return (int)esize;
}

struct Array {
  Span span;
  const char* what;
  bool out;
};
Array array(const void* p, int64_t bytes, const char* what, bool out) { return Array{array_span(p, bytes), what, out}; }
Array matrix(const void* p, int64_t rows, int64_t width, int64_t pitch, const char* what, bool out) {
  return Array{matrix_span(p, rows, width, pitch), what, out};
}
bool off(const void* p, uintptr_t e) { return reinterpret_cast<uintptr_t>(p) % e != 0; }


}  // namespace
}  // namespace relay
