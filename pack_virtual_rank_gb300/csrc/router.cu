// router.cu -- relay_router_forward, relay_balance_loss, relay_router_backward.
//
// One warp per row. Lane l holds the row's experts [l * N, (l + 1) * N) in registers, so that
// the lowest lane of a tie holds the lowest expert. The forward pass accumulates the softmax per
// expert in registers over the rows its warp walks (a fixed assignment), joins the warps of a
// block in shared memory in order, and a second launch joins the blocks in order: the sums have
// one order, without atomics on floats.
#include <limits.h>
#include <math.h>

#include <algorithm>
#include <string>

#include "device.cuh"
#include "program.h"

namespace relay {
namespace {

constexpr int kRouterThreads = 256, kRouterWarps = kRouterThreads / 32;
constexpr uint32_t kKeyNegInf = 0x007fffffu;  // order_key(-inf)

__device__ __forceinline__ float ld1(const float* p) { return *p; }
__device__ __forceinline__ float ld1(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
__device__ __forceinline__ void st1(float* p, float v) { *p = v; }
__device__ __forceinline__ void st1(uint16_t* p, float v) { *p = (uint16_t)(bf16x2_rn(v, 0.0f) & 0xffffu); }

// An unsigned key in the order of the value: +0 and -0 equal, NaN below -inf (1), 0 left for
// "no expert here, or already chosen".
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(__fadd_rn(v, 0.0f));
  const uint32_t k = (u >> 31) ? ~u : u | 0x80000000u;
  return v != v ? 1u : k;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k >> 31) ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ float sum_warp(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

struct ForwardArgs {
  const void* logits;
  int64_t ld, tokens;
  int experts, top, normalize;
  const uint8_t* mask;
  int32_t* index;
  float* gate;
  int32_t* part_count;  // [blocks][experts], or the result when one block runs
  float* part_prob;
};

template <class T, int N>
__global__ void __launch_bounds__(kRouterThreads) router_forward_kernel(const ForwardArgs a) {
  extern __shared__ float s_prob[];  // [warps][experts], then the counts [experts]
  int32_t* s_count = reinterpret_cast<int32_t*>(s_prob + kRouterWarps * a.experts);
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  for (int e = threadIdx.x; e < a.experts; e += kRouterThreads) s_count[e] = 0;
  __syncthreads();
  float psum[N];
#pragma unroll
  for (int i = 0; i < N; ++i) psum[i] = 0.0f;
  const int64_t stride = (int64_t)gridDim.x * kRouterWarps;
  for (int64_t row = (int64_t)blockIdx.x * kRouterWarps + warp; row < a.tokens; row += stride) {
    const T* x = static_cast<const T*>(a.logits) + row * a.ld;
    const bool counted = a.mask == nullptr || a.mask[row] != 0;
    float v[N];
    uint32_t key[N];
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = lane * N + i;
      const bool in = counted && e < a.experts;
      v[i] = in ? ld1(x + e) : -INFINITY;
      key[i] = in ? order_key(v[i]) : 0u;
      best = max(best, key[i]);
    }
    const uint32_t first = __reduce_max_sync(~0u, best);
    if (first <= kKeyNegInf) {  // masked out, or no logit above -inf
      if (lane < a.top) {
        a.index[row * a.top + lane] = -1;
        a.gate[row * a.top + lane] = 0.0f;
      }
      continue;
    }
    const float m = key_value(first);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = expf(v[i] - m);
      sum += v[i];
    }
    sum = sum_warp(sum);
    const float inv = 1.0f / sum;
#pragma unroll
    for (int i = 0; i < N; ++i) psum[i] += v[i] * inv;
    int chosen = -1;
    float val = 0.0f;
    uint32_t win = first;
    for (int j = 0; j < a.top; ++j) {
      const int owner = __ffs(__ballot_sync(~0u, best == win)) - 1;
      int e = 0;
      if (lane == owner) {
        bool open = true;
        best = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          if (open && key[i] == win) {
            open = false;
            key[i] = 0;
            e = lane * N + i;
          }
          best = max(best, key[i]);
        }
        atomicAdd(&s_count[e], 1);  // integers: any order gives the same sum
      }
      e = __shfl_sync(~0u, e, owner);
      if (lane == j) {
        chosen = e;
        val = win <= 1u ? NAN : expf(key_value(win) - m);
      }
      win = __reduce_max_sync(~0u, best);
    }
    float scale = inv;
    if (a.normalize) scale = 1.0f / sum_warp(lane < a.top ? val : 0.0f);
    if (sum != sum) scale = sum;
    if (lane < a.top) {
      a.index[row * a.top + lane] = chosen;
      a.gate[row * a.top + lane] = val * scale;
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (lane * N + i < a.experts) s_prob[warp * a.experts + lane * N + i] = psum[i];
  __syncthreads();
  for (int e = threadIdx.x; e < a.experts; e += kRouterThreads) {
    float p = 0.0f;
    for (int i = 0; i < kRouterWarps; ++i) p += s_prob[i * a.experts + e];
    a.part_prob[(int64_t)blockIdx.x * a.experts + e] = p;
    a.part_count[(int64_t)blockIdx.x * a.experts + e] = s_count[e];
  }
}

// Joins the blocks' partial sums: a block takes 32 experts, its warps stride over the partials.
constexpr int kJoinWarps = 16;
__global__ void __launch_bounds__(32 * kJoinWarps)
    router_join_kernel(const int32_t* part_count, const float* part_prob, int blocks, int experts,
                       int32_t* counts, float* prob_sum) {
  __shared__ float s_p[kJoinWarps][32];
  __shared__ int32_t s_c[kJoinWarps][32];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, e = blockIdx.x * 32 + lane;
  float p = 0.0f;
  int32_t c = 0;
  if (e < experts)
    for (int b = warp; b < blocks; b += kJoinWarps) {
      p += part_prob[(int64_t)b * experts + e];
      c += part_count[(int64_t)b * experts + e];
    }
  s_p[warp][lane] = p;
  s_c[warp][lane] = c;
  __syncthreads();
  if (warp != 0 || e >= experts) return;
  for (int i = 1; i < kJoinWarps; ++i) {
    p += s_p[i][lane];
    c += s_c[i][lane];
  }
  prob_sum[e] = p;
  counts[e] = c;
}

constexpr int kBalanceThreads = 256;
__global__ void __launch_bounds__(kBalanceThreads)
    balance_kernel(const int32_t* counts, const float* prob_sum, int experts, int top, float coef,
                   float* loss, float* d_prob) {
  __shared__ long long s_total[kBalanceThreads / 32];
  __shared__ float s_loss[kBalanceThreads / 32];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  long long total = 0;
  for (int e = threadIdx.x; e < experts; e += kBalanceThreads) total += counts[e];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(~0u, total, o);
  if (lane == 0) s_total[warp] = total;
  __syncthreads();
  total = 0;
  for (int i = 0; i < kBalanceThreads / 32; ++i) total += s_total[i];
  const float n = (float)((double)total / top);  // counted tokens
  float sum = 0.0f;
  for (int e = threadIdx.x; e < experts; e += kBalanceThreads) {
    const float d = total > 0 ? coef * experts * ((float)counts[e] / ((float)top * n)) / n : 0.0f;
    d_prob[e] = d;
    if (total > 0) sum += d * prob_sum[e];
  }
  sum = sum_warp(sum);
  if (lane == 0) s_loss[warp] = sum;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int i = 1; i < kBalanceThreads / 32; ++i) sum += s_loss[i];
  loss[0] = sum;
}

struct BackwardArgs {
  const void* logits;
  void* d_logits;
  int64_t ld, d_ld, tokens;
  int experts, top, normalize;
  const int32_t* index;
  const float* d_gate;
  const float* d_prob;
};

template <class T, int N>
__global__ void __launch_bounds__(kRouterThreads) router_backward_kernel(const BackwardArgs a) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t row = (int64_t)blockIdx.x * kRouterWarps + warp;
  if (row >= a.tokens) return;
  const T* x = static_cast<const T*>(a.logits) + row * a.ld;
  T* dx = static_cast<T*>(a.d_logits) + row * a.d_ld;
  const int mine = lane < a.top ? a.index[row * a.top + lane] : 0;
  if (__shfl_sync(~0u, mine, 0) < 0) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (lane * N + i < a.experts) st1(dx + lane * N + i, 0.0f);
    return;
  }
  float p[N], g[N], m = -INFINITY;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = lane * N + i;
    p[i] = e < a.experts ? ld1(x + e) : -INFINITY;
    g[i] = e < a.experts && a.d_prob != nullptr ? a.d_prob[e] : 0.0f;
    m = fmaxf(m, p[i]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    p[i] = expf(p[i] - m);
    sum += p[i];
  }
  const float inv = 1.0f / sum_warp(sum);
#pragma unroll
  for (int i = 0; i < N; ++i) p[i] *= inv;
  // what each chosen expert adds: to dL/dp, or (normalize) straight to its logit's gradient
  float dg = lane < a.top && a.d_gate != nullptr ? a.d_gate[row * a.top + lane] : 0.0f;
  if (a.normalize) {
    float c = lane < a.top && mine >= 0 && mine < a.experts ? expf(ld1(x + mine) - m) : 0.0f;
    c = c / sum_warp(c);
    const float inner = sum_warp(c * dg);
    dg = c * (dg - inner);
  }
  float extra[N];
#pragma unroll
  for (int i = 0; i < N; ++i) extra[i] = 0.0f;
  for (int j = 0; j < a.top; ++j) {
    const int e = __shfl_sync(~0u, mine, j);
    const float d = __shfl_sync(~0u, dg, j);
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (lane * N + i == e) extra[i] += d;
  }
  float dot = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (!a.normalize) g[i] += extra[i];
    dot += p[i] * g[i];
  }
  dot = sum_warp(dot);
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (lane * N + i < a.experts)
      st1(dx + lane * N + i, p[i] * (g[i] - dot) + (a.normalize ? extra[i] : 0.0f));
}

// Registers per lane for a number of experts.
template <class F>
cudaError_t by_width(int experts, F f) {
  if (experts <= 32) return f(std::integral_constant<int, 1>());
  if (experts <= 64) return f(std::integral_constant<int, 2>());
  if (experts <= 128) return f(std::integral_constant<int, 4>());
  if (experts <= 256) return f(std::integral_constant<int, 8>());
  if (experts <= 512) return f(std::integral_constant<int, 16>());
  return f(std::integral_constant<int, 32>());
}

int64_t forward_blocks(int64_t tokens) {
  return std::max<int64_t>(1, std::min<int64_t>((tokens + kRouterWarps - 1) / kRouterWarps, 4 * 152));
}

relay_status_t bad(const std::string& msg) {
  return report_error(RELAY_ERR_INVALID_ARGUMENT, "relay_router: " + msg);
}
relay_status_t done(cudaError_t e) {
  if (e == cudaSuccess) return RELAY_OK;
  return report_error(RELAY_ERR_CUDA, std::string("relay_router: ") + cudaGetErrorString(e));
}

relay_status_t check_shape(relay_dtype_t dtype, int64_t tokens, int experts, int top) {
  if (dtype != RELAY_F32 && dtype != RELAY_BF16) return bad("dtype must be RELAY_F32 or RELAY_BF16");
  if (tokens < 0 || tokens > INT32_MAX) return bad("tokens out of range");
  if (experts < 1 || experts > RELAY_ROUTER_MAX_EXPERTS) return bad("experts must be 1..1024");
  if (top < 1 || top > experts || top > RELAY_ROUTER_MAX_TOP) return bad("top must be 1..min(experts, 32)");
  return RELAY_OK;
}

struct Span {
  uintptr_t lo, hi;
  const char* what;
  bool out;
};
Span span(const void* p, int64_t bytes, const char* what, bool out) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return Span{lo, lo + (uintptr_t)(p != nullptr ? bytes : 0), what, out};
}
relay_status_t check_spans(const Span* s, int n) {
  for (int i = 0; i < n; ++i)
    for (int j = i + 1; j < n; ++j)
      if ((s[i].out || s[j].out) && s[i].lo < s[j].hi && s[j].lo < s[i].hi)
        return bad(std::string(s[i].what) + " overlaps " + s[j].what);
  return RELAY_OK;
}
bool off(const void* p, uintptr_t e) { return reinterpret_cast<uintptr_t>(p) % e != 0; }

}  // namespace
}  // namespace relay

extern "C" {

int64_t relay_router_workspace_size(int64_t tokens, int experts) {
  using namespace relay;
  if (tokens < 0 || tokens > INT32_MAX || experts < 1 || experts > RELAY_ROUTER_MAX_EXPERTS) {
    bad("tokens or experts out of range");
    return -1;
  }
  return forward_blocks(tokens) * experts * 8 + 16;
}

relay_status_t relay_router_forward(const void* logits, int64_t row_stride, relay_dtype_t dtype,
                                    int64_t tokens, int experts, int top, int normalize,
                                    const uint8_t* mask, int32_t* index, float* gate,
                                    int32_t* counts, float* prob_sum, void* workspace,
                                    int64_t workspace_bytes, cudaStream_t stream) {
  using namespace relay;
  relay_status_t st = check_shape(dtype, tokens, experts, top);
  if (st != RELAY_OK) return st;
  if (counts == nullptr || prob_sum == nullptr) return bad("counts or prob_sum is NULL");
  if (tokens > 0 && (logits == nullptr || index == nullptr || gate == nullptr))
    return bad("logits, index or gate is NULL");
  if (tokens > 0 && (row_stride < experts || row_stride > (1ll << 31))) return bad("row_stride is less than experts or more than 2^31");
  const int E = esize_of(dtype);
  if (off(logits, E) || off(index, 4) || off(gate, 4) || off(counts, 4) || off(prob_sum, 4))
    return bad("an array is not element-aligned");
  const int64_t need = relay_router_workspace_size(tokens, experts);
  if (workspace == nullptr) return bad("workspace is NULL");
  if (workspace_bytes < need)
    return bad("the workspace holds " + std::to_string(workspace_bytes) + " bytes, " + std::to_string(need) + " are needed");
  const Span s[] = {span(logits, tokens ? ((tokens - 1) * row_stride + experts) * E : 0, "logits", false),
                    span(mask, tokens, "mask", false),
                    span(index, tokens * top * 4, "index", true),
                    span(gate, tokens * top * 4, "gate", true),
                    span(counts, experts * 4, "counts", true),
                    span(prob_sum, experts * 4, "prob_sum", true),
                    span(workspace, need, "workspace", true)};
  st = check_spans(s, 7);
  if (st != RELAY_OK) return st;
  const int blocks = (int)forward_blocks(tokens);
  int32_t* part_count = reinterpret_cast<int32_t*>((reinterpret_cast<uintptr_t>(workspace) + 15) & ~(uintptr_t)15);
  float* part_prob = reinterpret_cast<float*>(part_count + (int64_t)blocks * experts);
  const ForwardArgs a{logits, row_stride, tokens, experts, top, normalize, mask, index, gate,
                      blocks == 1 ? counts : part_count, blocks == 1 ? prob_sum : part_prob};
  const size_t smem = (size_t)(kRouterWarps + 1) * experts * 4;
  cudaError_t e = by_width(experts, [&](auto n) {
    constexpr int N = decltype(n)::value;
    if (dtype == RELAY_BF16)
      router_forward_kernel<uint16_t, N><<<blocks, kRouterThreads, smem, stream>>>(a);
    else
      router_forward_kernel<float, N><<<blocks, kRouterThreads, smem, stream>>>(a);
    return cudaGetLastError();
  });
  if (e == cudaSuccess && blocks > 1) {
    router_join_kernel<<<(experts + 31) / 32, 32 * kJoinWarps, 0, stream>>>(part_count, part_prob, blocks,
                                                                           experts, counts, prob_sum);
    e = cudaGetLastError();
  }
  return done(e);
}

relay_status_t relay_balance_loss(const int32_t* counts, const float* prob_sum, int experts, int top,
                                  float coef, float* loss, float* d_prob, cudaStream_t stream) {
  using namespace relay;
  relay_status_t st = check_shape(RELAY_F32, 0, experts, top);
  if (st != RELAY_OK) return st;
  if (counts == nullptr || prob_sum == nullptr || loss == nullptr || d_prob == nullptr)
    return bad("counts, prob_sum, loss or d_prob is NULL");
  if (off(counts, 4) || off(prob_sum, 4) || off(loss, 4) || off(d_prob, 4)) return bad("an array is not element-aligned");
  const Span s[] = {span(counts, experts * 4, "counts", false), span(prob_sum, experts * 4, "prob_sum", false),
                    span(loss, 4, "loss", true), span(d_prob, experts * 4, "d_prob", true)};
  st = check_spans(s, 4);
  if (st != RELAY_OK) return st;
  balance_kernel<<<1, kBalanceThreads, 0, stream>>>(counts, prob_sum, experts, top, coef, loss, d_prob);
  return done(cudaGetLastError());
}

relay_status_t relay_router_backward(const void* logits, int64_t row_stride, relay_dtype_t dtype,
                                     int64_t tokens, int experts, int top, int normalize,
                                     const int32_t* index, const float* d_gate, const float* d_prob,
                                     void* d_logits, int64_t d_row_stride, cudaStream_t stream) {
  using namespace relay;
  relay_status_t st = check_shape(dtype, tokens, experts, top);
  if (st != RELAY_OK) return st;
  if (tokens == 0) return RELAY_OK;
  if (logits == nullptr || index == nullptr || d_logits == nullptr) return bad("logits, index or d_logits is NULL");
  if (row_stride < experts || d_row_stride < experts || row_stride > (1ll << 31) || d_row_stride > (1ll << 31))
    return bad("a row stride is less than experts or more than 2^31");
  const int E = esize_of(dtype);
  if (off(logits, E) || off(d_logits, E) || off(index, 4) || off(d_gate, 4) || off(d_prob, 4))
    return bad("an array is not element-aligned");
  const Span s[] = {span(logits, ((tokens - 1) * row_stride + experts) * E, "logits", false),
                    span(index, tokens * top * 4, "index", false),
                    span(d_gate, tokens * top * 4, "d_gate", false),
                    span(d_prob, experts * 4, "d_prob", false),
                    span(d_logits, ((tokens - 1) * d_row_stride + experts) * E, "d_logits", true)};
  st = check_spans(s, 5);
  if (st != RELAY_OK) return st;
  const BackwardArgs a{logits, d_logits, row_stride, d_row_stride, tokens, experts, top, normalize, index, d_gate, d_prob};
  const unsigned blocks = (unsigned)((tokens + kRouterWarps - 1) / kRouterWarps);
  return done(by_width(experts, [&](auto n) {
    constexpr int N = decltype(n)::value;
    if (dtype == RELAY_BF16)
      router_backward_kernel<uint16_t, N><<<blocks, kRouterThreads, 0, stream>>>(a);
    else
      router_backward_kernel<float, N><<<blocks, kRouterThreads, 0, stream>>>(a);
    return cudaGetLastError();
  }));
}

}  // extern "C"
