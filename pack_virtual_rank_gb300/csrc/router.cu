// router.cu -- relay_router_forward, relay_balance_loss, relay_router_backward.
//
// One warp per row. Lane l holds the row's experts [l * N, (l + 1) * N) in registers, read with
// 16-byte loads where the rows allow it; the lowest lane of a tie holds the lowest expert.
//
// Forward. Choosing k of E takes k rounds of: the largest of the lanes' best (one warp-wide
// integer maximum over keys in the order of the values), the lowest lane that holds it steps to
// its next. A lane finds its two best up front; only a lane chosen from twice, about one row in
// two at 8 of 256, scans its values again, for the largest after the last one taken. Clearing
// and rescanning in every round took three times the instructions. The softmax per expert adds up in registers over the rows
// that a warp walks (a fixed assignment); warps join in shared memory in order and a second
// launch joins the blocks in order: no sum of floats depends on timing.
//
// Backward. p (a - sum p a) with a = d_prob plus d_gate at the chosen. The chosen are k of E, so the
// row is written from d_prob alone and lane j then completes the j-th chosen expert: comparing
// every value with every chosen index was most of the instructions.
#include <limits.h>
#include <math.h>

#include <algorithm>
#include <string>

#include "device.cuh"
#include "launch.cuh"
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

// exp(x - m). The difference first: x and m may be the type's lowest value, which has no log2.
__device__ __forceinline__ float exp_below(float x, float m) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"((x - m) * 1.4426950408889634f));
  return y;
}

// The lane's N values of a row; -inf past the last expert. vec: the rows are aligned to a lane's
// values (at most 16 bytes) and a lane holds N experts or none.
__device__ __forceinline__ uint4 ld16(const void* p) {
  uint4 r;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}
template <int N>
__device__ __forceinline__ void load_row(float (&v)[N], const float* x, int lane, int experts, bool vec) {
  const int e0 = lane * N;
  if (vec) {
    if constexpr (N >= 4) {
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        const uint4 u = e0 < experts ? ld16(x + e0 + i) : make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u);
        TF32::unpack(u, v + i);
      }
      return;
    } else if constexpr (N == 2) {
      const float2 u = e0 < experts ? *reinterpret_cast<const float2*>(x + e0) : make_float2(-INFINITY, -INFINITY);
      v[0] = u.x;
      v[1] = u.y;
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = e0 + i < experts ? x[e0 + i] : -INFINITY;
}
template <int N>
__device__ __forceinline__ void load_row(float (&v)[N], const uint16_t* x, int lane, int experts, bool vec) {
  const int e0 = lane * N;
  if (vec) {
    if constexpr (N >= 8) {
#pragma unroll
      for (int i = 0; i < N; i += 8) {
        const uint4 u = e0 < experts ? ld16(x + e0 + i) : make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
        TBF16::unpack(u, v + i);
      }
      return;
    } else if constexpr (N >= 2) {
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const uint32_t u = e0 < experts ? *reinterpret_cast<const uint32_t*>(x + e0 + i) : 0xff80ff80u;
        v[i] = __uint_as_float(u << 16);
        v[i + 1] = __uint_as_float(u & 0xffff0000u);
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = e0 + i < experts ? ld1(x + e0 + i) : -INFINITY;
}
template <int N>
__device__ __forceinline__ void store_row(float* x, const float (&v)[N], int lane, int experts, bool vec) {
  const int e0 = lane * N;
  if (e0 >= experts) return;
  if (vec) {
    if constexpr (N >= 4) {
#pragma unroll
      for (int i = 0; i < N; i += 4)
        *reinterpret_cast<float4*>(x + e0 + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
      return;
    } else if constexpr (N == 2) {
      *reinterpret_cast<float2*>(x + e0) = make_float2(v[0], v[1]);
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (e0 + i < experts) x[e0 + i] = v[i];
}
template <int N>
__device__ __forceinline__ void store_row(uint16_t* x, const float (&v)[N], int lane, int experts, bool vec) {
  const int e0 = lane * N;
  if (e0 >= experts) return;
  if (vec) {
    if constexpr (N >= 8) {
#pragma unroll
      for (int i = 0; i < N; i += 8) *reinterpret_cast<uint4*>(x + e0 + i) = TBF16::pack(v + i);
      return;
    } else if constexpr (N >= 2) {
#pragma unroll
      for (int i = 0; i < N; i += 2) *reinterpret_cast<uint32_t*>(x + e0 + i) = bf16x2_rn(v[i], v[i + 1]);
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (e0 + i < experts) st1(x + e0 + i, v[i]);
}

struct ForwardArgs {
  const void* logits;
  int64_t ld, tokens;
  int experts, top, normalize, vec;
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
  dep_launch();
  for (int e = threadIdx.x; e < a.experts; e += kRouterThreads) s_count[e] = 0;
  dep_wait();
  __syncthreads();
  float psum[N];
#pragma unroll
  for (int i = 0; i < N; ++i) psum[i] = 0.0f;
  const unsigned below = (1u << lane) - 1;
  const int64_t stride = (int64_t)gridDim.x * kRouterWarps;
  for (int64_t row = (int64_t)blockIdx.x * kRouterWarps + warp; row < a.tokens; row += stride) {
    int32_t* index = a.index + row * a.top;
    float* gate = a.gate + row * a.top;
    uint32_t key[N], best = 0, second = 0;
    int best_i = 0, second_i = 0;
    float v[N];
    bool counted = a.mask == nullptr || a.mask[row] != 0;
    if (counted) {
      load_row<N>(v, static_cast<const T*>(a.logits) + row * a.ld, lane, a.experts, a.vec);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        key[i] = lane * N + i < a.experts ? order_key(v[i]) : 0u;
        // equal keys: the lower expert stays ahead
        if (key[i] > best) {
          second = best;
          second_i = best_i;
          best = key[i];
          best_i = i;
        } else if (key[i] > second) {
          second = key[i];
          second_i = i;
        }
      }
    }
    uint32_t win = counted ? __reduce_max_sync(~0u, best) : 0u;
    if (win <= kKeyNegInf) {  // masked out, or no logit above -inf
      if (lane < a.top) {
        index[lane] = -1;
        gate[lane] = 0.0f;
      }
      continue;
    }
    const float m = key_value(win);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = exp_below(v[i], m);
      sum += v[i];
    }
    sum = sum_warp(sum);
    const float inv = 1.0f / sum;
#pragma unroll
    for (int i = 0; i < N; ++i) psum[i] = fmaf(v[i], inv, psum[i]);
    bool again = false;  // the lane's second best is its best now
    float mine = 0.0f, chosen_sum = 0.0f;
    for (int j = 0; j < a.top; ++j) {
      const float val = win <= 1u ? NAN : exp_below(key_value(win), m);
      chosen_sum += val;
      if (lane == j) mine = val;
      const unsigned holders = __ballot_sync(~0u, best == win);
      if (best == win && (holders & below) == 0) {
        const int e = lane * N + best_i;
        index[j] = e;
        atomicAdd(&s_count[e], 1);  // integers: any order gives the same sum
        if (!again) {
          again = true;
          best = second;
          best_i = second_i;
        } else {
          // the largest after the one just taken
          uint32_t k = 0;
          int at = 0;
#pragma unroll
          for (int i = 0; i < N; ++i)
            if ((key[i] < win || (key[i] == win && i > best_i)) && key[i] > k) {
              k = key[i];
              at = i;
            }
          best = k;
          best_i = at;
        }
      }
      win = __reduce_max_sync(~0u, best);
    }
    float scale = a.normalize ? 1.0f / chosen_sum : inv;
    if (sum != sum) scale = sum;
    if (lane < a.top) gate[lane] = mine * scale;
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
constexpr int kJoinWarps = 32;
__global__ void __launch_bounds__(32 * kJoinWarps)
    router_join_kernel(const int32_t* part_count, const float* part_prob, int blocks, int experts,
                       int32_t* counts, float* prob_sum) {
  __shared__ float s_p[kJoinWarps][33];
  __shared__ int32_t s_c[kJoinWarps][33];
  dep_launch();
  dep_wait();
  // eight experts to a block: a warp reads four blocks' partials at a time
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, e = blockIdx.x * 8 + lane % 8;
  float p = 0.0f;
  int32_t c = 0;
  if (e < experts) {
#pragma unroll 4
    for (int b = warp * 4 + lane / 8; b < blocks; b += 4 * kJoinWarps) {
      p += part_prob[(int64_t)b * experts + e];
      c += part_count[(int64_t)b * experts + e];
    }
  }
#pragma unroll
  for (int o = 8; o < 32; o <<= 1) {
    p += __shfl_xor_sync(~0u, p, o);
    c += __shfl_xor_sync(~0u, c, o);
  }
  s_p[lane % 8][warp] = p;
  s_c[lane % 8][warp] = c;
  __syncthreads();
  if (warp >= 8 || blockIdx.x * 8 + warp >= experts) return;
  p = sum_warp(s_p[warp][lane]);
  c = __reduce_add_sync(~0u, s_c[warp][lane]);
  if (lane == 0) {
    prob_sum[blockIdx.x * 8 + warp] = p;
    counts[blockIdx.x * 8 + warp] = c;
  }
}

constexpr int kBalanceThreads = 256;
__global__ void __launch_bounds__(kBalanceThreads)
    balance_kernel(const int32_t* counts, const float* prob_sum, int experts, int top, float coef,
                   float* loss, float* d_prob) {
  __shared__ long long s_total[kBalanceThreads / 32];
  __shared__ float s_loss[kBalanceThreads / 32];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  dep_launch();
  dep_wait();
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
  int experts, top, normalize, vec, d_vec;
  const int32_t* index;
  const float* d_gate;
  const float* d_prob;
};

template <class T, int N>
__global__ void __launch_bounds__(kRouterThreads) router_backward_kernel(const BackwardArgs a) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  dep_launch();
  dep_wait();
  float g[N];
#pragma unroll
  for (int i = 0; i < N; ++i)
    g[i] = lane * N + i < a.experts && a.d_prob != nullptr ? a.d_prob[lane * N + i] : 0.0f;
  const int64_t stride = (int64_t)gridDim.x * kRouterWarps;
  for (int64_t row = (int64_t)blockIdx.x * kRouterWarps + warp; row < a.tokens; row += stride) {
    const T* x = static_cast<const T*>(a.logits) + row * a.ld;
    T* dx = static_cast<T*>(a.d_logits) + row * a.d_ld;
    const int mine = lane < a.top ? a.index[row * a.top + lane] : -1;
    const float dg = lane < a.top && a.d_gate != nullptr ? a.d_gate[row * a.top + lane] : 0.0f;
    float p[N];
    if (__shfl_sync(~0u, mine, 0) < 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) p[i] = 0.0f;
      store_row<N>(dx, p, lane, a.experts, a.d_vec);
      continue;
    }
    load_row<N>(p, x, lane, a.experts, a.vec);
    const bool holds = mine >= 0 && mine < a.experts;
    const float own = holds ? ld1(x + mine) : -INFINITY;
    // the first chosen logit is the row's largest, but the index is the caller's
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i) m = fmaxf(m, p[i]);
    m = key_value(__reduce_max_sync(~0u, order_key(m)));
    float sum = 0.0f, dot = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      p[i] = exp_below(p[i], m);
      sum += p[i];
      dot = fmaf(p[i], g[i], dot);
    }
    const float e = exp_below(own, m);  // 0 for a lane without a choice
    const float own_prob = holds && a.d_prob != nullptr ? a.d_prob[mine] : 0.0f;
    const float inv = 1.0f / sum_warp(sum);
    const float own_p = e * inv;
    if (!a.normalize) dot = fmaf(e, dg, dot);
    dot = sum_warp(dot) * inv;
    float extra;
    if (a.normalize) {
      const float c = e / sum_warp(e), inner = sum_warp(c * dg);
      extra = c * (dg - inner);
    } else {
      extra = own_p * dg;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = p[i] * inv * (g[i] - dot);
    store_row<N>(dx, p, lane, a.experts, a.d_vec);
    __syncwarp();  // orders the row's stores before the chosen experts'
    if (holds) st1(dx + mine, own_p * (own_prob - dot) + extra);
  }
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

// Blocks of the forward pass, whose statistics are joined afterwards: at most four an SM of the
// GB300's 152 (also with another device current, so that the workspace is one size).
int64_t forward_blocks(int64_t tokens) {
  return std::max<int64_t>(1, std::min<int64_t>((tokens + kRouterWarps - 1) / kRouterWarps, 4 * 152));
}

// Rows a lane's values can be read from (or written to) whole: see load_row.
int whole_lanes(const void* p, int64_t ld, int64_t esize, int experts) {
  int n = 1;
  while (n * 32 < experts) n *= 2;
  const int64_t bytes = std::min<int64_t>(16, n * esize);
  return experts % n == 0 && reinterpret_cast<uintptr_t>(p) % bytes == 0 && ld * esize % bytes == 0;
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
  const ForwardArgs a{logits, row_stride, tokens, experts, top, normalize, whole_lanes(logits, row_stride, E, experts),
                      mask, index, gate,
                      blocks == 1 ? counts : part_count, blocks == 1 ? prob_sum : part_prob};
  const size_t smem = (size_t)(kRouterWarps + 1) * experts * 4;
  cudaError_t e = by_width(experts, [&](auto n) {
    constexpr int N = decltype(n)::value;
    return launch_chained(dtype == RELAY_BF16 ? router_forward_kernel<uint16_t, N> : router_forward_kernel<float, N>,
                          blocks, kRouterThreads, smem, stream, a);
  });
  if (e == cudaSuccess && blocks > 1) {
    e = launch_chained(router_join_kernel, (experts + 7) / 8, 32 * kJoinWarps, 0, stream, part_count, part_prob, blocks,
                       experts, counts, prob_sum);
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
  return done(launch_chained(balance_kernel, 1, kBalanceThreads, 0, stream, counts, prob_sum, experts, top, coef, loss,
                             d_prob));
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
  const BackwardArgs a{logits, d_logits, row_stride, d_row_stride, tokens, experts, top, normalize,
                       whole_lanes(logits, row_stride, E, experts), whole_lanes(d_logits, d_row_stride, E, experts),
                       index, d_gate, d_prob};
  const int blocks = (int)std::min<int64_t>((tokens + kRouterWarps - 1) / kRouterWarps, 8 * 152);
  return done(by_width(experts, [&](auto n) {
    constexpr int N = decltype(n)::value;
    return launch_chained(dtype == RELAY_BF16 ? router_backward_kernel<uint16_t, N> : router_backward_kernel<float, N>,
                          blocks, kRouterThreads, 0, stream, a);
  }));
}

}  // extern "C"
