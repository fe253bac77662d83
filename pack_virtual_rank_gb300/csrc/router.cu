// router.cu -- relay_router_forward, relay_balance_loss, relay_router_backward.
//
// L lanes of a warp share a row (32 / L rows to a warp); a lane holds N neighbouring experts in
// registers, so the lowest lane of a tie holds the lowest expert. Up to 256 experts N is 8, so
// that a lane's values are one or two 16-byte loads where the rows allow it, and a warp's reductions
// serve as many rows as fit. The next rows are loaded while the present ones are worked on.
//
// Forward. The time goes into choosing, not into memory. Choosing takes k rounds of: the
// largest of the lanes' best, over unsigned keys in the order of the values; the lane that holds
// it steps to its next. A key is the value's upper 22 bits in order and the expert counted down,
// so keys are unique, a tie goes to the lower expert, and a round needs neither the holder's lane
// nor its index. That is exact for bf16. For fp32 it is exact unless two of the k + 1 largest
// agree in their upper 22 bits; such a row, and one with a NaN, chooses again by whole values
// (choose_exact). A lane finds its two best up front; only a lane chosen from twice, about one
// row in two at 8 of 256, scans its values again. The softmax
// per expert adds up in registers over the rows that a lane walks (a fixed assignment); lanes of a block join
// in shared memory in order and a second launch joins the blocks in order: no sum of floats
// depends on timing.
//
// Backward. p (a - sum p a) with a = d_prob plus d_gate at the chosen. The chosen are k of E, so the
// row is written from d_prob alone and lane j then completes the j-th chosen expert: comparing
// every value with every chosen index was most of the instructions.
#include <limits.h>
#include <math.h>
#include <string.h>

#include <algorithm>
#include <string>

#include "router.cuh"

namespace relay {
namespace {

struct ForwardArgs {
  const void* logits;
  int64_t ld, tokens;
  int experts, top, normalize, bytes;
  const uint8_t* mask;
  int32_t* index;
  float* gate;
  int32_t* part_count;  // [blocks][experts], or the result when one block runs
  float* part_prob;
};

// Chooses by whole values, NaN below -inf, for the L lanes of a row: lane j gets the j-th expert.
// Returns whether the row has a logit above -inf, or a NaN: a row that a NaN has reached is counted, and shows
// it. Rare, and kept out of the kernel's registers.
template <class T, int N, int L>
__device__ __noinline__ bool choose_exact(const T* x, int experts, int top, bool counted, int* chosen) {
  const int lane = threadIdx.x % 32, sub = lane % L;
  uint32_t last = ~0u;
  int last_e = -1;
  bool live = false, nan = false;
  for (int j = 0; j < top; ++j) {
    uint32_t best = 0;
    int best_e = 0;
    for (int i = 0; i < N && counted; ++i) {
      const int e = sub * N + i;
      if (e >= experts) break;
      const float v = ld1(x + e);
      nan |= v != v;
      const uint32_t k = v != v ? 1u : order_key(v);
      if ((k < last || (k == last && e > last_e)) && k > best) {
        best = k;
        best_e = e;
      }
    }
    const uint32_t win = max_row<L>(best);
    const unsigned holders = __ballot_sync(~0u, best == win) >> (lane - sub) & (L == 32 ? ~0u : (1u << (L % 32)) - 1);
    last_e = __shfl_sync(~0u, best_e, lane - sub + __ffs(holders) - 1);
    last = win;
    if (j == 0) live = max_row<L>(nan ? ~0u : win) > kKeyNegInf;
    if (sub == j) *chosen = last_e;
  }
  return live;
}

template <class T, int N, int L>
__global__ void __launch_bounds__(kRouterThreads, N == 8 ? 4 : 1) router_forward_kernel(const ForwardArgs a) {
  constexpr int kRows = 32 / L;
  constexpr int kTracked = L < 32 ? 3 : 2;  // a lane's best keys kept in order: fewer lanes are chosen from more often
  extern __shared__ float s_prob[];  // [warps * kRows][experts], then the counts [experts]
  int32_t* s_count = reinterpret_cast<int32_t*>(s_prob + kRouterWarps * kRows * a.experts);
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, sub = lane % L, e0 = sub * N;
  dep_launch();
  for (int e = threadIdx.x; e < a.experts; e += kRouterThreads) s_count[e] = 0;
  dep_wait();
  __syncthreads();
  float psum[N];
#pragma unroll
  for (int i = 0; i < N; ++i) psum[i] = 0.0f;
  const int64_t stride = (int64_t)gridDim.x * kRouterWarps * kRows;
  int64_t row = ((int64_t)blockIdx.x * kRouterWarps + warp) * kRows + lane / L;
  const T* x = static_cast<const T*>(a.logits);
  Lane<T, N> next;
  bool next_counted = false;
  auto fetch = [&](int64_t r) {
    next_counted = r < a.tokens && (a.mask == nullptr || a.mask[r] != 0);
    if (r < a.tokens) next.load(x + r * a.ld, e0, a.experts, a.bytes);
  };
  fetch(row);
  const bool full = a.experts == N * L;
  for (; row - lane / L < a.tokens; row += stride) {
    float v[N];
    next.values(v);
    const bool counted = next_counted;
    fetch(row + stride);
    uint32_t key[N], best = 0, second = 0, third = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      key[i] = unique_key(v[i], e0 + i);
      if (!full && e0 + i >= a.experts) key[i] = 0u;
      if (kTracked == 3) third = max(third, min(second, key[i]));
      second = max(second, min(best, key[i]));
      best = max(best, key[i]);
    }
    if (!counted) best = second = third = 0;
    uint32_t win = max_row<L>(best);
    bool live = win > (kKeyNegInf | kExpertMask);  // else masked out, or no logit above -inf (NaN: choose_exact)
    // the largest value: a bf16 key holds all of it
    float m;
    if (sizeof(T) == 2) {
      m = __uint_as_float(__float_as_uint(key_value(win)) & 0xffff0000u);
    } else {
      m = v[0];
#pragma unroll
      for (int i = 1; i < N; ++i) m = fmaxf(m, v[i]);
      m = key_value(max_row<L>(order_key(m)));
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = exp_below(v[i], m);
      sum += v[i];
    }
    sum = sum_row<L>(sum);
    const float inv = 1.0f / sum;
    int taken = 0;        // of the lane's kTracked best
    bool close = false;   // two of the largest agree in their upper bits
    uint32_t mine = 0;    // lane j: the key chosen j-th
#pragma unroll 4
    for (int j = 0; j < a.top; ++j) {
      const bool holder = best == win;
      if (sub == j) mine = win;
      uint32_t after = second;
      // the largest after the one just taken; a vote, so that it is a branch and not predicated
      // into every round
      if (__any_sync(~0u, holder && taken == kTracked - 1)) {
        uint32_t left = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) left = max(left, key[i] < win ? key[i] : 0u);
        if (taken == kTracked - 1) after = left;
      }
      if (holder) {
        best = after;
        if (kTracked == 3) second = third;
        taken = min(taken + 1, kTracked - 1);
      }
      win = max_row<L>(best);
    }
    if (sizeof(T) == 4) {
      const uint32_t after = __shfl_down_sync(~0u, mine, 1, L);
      close = sub < a.top && (mine ^ (sub + 1 == a.top ? win : after)) <= kExpertMask;
    }
    int chosen = key_expert(mine);
    if (__any_sync(~0u, counted && (close || sum != sum)))
      live = choose_exact<T, N, L>(x + (row < a.tokens ? row : 0) * a.ld, a.experts, a.top, counted, &chosen);
    if (live) {
#pragma unroll
      for (int i = 0; i < N; ++i) psum[i] = fmaf(v[i], inv, psum[i]);
    }
    const bool chose = live && sub < a.top;
    // the key lost the value's lower bits (fp32): read it again
    const float val = chose ? exp_below(ld1(x + row * a.ld + chosen), m) : 0.0f;
    float scale = inv;
    if (a.normalize) scale = 1.0f / sum_row<L>(val);
    if (sum != sum) scale = sum;
    if (sub < a.top && row < a.tokens) {
      a.index[row * a.top + sub] = live ? chosen : -1;
      a.gate[row * a.top + sub] = live ? val * scale : 0.0f;
      if (live) atomicAdd(&s_count[chosen], 1);  // integers: any order gives the same sum
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (e0 + i < a.experts) s_prob[(warp * kRows + lane / L) * a.experts + e0 + i] = psum[i];
  __syncthreads();
  for (int e = threadIdx.x; e < a.experts; e += kRouterThreads) {
    float p = 0.0f;
    for (int i = 0; i < kRouterWarps * kRows; ++i) p += s_prob[i * a.experts + e];
    a.part_prob[(int64_t)blockIdx.x * a.experts + e] = p;
    a.part_count[(int64_t)blockIdx.x * a.experts + e] = s_count[e];
  }
}

// Joins the blocks' partial sums: a block takes eight experts, its warps stride over the partials.
constexpr int kJoinWarps = 32;
__global__ void __launch_bounds__(32 * kJoinWarps)
    router_join_kernel(const int32_t* part_count, const float* part_prob, int blocks, int experts,
                       int32_t* counts, float* prob_sum) {
  __shared__ float s_p[kJoinWarps][33];
  __shared__ int32_t s_c[kJoinWarps][33];
  dep_launch();
  dep_wait();
  // a warp reads four blocks' partials at a time
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
  int experts, top, normalize, bytes, d_bytes;
  float scale;  // of the gates
  const int32_t* index;
  const float* d_gate;
  const float* d_prob;
};

template <class T, int N, int L>
__global__ void __launch_bounds__(kRouterThreads) router_backward_kernel(const BackwardArgs a) {
  constexpr int kRows = 32 / L;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, sub = lane % L, e0 = sub * N;
  dep_launch();
  dep_wait();
  float g[N];
#pragma unroll
  for (int i = 0; i < N; ++i) g[i] = e0 + i < a.experts && a.d_prob != nullptr ? a.d_prob[e0 + i] : 0.0f;
  const int64_t stride = (int64_t)gridDim.x * kRouterWarps * kRows;
  int64_t row = ((int64_t)blockIdx.x * kRouterWarps + warp) * kRows + lane / L;
  const T* x = static_cast<const T*>(a.logits);
  Lane<T, N> next;
  int next_index = -1;
  float next_dg = 0.0f;
  auto fetch = [&](int64_t r) {
    next_index = -1;
    next_dg = 0.0f;
    if (r >= a.tokens) return;
    next.load(x + r * a.ld, e0, a.experts, a.bytes);
    if (sub < a.top) {
      next_index = a.index[r * a.top + sub];
      if (a.d_gate != nullptr) next_dg = a.d_gate[r * a.top + sub] * a.scale;
    }
  };
  fetch(row);
  for (; row - lane / L < a.tokens; row += stride) {
    float p[N];
    next.values(p);
    const int mine = next_index;
    const float dg = next_dg;
    fetch(row + stride);
    const bool in = row < a.tokens, live = __shfl_sync(~0u, mine, lane - sub) >= 0;
    const bool holds = live && mine >= 0 && mine < a.experts;
    const float own = holds ? ld1(x + row * a.ld + mine) : -INFINITY;
    const float own_g = holds && a.d_prob != nullptr ? a.d_prob[mine] : 0.0f;
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i) m = fmaxf(m, p[i]);
    m = key_value(max_row<L>(order_key(m)));
    float sum = 0.0f, dot = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      p[i] = exp_below(p[i], m);
      sum += p[i];
      dot = fmaf(p[i], g[i], dot);
    }
    const float e = holds ? exp_below(own, m) : 0.0f;
    const float inv = 1.0f / sum_row<L>(sum);
    if (!a.normalize) dot = fmaf(e, dg, dot);
    dot = sum_row<L>(dot) * inv;
    float extra = e * inv * dg;
    if (a.normalize) {
      // chosen scores of 0 (relay_grouped_router_forward chooses by more than the score) have gates of 0
      const float z = sum_row<L>(e), c = z == 0.0f ? 0.0f : e / z, inner = sum_row<L>(c * dg);
      extra = c * (dg - inner);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = live ? p[i] * inv * (g[i] - dot) : 0.0f;
    T* dx = static_cast<T*>(a.d_logits) + row * a.d_ld;
    if (in) Lane<T, N>::store(dx, p, e0, a.experts, a.d_bytes);
    __syncwarp();  // orders the row's stores before the chosen experts'
    if (in && holds) st1(dx + mine, e * inv * (own_g - dot) + extra);
  }
}

// Values per lane and lanes per row: 8 and as few lanes as hold the experts and the choice.
template <class F>
cudaError_t by_width(int experts, int top, F f) {
  using std::integral_constant;
  const int lanes = std::max((experts + 7) / 8, top);
  if (lanes <= 4) return f(integral_constant<int, 8>(), integral_constant<int, 4>());
  if (lanes <= 8) return f(integral_constant<int, 8>(), integral_constant<int, 8>());
  if (lanes <= 16) return f(integral_constant<int, 8>(), integral_constant<int, 16>());
  if (lanes <= 32) return f(integral_constant<int, 8>(), integral_constant<int, 32>());
  if (lanes <= 64) return f(integral_constant<int, 16>(), integral_constant<int, 32>());
  return f(integral_constant<int, 32>(), integral_constant<int, 32>());
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

relay_status_t check_overlaps(const Array* s, int n) {
  for (int i = 0; i < n; ++i)
    for (int j = i + 1; j < n; ++j)
      if ((s[i].out || s[j].out) && overlap(s[i].span, s[j].span))
        return bad(std::string(s[i].what) + " overlaps " + s[j].what);
  return RELAY_OK;
}
}  // namespace

cudaError_t router_join(const int32_t* part_count, const float* part_prob, int blocks, int experts, int32_t* counts,
                        float* prob_sum, cudaStream_t stream) {
  return launch_chained(router_join_kernel, (experts + 7) / 8, 32 * kJoinWarps, 0, stream, part_count, part_prob, blocks, experts,
                        counts, prob_sum);
}

cudaError_t router_softmax_backward(const SoftmaxBackward& b, cudaStream_t stream) {
  const int64_t E = esize_of(b.dtype);
  const BackwardArgs a{b.logits, b.d_logits, b.ld, b.d_ld, b.tokens, b.experts, b.top, b.normalize,
                       load_bytes(b.logits, b.ld, E, b.experts), load_bytes(b.d_logits, b.d_ld, E, b.experts), b.scale,
                       b.index, b.d_gate, b.d_prob};
  // Four blocks an SM, whose warps load their next rows under the present ones (16 an SM: 2% slower at 131072 x 256
  // fp32). They are all resident where a thread has 64 registers at most: bf16 up to 256 experts, fp32 from 129 to
  // 256. fp32 up to 128 experts has 71 (three blocks an SM), 257 to 512 experts 91 (fp32) and 78, more 141 and 128:
  // there the last blocks start when the first end.
  const int blocks = (int)std::min<int64_t>((b.tokens + kRouterWarps - 1) / kRouterWarps, 4 * 152);
  return by_width(b.experts, b.top, [&](auto n, auto l) {
    constexpr int N = decltype(n)::value, L = decltype(l)::value;
    return launch_chained(b.dtype == RELAY_BF16 ? router_backward_kernel<uint16_t, N, L> : router_backward_kernel<float, N, L>,
                          blocks, kRouterThreads, 0, stream, a);
  });
}

}  // namespace relay

extern "C" {

int64_t relay_router_workspace_size(int64_t tokens, int experts) {
  using namespace relay;
  if (tokens < 0 || tokens > INT32_MAX || experts < 1 || experts > RELAY_ROUTER_MAX_EXPERTS) {
    guarded([] { return bad("tokens or experts out of range"); });
    return -1;
  }
  return forward_blocks(tokens, kRouterWarps) * experts * 8 + 16;  // a row to a warp: the most blocks
}

relay_status_t relay_router_forward(const void* logits, int64_t row_stride, relay_dtype_t dtype,
                                    int64_t tokens, int experts, int top, int normalize,
                                    const uint8_t* mask, int32_t* index, float* gate,
                                    int32_t* counts, float* prob_sum, void* workspace,
                                    int64_t workspace_bytes, cudaStream_t stream) {
  using namespace relay;
  return guarded([&]() -> relay_status_t {
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
    const Array s[] = {matrix(logits, tokens, experts * E, row_stride * E, "logits", false),
                      array(mask, tokens, "mask", false),
                      array(index, tokens * top * 4, "index", true),
                      array(gate, tokens * top * 4, "gate", true),
                      array(counts, experts * 4, "counts", true),
                      array(prob_sum, experts * 4, "prob_sum", true),
                      array(workspace, need, "workspace", true)};
    st = check_overlaps(s, 7);
    if (st != RELAY_OK) return st;
    int rows = kRouterWarps;
    by_width(experts, top, [&](auto, auto l) {
      rows *= 32 / decltype(l)::value;
      return cudaSuccess;
    });
    const int blocks = (int)forward_blocks(tokens, rows);
    int32_t* part_count = reinterpret_cast<int32_t*>((reinterpret_cast<uintptr_t>(workspace) + 15) & ~(uintptr_t)15);
    float* part_prob = reinterpret_cast<float*>(part_count + (int64_t)blocks * experts);
    const ForwardArgs a{logits, row_stride, tokens, experts, top, normalize, load_bytes(logits, row_stride, E, experts),
                        mask, index, gate,
                        blocks == 1 ? counts : part_count, blocks == 1 ? prob_sum : part_prob};
    cudaError_t e = by_width(experts, top, [&](auto n, auto l) {
      constexpr int N = decltype(n)::value, L = decltype(l)::value;
      const size_t smem = (size_t)(kRouterWarps * (32 / L) + 1) * experts * 4;
      return launch_chained(dtype == RELAY_BF16 ? router_forward_kernel<uint16_t, N, L> : router_forward_kernel<float, N, L>,
                            blocks, kRouterThreads, smem, stream, a);
    });
    if (e == cudaSuccess && blocks > 1) {
      e = router_join(part_count, part_prob, blocks, experts, counts, prob_sum, stream);
    }
    return done(e);
  });
}

relay_status_t relay_balance_loss(const int32_t* counts, const float* prob_sum, int experts, int top,
                                  float coef, float* loss, float* d_prob, cudaStream_t stream) {
  using namespace relay;
  return guarded([&]() -> relay_status_t {
    relay_status_t st = check_shape(RELAY_F32, 0, experts, top);
    if (st != RELAY_OK) return st;
    if (counts == nullptr || prob_sum == nullptr || loss == nullptr || d_prob == nullptr)
      return bad("counts, prob_sum, loss or d_prob is NULL");
    if (off(counts, 4) || off(prob_sum, 4) || off(loss, 4) || off(d_prob, 4)) return bad("an array is not element-aligned");
    const Array s[] = {array(counts, experts * 4, "counts", false), array(prob_sum, experts * 4, "prob_sum", false),
                      array(loss, 4, "loss", true), array(d_prob, experts * 4, "d_prob", true)};
    st = check_overlaps(s, 4);
    if (st != RELAY_OK) return st;
    return done(launch_chained(balance_kernel, 1, kBalanceThreads, 0, stream, counts, prob_sum, experts, top, coef, loss,
                               d_prob));
  });
}

relay_status_t relay_router_backward(const void* logits, int64_t row_stride, relay_dtype_t dtype,
                                     int64_t tokens, int experts, int top, int normalize,
                                     const int32_t* index, const float* d_gate, const float* d_prob,
                                     void* d_logits, int64_t d_row_stride, cudaStream_t stream) {
  using namespace relay;
  return guarded([&]() -> relay_status_t {
    relay_status_t st = check_shape(dtype, tokens, experts, top);
    if (st != RELAY_OK) return st;
    if (tokens == 0) return RELAY_OK;
    if (logits == nullptr || index == nullptr || d_logits == nullptr) return bad("logits, index or d_logits is NULL");
    if (row_stride < experts || d_row_stride < experts || row_stride > (1ll << 31) || d_row_stride > (1ll << 31))
      return bad("a row stride is less than experts or more than 2^31");
    const int E = esize_of(dtype);
    if (off(logits, E) || off(d_logits, E) || off(index, 4) || off(d_gate, 4) || off(d_prob, 4))
      return bad("an array is not element-aligned");
    const Array s[] = {matrix(logits, tokens, experts * E, row_stride * E, "logits", false),
                      array(index, tokens * top * 4, "index", false),
                      array(d_gate, tokens * top * 4, "d_gate", false),
                      array(d_prob, experts * 4, "d_prob", false),
                      matrix(d_logits, tokens, experts * E, d_row_stride * E, "d_logits", true)};
    st = check_overlaps(s, 5);
    if (st != RELAY_OK) return st;
    return done(router_softmax_backward(SoftmaxBackward{logits, d_logits, row_stride, d_row_stride, tokens, (int)dtype, experts, top,
                                                        normalize, 1.0f, index, d_gate, d_prob},
                                        stream));
  });
}

}  // extern "C"

namespace {
// A word as an int: out of range is -1, which every check refuses.
int word(int64_t v) { return v < INT_MIN || v > INT_MAX ? -1 : (int)v; }
}  // namespace

extern "C" {

// The same calls with their arguments, in order, as one block of 8-byte words (the coefficient as the
// bits of a double): for a caller whose foreign-function layer pays per argument.
relay_status_t relay_packed_router_forward(const int64_t* a) {
  return relay_router_forward(reinterpret_cast<const void*>(a[0]), a[1], (relay_dtype_t)a[2], a[3], word(a[4]), word(a[5]),
                              (int)a[6], reinterpret_cast<const uint8_t*>(a[7]), reinterpret_cast<int32_t*>(a[8]),
                              reinterpret_cast<float*>(a[9]), reinterpret_cast<int32_t*>(a[10]),
                              reinterpret_cast<float*>(a[11]), reinterpret_cast<void*>(a[12]), a[13],
                              reinterpret_cast<cudaStream_t>(a[14]));
}
relay_status_t relay_packed_router_balance(const int64_t* a) {
  double coef;
  memcpy(&coef, a + 4, sizeof coef);
  return relay_balance_loss(reinterpret_cast<const int32_t*>(a[0]), reinterpret_cast<const float*>(a[1]), word(a[2]),
                            word(a[3]), (float)coef, reinterpret_cast<float*>(a[5]), reinterpret_cast<float*>(a[6]),
                            reinterpret_cast<cudaStream_t>(a[7]));
}
relay_status_t relay_packed_router_backward(const int64_t* a) {
  return relay_router_backward(reinterpret_cast<const void*>(a[0]), a[1], (relay_dtype_t)a[2], a[3], word(a[4]),
                               word(a[5]), (int)a[6], reinterpret_cast<const int32_t*>(a[7]),
                               reinterpret_cast<const float*>(a[8]), reinterpret_cast<const float*>(a[9]),
                               reinterpret_cast<void*>(a[10]), a[11], reinterpret_cast<cudaStream_t>(a[12]));
}

}  // extern "C"
