// grouped_router.cu -- relay_grouped_router_forward, relay_grouped_router_backward, relay_router_bias_update.
//
//   s = 1 / (1 + exp(-x)) or softmax(x);  c = s + bias
//   a group's value = the sum of its one or two largest c; the `kept` largest groups stay
//   index = the top largest c of the groups that stayed; gate = scale * s, or scale * s / sum of the row's chosen s
//
// The rows lie in registers as in router.cu, with one more rule: a lane's experts are of one group. A group takes P lanes (a
// power of two), so its two largest come out of log2 P exchanges, and each lane counts how many groups are before
// its own.
//
// The choice is by exact values: of two near ones the larger, of equal ones the lower expert. Without a bias the order
// of c is that of x, and the keys are router.cu's. With one, c is computed in fp32, and a key is 22 bits of its distance below the
// row's largest, in steps of 2^-21 of the largest score (2 of it in all; what is further below is only known to be). Where two
// neighbours in the choice are nearer than fp32's error allows, and not equal in logit and bias (one row in some hundred), the
// chosen and a few candidates more are ranked by their values in 64 bits, one to a lane; groups as near to one another are compared
// by the 64-bit values of their largest. What that does not settle is chosen again in 64 bits as a whole (choose_slow). (All near rows
// chosen again as a whole: 99 us at 65536 x 256 bf16, eight groups, and not 73.)
//
// Bound by chains of dependent instructions: a round of the choice is a maximum over the row's lanes, a vote and a selection, and 24
// warps an SM do not hide one another's (the busiest unit is busy 59% of the time; most stalls are waits for a fixed latency). 65536
// x 256 bf16, 8 of 256 from 4 of 8 groups with a bias: 73 us, its bytes 5. The backward pass waits for memory, the row and then its
// chosen experts' logits, and for its sums over the row, one behind the other: 24 us, its bytes 10.
#include <float.h>
#include <limits.h>
#include <math.h>
#include <string.h>

#include <algorithm>
#include <string>
#include <type_traits>

#include "router.cuh"

namespace relay {
namespace {

struct GroupArgs {
  const void* logits;
  int64_t ld, tokens;
  int experts, groups, size, kept, lanes, top, group_sum, normalize, bytes;  // groups of `size` experts on `lanes` lanes each
  float scale;
  const float* bias;
  const uint8_t* mask;
  int32_t* index;
  float* gate;
  int32_t* part_count;  // [blocks][experts], or the result when one block runs
  float* part_prob;
};

__device__ __forceinline__ float reciprocal(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float exp2_near(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 0 at -inf, 1 at +inf. The exponent's rounding is 2^-24 of it: |x| 2^-23 of exp(-x).
__device__ __forceinline__ float sigmoid_near(float x) { return reciprocal(1.0f + exp2_near(x * -1.4426950408889634f)); }

// A lane's place in its row.
struct Place {
  int sub, group, e0, end;  // lane of the row, its group (a.groups and more: idle), its experts e0 .. end - 1 (at most N)
};
template <int N>
__device__ __forceinline__ Place place_of(const GroupArgs& a, int sub) {
  Place p;
  p.sub = sub;
  p.group = sub / a.lanes;
  p.end = min((p.group + 1) * a.size, a.experts);
  p.e0 = p.group < a.groups ? p.group * a.size + sub % a.lanes * N : p.end;
  return p;
}

__device__ __forceinline__ double exchange(double v, int o) { return __shfl_xor_sync(~0u, v, o); }
__device__ __forceinline__ float exchange(float v, int o) { return __shfl_xor_sync(~0u, v, o); }
__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ float smaller(float a, float b) { return fminf(a, b); }
__device__ __forceinline__ double larger(double a, double b) { return fmax(a, b); }
__device__ __forceinline__ double smaller(double a, double b) { return fmin(a, b); }
// The two largest over the lanes of a group.
template <class F>
__device__ __forceinline__ void join_two(F& one, F& two, int lanes) {
  for (int o = lanes / 2; o > 0; o >>= 1) {
    const F x = exchange(one, o), y = exchange(two, o);
    two = larger(smaller(one, x), larger(two, y));
    one = larger(one, x);
  }
}
// Groups before the lane's own: of a larger value, or an equal one and a lower number.
template <class F>
__device__ __forceinline__ int groups_before(const GroupArgs& a, F value, int group, int lane0) {
  int n = 0;
  for (int q = 0; q < a.groups; ++q) {
    const F other = __shfl_sync(~0u, value, lane0 + q * a.lanes);
    n += other > value || (other == value && q < group);
  }
  return n;
}

// The choice of a row in 64 bits: the chosen expert of lane j, or -1. Scores that are NaN stand below all others that can be
// chosen: a softmax is taken over the logits that are numbers, so that a NaN logit makes its own score NaN and no other's. Of
// logits of +inf each has an equal share. Rare, and kept out of the kernel's registers.
template <class T, int N, int L, bool SIGMOID>
__device__ __noinline__ int choose_slow(const GroupArgs& a, const T* x, bool counted, int sub) {
  const int lane0 = threadIdx.x % 32 - sub;
  const Place at = place_of<N>(a, sub);
  double c[N], top = -INFINITY, sum = 0.0;
  uint32_t can = 0;  // experts that can be chosen
  for (int i = 0; i < N; ++i) {
    c[i] = counted && at.e0 + i < at.end ? (double)ld1(x + at.e0 + i) : -INFINITY;
    if (!(c[i] == -INFINITY)) can |= 1u << i;
    top = fmax(top, c[i]);
  }
  auto below = [&](double v) { return v == top ? 1.0 : exp(v - top); };  // also at +inf
  if (!SIGMOID && (a.bias != nullptr || a.group_sum > 1)) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) top = fmax(top, exchange(top, o));
    for (int i = 0; i < N; ++i)
      if ((can >> i & 1) && c[i] == c[i]) sum += below(c[i]);
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) sum += exchange(sum, o);
  }
  auto score = [&](double v) { return SIGMOID ? 1.0 / (1.0 + exp(-v)) : below(v) / sum; };
  auto ordered = [](double v) { return v != v ? -DBL_MAX / 2 : v; };  // two of them still stand above a group of which nothing can be chosen
  double one = -INFINITY, two = -INFINITY;
  for (int i = 0; i < N; ++i) {
    if (!(can >> i & 1)) continue;
    double v = c[i];  // as the groups are compared
    if (a.bias != nullptr) {
      const float b = a.bias[at.e0 + i];
      v = c[i] = b == -INFINITY ? -INFINITY : score(c[i]) + b;
      if (c[i] == -INFINITY) {
        can &= ~(1u << i);
        continue;
      }
    } else if (a.group_sum > 1) {
      v = score(v);
    }
    c[i] = ordered(c[i]);
    v = ordered(v);
    two = fmax(two, fmin(one, v));
    one = fmax(one, v);
  }
  if (a.groups > 1) {
    join_two(one, two, a.lanes);
    if (a.group_sum > 1 && two > -INFINITY) one += two;
    if (groups_before(a, one, at.group, lane0) >= a.kept) can = 0;
  }
  int chosen = -1;
  for (int j = 0; j < a.top; ++j) {
    double best = -INFINITY;
    int e = INT_MAX;
    for (int i = 0; i < N; ++i)
      if ((can >> i & 1) && (e == INT_MAX || c[i] > best)) {
        best = c[i];
        e = at.e0 + i;
      }
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) {
      const double other = exchange(best, o);
      const int other_e = __shfl_xor_sync(~0u, e, o);
      if (other_e != INT_MAX && (e == INT_MAX || other > best || (other == best && other_e < e))) {
        best = other;
        e = other_e;
      }
    }
    if (e >= at.e0 && e < at.e0 + N && e < at.end) can &= ~(1u << (e - at.e0));
    if (sub == j && e != INT_MAX) chosen = e;
  }
  return chosen;
}

// Blocks an SM holds. Registers that the 64-bit paths want spill at each of these bounds (60 to 140 bytes at three blocks of 8 values a
// lane); more blocks spill more and are slower, and fewer too: one of 16 values takes 138 us and not 101 at 65536 x 512 bf16, eight groups.
constexpr int resident(int values) { return values == 8 ? 3 : values == 16 ? 2 : 1; }

template <class T, int N, int L, bool SIGMOID>
__global__ void __launch_bounds__(kRouterThreads, resident(N)) grouped_forward_kernel(const GroupArgs a) {
  constexpr int kRows = 32 / L;
  constexpr int kTracked = L < 32 ? 3 : 2;  // a lane's best keys kept in order: fewer lanes are chosen from more often
  extern __shared__ float s_prob[];         // [warps * kRows][experts], then the counts [experts]
  int32_t* s_count = reinterpret_cast<int32_t*>(s_prob + kRouterWarps * kRows * a.experts);
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, sub = lane % L, lane0 = lane - sub;
  const Place at = place_of<N>(a, sub);
  dep_launch();
  for (int e = threadIdx.x; e < a.experts; e += kRouterThreads) s_count[e] = 0;
  dep_wait();
  __syncthreads();
  const bool biased = a.bias != nullptr;
  float psum[N], bias[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    psum[i] = 0.0f;
    bias[i] = biased && at.e0 + i < at.end ? a.bias[at.e0 + i] : 0.0f;
  }
  const int64_t stride = (int64_t)gridDim.x * kRouterWarps * kRows;
  int64_t row = ((int64_t)blockIdx.x * kRouterWarps + warp) * kRows + lane / L;
  const T* x = static_cast<const T*>(a.logits);
  Lane<T, N> next;
  bool next_counted = false;
  auto fetch = [&](int64_t r) {
    next_counted = r < a.tokens && (a.mask == nullptr || a.mask[r] != 0);
    if (r < a.tokens) next.load(x + r * a.ld, at.e0, at.end, a.bytes);
  };
  fetch(row);
  const bool full = a.size == N * a.lanes && a.groups * a.lanes == L;  // every lane has N experts
  for (; row - lane / L < a.tokens; row += stride) {
    float c[N], s[N];
    next.values(c);
    const bool counted = next_counted;
    fetch(row + stride);
    // scores, and what the choice is by
    float m = 0.0f, total = 0.0f;
    if (!SIGMOID) {
      m = c[0];
#pragma unroll
      for (int i = 1; i < N; ++i) m = fmaxf(m, c[i]);
      m = key_value(max_row<L>(order_key(m)));
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (!full && at.e0 + i >= at.end) c[i] = -INFINITY;  // also where a row's load brought more than the lane's own
      s[i] = SIGMOID ? sigmoid_near(c[i]) : exp_below(c[i], m);
      if (!SIGMOID && c[i] == -INFINITY) s[i] = 0.0f;
      total += s[i];
    }
    total = sum_row<L>(total);
    const float inv = total == 0.0f ? 0.0f : 1.0f / total, largest = SIGMOID ? 1.0f : inv;
    if (!SIGMOID) {
#pragma unroll
      for (int i = 0; i < N; ++i) s[i] *= inv;
    }
    if (biased) {
#pragma unroll
      for (int i = 0; i < N; ++i) c[i] = c[i] == -INFINITY ? -INFINITY : s[i] + bias[i];
    }
    bool close = false, stays = true;
    if (a.groups > 1) {
      float one = -INFINITY, two = -INFINITY;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        two = fmaxf(two, fminf(one, c[i]));
        one = fmaxf(one, c[i]);
      }
      join_two(one, two, a.lanes);
      float value = one, error = 0.0f;
      const bool computed = biased || a.group_sum > 1;  // logits compare exactly
      if (computed) {
        const float near = one > -INFINITY ? fmaxf(fabsf(one), fabsf(two > -INFINITY ? two : 0.0f)) : 0.0f;
        if (biased) {
          if (a.group_sum > 1 && two > -INFINITY) value = one + two;
          error = 2e-6f * largest + 0x1p-21f * near;
        } else {
          value = one == -INFINITY ? -INFINITY
                  : SIGMOID ? sigmoid_near(one) + sigmoid_near(two)
                            : (exp_below(one, m) + (two > -INFINITY ? exp_below(two, m) : 0.0f)) * inv;
          error = 2e-6f * largest;
        }
      }
      stays = groups_before(a, value, at.group, lane0) < a.kept && at.group < a.groups;
      if (computed) {
        // the least that stays against the largest that does not
        const float least = key_value(~max_row<L>(stays ? ~order_key(value) : 0u));
        const float most = key_value(max_row<L>(!stays && at.group < a.groups ? order_key(value) : kKeyNegInf));
        error = key_value(max_row<L>(order_key(error)));
        close = most > -INFINITY && !(least - most > error);
        if (__any_sync(~0u, counted && close)) {
          if (SIGMOID || !biased) {
            // the groups' values in 64 bits, from the experts that may be their largest (a softmax's without its sum)
            const float from = (a.group_sum > 1 && two > -INFINITY ? two : one) - (biased ? error : 0.0f);  // logits are exact
            uint32_t may = 0;
#pragma unroll
            for (int i = 0; i < N; ++i) may |= (uint32_t)(c[i] >= from && c[i] > -INFINITY) << i;
            double first = -INFINITY, second = -INFINITY;
            const T* xr = x + (row < a.tokens ? row : 0) * a.ld;
            while (may != 0) {
              const int e = at.e0 + __ffs(may) - 1;
              may &= may - 1;
              const double v = (double)ld1(xr + e);
              const double score = SIGMOID ? 1.0 / (1.0 + exp(-v)) + (biased ? (double)a.bias[e] : 0.0) : exp(v - m);
              second = larger(second, smaller(first, score));
              first = larger(first, score);
            }
            __syncwarp();
            join_two(first, second, a.lanes);
            if (a.group_sum > 1 && second > -INFINITY) first += second;
            stays = groups_before(a, first, at.group, lane0) < a.kept && at.group < a.groups;
            close = false;
          }  // the softmax's sum is wanted in 64 bits: choose_slow
        }
      }
    }
    // keys
    uint32_t key[N], best = 0, second = 0, third = 0;
    float far = 0.0f;  // steps in which fp32 may be wrong
    if (biased) {
      float most = -INFINITY;
#pragma unroll
      for (int i = 0; i < N; ++i) most = fmaxf(most, c[i]);
      most = key_value(max_row<L>(stays ? order_key(most) : kKeyNegInf));
      const float steps = SIGMOID ? 0x1p21f : 0x1p21f * total;
      far = 6.0f + fabsf(most) * (SIGMOID ? 1.0f : total);
      close |= !(most < INFINITY);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        // added to 2^23 the steps are the fraction's low bits; what is above them leaves by the shift
        const float below = fmaxf(fmaf(c[i] - most, steps, 4194303.0f), 1.0f) + 8388608.0f;
        key[i] = c[i] == -INFINITY || !stays ? 0u : __float_as_uint(below) << 10 | (kExpertMask - (uint32_t)(at.e0 + i));
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) key[i] = c[i] == -INFINITY || !stays ? 0u : unique_key(c[i], at.e0 + i);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (kTracked == 3) third = max(third, min(second, key[i]));
      second = max(second, min(best, key[i]));
      best = max(best, key[i]);
    }
    if (!counted) best = second = third = 0;
    uint32_t win = max_row<L>(best);
    int taken = 0;      // of the lane's kTracked best
    uint32_t mine = 0;  // lane j: the key chosen j-th, 0 when there are no more
    auto choose = [&](int j) {
      const bool holder = best == win;
      if (sub == j) mine = win;
      uint32_t after = second;
      // the largest after the one just taken; a vote, so that it is a branch and not predicated into every round
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
    };
#pragma unroll 4
    for (int j = 0; j < a.top; ++j) choose(j);
    const T* xr = x + (row < a.tokens ? row : 0) * a.ld;
    int place = sub;  // of the lane's key in the choice
    if (biased || sizeof(T) == 4) {
      // keys that do not tell which is larger
      auto alike = [&](uint32_t k, uint32_t below) {
        return biased ? (float)((k >> 10) - (below >> 10)) <= far : (k ^ below) <= kExpertMask;
      };
      const uint32_t down = __shfl_down_sync(~0u, mine, 1, L), after = sub + 1 == a.top ? win : down;
      bool near = sub < a.top && mine != 0 && after != 0 && alike(mine, after);
      bool same = false;  // the last one chosen and the first one left
      if (near) {  // equal ones are in the order of their experts
        const int e = key_expert(mine), f = key_expert(after);
        near = ld1(xr + e) != ld1(xr + f) || (biased && a.bias[e] != a.bias[f]);
        same = !near && sub + 1 == a.top;
      }
      if (__any_sync(~0u, counted && same)) {
        // one that is larger may stand behind equal ones
        const uint32_t last = __shfl_sync(~0u, mine, lane0 + a.top - 1);
        if (__shfl_sync(~0u, (int)same, lane0 + a.top - 1)) {
          const int e = key_expert(last);
          const float v = ld1(xr + e), b = biased ? a.bias[e] : 0.0f;
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (key[i] != 0 && key[i] < last && alike(last, key[i])) near |= ld1(xr + at.e0 + i) != v || (biased && a.bias[at.e0 + i] != b);
        }
      }
      if (__any_sync(~0u, counted && near)) {
        if (SIGMOID || !biased) {
          // a few more candidates, ranked by their exact values
          const int many = min(L, a.top + 4);
          for (int j = a.top; j < many; ++j) choose(j);
          const uint32_t last = __shfl_sync(~0u, mine, lane0 + a.top - 1);
          close |= last != 0 && win != 0 && alike(last, win);  // not enough of them
          double value = -INFINITY;
          if (mine != 0) {
            const double v = (double)ld1(xr + key_expert(mine));
            value = biased ? 1.0 / (1.0 + exp(-v)) + (double)a.bias[key_expert(mine)] : v;
          }
          place = mine != 0 ? 0 : sub < a.top ? sub : 32;
          for (int j = 0; j < many; ++j) {
            const double v = __shfl_sync(~0u, value, lane0 + j);
            const uint32_t k = __shfl_sync(~0u, mine, lane0 + j);
            if (mine != 0 && k != 0) place += v > value || (v == value && key_expert(k) < key_expert(mine));
          }
        } else {
          close |= near;  // the softmax's sum is wanted in 64 bits
        }
      }
    }
    int chosen = mine != 0 && place < a.top ? key_expert(mine) : -1;
    bool live = __shfl_sync(~0u, mine, lane0) != 0;  // something was chosen
    if (__any_sync(~0u, counted && (close || total != total))) {
      chosen = choose_slow<T, N, L, SIGMOID>(a, xr, counted, sub);
      place = sub;
      live = __shfl_sync(~0u, chosen, lane0) >= 0;
    }
    if (live) {
#pragma unroll
      for (int i = 0; i < N; ++i) psum[i] = SIGMOID ? fmaf(s[i], inv, psum[i]) : psum[i] + s[i];
    }
    const bool chose = chosen >= 0;
    // the scores of the chosen, to fp32's rounding; of a softmax before the division by its sum. What is below the normal
    // range is 0, as in the gradient
    float own = 0.0f;
    if (chose) {
      const float v = ld1(xr + chosen);
      own = SIGMOID ? 1.0f / (1.0f + expf(-v)) : expf(v - m);
      if (own < FLT_MIN) own = 0.0f;
    }
    if (a.normalize) {
      const float z = sum_row<L>(own);
      own = z == 0.0f ? 0.0f : own / z;
    } else if (!SIGMOID) {
      own *= inv;
    }
    own *= a.scale;
    if (total != total) own = total;
    if (place < a.top && row < a.tokens) {
      a.index[row * a.top + place] = chosen;
      a.gate[row * a.top + place] = chose ? own : 0.0f;
      if (chose) atomicAdd(&s_count[chosen], 1);  // integers: any order gives the same sum
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (at.e0 + i < at.end) s_prob[(warp * kRows + lane / L) * a.experts + at.e0 + i] = psum[i];
  __syncthreads();
  for (int e = threadIdx.x; e < a.experts; e += kRouterThreads) {
    float p = 0.0f;
    for (int i = 0; i < kRouterWarps * kRows; ++i) p += s_prob[i * a.experts + e];
    a.part_prob[(int64_t)blockIdx.x * a.experts + e] = p;
    a.part_count[(int64_t)blockIdx.x * a.experts + e] = s_count[e];
  }
}

// The gradient of sigmoid scores. With q = dL/ds, dx = q s (1 - s); 1 - s without cancellation. As in router.cu the
// row is written from the probabilities' gradient alone, and lane j completes the j-th chosen expert.
struct SigmoidArgs {
  const void* logits;
  void* d_logits;
  int64_t ld, d_ld, tokens;
  int experts, top, normalize, bytes, d_bytes;
  float scale;
  const int32_t* index;
  const float* d_gate;
  const float* d_prob;
};
// s, and its derivative.
__device__ __forceinline__ float sigmoid_slope(float x, float* slope) {
  const float t = exp2_near(fabsf(x) * -1.4426950408889634f), r = reciprocal(1.0f + t);
  *slope = t * r * r;
  return x >= 0.0f ? r : t * r;
}

// Four blocks an SM of 8 values a lane. Of more there are as many as fit: 16 values in fp32 have 133 registers, one block (65536 x 512:
// 93 us, its bytes 40; bf16 51), 32 values one block (32768 x 1024: 97 us, bf16 71).
template <class T, int N, int L>
__global__ void __launch_bounds__(kRouterThreads, N == 8 ? 4 : 1) sigmoid_backward_kernel(const SigmoidArgs a) {
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
    float v[N];
    next.values(v);
    const int mine = next_index;
    const float dg = next_dg;
    fetch(row + stride);
    const bool in = row < a.tokens, live = __shfl_sync(~0u, mine, lane - sub) >= 0;
    const bool holds = live && mine >= 0 && mine < a.experts;
    const float own = holds ? ld1(x + row * a.ld + mine) : -INFINITY;
    const float own_g = holds && a.d_prob != nullptr ? a.d_prob[mine] : 0.0f;
    float sum = 0.0f, dot = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float slope;
      const float s = sigmoid_slope(v[i], &slope);
      sum += s;
      dot = fmaf(s, g[i], dot);
      v[i] = slope;
    }
    sum = sum_row<L>(sum);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    dot = sum_row<L>(dot) * inv;
    const bool small = in && sum < 0x1p-40f;
    if (__any_sync(~0u, small)) {
      // scores whose products with small d_prob leave fp32's range: by their shares (a slope is the score where it is small)
      float by_share = 0.0f;
#pragma unroll
      for (int i = 0; i < N; ++i) by_share = fmaf(v[i] * inv, g[i], by_share);
      by_share = sum_row<L>(by_share);
      if (small) dot = by_share;
    }
    float own_slope, q = dg;
    const float own_s = holds ? sigmoid_slope(own, &own_slope) : 0.0f;
    if (!holds) q = own_slope = 0.0f;
    float gate_slope = own_slope;
    if (a.normalize) {
      // a row's only chosen expert has a share of exactly 1: its difference is 0
      const float z = sum_row<L>(own_s), zi = z == 0.0f ? 0.0f : 1.0f / z, share = own_s == z ? 1.0f : own_s * zi;
      q -= sum_row<L>(share * q);
      gate_slope *= zi;
    }
    // in this order: 1 / sum and 1 / z are up to 2^126, a slope's product with them is at most 1
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = live ? v[i] * inv * (g[i] - dot) : 0.0f;
    T* dx = static_cast<T*>(a.d_logits) + row * a.d_ld;
    if (in) Lane<T, N>::store(dx, v, e0, a.experts, a.d_bytes);
    __syncwarp();  // orders the row's stores before the chosen experts'
    if (in && holds) st1(dx + mine, own_slope * inv * (own_g - dot) + gate_slope * q);
  }
}

constexpr int kBiasThreads = 256;
__global__ void __launch_bounds__(kBiasThreads)
    bias_update_kernel(const int32_t* counts, const float* bias, int experts, float rate, float* out) {
  __shared__ long long s_total[kBiasThreads / 32];
  dep_launch();
  dep_wait();
  long long total = 0;
  for (int e = threadIdx.x; e < experts; e += kBiasThreads) total += counts[e];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(~0u, total, o);
  if (threadIdx.x % 32 == 0) s_total[threadIdx.x / 32] = total;
  __syncthreads();
  total = 0;
  for (int i = 0; i < kBiasThreads / 32; ++i) total += s_total[i];
  for (int e = threadIdx.x; e < experts; e += kBiasThreads) {
    const long long less = total - (long long)experts * counts[e];  // exact
    out[e] = less > 0 ? bias[e] + rate : less < 0 ? bias[e] - rate : bias[e];
  }
}

// ------------------------------------------------------------------ host side --

relay_status_t bad(const std::string& msg) {
  return report_error(RELAY_ERR_INVALID_ARGUMENT, "relay_grouped_router: " + msg);
}
relay_status_t done(cudaError_t e) {
  if (e == cudaSuccess) return RELAY_OK;
  return report_error(RELAY_ERR_CUDA, std::string("relay_grouped_router: ") + cudaGetErrorString(e));
}
relay_status_t check_overlaps(const Array* s, int n) {
  for (int i = 0; i < n; ++i)
    for (int j = i + 1; j < n; ++j)
      if ((s[i].out || s[j].out) && overlap(s[i].span, s[j].span))
        return bad(std::string(s[i].what) + " overlaps " + s[j].what);
  return RELAY_OK;
}

int power_of_two(int n) {  // not below n
  int p = 1;
  while (p < n) p *= 2;
  return p;
}

relay_status_t check_routing(const relay_routing_t* h, relay_dtype_t dtype, int64_t tokens) {
  if (h == nullptr) return bad("the description is NULL");
  if (dtype != RELAY_F32 && dtype != RELAY_BF16) return bad("dtype must be RELAY_F32 or RELAY_BF16");
  if (tokens < 0 || tokens > INT32_MAX) return bad("tokens out of range");
  if (h->score != RELAY_SCORE_SOFTMAX && h->score != RELAY_SCORE_SIGMOID) return bad("score must be softmax or sigmoid");
  if (h->experts < 1 || h->experts > RELAY_ROUTER_MAX_EXPERTS) return bad("experts must be 1..1024");
  if (h->groups < 1 || h->groups > RELAY_ROUTER_MAX_GROUPS || h->experts % h->groups) return bad("groups must be 1..32 and divide the experts");
  if (h->kept < 1 || h->kept > h->groups) return bad("kept must be 1..groups");
  if (h->kept < h->groups && h->experts > RELAY_ROUTER_MAX_GROUPED) return bad("groups are chosen among up to 512 experts");
  if (h->group_sum != 1 && h->group_sum != 2) return bad("group_sum must be 1 or 2");
  if (h->top < 1 || h->top > RELAY_ROUTER_MAX_TOP || h->top > h->kept * (h->experts / h->groups))
    return bad("top must be 1..32, and no more than the experts of the kept groups");
  if (!std::isfinite(h->scale)) return bad("scale must be finite");
  return RELAY_OK;
}

// Values per lane (8, 16 or 32), lanes of a group and of a row.
struct Width {
  int values, group_lanes, lanes;
};
Width width_of(int groups, int size, int top) {
  for (int n : {8, 16, 32}) {
    const int p = power_of_two((size + n - 1) / n);
    if (p * groups > 32) continue;
    int lanes = std::max(4, power_of_two(std::max(p * groups, top)));
    if (n > 8) lanes = 32;
    return Width{n, groups == 1 ? lanes : p, lanes};
  }
  return Width{0, 0, 0};  // not for sizes that check_routing passes
}
template <class F>
cudaError_t by_lanes(const Width& w, F f) {
  using std::integral_constant;
  if (w.values == 32) return f(integral_constant<int, 32>(), integral_constant<int, 32>());
  if (w.values == 16) return f(integral_constant<int, 16>(), integral_constant<int, 32>());
  if (w.values != 8) return cudaErrorInvalidConfiguration;
  if (w.lanes == 4) return f(integral_constant<int, 8>(), integral_constant<int, 4>());
  if (w.lanes == 8) return f(integral_constant<int, 8>(), integral_constant<int, 8>());
  if (w.lanes == 16) return f(integral_constant<int, 8>(), integral_constant<int, 16>());
  return f(integral_constant<int, 8>(), integral_constant<int, 32>());
}

template <class T, int N, int L>
cudaError_t launch_forward(bool sigmoid, int blocks, size_t smem, const GroupArgs& a, cudaStream_t s) {
  return launch_chained(sigmoid ? grouped_forward_kernel<T, N, L, true> : grouped_forward_kernel<T, N, L, false>, blocks,
                        kRouterThreads, smem, s, a);
}

}  // namespace
}  // namespace relay

extern "C" {

relay_status_t relay_grouped_router_forward(const relay_routing_t* how, const void* logits, int64_t row_stride, relay_dtype_t dtype,
                                            int64_t tokens, const float* bias, const uint8_t* mask, int32_t* index, float* gate,
                                            int32_t* counts, float* prob_sum, void* workspace, int64_t workspace_bytes,
                                            cudaStream_t stream) {
  using namespace relay;
  return guarded([&]() -> relay_status_t {
    relay_status_t st = check_routing(how, dtype, tokens);
    if (st != RELAY_OK) return st;
    const int experts = how->experts, top = how->top;
    if (counts == nullptr || prob_sum == nullptr) return bad("counts or prob_sum is NULL");
    if (tokens > 0 && (logits == nullptr || index == nullptr || gate == nullptr)) return bad("logits, index or gate is NULL");
    if (tokens > 0 && (row_stride < experts || row_stride > (1ll << 31))) return bad("row_stride is less than experts or more than 2^31");
    const int E = esize_of(dtype);
    if (off(logits, E) || off(bias, 4) || off(index, 4) || off(gate, 4) || off(counts, 4) || off(prob_sum, 4))
      return bad("an array is not element-aligned");
    const int64_t need = relay_router_workspace_size(tokens, experts);
    if (workspace == nullptr) return bad("workspace is NULL");
    if (workspace_bytes < need)
      return bad("the workspace holds " + std::to_string(workspace_bytes) + " bytes, " + std::to_string(need) + " are needed");
    const Array s[] = {matrix(logits, tokens, experts * E, row_stride * E, "logits", false),
                       array(bias, experts * 4, "bias", false),
                       array(mask, tokens, "mask", false),
                       array(index, tokens * top * 4, "index", true),
                       array(gate, tokens * top * 4, "gate", true),
                       array(counts, experts * 4, "counts", true),
                       array(prob_sum, experts * 4, "prob_sum", true),
                       array(workspace, need, "workspace", true)};
    st = check_overlaps(s, 8);
    if (st != RELAY_OK) return st;
    // where all groups stay there is nothing to choose between them
    const int groups = how->kept < how->groups ? how->groups : 1, size = experts / groups;
    const Width w = width_of(groups, size, top);
    // as many blocks as are resident at once, within the workspace's number
    const int blocks = (int)std::min<int64_t>(resident(w.values) * 152, forward_blocks(tokens, kRouterWarps * (32 / std::max(w.lanes, 1))));
    int32_t* part_count = reinterpret_cast<int32_t*>((reinterpret_cast<uintptr_t>(workspace) + 15) & ~(uintptr_t)15);
    float* part_prob = reinterpret_cast<float*>(part_count + (int64_t)blocks * experts);
    GroupArgs a{};
    a.logits = logits;
    a.ld = row_stride;
    a.tokens = tokens;
    a.experts = experts;
    a.groups = groups;
    a.size = size;
    a.kept = std::min(how->kept, groups);
    a.lanes = w.group_lanes;
    a.top = top;
    a.group_sum = how->group_sum;
    a.normalize = how->normalize;
    a.bytes = load_bytes(logits, row_stride, E, size);  // groups start at multiples of their size
    a.scale = how->scale;
    a.bias = bias;
    a.mask = mask;
    a.index = index;
    a.gate = gate;
    a.part_count = blocks == 1 ? counts : part_count;
    a.part_prob = blocks == 1 ? prob_sum : part_prob;
    const bool sigmoid = how->score == RELAY_SCORE_SIGMOID;
    cudaError_t e = by_lanes(w, [&](auto n, auto l) {
      constexpr int N = decltype(n)::value, L = decltype(l)::value;
      const size_t smem = (size_t)(kRouterWarps * (32 / L) + 1) * experts * 4;
      return dtype == RELAY_BF16 ? launch_forward<uint16_t, N, L>(sigmoid, blocks, smem, a, stream)
                                 : launch_forward<float, N, L>(sigmoid, blocks, smem, a, stream);
    });
    if (e == cudaSuccess && blocks > 1) e = router_join(part_count, part_prob, blocks, experts, counts, prob_sum, stream);
    return done(e);
  });
}

relay_status_t relay_grouped_router_backward(const relay_routing_t* how, const void* logits, int64_t row_stride, relay_dtype_t dtype,
                                             int64_t tokens, const int32_t* index, const float* d_gate, const float* d_prob,
                                             void* d_logits, int64_t d_row_stride, cudaStream_t stream) {
  using namespace relay;
  return guarded([&]() -> relay_status_t {
    relay_status_t st = check_routing(how, dtype, tokens);
    if (st != RELAY_OK) return st;
    if (tokens == 0) return RELAY_OK;
    const int experts = how->experts, top = how->top;
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
    if (how->score == RELAY_SCORE_SOFTMAX)
      return done(router_softmax_backward(SoftmaxBackward{logits, d_logits, row_stride, d_row_stride, tokens, (int)dtype, experts, top,
                                                          how->normalize, how->scale, index, d_gate, d_prob},
                                          stream));
    const SigmoidArgs a{logits, d_logits, row_stride, d_row_stride, tokens, experts, top, how->normalize,
                        load_bytes(logits, row_stride, E, experts), load_bytes(d_logits, d_row_stride, E, experts),
                        how->scale, index, d_gate, d_prob};
    const int blocks = (int)std::min<int64_t>((tokens + kRouterWarps - 1) / kRouterWarps, 4 * 152);
    return done(by_lanes(width_of(1, experts, top), [&](auto n, auto l) {
      constexpr int N = decltype(n)::value, L = decltype(l)::value;
      return launch_chained(dtype == RELAY_BF16 ? sigmoid_backward_kernel<uint16_t, N, L> : sigmoid_backward_kernel<float, N, L>,
                            blocks, kRouterThreads, 0, stream, a);
    }));
  });
}

relay_status_t relay_router_bias_update(const int32_t* counts, const float* bias, int experts, float rate, float* bias_out,
                                        cudaStream_t stream) {
  using namespace relay;
  return guarded([&]() -> relay_status_t {
    if (experts < 1 || experts > RELAY_ROUTER_MAX_EXPERTS) return bad("experts must be 1..1024");
    if (!std::isfinite(rate)) return bad("rate must be finite");
    if (counts == nullptr || bias == nullptr || bias_out == nullptr) return bad("counts, bias or bias_out is NULL");
    if (off(counts, 4) || off(bias, 4) || off(bias_out, 4)) return bad("an array is not element-aligned");
    const Array s[] = {array(counts, experts * 4, "counts", false),
                       array(bias == bias_out ? nullptr : bias, experts * 4, "bias", false),  // in place
                       array(bias_out, experts * 4, "bias_out", true)};
    const relay_status_t st = check_overlaps(s, 3);
    if (st != RELAY_OK) return st;
    return done(launch_chained(bias_update_kernel, 1, kBiasThreads, 0, stream, counts, bias, experts, rate, bias_out));
  });
}

// The same calls with their arguments, in order, as one block of 8-byte words behind the description: for a caller whose
// foreign-function layer pays per argument.
relay_status_t relay_packed_grouped_forward(const relay_routing_t* how, const int64_t* a) {
  return relay_grouped_router_forward(how, reinterpret_cast<const void*>(a[0]), a[1], (relay_dtype_t)a[2], a[3],
                                      reinterpret_cast<const float*>(a[4]), reinterpret_cast<const uint8_t*>(a[5]),
                                      reinterpret_cast<int32_t*>(a[6]), reinterpret_cast<float*>(a[7]),
                                      reinterpret_cast<int32_t*>(a[8]), reinterpret_cast<float*>(a[9]),
                                      reinterpret_cast<void*>(a[10]), a[11], reinterpret_cast<cudaStream_t>(a[12]));
}
relay_status_t relay_packed_grouped_backward(const relay_routing_t* how, const int64_t* a) {
  return relay_grouped_router_backward(how, reinterpret_cast<const void*>(a[0]), a[1], (relay_dtype_t)a[2], a[3],
                                       reinterpret_cast<const int32_t*>(a[4]), reinterpret_cast<const float*>(a[5]),
                                       reinterpret_cast<const float*>(a[6]), reinterpret_cast<void*>(a[7]), a[8],
                                       reinterpret_cast<cudaStream_t>(a[9]));
}

}  // extern "C"
