// grads.cu -- relay_grad_norm, relay_grad_clip: the 2-norm over all of a list of tensors, and their scaling.
//
//   norm = sqrt(sum x^2);  out = x * min(1, max_norm / (norm + 1e-6))
//
// Both are bound by memory. A list is cut into chunks of 32 KiB that never span two tensors; blocks stride over the chunks,
// a thread holds eight 16-byte vectors of one in flight. The list's table travels in the launch's parameters (constant
// memory): no copy to the device, and a captured call holds all it needs. 3.4 GB of bf16 take 469 us for the norm (7.1 TB/s)
// and 973 us to scale out of place (6.9 TB/s).
//
// Sums. A thread squares and adds the values of a chunk (64 bf16, 32 fp32) in fp32, and the chunks' sums in two floats, the
// second with what the first's roundings lost; squares that fp32 cannot hold (a chunk's sum below 2^-90 or above 2^100) are
// summed again, scaled, into a double. (A launch has 2^30 chunks and 456 blocks: with fewer than 2^22 of them a thread's sum stays
// below 2^122.) Threads, then blocks join in doubles in a fixed order: equal calls give equal bits. A chunk's sum is the joint of four chains
// of up to 16 squares: the norm is within 10 roundings of fp32 (10 x 2^-24) of its value.
//
// Clipping walks the chunks from the last to the first: what the norm read last is still in L2.
#include <float.h>
#include <math.h>

#include <algorithm>
#include <string>
#include <vector>

#include "device.cuh"
#include "launch.cuh"
#include "program.h"

namespace relay {
namespace {

constexpr int kGradThreads = 256, kVectors = 8;
constexpr int kChunkBytes = kGradThreads * kVectors * 16;

// A tensor's first chunk in the launch; its elements, negative for bf16.
template <int MAX>
struct Table {
  int32_t n, chunks;
  int32_t first[MAX];
  int64_t count[MAX];
  const void* in[MAX];
};
template <int MAX>
struct ClipTable {
  Table<MAX> t;
  void* out[MAX];
};
constexpr int kFewTensors = 48, kMostTensors = 512;  // of one launch: 4 KB of parameters at most, or 16 KB

// The tensor that holds a chunk: the last whose first chunk is not behind it (tensors without elements are not in the table).
template <int MAX>
__device__ __forceinline__ int tensor_of(const Table<MAX>& t, int chunk) {
  int lo = 0, hi = t.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (t.first[mid] <= chunk) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Vector v of a tensor is the 16 bytes v * 16 behind its address rounded down to 16; of the first and the last only the
// tensor's own elements are touched.
template <class T>
__device__ __forceinline__ uint4 load_vector(const typename T::Elem* x, int64_t n, int skip, int64_t v) {
  constexpr int L = T::P::kLanes;
  const int64_t at = v * L - skip;
  if (at >= 0 && at + L <= n) return ld_once(x + at);
  float f[L];
#pragma unroll
  for (int i = 0; i < L; ++i) f[i] = at + i >= 0 && at + i < n ? ld_value(x + at + i) : 0.0f;
  return T::P::pack(f);
}
struct F32 {
  using P = TF32;
  using Elem = uint32_t;
};
struct Bf16 {
  using P = TBF16;
  using Elem = uint16_t;
};

// The sum of squares of a thread's vectors, of the values times `by`.
template <class T>
__device__ __forceinline__ float squares(const uint4 (&u)[kVectors], float by) {
  constexpr int L = T::P::kLanes;
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int j = 0; j < kVectors; ++j) {
    float f[L];
    T::P::unpack(u[j], f);
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const float x = f[i] * by;
      s[i & 3] = fmaf(x, x, s[i & 3]);
    }
  }
  return (s[0] + s[1]) + (s[2] + s[3]);
}

// The largest sum of a chunk that `hi` takes: with all of a thread's it stays finite.
constexpr float kMostSum = 0x1p100f;

struct Sum {
  float hi = 0.0f, lo = 0.0f;
  double rare = 0.0;
  __device__ __forceinline__ void add(float s) {
    const float t = hi + s, b = t - hi;
    lo += (hi - (t - b)) + (s - b);
    hi = t;
  }
};

template <class T>
__device__ __forceinline__ void sum_chunk(const void* in, int64_t n, int64_t chunk, Sum& sum) {
  const auto* x = static_cast<const typename T::Elem*>(in);
  const int skip = (int)(reinterpret_cast<uintptr_t>(in) % 16 / sizeof(typename T::Elem));
  const int64_t v0 = chunk * (kGradThreads * kVectors) + threadIdx.x;
  uint4 u[kVectors];
#pragma unroll
  for (int j = 0; j < kVectors; ++j) u[j] = load_vector<T>(x, n, skip, v0 + j * kGradThreads);
  const float s = squares<T>(u, 1.0f);
  if (s >= 0x1p-90f && s <= kMostSum) {
    sum.add(s);
    return;
  }
  // values whose squares leave fp32's range, zeros, infinities, NaN
  const bool small = s < 0x1p-90f;
  sum.rare += (double)squares<T>(u, small ? 0x1p100f : 0x1p-100f) * (small ? 0x1p-200 : 0x1p200);
}

// A block's sum, in thread 0.
__device__ __forceinline__ double sum_block(double v, double* s_part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  if (threadIdx.x % 32 == 0) s_part[threadIdx.x / 32] = v;
  __syncthreads();
  if (threadIdx.x == 0)
    for (int i = 1; i < (int)blockDim.x / 32; ++i) v += s_part[i];
  return v;
}

// norm: where one block does it all, and otherwise NULL.
template <int MAX>
__global__ void __launch_bounds__(kGradThreads) grad_sum_kernel(const __grid_constant__ Table<MAX> t, double* part, float* norm) {
  __shared__ double s_part[kGradThreads / 32];
  dep_launch();
  dep_wait();
  Sum sum;
  for (int c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    const int i = tensor_of(t, c);
    const int64_t n = t.count[i];
    if (n < 0) sum_chunk<Bf16>(t.in[i], -n, c - t.first[i], sum);
    else sum_chunk<F32>(t.in[i], n, c - t.first[i], sum);
  }
  const double v = sum_block((double)sum.hi + (double)sum.lo + sum.rare, s_part);
  if (threadIdx.x != 0) return;
  if (norm != nullptr) *norm = (float)sqrt(v);
  else part[blockIdx.x] = v;
}

constexpr int kJoinThreads = 256;  // 1024: 1.7 us more
__global__ void __launch_bounds__(kJoinThreads) grad_join_kernel(const double* part, int parts, float* norm) {
  __shared__ double s_part[kJoinThreads / 32];
  dep_launch();
  dep_wait();
  double v = 0.0;
  for (int i = threadIdx.x; i < parts; i += kJoinThreads) v += part[i];
  v = sum_block(v, s_part);
  if (threadIdx.x == 0) *norm = (float)sqrt(v);
}

// A value is multiplied by factor. Where that is below fp32's normal range: by a power of two, 2^200 times the factor, and the power
// again, so that neither leaves the range (of a value that the first takes below it nothing is left).
struct Factor {
  float factor, power;
};

template <class T>
__device__ __forceinline__ void clip_chunk(const void* in, void* out, int64_t n, int64_t chunk, const Factor& by) {
  using E = typename T::Elem;
  constexpr int L = T::P::kLanes;
  const auto* x = static_cast<const E*>(in);
  auto* y = static_cast<E*>(out);
  const int skip = (int)(reinterpret_cast<uintptr_t>(in) % 16 / sizeof(E));
  const int64_t v0 = chunk * (kGradThreads * kVectors) + threadIdx.x;
  if ((reinterpret_cast<uintptr_t>(in) ^ reinterpret_cast<uintptr_t>(out)) % 16 != 0 || by.power != 1.0f) {
    // the two lie differently on the 16-byte grid, or the factor is a rare one (here alone, it costs the rest nothing:
    // 1% otherwise): neighbouring threads take neighbouring elements
    const int64_t lo = max((int64_t)0, chunk * (kGradThreads * kVectors * L) - skip);
    const int64_t hi = min(n, (chunk + 1) * (kGradThreads * kVectors * L) - skip);
#pragma unroll 8
    for (int64_t e = lo + threadIdx.x; e < hi; e += kGradThreads)
      T::P::store1(y + e, __fmul_rn(__fmul_rn(__fmul_rn(T::P::template load1<true>(x + e), by.power), by.factor), by.power));
    return;
  }
  uint4 u[kVectors];
#pragma unroll
  for (int j = 0; j < kVectors; ++j) {
    const int64_t at = (v0 + j * kGradThreads) * L - skip;
    if (at >= 0 && at + L <= n) u[j] = Mem<true>::v4(x + at);
  }
#pragma unroll
  for (int j = 0; j < kVectors; ++j) {
    const int64_t at = (v0 + j * kGradThreads) * L - skip;
    if (at >= 0 && at + L <= n) {
      float f[L];
      T::P::unpack(u[j], f);
#pragma unroll
      for (int i = 0; i < L; ++i) f[i] = __fmul_rn(f[i], by.factor);
      st_v4(y + at, T::P::pack(f));
    } else {
#pragma unroll
      for (int i = 0; i < L; ++i)
        if (at + i >= 0 && at + i < n) T::P::store1(y + at + i, __fmul_rn(T::P::template load1<true>(x + at + i), by.factor));
    }
  }
}

template <int MAX>
__global__ void __launch_bounds__(kGradThreads) grad_clip_kernel(const __grid_constant__ ClipTable<MAX> c, const float* norm,
                                                                 float max_norm, int in_place) {
  const Table<MAX>& t = c.t;
  dep_launch();
  dep_wait();
  const float total = *norm;
  Factor by{max_norm / (total + 1e-6f), 1.0f};
  // nothing to clip, or a norm that says that something is wrong: the values stay as they are
  const bool clips = by.factor < 1.0f && total < INFINITY;
  if (!clips && in_place) return;
  if (!clips) by.factor = 1.0f;
  // max_norm is below 4 here, and total above 2^-24
  else if (by.factor < FLT_MIN) by = Factor{max_norm * 0x1p100f / ((total + 1e-6f) * 0x1p-100f), 0x1p-100f};
  for (int k = blockIdx.x; k < t.chunks; k += gridDim.x) {
    const int chunk = t.chunks - 1 - k, i = tensor_of(t, chunk);
    const int64_t n = t.count[i];
    if (n < 0) clip_chunk<Bf16>(t.in[i], c.out[i], -n, chunk - t.first[i], by);
    else clip_chunk<F32>(t.in[i], c.out[i], n, chunk - t.first[i], by);
  }
}

// ------------------------------------------------------------------ host side --

relay_status_t bad(const std::string& msg) { return report_error(RELAY_ERR_INVALID_ARGUMENT, "relay_grad: " + msg); }
relay_status_t done(cudaError_t e) {
  if (e == cudaSuccess) return RELAY_OK;
  return report_error(RELAY_ERR_CUDA, std::string("relay_grad: ") + cudaGetErrorString(e));
}

relay_status_t check_list(const relay_grads_t* g, const char* name) {
  const std::string who = name;
  if (g == nullptr) return bad(who + " is NULL");
  if (g->n < 0 || g->n > RELAY_GRADS_MAX) return bad(who + " has a number of tensors out of range");
  if (g->n > 0 && (g->grad == nullptr || g->count == nullptr || g->dtype == nullptr)) return bad(who + ": an array is NULL");
  for (int i = 0; i < g->n; ++i) {
    if (g->dtype[i] != RELAY_F32 && g->dtype[i] != RELAY_BF16)
      return bad(who + "[" + std::to_string(i) + "]: dtype must be RELAY_F32 or RELAY_BF16");
    if (g->count[i] > (1ull << 42)) return bad(who + "[" + std::to_string(i) + "]: more than 2^42 elements");
    if (g->count[i] == 0) continue;
    if (g->grad[i] == nullptr) return bad(who + "[" + std::to_string(i) + "] is NULL");
    if (reinterpret_cast<uintptr_t>(g->grad[i]) % (uintptr_t)esize_of(g->dtype[i]) != 0)
      return bad(who + "[" + std::to_string(i) + "] is not element-aligned");
  }
  return RELAY_OK;
}

struct Range {
  uintptr_t lo, hi;
  bool written;
};
// Whether bytes that are written belong to two of the ranges.
bool clash(std::vector<Range>& r) {
  auto before = [](const Range& a, const Range& b) { return a.lo < b.lo; };
  if (!std::is_sorted(r.begin(), r.end(), before)) std::sort(r.begin(), r.end(), before);
  uintptr_t any = 0, written = 0;
  for (const Range& x : r) {
    if (x.lo < (x.written ? any : written)) return true;
    any = std::max(any, x.hi);
    if (x.written) written = std::max(written, x.hi);
  }
  return false;
}
void put(std::vector<Range>* r, const void* p, size_t bytes, bool written) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  if (bytes > 0) r->push_back(Range{lo, lo + bytes, written});
}

int64_t chunks_of(const relay_grads_t& g, int i) {
  if (g.count[i] == 0) return 0;
  const int64_t e = esize_of(g.dtype[i]), skip = (int64_t)(reinterpret_cast<uintptr_t>(g.grad[i]) % 16);
  return ((int64_t)g.count[i] * e + skip + kChunkBytes - 1) / kChunkBytes;
}

// Blocks of the sum: as many as are resident (3 an SM; 6 an SM take 20.4 us and not 18.3 at 64 MB, the same from 300 MB on). The
// scaling's end with few chunks each (2 to 200 an SM: within 4%).
int sum_blocks(int64_t chunks) { return (int)std::min<int64_t>(chunks, 3 * 152); }
int clip_blocks(int64_t chunks) { return (int)std::min<int64_t>(chunks, 40 * 152); }
// So few chunks that one block is done before a second launch would be.
constexpr int64_t kOneBlockChunks = 4;
constexpr int64_t kMostChunks = 1ll << 30;  // of a launch
static_assert((double)kMostSum * (kMostChunks / (3 * 152) + kOneBlockChunks) < 0x1p127, "a thread's sum of chunks is finite");

// Tensors of one launch: a piece of the list with at most kMostTensors tensors and kMostChunks chunks.
struct Piece {
  int lo, hi;
  int64_t chunks;
};
relay_status_t pieces_of(const relay_grads_t& g, std::vector<Piece>* out) {
  Piece p{0, 0, 0};
  for (int i = 0; i < g.n; ++i) {
    const int64_t c = chunks_of(g, i);
    if (c > kMostChunks) return bad("a tensor is too large");
    if (p.hi - p.lo == kMostTensors || p.chunks + c > kMostChunks) {
      if (p.chunks > 0) out->push_back(p);
      p = Piece{i, i, 0};
    }
    p.chunks += c;
    p.hi = i + 1;
  }
  if (p.chunks > 0 || out->empty()) out->push_back(p);
  return RELAY_OK;
}

template <int MAX>
void fill(Table<MAX>* t, const relay_grads_t& g, const Piece& p) {
  t->n = 0;
  int64_t chunks = 0;
  for (int i = p.lo; i < p.hi; ++i) {
    if (g.count[i] == 0) continue;
    t->first[t->n] = (int32_t)chunks;
    t->count[t->n] = g.dtype[i] == RELAY_BF16 ? -(int64_t)g.count[i] : (int64_t)g.count[i];
    t->in[t->n++] = g.grad[i];
    chunks += chunks_of(g, i);
  }
  t->chunks = (int32_t)chunks;
}

template <int MAX>
cudaError_t launch_sum(const relay_grads_t& g, const Piece& p, double* part, float* norm, cudaStream_t s) {
  Table<MAX> t;
  fill(&t, g, p);
  return launch_chained(grad_sum_kernel<MAX>, norm != nullptr ? 1 : sum_blocks(p.chunks), kGradThreads, 0, s, t, part, norm);
}
template <int MAX>
cudaError_t launch_clip(const relay_grads_t& g, const relay_grads_t& out, const Piece& p, const float* norm, float max_norm,
                        int in_place, cudaStream_t s) {
  ClipTable<MAX> c;
  fill(&c.t, g, p);
  for (int i = p.lo, k = 0; i < p.hi; ++i)
    if (g.count[i] != 0) c.out[k++] = out.grad[i];
  return launch_chained(grad_clip_kernel<MAX>, clip_blocks(p.chunks), kGradThreads, 0, s, c, norm, max_norm, in_place);
}

// A double for every block of every launch.
int64_t grad_need(const std::vector<Piece>& pieces) {
  int64_t parts = 0;
  for (const Piece& p : pieces) parts += sum_blocks(p.chunks);
  return 8 * parts + 8;
}

}  // namespace
}  // namespace relay

extern "C" {

int64_t relay_grad_workspace_size(const relay_grads_t* grads) {
  using namespace relay;
  int64_t bytes = -1;
  guarded([&]() -> relay_status_t {
    relay_status_t st = check_list(grads, "grads");
    if (st != RELAY_OK) return st;
    std::vector<Piece> pieces;
    st = pieces_of(*grads, &pieces);
    if (st == RELAY_OK) bytes = grad_need(pieces);
    return st;
  });
  return bytes;
}

relay_status_t relay_grad_norm(const relay_grads_t* grads, float* norm, void* workspace, int64_t workspace_bytes,
                               cudaStream_t stream) {
  using namespace relay;
  return guarded([&]() -> relay_status_t {
    relay_status_t st = check_list(grads, "grads");
    if (st != RELAY_OK) return st;
    if (norm == nullptr || reinterpret_cast<uintptr_t>(norm) % 4) return bad("norm is NULL or not element-aligned");
    std::vector<Piece> pieces;
    st = pieces_of(*grads, &pieces);
    if (st != RELAY_OK) return st;
    const int64_t need = grad_need(pieces);
    if (workspace == nullptr) return bad("workspace is NULL");
    if (workspace_bytes < need)
      return bad("the workspace holds " + std::to_string(workspace_bytes) + " bytes, " + std::to_string(need) + " are needed");
    std::vector<Range> ranges;
    ranges.reserve(grads->n + 2);
    put(&ranges, norm, 4, true);
    put(&ranges, workspace, need, true);
    // the tensors are only read: two of them may share bytes
    for (int i = 0; i < grads->n; ++i) put(&ranges, grads->grad[i], grads->count[i] * esize_of(grads->dtype[i]), false);
    if (clash(ranges)) return bad("norm, the workspace and the tensors overlap");
    double* part = reinterpret_cast<double*>((reinterpret_cast<uintptr_t>(workspace) + 7) & ~(uintptr_t)7);
    const bool one = pieces.size() == 1 && pieces[0].chunks <= kOneBlockChunks;
    int parts = 0;
    for (const Piece& p : pieces) {
      const cudaError_t e = p.hi - p.lo <= kFewTensors ? launch_sum<kFewTensors>(*grads, p, part + parts, one ? norm : nullptr, stream)
                                                       : launch_sum<kMostTensors>(*grads, p, part + parts, one ? norm : nullptr, stream);
      if (e != cudaSuccess) return done(e);
      parts += sum_blocks(p.chunks);
    }
    if (one) return RELAY_OK;
    return done(launch_chained(grad_join_kernel, 1, kJoinThreads, 0, stream, part, parts, norm));
  });
}

relay_status_t relay_grad_clip(const relay_grads_t* grads, const relay_grads_t* out, const float* norm, float max_norm,
                               cudaStream_t stream) {
  using namespace relay;
  return guarded([&]() -> relay_status_t {
    relay_status_t st = check_list(grads, "grads");
    if (st != RELAY_OK) return st;
    if (out != nullptr) {
      st = check_list(out, "out");
      if (st != RELAY_OK) return st;
      if (out->n != grads->n) return bad("out must have as many tensors as grads");
      for (int i = 0; i < grads->n; ++i)
        if (out->count[i] != grads->count[i] || out->dtype[i] != grads->dtype[i])
          return bad("out[" + std::to_string(i) + "] must have the size and dtype of grads'");
    }
    if (norm == nullptr || reinterpret_cast<uintptr_t>(norm) % 4) return bad("norm is NULL or not element-aligned");
    if (!(max_norm > 0.0f) || !std::isfinite(max_norm)) return bad("max_norm must be finite and positive");
    std::vector<Range> ranges;
    ranges.reserve(2 * grads->n + 1);
    put(&ranges, norm, 4, false);
    const relay_grads_t& to = out != nullptr ? *out : *grads;
    bool in_place = true;
    for (int i = 0; i < grads->n; ++i) {
      const size_t bytes = grads->count[i] * esize_of(grads->dtype[i]);
      if (bytes > 0 && to.grad[i] != grads->grad[i]) {
        put(&ranges, grads->grad[i], bytes, false);
        in_place = false;
      }
      put(&ranges, to.grad[i], bytes, true);
    }
    if (clash(ranges)) return bad("a tensor that is written overlaps another, or norm");
    std::vector<Piece> pieces;
    st = pieces_of(*grads, &pieces);
    if (st != RELAY_OK) return st;
    for (size_t k = pieces.size(); k-- > 0;) {
      const Piece& p = pieces[k];
      if (p.chunks == 0) continue;
      const cudaError_t e = p.hi - p.lo <= kFewTensors ? launch_clip<kFewTensors>(*grads, to, p, norm, max_norm, in_place, stream)
                                                       : launch_clip<kMostTensors>(*grads, to, p, norm, max_norm, in_place, stream);
      if (e != cudaSuccess) return done(e);
    }
    return RELAY_OK;
  });
}

}  // extern "C"
