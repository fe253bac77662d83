// fp8_quantize.cu -- relay_quantize_fp8: values to 8 bits (e4m3) with a power of two for each block of 128.
//
//   2^k, the least power of two with amax / 2^k <= 448 (1 for a block of zeros);  q = round(x / 2^k), ties to even
//
// A power of two makes the division exact: q is rounded once, and the same block quantized along the other dimension
// has the same values. A block holds 128 neighbours of a row, or 128 x 128.
//
// Bound by memory: a CTA reads 128 x 128 values once, keeps them in registers as they lie (64 a thread: eight rows of eight
// columns; bf16 in 32 registers, so that four CTAs an SM keep enough reads on their way), and writes what is asked for of the
// tile, its transpose, and both's scales. The transpose goes through shared memory as 8-byte pieces of eight rows, placed
// so that neither side meets a bank twice.
#include <algorithm>
#include <string>

#include "device.cuh"
#include "fp8.h"
#include "launch.cuh"
#include "program.h"
#include "spans.h"

namespace relay {
namespace {

constexpr int kQuantThreads = 256;
constexpr float kUnitRange = 448.0f;  // e4m3's largest value: 1.75 * 2^8
static_assert(kUnitRange == 1.75f * 256.0f, "scale_of rests on it");

struct QuantArgs {
  const void* x;
  int64_t ld;
  int32_t rows, cols, groups;
  int32_t vectors;                 // x's rows take 16-byte loads
  uint8_t* q;                      // [batch][rows][cols], row stride q_ld; NULL: not wanted
  int64_t q_ld;
  float* scale;                    // [blocks of cols][rows], or tiles: [batch][blocks of rows][blocks of cols]
  int32_t tiles;
  uint8_t* qt;                     // [batch][cols][depth], row stride qt_ld; NULL: not wanted
  int64_t qt_ld;
  float* scale_t;                  // [depth blocks][cols], or tiles: [batch][blocks of cols][depth blocks]
  int32_t tiles_t;
  int32_t depth_blocks;            // of the transpose: blocks of rows, or of all groups' rows
  const int32_t* offset;
};

// The scale of a block whose largest magnitude has these bits, and its reciprocal: both exact. A block that holds
// an infinity or a NaN has scale NaN: what it is multiplied into shows it.
__device__ __forceinline__ float scale_of(uint32_t top, float* inverse) {
  if (top >= 0x7f800000u) {
    *inverse = __uint_as_float(0x7fffffffu);
    return *inverse;
  }
  int e = (int)(top >> 23) - 127 - ((top & 0x7fffffu) <= 0x600000u ? 8 : 7);
  e = top == 0 ? 0 : max(e, -126);
  *inverse = __uint_as_float((uint32_t)(127 - e) << 23);
  return __uint_as_float((uint32_t)(127 + e) << 23);
}
// Two values to e4m3, the first in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint2 e4m3x8(const float (&v)[8]) {
  return make_uint2(e4m3x2(v[0], v[1]) | e4m3x2(v[2], v[3]) << 16, e4m3x2(v[4], v[5]) | e4m3x2(v[6], v[7]) << 16);
}
// n of the 8 bytes.
__device__ __forceinline__ void store_bytes(uint8_t* to, uint2 b, int n) {
  if (n >= 8) {
    *reinterpret_cast<uint2*>(to) = b;
    return;
  }
  const uint64_t all = (uint64_t)b.y << 32 | b.x;
  for (int i = 0; i < n; ++i) to[i] = (uint8_t)(all >> (8 * i));
}

// Eight rows of eight bytes to eight columns.
__device__ __forceinline__ void turn4(uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  const uint32_t e = __byte_perm(a, b, 0x5140), f = __byte_perm(c, d, 0x5140), g = __byte_perm(a, b, 0x7362), h = __byte_perm(c, d, 0x7362);
  a = __byte_perm(e, f, 0x5410);
  b = __byte_perm(e, f, 0x7632);
  c = __byte_perm(g, h, 0x5410);
  d = __byte_perm(g, h, 0x7632);
}
__device__ __forceinline__ void turn(uint2 (&r)[8]) {
  turn4(r[0].x, r[1].x, r[2].x, r[3].x);
  turn4(r[4].x, r[5].x, r[6].x, r[7].x);
  turn4(r[0].y, r[1].y, r[2].y, r[3].y);
  turn4(r[4].y, r[5].y, r[6].y, r[7].y);
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // the corners change places
    const uint32_t t = r[i].y;
    r[i].y = r[4 + i].x;
    r[4 + i].x = t;
  }
}

// Eight neighbours of a row as they lie. Magnitudes compare as integers, two bf16 at once.
template <class T>
struct Eight;
template <>
struct Eight<float> {
  static constexpr int kWords = 8;
  static __device__ __forceinline__ uint32_t magnitude(uint32_t w) { return w & 0x7fffffffu; }
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return max(a, b); }
  static __device__ __forceinline__ uint32_t fold(uint32_t a) { return a; }  // as fp32 bits
  static __device__ __forceinline__ uint32_t column(const uint32_t (&m)[8], int k) { return m[k]; }
  static __device__ __forceinline__ float value(const uint32_t (&w)[8], int k) { return __uint_as_float(w[k]); }
  static __device__ __forceinline__ void set(uint32_t (&w)[8], int k, float v) { w[k] = __float_as_uint(v); }
};
template <>
struct Eight<uint16_t> {
  static constexpr int kWords = 4;
  static __device__ __forceinline__ uint32_t magnitude(uint32_t w) { return w & 0x7fff7fffu; }
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }
  static __device__ __forceinline__ uint32_t fold(uint32_t a) { return max(a << 16, a & 0xffff0000u); }
  static __device__ __forceinline__ uint32_t column(const uint32_t (&m)[4], int k) { return k % 2 ? m[k / 2] & 0xffff0000u : m[k / 2] << 16; }
  static __device__ __forceinline__ float value(const uint32_t (&w)[4], int k) { return __uint_as_float(column(w, k)); }
  static __device__ __forceinline__ void set(uint32_t (&w)[4], int k, float v) {
    const uint32_t b = __float_as_uint(v) >> 16;  // v is a bf16 value
    w[k / 2] = k % 2 ? (w[k / 2] & 0xffffu) | b << 16 : (w[k / 2] & 0xffff0000u) | b;
  }
};

// EDGES: rows of x or of an output may end inside 8 values, or be off the 16-byte grid. Without, the program is short enough for the
// instruction caches.
template <class T, bool EDGES>
__global__ void __launch_bounds__(kQuantThreads, sizeof(T) == 2 ? 4 : 2) fp8_quantize_kernel(const QuantArgs a) {
  using V = Eight<T>;
  constexpr int W = V::kWords;
  __shared__ __align__(16) uint8_t s_t[kBlock * kBlock];
  __shared__ uint32_t s_col[kQuantThreads / 32][kBlock];
  __shared__ uint32_t s_top[kQuantThreads / 32];
  __shared__ __align__(16) float s_inverse[kBlock];  // of the columns' scales
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int piece = threadIdx.x / 16, row8 = piece * 8, col8 = threadIdx.x % 16 * 8;  // the thread's first row and column
  dep_launch();
  dep_wait();
  const int batch = blockIdx.z, cb = blockIdx.x, db = blockIdx.y, c0 = cb * kBlock;
  // the block's rows: a stretch of the matrix, or of the group that block db of all groups belongs to
  int r0 = db * kBlock, r_end = min(a.rows, r0 + kBlock);
  if (a.offset != nullptr) {
    int first = 0, found = -1, lo = 0, hi = 0, start = 0;
    for (int base = 0; base < a.groups && found < 0; base += 32) {
      const int g = base + lane;
      const int from = g < a.groups ? offset_at(a.offset, g, a.rows) : 0, to = g < a.groups ? offset_at(a.offset, g + 1, a.rows) : 0;
      int n = to > from ? (to - from + kBlock - 1) / kBlock : 0, sum = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int before = __shfl_up_sync(~0u, sum, o);
        if (lane >= o) sum += before;
      }
      const unsigned past = __ballot_sync(~0u, db < first + sum);
      if (past != 0) {
        const int at = __ffs(past) - 1;
        found = base + at;
        lo = __shfl_sync(~0u, from, at);
        hi = __shfl_sync(~0u, to, at);
        start = first + __shfl_sync(~0u, sum - n, at);
      }
      first += __shfl_sync(~0u, sum, 31);
    }
    if (found < 0) return;  // behind the last group's blocks
    r0 = lo + (db - start) * kBlock;
    r_end = min(hi, r0 + kBlock);
  }
  const T* x = static_cast<const T*>(a.x) + (int64_t)batch * a.rows * a.ld;
  uint32_t v[8][W];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + row8 + i, c = c0 + col8;
    const T* from = x + (int64_t)r * a.ld + c;
    if (r < r_end && (!EDGES || (a.vectors && c + 8 <= a.cols))) {
#pragma unroll
      for (int k = 0; k < W; k += 4) {
        const uint4 u = ld_once(reinterpret_cast<const uint32_t*>(from) + k);
        v[i][k] = u.x; v[i][k + 1] = u.y; v[i][k + 2] = u.z; v[i][k + 3] = u.w;
      }
    } else {
#pragma unroll
      for (int k = 0; k < W; ++k) v[i][k] = 0;
      if (EDGES && r < r_end) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (c + k < a.cols) V::set(v[i], k, ld_value(from + k));
      }
    }
  }
  const bool need_cols = a.qt != nullptr && !a.tiles_t, need_tile = (a.q != nullptr && a.tiles) || (a.qt != nullptr && a.tiles_t);
  uint32_t all = 0;
  if (need_cols || need_tile) {
    uint32_t m[W];  // of the thread's columns
#pragma unroll
    for (int j = 0; j < W; ++j) {
      m[j] = V::magnitude(v[0][j]);
#pragma unroll
      for (int i = 1; i < 8; ++i) m[j] = V::larger(m[j], V::magnitude(v[i][j]));
      all = j == 0 ? m[j] : V::larger(all, m[j]);
    }
    all = V::fold(all);
    if (need_cols) {
#pragma unroll
      for (int j = 0; j < W; ++j) m[j] = V::larger(m[j], __shfl_xor_sync(~0u, m[j], 16));
      if (lane < 16) {
#pragma unroll
        for (int k = 0; k < 8; ++k) s_col[warp][col8 + k] = V::column(m, k);
      }
    }
  }
  if (need_tile) {
    all = __reduce_max_sync(~0u, all);
    if (lane == 0) s_top[warp] = all;
  }
  if (need_cols || need_tile) __syncthreads();
  float tile_inverse = 1.0f;
  if (need_tile) {
    all = 0;
#pragma unroll
    for (int i = 0; i < kQuantThreads / 32; ++i) all = max(all, s_top[i]);
    const float s = scale_of(all, &tile_inverse);
    const int64_t row_blocks = (a.rows + kBlock - 1) / kBlock, col_blocks = gridDim.x;
    if (threadIdx.x == 0 && a.q != nullptr && a.tiles) a.scale[(batch * row_blocks + db) * col_blocks + cb] = s;
    if (threadIdx.x == 32 && a.qt != nullptr && a.tiles_t) a.scale_t[(batch * col_blocks + cb) * a.depth_blocks + db] = s;
  }
  if (need_cols) {
    if (threadIdx.x < kBlock) {
      const int c = threadIdx.x;
      uint32_t t = 0;
#pragma unroll
      for (int i = 0; i < kQuantThreads / 32; ++i) t = max(t, s_col[i][c]);
      float inverse;
      const float s = scale_of(t, &inverse);
      s_inverse[c] = inverse;
      if (!EDGES || c0 + c < a.cols) a.scale_t[(int64_t)db * a.cols + c0 + c] = s;
    }
    __syncthreads();
  }
  const bool same = a.q != nullptr && a.tiles && a.tiles_t;  // the transpose holds the same bytes
  uint2 bytes[8];
  if (a.q != nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = r0 + row8 + i;
      float inverse = tile_inverse;
      if (!a.tiles) {
        uint32_t t = V::magnitude(v[i][0]);
#pragma unroll
        for (int j = 1; j < W; ++j) t = V::larger(t, V::magnitude(v[i][j]));
        t = V::fold(t);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) t = max(t, __shfl_xor_sync(~0u, t, o));
        const float s = scale_of(t, &inverse);
        if (lane % 16 == 0 && r < r_end) a.scale[(int64_t)cb * a.rows + r] = s;
      }
      float y[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] = V::value(v[i], k) * inverse;
      bytes[i] = e4m3x8(y);
      if (r < r_end) store_bytes(a.q + ((int64_t)batch * a.rows + r) * a.q_ld + c0 + col8, bytes[i], EDGES ? a.cols - c0 - col8 : 8);
    }
  }
  if (a.qt == nullptr) return;
  // eight rows of a column: 8 bytes, at another place in each group of eight columns
  auto put = [&](int k, uint2 column) {
    *reinterpret_cast<uint2*>(s_t + (col8 + k) * kBlock + (piece ^ (col8 / 8)) * 8) = column;
  };
  if (same) {
    turn(bytes);
#pragma unroll
    for (int k = 0; k < 8; ++k) put(k, bytes[k]);
  } else {
    float inverse[8];
#pragma unroll
    for (int k = 0; k < 8; k += 4) {
      const float4 u = a.tiles_t ? make_float4(tile_inverse, tile_inverse, tile_inverse, tile_inverse)
                                 : *reinterpret_cast<const float4*>(s_inverse + col8 + k);
      inverse[k] = u.x; inverse[k + 1] = u.y; inverse[k + 2] = u.z; inverse[k + 3] = u.w;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = V::value(v[i], k) * inverse[k];
      put(k, e4m3x8(y));
    }
  }
  __syncthreads();
  // along the rows: all 128 of a group's block (zeros behind its last row), or what the matrix has
  const int64_t d0 = (int64_t)db * kBlock;
  const int width = a.offset != nullptr ? kBlock : r_end - r0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = i * 16 + piece, at = threadIdx.x % 16;
    if (EDGES && c0 + c >= a.cols) break;
    const uint2 b = *reinterpret_cast<const uint2*>(s_t + c * kBlock + (at ^ (c / 8)) * 8);
    store_bytes(a.qt + ((int64_t)batch * a.cols + c0 + c) * a.qt_ld + d0 + at * 8, b, EDGES ? width - at * 8 : 8);
  }
}

relay_status_t bad(const std::string& msg) { return report_error(RELAY_ERR_INVALID_ARGUMENT, "relay_quantize_fp8: " + msg); }

}  // namespace
}  // namespace relay

extern "C" {

int64_t relay_fp8_depth(int64_t rows, int groups) {
  using namespace relay;
  if (rows < 0 || rows > RELAY_FP8_MAX_ROWS || groups < 0 || groups > RELAY_FP8_MAX_GROUPS) {
    guarded([] { return bad("rows or groups out of range"); });
    return -1;
  }
  return groups == 0 ? rows : kBlock * (rows / kBlock + std::min<int64_t>(groups, rows));
}

relay_status_t relay_quantize_fp8(const relay_fp8_quantize_t* p, cudaStream_t stream) {
  using namespace relay;
  return guarded([&]() -> relay_status_t {
    if (p == nullptr) return bad("the description is NULL");
    if (p->dtype != RELAY_F32 && p->dtype != RELAY_BF16) return bad("dtype must be RELAY_F32 or RELAY_BF16");
    if (p->rows < 0 || p->rows > RELAY_FP8_MAX_ROWS || p->cols < 1 || p->cols > RELAY_FP8_MAX_ROWS) return bad("rows or cols out of range");
    if (p->batch < 0 || p->batch > RELAY_FP8_MAX_GROUPS) return bad("batch out of range");
    if (p->groups < 0 || p->groups > RELAY_FP8_MAX_GROUPS) return bad("groups out of range");
    const bool grouped = p->offset != nullptr;
    if (grouped != (p->groups > 0)) return bad("groups and offset go together");
    if (p->q == nullptr && p->qt == nullptr) return bad("neither q nor qt is given");
    if ((p->q != nullptr && p->scale == nullptr) || (p->qt != nullptr && p->scale_t == nullptr)) return bad("a scale is NULL");
    if (p->batch != 1 && ((p->q != nullptr && !p->tiles) || (p->qt != nullptr && !p->tiles_t) || grouped))
      return bad("a batch of matrices has tiles, and no groups");
    if (grouped && p->q != nullptr && p->tiles) return bad("tiles of rows in groups: only of the transpose");
    if (p->rows == 0 || p->batch == 0) return RELAY_OK;
    if (p->x == nullptr) return bad("x is NULL");
    const int64_t E = esize_of(p->dtype), limit = 1ll << 32;
    const int64_t depth = relay_fp8_depth(p->rows, p->groups), rb = blocks_of(p->rows), cb = blocks_of(p->cols), dblocks = blocks_of(depth);
    if (p->x_stride < p->cols || p->x_stride > limit) return bad("x_stride is less than cols or more than 2^32");
    if (p->q != nullptr && (p->q_stride < p->cols || p->q_stride > limit || p->q_stride % 16)) return bad("q_stride is less than cols, more than 2^32 or no multiple of 16");
    if (p->qt != nullptr && (p->qt_stride < depth || p->qt_stride > limit || p->qt_stride % 16)) return bad("qt_stride is less than the depth, more than 2^32 or no multiple of 16");
    auto off = [](const void* q, uintptr_t e) { return reinterpret_cast<uintptr_t>(q) % e != 0; };
    if (off(p->x, E) || off(p->scale, 4) || off(p->scale_t, 4) || off(p->offset, 4)) return bad("an array is not element-aligned");
    if (off(p->q, 16) || off(p->qt, 16)) return bad("q or qt is not on a 16-byte boundary");
    struct {
      Span span;
      const char* what;
      bool out;
    } s[] = {{matrix_span(p->x, p->batch * p->rows, p->cols * E, p->x_stride * E), "x", false},
             {array_span(p->offset, 4ll * (p->groups + 1)), "offset", false},
             {matrix_span(p->q, p->batch * p->rows, p->cols, p->q_stride), "q", true},
             {array_span(p->q != nullptr ? p->scale : nullptr, p->tiles ? 4 * p->batch * rb * cb : 4 * cb * p->rows), "scale", true},
             {matrix_span(p->qt, p->batch * p->cols, depth, p->qt_stride), "qt", true},
             {array_span(p->qt != nullptr ? p->scale_t : nullptr, p->tiles_t ? 4 * p->batch * cb * dblocks : 4 * dblocks * p->cols), "scale_t", true}};
    for (int i = 0; i < 6; ++i)
      for (int j = i + 1; j < 6; ++j)
        if ((s[i].out || s[j].out) && overlap(s[i].span, s[j].span)) return bad(std::string(s[i].what) + " overlaps " + s[j].what);
    QuantArgs a{};
    a.x = p->x;
    a.ld = p->x_stride;
    a.rows = (int32_t)p->rows;
    a.cols = (int32_t)p->cols;
    a.groups = p->groups;
    a.vectors = !off(p->x, 16) && p->x_stride * E % 16 == 0;
    a.q = static_cast<uint8_t*>(p->q);
    a.q_ld = p->q_stride;
    a.scale = p->scale;
    a.tiles = p->tiles;
    a.qt = static_cast<uint8_t*>(p->qt);
    a.qt_ld = p->qt_stride;
    a.scale_t = p->scale_t;
    a.tiles_t = p->tiles_t;
    a.depth_blocks = (int32_t)dblocks;
    a.offset = p->offset;
    const dim3 grid((unsigned)cb, (unsigned)(grouped ? dblocks : rb), (unsigned)p->batch);
    const bool edges = !a.vectors || a.cols % kBlock != 0 || (a.qt != nullptr && !grouped && a.rows % kBlock != 0);
    auto* kernel = p->dtype == RELAY_BF16 ? (edges ? fp8_quantize_kernel<uint16_t, true> : fp8_quantize_kernel<uint16_t, false>)
                                          : (edges ? fp8_quantize_kernel<float, true> : fp8_quantize_kernel<float, false>);
    const cudaError_t e = launch_chained(kernel, grid, kQuantThreads, 0, stream, a);
    if (e != cudaSuccess) return report_error(RELAY_ERR_CUDA, std::string("relay_quantize_fp8: ") + cudaGetErrorString(e));
    return RELAY_OK;
  });
}

}  // extern "C"
