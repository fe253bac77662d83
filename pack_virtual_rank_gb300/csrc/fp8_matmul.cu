// fp8_matmul.cu -- relay_matmul_fp8: products of e4m3 matrices with a scale for each block of 128 of the inner dimension.
//
//   out[r][n] = sum over blocks k of  a_scale[k][r] b_scale[n / 128][k] * sum over d in k of a[r][d] b[n][d]
//
// The fifth-generation tensor cores multiply a block of 128 (four products of 32) into tensor memory; its sum then moves
// into registers with the block's scales, one fused multiply-add a value, while the next block is multiplied into
// another part of tensor memory.
//
// A pair of CTAs walks tiles of 256 x 256 of out: a's rows are the product's M, one to a lane of the accumulator, and a thread
// finishes the 128 columns of one of b's tiles, so that a block's scales are one number a thread. 8192 x 8192 x 4096: 190 us, 2.9
// PFLOP/s, tensor pipe 66% busy. What bounds it is the hand-over: reading the sums and the multiply-adds take about 480 cycles a
// block, the way there and back 250, the products 512, and tensor memory holds two blocks.
//
// Few rows are multiplied transposed, by single CTAs: b's rows (out's columns) are M and a's rows N, as many as there are (16 to
// 128) and not padded to 128. The scale of b is then one number for the tile, that of a one number per column
// of the accumulator, read from shared memory four at a time. (At 256 x 256 that reading was a third of
// the time: 276 us against 203 at 8192 x 8192 x 4096.) A cluster splits the inner dimension where the tiles are few.
#include <limits.h>
#include <math.h>

#include <algorithm>
#include <cmath>
#include <string>

#include "device.cuh"
#include "fp8.h"
#include "launch.cuh"
#include "maps.h"
#include "program.h"
#include "spans.h"
#include "tc.cuh"

namespace relay {
namespace {

// Bit 0: a wait ran out, the call's output is unspecified.
__device__ unsigned g_fp8_fault;

constexpr int kHalf = 128;                     // rows of the product's first operand in one CTA
constexpr int kFinishWarps = 8, kScaleWarps = 2;
constexpr int kProductThreads = 128 + 32 * kFinishWarps;
constexpr int kScaleStages = 4;                // blocks whose scales wait in shared memory
constexpr int kMostSplits = 8;                 // CTAs of a cluster that share a tile's inner dimension
constexpr int kAhead = 4;                      // blocks whose scales are on their way there

// CTAS 2: a pair's 256 of a's rows by NT = 256 of b's. CTAS 1: 128 of b's rows by NT of a's; splits of the inner dimension are
// a cluster that joins its sums in shared memory.
template <int CTAS, int NT>
struct Shape {
  static constexpr bool kPair = CTAS == 2;
  static constexpr int kRows = kPair ? 256 : NT, kCols = kPair ? NT : kHalf;  // of out
  static constexpr int kShare = NT / CTAS;     // rows of the second operand one CTA brings
  static constexpr int kFirstBytes = kHalf * kBlock, kStageBytes = kFirstBytes + kShare * kBlock;
  static constexpr int kPerSm = NT <= 64 ? 2 : 1;  // CTAs an SM holds: one's start and end under the other's products
  static constexpr int kStages = kPair ? 4 : NT >= 128 ? 6 : NT >= 64 ? 4 : 5;
  static constexpr int kAcc = NT >= 256 ? 2 : 4;          // blocks in tensor memory
  static constexpr int kTmem = kAcc * NT < 32 ? 32 : kAcc * NT;
  static constexpr int kMine = NT / 2;         // columns of the accumulator one thread finishes
  static constexpr int kAScales = kPair ? kHalf : NT, kBScales = kPair ? 2 : 1;  // of a block, in one CTA
  static constexpr int kScales = kAScales * kBScales;
  static constexpr int kRing = kStages * kStageBytes, kScaleBytes = kScaleStages * kScales * 4;
  static constexpr int kRawBytes = (kAScales + 4) * 4;  // a block's scales as they lie, b's behind them
  static constexpr int kStoreBytes = kPair ? 8192 : 1024;  // of a finishing warp
  static constexpr int kFinishBytes = kFinishWarps * kStoreBytes;
  static constexpr int kSmem = 1024 + kRing + kFinishBytes + kScaleBytes + kAhead * kRawBytes;  // without the groups' table
  // A CTA of the next call may start beside the last of this one and takes its tensor memory at once: what fits an SM's
  // shared memory together has to fit its tensor memory, or the two would wait for one another.
  static_assert(kPerSm * kTmem <= 512 && (kPerSm + 1) * kSmem > 228 * 1024, "tensor memory has 512 columns");
  static_assert(kStageBytes % 1024 == 0 && kFirstBytes % 1024 == 0, "operands on 1024-byte addresses");
};

// A pair's finishing threads hold 128 sums each, and registers move to them from the four warps that load and multiply: at
// launch every thread has kLaunchRegs. The launch checks that the kernel was given exactly that many.
constexpr int kLaunchRegs = 168, kFeedRegs = 56, kFinishRegs = 224;
static_assert(kFeedRegs + 2 * kFinishRegs == 3 * kLaunchRegs, "the groups' registers add up to the launch's");

struct ProductArgs {
  CUtensorMap a, b, c;                       // c: out, where out_map
  const float* a_scale;
  const float* b_scale;
  void* out;
  const int32_t* offset;
  int64_t out_ld;
  int32_t rows, cols, depth_blocks, groups;  // groups 1 where there are none
  int32_t by_depth, wide_out, splits;
  int32_t vectors;                           // out's rows take 16-byte stores
  int32_t out_map;                           // and end on 16 bytes: they can be stored through a map
  int32_t extra;                             // bytes a stage waits for that no load brings (test of the bounded waits)
};

// One tile of out: rows r0 .. r_end - 1, columns from n0 on, blocks k_lo .. k_hi - 1.
struct Tile {
  int group, r0, r_end, n0, k_lo, k_hi;
};

// Groups in shared memory: first[g] the tiles before group g; at[g] its first row, or first block of the depth (groups + 1 of
// both: a group ends where the next begins).
struct Groups {
  const int* first;
  const int* at;
  int nt;  // tiles along out's columns
};

template <int CTAS, int NT>
__device__ __forceinline__ Tile tile_at(const ProductArgs& p, const Groups& s, int i) {
  using S = Shape<CTAS, NT>;
  int lo = 0, hi = p.groups;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (s.first[mid] <= i) lo = mid;
    else hi = mid;
  }
  Tile t;
  t.group = lo;
  const int within = i - s.first[lo], mt = (s.first[lo + 1] - s.first[lo]) / s.nt;
  const int r = within % mt;
  t.n0 = within / mt * S::kCols;
  if (p.by_depth) {
    t.r0 = r * S::kRows;
    t.r_end = min(p.rows, t.r0 + S::kRows);
    t.k_lo = s.at[lo];
    t.k_hi = s.at[lo + 1];
  } else {
    t.r0 = s.at[lo] + r * S::kRows;
    t.r_end = min(s.at[lo + 1], t.r0 + S::kRows);
    t.k_lo = 0;
    t.k_hi = p.depth_blocks;
  }
  return t;
}

// Fills the table; the first warp. Whatever the offsets hold, the groups lie one behind the other inside the rows (or
// blocks of the depth).
template <int CTAS, int NT>
__device__ __forceinline__ void read_groups(const ProductArgs& p, int* first, int* at, int nt) {
  using S = Shape<CTAS, NT>;
  const int lane = threadIdx.x;
  auto sum_to = [lane](int v) {  // over the lanes up to this one
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int before = __shfl_up_sync(~0u, v, o);
      if (lane >= o) v += before;
    }
    return v;
  };
  const int last = p.by_depth ? INT_MAX - kBlock : p.rows;  // of a row's number
  const int begin = p.by_depth || p.offset == nullptr ? 0 : offset_at(p.offset, 0, last);
  const int most = (p.by_depth ? p.depth_blocks : p.rows) - begin;  // in all groups
  int tiles = 0, before = 0;
  for (int base = 0; base < p.groups; base += 32) {
    const int g = base + lane;
    int n = 0;
    if (g < p.groups) {
      n = most;
      if (p.offset != nullptr) {
        n = max(0, offset_at(p.offset, g + 1, last) - offset_at(p.offset, g, last));
        if (p.by_depth) n = (n + kBlock - 1) / kBlock;
        n = min(n, most);
      }
    }
    const int sum = sum_to(n), start = min(before + sum - n, most);
    n = min(n, most - start);
    const int mine = g < p.groups ? ((p.by_depth ? p.rows : n) + S::kRows - 1) / S::kRows * nt : 0, tsum = sum_to(mine);
    if (g < p.groups) {
      first[g] = tiles + tsum - mine;
      at[g] = begin + start;
    }
    tiles += __shfl_sync(~0u, tsum, 31);
    before = min(before + __shfl_sync(~0u, sum, 31), most);
  }
  if (lane == 0) {
    first[p.groups] = tiles;
    at[p.groups] = begin + before;
  }
}

template <int CTAS>
__device__ __forceinline__ void fp8_product(uint32_t tmem, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  if constexpr (CTAS == 2)
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(tmem),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
  else
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(tmem),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}
// fp32 accumulator, both operands e4m3 with the inner dimension contiguous, M x N.
__host__ __device__ constexpr uint32_t fp8_desc(int m, int n) { return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24); }

// W columns of 32 lanes (lane i of the warp: row i) of tensor memory; the values are there after tmem_wait on them.
template <int W>
__device__ __forceinline__ void tmem_load(uint32_t tmem, float (&v)[W]) {
  if constexpr (W == 32) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, "
        "%19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
          "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(tmem)
        : "memory");
  } else if constexpr (W == 16) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(tmem)
        : "memory");
  } else {
    static_assert(W == 8, "8, 16 or 32 columns");
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "r"(tmem)
                 : "memory");
  }
}
// Waits for all loads of the warp; v is not read before.
template <int W>
__device__ __forceinline__ void tmem_wait(float (&v)[W]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < W; ++i) asm volatile("" : "+f"(v[i]));
}

// c += a * b, two at once, each a fused multiply-add.
__device__ __forceinline__ void fma2(float& c0, float& c1, float a0, float a1, float b0, float b1) {
  asm("{\n.reg .b64 a, b, c;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nmov.b64 c, {%0, %1};\n"
      "fma.rn.f32x2 c, a, b, c;\nmov.b64 {%0, %1}, c;\n}"
      : "+f"(c0), "+f"(c1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ float4 lds4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void sts1(uint32_t addr, float v) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory"); }
__device__ __forceinline__ float lds1(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
// From memory to shared memory, in the background; where there is none, 0 and nothing is read.
__device__ __forceinline__ void copy_float(uint32_t dst, const float* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(there ? 4 : 0) : "memory");
}
// At a barrier of either CTA of the pair: tensor memory has been read (ordered by tcgen05.fence, not by the arrival).
__device__ __forceinline__ void bar_arrive_other(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("{\n.reg .b64 s;\nmbarrier.arrive.shared::cta.b64 s, [%0];\n}" ::"r"(bar) : "memory");
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ void store_out(const ProductArgs& p, int group, int row, int n, float v) {
  const int64_t at = ((int64_t)(p.by_depth ? group : 0) * p.rows + row) * p.out_ld + n;
  if (p.wide_out) static_cast<float*>(p.out)[at] = v;
  else static_cast<uint16_t*>(p.out)[at] = (uint16_t)(bf16x2_rn(v, 0.0f) & 0xffffu);
}

// 16 bytes of a row of out from column n on, of which the row may have fewer.
template <class T>
__device__ __forceinline__ void store_piece(T* to, float4 x, int columns) {
  constexpr int kLanes = 16 / (int)sizeof(T);
  if (columns >= kLanes) {
    *reinterpret_cast<float4*>(to) = x;
    return;
  }
  const uint32_t e[4] = {__float_as_uint(x.x), __float_as_uint(x.y), __float_as_uint(x.z), __float_as_uint(x.w)};
#pragma unroll
  for (int k = 0; k < kLanes; ++k)
    if (k < columns) {
      if constexpr (sizeof(T) == 4) to[k] = __uint_as_float(e[k]);
      else to[k] = (T)(e[k / 2] >> (k % 2 * 16));
    }
}

// A warp's N rows of 32 columns, v[j] row r0 + j, column n + lane. Through the warp's buffer they turn into 16 bytes a thread.
// (Stored as they are, 32 neighbours of 2 bytes at a time, 128 rows took 14,500 cycles and not 3,900.)
template <class T, int N>
__device__ __forceinline__ void store_columns(const ProductArgs& p, const Tile& t, int r0, int n, uint32_t buf, const float (&v)[N]) {
  constexpr int kFit = 1024 / 32 / (int)sizeof(T), kRows = N < kFit ? N : kFit;  // rows in the buffer
  constexpr int kPieces = 2 * (int)sizeof(T);                                     // 16-byte pieces of a row
  const int lane = threadIdx.x % 32;
  if (n >= p.cols || r0 >= t.r_end) return;
  if (!p.vectors) {
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (r0 + j < t.r_end && n + lane < p.cols) store_out(p, t.group, r0 + j, n + lane, v[j]);
    return;
  }
  T* out = static_cast<T*>(p.out) + (int64_t)(p.by_depth ? t.group : 0) * p.rows * p.out_ld;
#pragma unroll
  for (int j0 = 0; j0 < N; j0 += kRows) {
    if (r0 + j0 >= t.r_end) break;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const uint32_t at = buf + (j * 32 + lane) * (int)sizeof(T);
      if constexpr (sizeof(T) == 4) sts1(at, v[j0 + j]);
      else asm volatile("st.shared.b16 [%0], %1;" ::"r"(at), "h"((uint16_t)(bf16x2_rn(v[j0 + j], 0.0f) & 0xffffu)) : "memory");
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kRows * kPieces / 32; ++i) {
      const int row = r0 + j0 + i * (32 / kPieces) + lane / kPieces, col = n + lane % kPieces * (16 / (int)sizeof(T));
      const float4 x = lds4(buf + i * 512 + lane * 16);
      if (row < t.r_end) store_piece(out + row * p.out_ld + col, x, p.cols - col);
    }
  }
}

// A warp's 32 rows of N columns, v[j] row r0 + lane, column n + j. Where all rows are the group's they leave through a tensor map
// while the next tile is multiplied, 128 bytes of each row to a box; else, 64 bytes of each row at a time, neighbouring
// threads get neighbouring pieces of a row.
template <class T, int N>
__device__ __forceinline__ void store_rows(const ProductArgs& p, const Tile& t, int r0, int n, uint32_t buf, const float (&v)[N]) {
  constexpr int kCols = 64 / (int)sizeof(T), kPiece = 16 / (int)sizeof(T);
  const int lane = threadIdx.x % 32;
  if (n >= p.cols || r0 >= t.r_end) return;
  auto free_buffer = [&] {  // the store before may still be reading it
    if (lane == 0) store_wait_read<0>();
    __syncwarp();
  };
  free_buffer();
  if (p.out_map && r0 + 32 <= t.r_end) {
    constexpr int kBox = 2 * kCols;  // columns of a box; two boxes fit the buffer
#pragma unroll
    for (int c = 0; c < N; c += 2 * kBox) {
      if (c > 0) {
        if (n + c >= p.cols) break;
        free_buffer();
      }
#pragma unroll
      for (int box = 0; box < 2; ++box)
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = c + box * kBox + q * kPiece;
            w[i] = sizeof(T) == 4 ? __float_as_uint(v[j + i]) : bf16x2_rn(v[j + 2 * i], v[j + 2 * i + 1]);
          }
          const uint32_t at = buf + box * 4096 + lane * 128 + ((q ^ (lane & 7)) << 4);
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
        }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        const int y = (p.by_depth ? t.group * p.rows : 0) + r0;
        map_store(&p.c, n + c, y, buf);
        if (n + c + kBox < p.cols) map_store(&p.c, n + c + kBox, y, buf + 4096);
        store_commit();
      }
    }
    return;
  }
  T* out = static_cast<T*>(p.out) + (int64_t)(p.by_depth ? t.group : 0) * p.rows * p.out_ld;
#pragma unroll
  for (int c = 0; c < N; c += kCols) {
    if (n + c >= p.cols) break;
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = sizeof(T) == 4 ? __float_as_uint(v[c + q * kPiece + i]) : bf16x2_rn(v[c + q * kPiece + 2 * i], v[c + q * kPiece + 2 * i + 1]);
      const uint32_t at = buf + lane * 64 + ((q ^ (lane >> 1 & 3)) << 4);
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
    }
    __syncwarp();
    if (p.vectors) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = i * 8 + lane / 4, col = n + c + lane % 4 * kPiece;
        const float4 x = lds4(buf + r * 64 + (((lane % 4) ^ (r >> 1 & 3)) << 4));
        if (r0 + r < t.r_end) store_piece(out + (int64_t)(r0 + r) * p.out_ld + col, x, p.cols - col);
      }
    } else {
      // rows off the 16-byte grid: neighbouring threads on neighbouring elements
#pragma unroll 4
      for (int i = 0; i < kCols; ++i) {
        const int e = i * 32 + lane, r = e / kCols, j = e % kCols;
        const uint32_t at = buf + r * 64 + (((j / kPiece) ^ (r >> 1 & 3)) << 4) + j % kPiece * (int)sizeof(T);
        if (r0 + r >= t.r_end || n + c + j >= p.cols) continue;
        T* to = out + (int64_t)(r0 + r) * p.out_ld + n + c + j;
        if constexpr (sizeof(T) == 4) {
          *to = lds1(at);
        } else {
          uint16_t h;
          asm volatile("ld.shared.b16 %0, [%1];" : "=h"(h) : "r"(at) : "memory");
          *to = h;
        }
      }
    }
  }
}

// One thread of a warp that runs as a whole, the same one every time.
__device__ __forceinline__ bool elected() {
  uint32_t yes;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(yes));
  return yes != 0;
}

struct Bars {
  uint32_t full, empty, acc_full, acc_empty, scale_full, scale_empty, drain;
};

// A CTA's loads; a whole warp, of which one thread acts: what it hands to the copy engine and the tensor cores is then uniform, and
// in uniform registers as it is. next(): the next tile, group -1 after the last.
template <int CTAS, int NT, class Next>
__device__ void produce(const ProductArgs& p, int rank, uint32_t ring, const Bars& bar, volatile int* gave_up, Next next) {
  using S = Shape<CTAS, NT>;
  const uint32_t pair_full = CTAS == 2 ? pair_addr(bar.full, 0) : bar.full;
  int stage = 0;
  uint32_t phase = 0;
  int64_t issued = 0;
  bool ok = true;
  for (Tile t = next(); ok && t.group >= 0; t = next()) {
    const int b_row = (p.by_depth ? 0 : t.group * p.cols) + t.n0 + (S::kPair ? rank * kHalf : 0);
    const int a_row = t.r0 + (S::kPair ? rank * kHalf : 0);
    const CUtensorMap* first = S::kPair ? &p.a : &p.b;
    const CUtensorMap* second = S::kPair ? &p.b : &p.a;
    for (int k = t.k_lo; k < t.k_hi; ++k) {
      if (!(ok = __all_sync(~0u, bar_wait<false>(bar.empty + 8 * stage, phase ^ 1, gave_up)))) break;  // the warp as one
      if (elected()) {
        if (CTAS == 1 || rank == 0) bar_expect(bar.full + 8 * stage, CTAS * S::kStageBytes + p.extra);
        const uint32_t at = ring + stage * S::kStageBytes, on = pair_full + 8 * stage;
        map_load<CTAS>(at, first, k * kBlock, S::kPair ? a_row : b_row, on);
        map_load<CTAS>(at + S::kFirstBytes, second, k * kBlock, S::kPair ? b_row : a_row, on);
      }
      ++issued;
      if (++stage == S::kStages) {
        stage = 0;
        phase ^= 1;
      }
    }
  }
  if (ok) return;
  // giving up: no load may still be on its way into shared memory when the CTA leaves. The first CTA's barriers count
  // both CTAs' loads, and the pair leaves together; what they do not count lands in microseconds.
  const uint64_t start = global_ns();
  for (int back = 0; (CTAS == 1 || rank == 0) && back < S::kStages && back < issued; ++back) {
    if (--stage < 0) {
      stage = S::kStages - 1;
      phase ^= 1;
    }
    while (!bar_try<false>(bar.full + 8 * stage, phase) && global_ns() - start < kWaitNs) {
    }
  }
  const uint64_t drained = global_ns();
  while (global_ns() - drained < 10000000ull) {
  }
}

template <int CTAS, int NT, class Next>
__device__ void multiply(uint32_t ring, const Bars& bar, uint32_t tmem, volatile int* gave_up, Next next) {
  using S = Shape<CTAS, NT>;
  constexpr uint32_t desc = fp8_desc(CTAS * kHalf, NT);
  int stage = 0;
  uint32_t phase = 0, n = 0;
  bool ok = true;
  for (Tile t = next(); ok && t.group >= 0; t = next()) {
    for (int k = t.k_lo; k < t.k_hi; ++k, ++n) {
      const uint32_t part = n % S::kAcc;
      const bool free = bar_wait<false>(bar.acc_empty + 8 * part, ((n / S::kAcc) & 1) ^ 1, gave_up);
      if (!(ok = __all_sync(~0u, bar_wait<false>(bar.full + 8 * stage, phase, gave_up) && free))) break;  // the warp as one
      tc_fence_after();
      if (elected()) {
        const uint32_t at = ring + stage * S::kStageBytes;
        const uint64_t d1 = operand_desc<64>(at, false), d2 = operand_desc<64>(at + S::kFirstBytes, false);
#pragma unroll
        for (int j = 0; j < kBlock / 32; ++j)
          fp8_product<CTAS>(tmem + part * NT, d1 + j * (32 >> 4), d2 + j * (32 >> 4), desc, j > 0);
        tc_commit<CTAS>(bar.acc_full + 8 * part);
        tc_commit<CTAS>(bar.empty + 8 * stage);
      }
      __syncwarp();
      if (++stage == S::kStages) {
        stage = 0;
        phase ^= 1;
      }
    }
  }
  // giving up: products still running write the tensor memory that is about to be freed
  if (!ok) {
    if (elected()) tc_commit<CTAS>(bar.drain);
    const uint64_t start = global_ns();
    while (!bar_try<false>(bar.drain, 0) && global_ns() - start < kWaitNs) {
    }
  }
}

// The scales' products of every block, one for each of the tile's rows (CTAS 2: of this CTA's, with each of b's two tiles), ahead of
// the sums that want them. The scales of the next kAhead blocks are on their way into shared memory (each thread reads
// what it asked for itself; b's come once for each warp), so that the loads' latency is not between two blocks.
template <int CTAS, int NT, class Next>
__device__ void bring_scales(const ProductArgs& p, int rank, uint32_t raw, uint32_t ring, const Bars& bar, volatile int* gave_up, Next next) {
  using S = Shape<CTAS, NT>;
  constexpr int kThreads = 32 * kScaleWarps, kEach = (S::kAScales + kThreads - 1) / kThreads;
  constexpr bool kAll = S::kAScales >= kThreads;  // every thread has one
  const int me = threadIdx.x - 64, lane = threadIdx.x % 32;
  const uint32_t mine = raw + me * 4, others = raw + (S::kAScales + me / 32 * S::kBScales) * 4;
  const int64_t row_blocks = (p.cols + kBlock - 1) / kBlock;
  Tile t = next();
  int k = t.k_lo, row = 0;
  const float* bs = nullptr;
  bool there = false;
  auto open = [&] {  // the first tile from t on that has blocks
    while (t.group >= 0 && k >= t.k_hi) {
      t = next();
      k = t.k_lo;
    }
    const int block = t.n0 / kBlock + (lane < S::kBScales ? lane : 0);
    there = t.group >= 0 && block < row_blocks;
    bs = p.b_scale + ((p.by_depth ? 0 : t.group * row_blocks) + block) * p.depth_blocks;
    row = t.r0 + (S::kPair ? rank * kHalf : 0) + me;
  };
  uint32_t asked = 0;
  auto ask = [&] {
    if (t.group >= 0) {
      const uint32_t at = asked % kAhead * S::kRawBytes;
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        const int r = row + kThreads * e;
        if (kAll || me < S::kAScales)
          copy_float(mine + at + kThreads * e * 4, p.a_scale + (int64_t)k * p.rows + (r < t.r_end ? r : 0), r < t.r_end);
      }
      if (lane < S::kBScales) copy_float(others + at + lane * 4, there ? bs + k : p.b_scale, there);
      ++asked;
      if (++k >= t.k_hi) open();
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  open();
  for (int i = 0; i < kAhead; ++i) ask();
  for (uint32_t n = 0; n < asked; ++n) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
    __syncwarp();
    const uint32_t at = n % kAhead * S::kRawBytes, s = n % kScaleStages;
    float f[S::kBScales][kEach];
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const float x = kAll || me < S::kAScales ? lds1(mine + at + kThreads * e * 4) : 0.0f;
#pragma unroll
      for (int j = 0; j < S::kBScales; ++j) f[j][e] = __fmul_rn(x, lds1(others + at + j * 4));
    }
    if (!__all_sync(~0u, bar_wait<false>(bar.scale_empty + 8 * s, ((n / kScaleStages) & 1) ^ 1, gave_up))) break;
#pragma unroll
    for (int j = 0; j < S::kBScales; ++j)
#pragma unroll
      for (int e = 0; e < kEach; ++e)
        if (kAll || me < S::kAScales) sts1(ring + (s * S::kScales + j * S::kAScales + me + kThreads * e) * 4, f[j][e]);
    __syncwarp();  // all of the warp have read and written theirs
    if (lane == 0) bar_arrive(bar.scale_full + 8 * s);
    ask();
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// A tile's sums. CTAS 2: v[j] is column n0 + part * 128 + j of out, in the row of the thread's lane; CTAS 1: row r0 + part * kMine + j,
// in the column of the lane. n: blocks before.
template <int CTAS, int NT>
__device__ __forceinline__ bool finish(const Tile& t, uint32_t& n, uint32_t scales, const Bars& bar, uint32_t tmem, int quarter, int part,
                                       volatile int* gave_up, float (&v)[Shape<CTAS, NT>::kMine]) {
  using S = Shape<CTAS, NT>;
  // columns read at a time: 32 of a pair's 128 take 190 us where 16 take 196 (8192 x 8192 x 4096); 64, or a read ahead, spill
  constexpr int W = S::kMine <= 16 ? S::kMine : NT == 64 ? 16 : 32;
  const int lane = threadIdx.x % 32;
  const uint32_t first_empty = S::kPair ? pair_addr(bar.acc_empty, 0) : bar.acc_empty;
#pragma unroll
  for (int j = 0; j < S::kMine; ++j) v[j] = 0.0f;
  for (int k = t.k_lo; k < t.k_hi; ++k, ++n) {
    const uint32_t acc = n % S::kAcc, s = n % kScaleStages;
    if (!__all_sync(~0u, bar_wait<false>(bar.scale_full + 8 * s, (n / kScaleStages) & 1, gave_up))) return false;
    if (!__all_sync(~0u, bar_wait<false>(bar.acc_full + 8 * acc, (n / S::kAcc) & 1, gave_up))) return false;
    tc_fence_after();
    const uint32_t from = tmem + acc * NT + part * S::kMine + ((uint32_t)(quarter * 32) << 16);
    const uint32_t f = scales + (s * S::kScales + part * S::kMine) * 4;  // CTAS 2: 128 rows with this part's tile
    const float own = S::kPair ? lds1(f + (quarter * 32 + lane) * 4) : 0.0f;
#pragma unroll
    for (int c = 0; c < S::kMine; c += W) {
      float x[W];
      tmem_load<W>(from + c, x);
      tmem_wait<W>(x);
#pragma unroll
      for (int j = 0; j < W; j += 4) {
        const float4 g = S::kPair ? make_float4(own, own, own, own) : lds4(f + (c + j) * 4);
        fma2(v[c + j], v[c + j + 1], x[j], x[j + 1], g.x, g.y);
        fma2(v[c + j + 2], v[c + j + 3], x[j + 2], x[j + 3], g.z, g.w);
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      bar_arrive(bar.scale_empty + 8 * s);
      if (S::kPair) bar_arrive_other(first_empty + 8 * acc);
      else bar_arrive(first_empty + 8 * acc);
    }
  }
  return true;
}

template <int CTAS, int NT>
__global__ void __launch_bounds__(kProductThreads, Shape<CTAS, NT>::kPerSm) fp8_product_kernel(const __grid_constant__ ProductArgs p) {
  using S = Shape<CTAS, NT>;
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t s_bar[2 * S::kStages + 2 * S::kAcc + 2 * kScaleStages + 1];
  __shared__ uint32_t s_tmem;
  __shared__ int s_gave_up;
  const int warp = __shfl_sync(~0u, (int)threadIdx.x / 32, 0), rank = (int)pair_rank();
  dep_launch();
  const uint32_t ring = (smem_addr(smem_raw) + 1023) & ~1023u, staging = ring + S::kRing, scales = staging + S::kFinishBytes;
  const uint32_t raw = scales + S::kScaleBytes;
  int* s_first = reinterpret_cast<int*>(smem_raw + (raw - smem_addr(smem_raw)) + kAhead * S::kRawBytes);
  Bars bar;
  bar.full = smem_addr(s_bar);
  bar.empty = bar.full + 8 * S::kStages;
  bar.acc_full = bar.empty + 8 * S::kStages;
  bar.acc_empty = bar.acc_full + 8 * S::kAcc;
  bar.scale_full = bar.acc_empty + 8 * S::kAcc;
  bar.scale_empty = bar.scale_full + 8 * kScaleStages;
  bar.drain = bar.scale_empty + 8 * kScaleStages;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      bar_init(bar.full + 8 * i, 1);
      bar_init(bar.empty + 8 * i, 1);
    }
    for (int i = 0; i < S::kAcc; ++i) {
      bar_init(bar.acc_full + 8 * i, 1);
      bar_init(bar.acc_empty + 8 * i, CTAS * kFinishWarps);  // of all CTAs, at the first's
    }
    for (int i = 0; i < kScaleStages; ++i) {
      bar_init(bar.scale_full + 8 * i, kScaleWarps);
      bar_init(bar.scale_empty + 8 * i, kFinishWarps);
    }
    bar_init(bar.drain, 1);
    s_gave_up = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    if (p.depth_blocks > 0) {  // else there are no maps
      map_prefetch(&p.a);
      map_prefetch(&p.b);
    }
    if (S::kPair && p.out_map) map_prefetch(&p.c);
  }
  if (warp == 1) tmem_alloc<CTAS>(smem_addr(&s_tmem), S::kTmem);
  dep_wait();
  const Groups groups{s_first, s_first + p.groups + 1, (p.cols + S::kCols - 1) / S::kCols};
  if (warp == 0) read_groups<CTAS, NT>(p, s_first, s_first + p.groups + 1, groups.nt);
  tc_fence_before();
  __syncthreads();
  const bool clustered = CTAS == 2 || p.splits > 1;
  if (clustered) pair_sync();  // the other CTAs' barriers are ready
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const int tiles = s_first[p.groups];
  // CTAS 2: every pair's tiles; CTAS 1: the one tile of a cluster, its share of the blocks
  int at = CTAS == 2 ? (int)blockIdx.x / 2 : (int)blockIdx.x / p.splits;
  const int step = CTAS == 2 ? (int)gridDim.x / 2 : INT_MAX / 2;  // none after the first
  const auto all = [&, at]() mutable {
    Tile t{-1, 0, 0, 0, 0, 0};
    if (at >= tiles) return t;
    t = tile_at<CTAS, NT>(p, groups, at);
    at += step;
    if (CTAS == 1 && p.splits > 1) {
      const int k = t.k_hi - t.k_lo;
      t.k_hi = t.k_lo + (int)((int64_t)k * (rank + 1) / p.splits);
      t.k_lo += (int)((int64_t)k * rank / p.splits);
    }
    return t;
  };
  auto next = all;
  if (CTAS == 2) {
    if (warp < 4) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFeedRegs));
    } else {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kFinishRegs));
    }
  }
  if (warp < 4) {
    if (warp == 0) produce<CTAS, NT>(p, rank, ring, bar, &s_gave_up, next);
    if (warp == 1 && (CTAS == 1 || rank == 0)) multiply<CTAS, NT>(ring, bar, tmem, &s_gave_up, next);
    if (warp >= 2) bring_scales<CTAS, NT>(p, rank, raw, scales, bar, &s_gave_up, next);
  } else {
    // warps 4 to 7 finish the accumulator's first half of columns, 8 to 11 the other; a warp reads the quarter of
    // tensor memory's lanes that its number gives it
    const int quarter = warp % 4, part = warp / 4 - 1, lane = threadIdx.x % 32;
    uint32_t n = 0;
    for (Tile t = next(); t.group >= 0; t = next()) {
      float v[S::kMine];
      if (!finish<CTAS, NT>(t, n, scales, bar, tmem, quarter, part, &s_gave_up, v)) break;
      const uint32_t buf = staging + (warp - 4) * S::kStoreBytes;
      if constexpr (S::kPair) {
        const int row = t.r0 + rank * kHalf + quarter * 32, col = t.n0 + part * S::kMine;
        if (p.wide_out) store_rows<float>(p, t, row, col, buf, v);
        else store_rows<uint16_t>(p, t, row, col, buf, v);
      } else if (p.splits > 1) {
        // the products are done with the ring: it takes the partial sums
#pragma unroll
        for (int j = 0; j < S::kMine; ++j) sts1(ring + ((part * S::kMine + j) * kHalf + quarter * 32 + lane) * 4, v[j]);
      } else {
        const int row = t.r0 + part * S::kMine, col = t.n0 + quarter * 32;
        if (p.wide_out) store_columns<float>(p, t, row, col, buf, v);
        else store_columns<uint16_t>(p, t, row, col, buf, v);
      }
    }
    if (S::kPair && lane == 0) store_wait_all();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (clustered) pair_sync();  // neither CTA's memory is used by the other's products any more; partial sums are there
  if (CTAS == 1 && p.splits > 1) {
    auto again = all;
    const Tile t = again();
    if (t.group >= 0 && !s_gave_up) {
      // each CTA joins its share of the tile's rows, in the order of the splits
      const int each = NT / p.splits;
      for (int e = threadIdx.x; e < each * kHalf; e += kProductThreads) {
        const int j = rank * each + e / kHalf, row = t.r0 + j, col = t.n0 + e % kHalf;
        float part[kMostSplits], sum = 0.0f;  // all asked for before the first is added
#pragma unroll
        for (int s = 0; s < kMostSplits; ++s)
          part[s] = s < p.splits ? ld_cluster(pair_addr(ring + (j * kHalf + e % kHalf) * 4, s)) : 0.0f;
#pragma unroll
        for (int s = 0; s < kMostSplits; ++s) sum = __fadd_rn(sum, part[s]);
        if (row < t.r_end && col < p.cols) store_out(p, t.group, row, col, sum);
      }
    }
    pair_sync();  // the partial sums stay until all have read them
  }
  if (threadIdx.x == 0 && s_gave_up) atomicOr(&g_fp8_fault, 1u);
  if (warp == 1) {
    tc_fence_after();
    tmem_free<CTAS>(tmem, S::kTmem);
  }
}

// ------------------------------------------------------------------ host side --

thread_local int t_extra = 0;

relay_status_t bad(const std::string& msg) { return report_error(RELAY_ERR_INVALID_ARGUMENT, "relay_matmul_fp8: " + msg); }

// out [rows][cols], written in boxes of 32 rows by 128 bytes (128-byte swizzle).
bool result_map(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, int64_t ld, bool wide) {
  const EncodeFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)ld * (wide ? 4 : 2)};
  const cuuint32_t box[2] = {wide ? 32u : 64u, 32u}, unit[2] = {1, 1};
  return fn(m, wide ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p), dims, strides, box, unit,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// A matrix [rows][bytes], read in boxes of box_rows by 128 bytes.
bool bytes_map(CUtensorMap* m, const void* p, int64_t rows, int64_t bytes, int64_t ld, int box_rows) {
  const EncodeFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)bytes, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)ld};
  const cuuint32_t box[2] = {(cuuint32_t)kBlock, (cuuint32_t)box_rows}, unit[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(p), dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The most tiles the rows can make, wherever the groups end.
int64_t most_tiles(const relay_fp8_matmul_t& w, int nt, int m) {
  const int64_t cols = (w.cols + m - 1) / m, groups = std::max(w.groups, 1);
  if (w.by_depth) return groups * ((w.rows + nt - 1) / nt) * cols;
  return (w.groups == 0 ? (w.rows + nt - 1) / nt : w.rows / nt + std::min<int64_t>(groups, w.rows)) * cols;
}

template <int CTAS, int NT>
cudaError_t launch(ProductArgs p, const relay_fp8_matmul_t& w, int splits, cudaStream_t s) {
  using S = Shape<CTAS, NT>;
  static thread_local int ready_device = -1;
  constexpr int kFixed = S::kSmem;
  constexpr int kMost = kFixed + 2 * (RELAY_FP8_MAX_GROUPS + 1) * 4;
  static_assert(kMost <= 227 * 1024 - 1024, "shared memory of a CTA");
  static_assert(S::kRing >= NT * kHalf * 4 || CTAS == 2, "the ring takes the partial sums");
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  auto* kernel = fp8_product_kernel<CTAS, NT>;
  if (ready_device != dev) {
    cudaFuncAttributes attr;
    e = cudaFuncGetAttributes(&attr, kernel);
    if (e != cudaSuccess) return e;
    if (CTAS == 2 && attr.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;  // the split would wait forever
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (e != cudaSuccess) return e;
    ready_device = dev;
  }
  const int64_t a_rows = w.rows, b_rows = w.by_depth ? w.cols : w.cols * std::max(w.groups, 1);
  if (w.depth > 0 && (!bytes_map(&p.a, w.a, a_rows, w.depth, w.a_stride, S::kPair ? kHalf : NT) ||
                      !bytes_map(&p.b, w.b, b_rows, w.depth, w.b_stride, kHalf)))
    return cudaErrorInvalidValue;
  if (S::kPair && p.out_map &&
      !result_map(&p.c, w.out, w.by_depth ? w.rows * std::max(w.groups, 1) : w.rows, w.cols, w.out_stride, p.wide_out != 0))
    return cudaErrorInvalidValue;
  const int64_t tiles = most_tiles(w, S::kRows, S::kCols);
  if (tiles * 8 > INT_MAX) return cudaErrorInvalidConfiguration;  // 2^28 tiles: refused before
  p.splits = splits;
  const int blocks = CTAS == 2 ? (int)std::min<int64_t>(2 * tiles, sm_count() / 2 * 2) : (int)(tiles * splits);
  return launch_chained_clusters(kernel, CTAS == 2 ? 2 : splits, blocks, kProductThreads, kFixed + 2 * (p.groups + 1) * 4, s, p);
}

// Which kernel. A round of CTAs takes `open` us and `step` us for every block of the inner dimension; the numbers are fitted to
// products of 8 to 8192 rows by 1536 to 8192 columns of 1024 to 4096 values, and to 96 to 16384 rows in 16 and 32 groups. On 35
// sizes, 28 of them others (1 to 5000 rows, 200 to 8192 columns, 200 to 16384 values, up to 32 groups of rows or of the depth), what
// it takes is within 8% of the best of ten, but for 512 rows in 32 groups: uneven ones take 16.0 us where 64 rows to a tile take 11.9,
// even ones 16.2 where 64 take 18.8. What it decides (us): 8 x 4096 x 4096: 16 rows split eight ways 7.3, whole 10.4, 32 rows whole
// 11.1; 256 x 1536 x 1024: 16 rows 5.3, 32 5.5, 64 6.3, 128 6.3, pairs 8.2; 400 x 4096 x 4096: 128 rows 14.1, pairs 17.0; 1024 x 4096
// x 4096: 128 rows 27.4, pairs 17.2; 96 rows of 32 groups by 1408 x 2048: 16 rows 8.8, 64 10.8; 2048 rows of 32 groups: 64 rows 21.6,
// 128 26.9, pairs 28.4.
struct Plan {
  bool pair;
  int rows, splits;
};
Plan choose(const relay_fp8_matmul_t& w) {
  const double sms = 152, blocks = (double)(w.depth + kBlock - 1) / kBlock;
  const double kb = w.by_depth ? blocks / std::max(w.groups, 1) : blocks;
  // tiles, when groups end anywhere
  auto tiles = [&](int rows, int cols) {
    const double across = (double)((w.cols + cols - 1) / cols), all = (double)((w.rows + rows - 1) / rows);
    if (w.by_depth) return across * all * std::max(w.groups, 1);
    if (w.groups == 0) return across * all;
    // some groups have no row, and the others' last tiles are half full
    return across * std::max((double)w.rows / rows + 0.4 * w.groups, 0.8 * (double)std::min<int64_t>(w.groups, w.rows));
  };
  Plan best{true, 256, 1};
  double least = 3.5 + std::ceil(tiles(256, 256) / (sms / 2)) * (1.5 + 0.41 * kb);
  const struct {
    int rows;
    double open, step;
  } one[] = {{16, 2.7, 0.23}, {32, 2.8, 0.26}, {64, 3.0, 0.40}, {128, 3.4, 0.31}};
  for (const auto& o : one) {
    const double t = tiles(o.rows, kHalf);
    for (int splits = 1; splits <= kMostSplits; splits *= 2) {
      if (splits > 1 && (o.rows > 32 || t * splits > 2 * sms)) break;
      const double rounds = t * splits / sms, step = o.step * kb / splits;
      // two CTAs an SM up to 64 rows; joining the splits costs about as much as a start
      double cost = o.rows == 128 ? std::ceil(rounds + (w.groups > 0 && !w.by_depth ? 0.3 : 0.0)) * (o.open + step)
                                  : std::max(1.0, std::ceil(rounds / 2)) * o.open + step * std::max(1.0, 0.85 * rounds);
      if (splits > 1) cost += 3.5;
      if (cost < least) {
        least = cost;
        best = Plan{false, o.rows, splits};
      }
    }
  }
  return best;
}

cudaError_t run(const ProductArgs& p, const relay_fp8_matmul_t& w, const Plan& c, cudaStream_t s) {
  if (c.pair) return launch<2, 256>(p, w, 1, s);
  switch (c.rows) {
    case 16: return launch<1, 16>(p, w, c.splits, s);
    case 32: return launch<1, 32>(p, w, c.splits, s);
    case 64: return launch<1, 64>(p, w, c.splits, s);
    default: return launch<1, 128>(p, w, c.splits, s);
  }
}

}  // namespace

cudaError_t fp8_read_fault(unsigned* fault) {
  cudaError_t e = cudaMemcpyFromSymbol(fault, g_fp8_fault, sizeof *fault);
  if (e != cudaSuccess || *fault == 0) return e;
  const unsigned zero = 0;
  return cudaMemcpyToSymbol(g_fp8_fault, &zero, sizeof zero);
}

}  // namespace relay

extern "C" {

relay_status_t relay_matmul_fp8(const relay_fp8_matmul_t* w, cudaStream_t stream) {
  using namespace relay;
  return guarded([&]() -> relay_status_t {
    if (w == nullptr) return bad("the description is NULL");
    if (w->out_dtype != RELAY_F32 && w->out_dtype != RELAY_BF16) return bad("out_dtype must be RELAY_F32 or RELAY_BF16");
    if (w->rows < 0 || w->rows > RELAY_FP8_MAX_ROWS || w->cols < 1 || w->cols > RELAY_FP8_MAX_ROWS) return bad("rows or cols out of range");
    if (w->depth < 0 || w->depth > 2 * RELAY_FP8_MAX_ROWS) return bad("depth out of range");
    if (w->groups < 0 || w->groups > RELAY_FP8_MAX_GROUPS) return bad("groups out of range");
    const bool grouped = w->offset != nullptr;
    if (grouped != (w->groups > 0)) return bad("groups and offset go together");
    if (w->by_depth && grouped && w->depth % kBlock) return bad("a depth of groups is made of whole blocks");
    if (w->rows == 0) return RELAY_OK;
    const int64_t groups = std::max(w->groups, 1), kb = blocks_of(w->depth), limit = 1ll << 32;
    const int64_t b_rows = w->by_depth ? w->cols : w->cols * groups, out_rows = w->by_depth ? w->rows * groups : w->rows;
    if (b_rows > INT_MAX || out_rows > INT_MAX) return bad("more than 2^31 - 1 rows over all groups");
    if (w->out == nullptr) return bad("out is NULL");
    if (w->depth > 0 && (w->a == nullptr || w->b == nullptr || w->a_scale == nullptr || w->b_scale == nullptr))
      return bad("a, b or a scale is NULL");
    auto off = [](const void* q, uintptr_t e) { return reinterpret_cast<uintptr_t>(q) % e != 0; };
    const int64_t E = esize_of(w->out_dtype);
    if (off(w->a, 16) || off(w->b, 16)) return bad("a or b is not on a 16-byte boundary");
    if (w->a_stride < w->depth || w->a_stride > limit || w->a_stride % 16) return bad("a_stride is less than depth, more than 2^32 or no multiple of 16");
    if (w->b_stride < w->depth || w->b_stride > limit || w->b_stride % 16) return bad("b_stride is less than depth, more than 2^32 or no multiple of 16");
    if (w->out_stride < w->cols || w->out_stride > limit) return bad("out_stride is less than cols or more than 2^32");
    if (off(w->a_scale, 4) || off(w->b_scale, 4) || off(w->offset, 4) || off(w->out, E)) return bad("an array is not element-aligned");
    const struct {
      Span span;
      const char* what;
    } in[] = {{matrix_span(w->a, w->rows, w->depth, w->a_stride), "a"},
              {matrix_span(w->b, b_rows, w->depth, w->b_stride), "b"},
              {array_span(w->a_scale, 4 * kb * w->rows), "a_scale"},
              {array_span(w->b_scale, 4 * kb * blocks_of(w->cols) * (w->by_depth ? 1 : groups)), "b_scale"},
              {array_span(w->offset, 4 * (groups + 1)), "offset"}};
    const Span out = matrix_span(w->out, out_rows, w->cols * E, w->out_stride * E);
    for (const auto& s : in)
      if (overlap(out, s.span)) return bad(std::string("out overlaps ") + s.what);
    ProductArgs p{};
    p.a_scale = w->a_scale;
    p.b_scale = w->b_scale;
    p.out = w->out;
    p.offset = w->offset;
    p.out_ld = w->out_stride;
    p.rows = (int32_t)w->rows;
    p.cols = (int32_t)w->cols;
    p.depth_blocks = (int32_t)kb;
    p.groups = (int32_t)groups;
    p.by_depth = w->by_depth != 0;
    p.wide_out = w->out_dtype == RELAY_F32;
    p.vectors = !off(w->out, 16) && w->out_stride * E % 16 == 0;
    // a store through a map writes 16 bytes at a time, also where the row ends inside them
    p.out_map = p.vectors && w->cols * E % 16 == 0;
    p.extra = t_extra;
    const Plan plan = choose(*w);
    const int64_t tiles = plan.pair ? most_tiles(*w, 256, 256) : most_tiles(*w, plan.rows, kHalf);
    if (tiles * 8 > INT_MAX) return report_error(RELAY_ERR_UNSUPPORTED, "relay_matmul_fp8: more than 2^28 tiles of out");
    const cudaError_t e = run(p, *w, plan, stream);
    if (e != cudaSuccess) return report_error(RELAY_ERR_CUDA, std::string("relay_matmul_fp8: ") + cudaGetErrorString(e));
    return RELAY_OK;
  });
}

relay_status_t relay_test_fp8_wait(const relay_fp8_matmul_t* what, int extra_bytes, cudaStream_t stream) {
  using namespace relay;
  return guarded([&]() -> relay_status_t {
    if (extra_bytes < 0 || extra_bytes > 65536) return bad("0 <= extra_bytes <= 65536");
    t_extra = extra_bytes;
    const relay_status_t st = relay_matmul_fp8(what, stream);
    t_extra = 0;
    return st;
  });
}

}  // extern "C"
