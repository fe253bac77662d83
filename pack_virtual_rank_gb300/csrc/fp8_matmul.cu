// fp8_matmul.cu -- relay_matmul_fp8: products of e4m3 matrices with a scale for each block of 128 of the inner dimension.
//
//   out[r][n] = sum over blocks k of  a_scale[k][r] b_scale[n / 128][k] * sum over d in k of a[r][d] b[n][d]
//
// The fifth-generation tensor cores multiply a block of 128 (four products of 32) into tensor memory; its sum then moves
// into registers with the block's scales, one fused multiply-add a value, while the next block is multiplied into
// another part of tensor memory.
//
// out is made transposed: b's rows (out's columns) are the product's M, one to a lane of the accumulator, and a's rows its N. So
// the scale of b is one number for the whole tile of 128, that of a one number per column of the accumulator, read
// from shared memory four at a time; few rows make a narrow product without padding them to 128; and a warp stores a
// row of out as 32 neighbours, whatever its address and wherever a group ends.
#include <limits.h>

#include <algorithm>
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

constexpr int kBM = 128;                       // b's rows of one CTA
constexpr int kFinishWarps = 8, kScaleWarps = 2;
constexpr int kProductThreads = 128 + 32 * kFinishWarps;
constexpr int kScaleStages = 8;                // blocks whose scales wait in shared memory

// CTAS make one product of 128 CTAS of b's rows by NT of a's. CTAS 1: splits of the inner dimension are a cluster that joins
// its sums in shared memory. CTAS 2: a pair walks tiles.
template <int CTAS, int NT>
struct Shape {
  static constexpr int kM = CTAS * kBM;
  static constexpr int kShare = NT / CTAS;     // a's rows one CTA brings
  static constexpr int kBBytes = kBM * kBlock, kABytes = kShare * kBlock, kStageBytes = kBBytes + kABytes;
  static constexpr int kStages = CTAS == 2 ? 6 : NT >= 128 ? 5 : NT >= 64 ? 7 : 8;
  static constexpr int kAcc = NT >= 256 ? 2 : 4;          // blocks in tensor memory
  static constexpr int kTmem = kAcc * NT < 32 ? 32 : kAcc * NT;
  static constexpr int kMine = NT / 2;         // columns of the accumulator one thread finishes
  static constexpr int kRing = kStages * kStageBytes, kScaleBytes = kScaleStages * NT * 4;
  static_assert(kTmem <= 512, "tensor memory has 512 columns");
  static_assert(kStageBytes % 1024 == 0 && kBBytes % 1024 == 0, "operands on 1024-byte addresses");
};

constexpr int kLaunchRegs = 168, kFeedRegs = 56, kFinishRegs = 224;
static_assert(kFeedRegs + 2 * kFinishRegs == 3 * kLaunchRegs, "the groups' registers add up to the launch's");

struct ProductArgs {
  CUtensorMap a, b;
  const float* a_scale;
  const float* b_scale;
  void* out;
  const int32_t* offset;
  int64_t out_ld;
  int32_t rows, cols, depth_blocks, groups;  // groups 1 where there are none
  int32_t by_depth, wide_out, splits;
  int32_t extra;                             // bytes a stage waits for that no load brings (test of the bounded waits)
};

// One tile of out: rows r0 .. r_end - 1 (at most NT), columns from n0 on, blocks k_lo .. k_hi - 1.
struct Tile {
  int group, r0, r_end, n0, k_lo, k_hi;
};

// Groups in shared memory: first[g] the tiles before group g; at[g] its first row, or first block of the depth.
struct Groups {
  const int* first;
  const int* at;
  const int* len;
  int nt;  // tiles along out's columns
};

template <int CTAS, int NT>
__device__ __forceinline__ Tile tile_at(const ProductArgs& p, const Groups& s, int i) {
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
  t.n0 = within / mt * Shape<CTAS, NT>::kM;
  if (p.by_depth) {
    t.r0 = r * NT;
    t.r_end = min(p.rows, t.r0 + NT);
    t.k_lo = s.at[lo];
    t.k_hi = s.at[lo] + s.len[lo];
  } else {
    t.r0 = s.at[lo] + r * NT;
    t.r_end = min(s.at[lo] + s.len[lo], t.r0 + NT);
    t.k_lo = 0;
    t.k_hi = p.depth_blocks;
  }
  return t;
}

// Fills the table; the first warp. Returns all tiles.
template <int CTAS, int NT>
__device__ __forceinline__ void read_groups(const ProductArgs& p, int* first, int* at, int* len, int nt) {
  const int lane = threadIdx.x;
  const int mt_all = (p.rows + NT - 1) / NT;
  auto sum_to = [lane](int v) {  // over the lanes up to this one
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int before = __shfl_up_sync(~0u, v, o);
      if (lane >= o) v += before;
    }
    return v;
  };
  // rows, or blocks of the depth; all groups together have no more, whatever the offsets say
  const int most = p.by_depth ? p.depth_blocks : p.rows;
  int tiles = 0, before = 0;
  for (int base = 0; base < p.groups; base += 32) {
    const int g = base + lane;
    int from = 0, n = 0;
    if (g < p.groups) {
      if (p.offset == nullptr) {
        n = most;
      } else {
        const int last = p.by_depth ? INT_MAX - kBlock : p.rows;
        from = offset_at(p.offset, g, last);
        n = max(0, offset_at(p.offset, g + 1, last) - from);
        if (p.by_depth) n = (n + kBlock - 1) / kBlock;
        n = min(n, most);
      }
    }
    const int sum = sum_to(n), start = min(before + sum - n, most);
    n = min(n, most - start);
    if (p.by_depth) from = start;  // a group's blocks follow those of the one before
    const int mine = g < p.groups ? (p.by_depth ? mt_all : (n + NT - 1) / NT) * nt : 0, tsum = sum_to(mine);
    if (g < p.groups) {
      first[g] = tiles + tsum - mine;
      at[g] = from;
      len[g] = n;
    }
    tiles += __shfl_sync(~0u, tsum, 31);
    before = min(before + __shfl_sync(~0u, sum, 31), most);
  }
  if (lane == 0) first[p.groups] = tiles;
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

struct Bars {
  uint32_t full, empty, acc_full, acc_empty, scale_full, scale_empty, drain;
};

// A CTA's loads. next(): the next tile, group -1 after the last.
template <int CTAS, int NT, class Next>
__device__ void produce(const ProductArgs& p, int rank, uint32_t ring, const Bars& bar, volatile int* gave_up, Next next) {
  using S = Shape<CTAS, NT>;
  const uint32_t pair_full = CTAS == 2 ? pair_addr(bar.full, 0) : bar.full;
  int stage = 0;
  uint32_t phase = 0;
  int64_t issued = 0;
  bool ok = true;
  for (Tile t = next(); ok && t.group >= 0; t = next()) {
    const int b_row = (p.by_depth ? 0 : t.group * p.cols) + t.n0 + (CTAS == 2 ? rank * kBM : 0);
    const int a_row = t.r0 + (CTAS == 2 ? rank * S::kShare : 0);
    for (int k = t.k_lo; k < t.k_hi; ++k) {
      if (!(ok = bar_wait(bar.empty + 8 * stage, phase ^ 1, gave_up))) break;
      if (CTAS == 1 || rank == 0) bar_expect(bar.full + 8 * stage, CTAS * S::kStageBytes + p.extra);
      ++issued;
      const uint32_t at = ring + stage * S::kStageBytes, on = pair_full + 8 * stage;
      map_load<CTAS>(at, &p.b, k * kBlock, b_row, on);
      map_load<CTAS>(at + S::kBBytes, &p.a, k * kBlock, a_row, on);
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
    while (!bar_try(bar.full + 8 * stage, phase) && global_ns() - start < kWaitNs) {
    }
  }
  const uint64_t drained = global_ns();
  while (global_ns() - drained < 10000000ull) {
  }
}

template <int CTAS, int NT, class Next>
__device__ void multiply(uint32_t ring, const Bars& bar, uint32_t tmem, volatile int* gave_up, Next next) {
  using S = Shape<CTAS, NT>;
  constexpr uint32_t desc = fp8_desc(S::kM, NT);
  int stage = 0;
  uint32_t phase = 0, n = 0;
  bool ok = true;
  for (Tile t = next(); ok && t.group >= 0; t = next()) {
    for (int k = t.k_lo; k < t.k_hi; ++k, ++n) {
      const uint32_t part = n % S::kAcc;
      if (!(ok = bar_wait(bar.acc_empty + 8 * part, ((n / S::kAcc) & 1) ^ 1, gave_up))) break;
      if (!(ok = bar_wait(bar.full + 8 * stage, phase, gave_up))) break;
      tc_fence_after();
      const uint32_t at = ring + stage * S::kStageBytes;
      const uint64_t db = operand_desc<64>(at, false), da = operand_desc<64>(at + S::kBBytes, false);
#pragma unroll
      for (int j = 0; j < kBlock / 32; ++j)
        fp8_product<CTAS>(tmem + part * NT, db + j * (32 >> 4), da + j * (32 >> 4), desc, j > 0);
      tc_commit<CTAS>(bar.empty + 8 * stage);
      tc_commit<CTAS>(bar.acc_full + 8 * part);
      if (++stage == S::kStages) {
        stage = 0;
        phase ^= 1;
      }
    }
  }
  // giving up: products still running write the tensor memory that is about to be freed
  if (!ok) {
    tc_commit<CTAS>(bar.drain);
    const uint64_t start = global_ns();
    while (!bar_try(bar.drain, 0) && global_ns() - start < kWaitNs) {
    }
  }
}

// The scales' products of every block, a row of the tile each, ahead of the sums that want them.
template <int CTAS, int NT, class Next>
__device__ void bring_scales(const ProductArgs& p, int rank, uint32_t ring, const Bars& bar, volatile int* gave_up, Next next) {
  constexpr int kEach = NT < 32 * kScaleWarps ? 1 : NT / (32 * kScaleWarps), kAhead = 4;
  const int me = threadIdx.x - 64;
  uint32_t n = 0;
  for (Tile t = next(); t.group >= 0; t = next()) {
    const int64_t row_blocks = (p.cols + kBlock - 1) / kBlock;
    const int block = t.n0 / kBlock + (CTAS == 2 ? rank : 0);
    const bool there = block < row_blocks;
    const float* bs = p.b_scale + ((p.by_depth ? 0 : t.group * row_blocks) + block) * p.depth_blocks;
    for (int k0 = t.k_lo; k0 < t.k_hi; k0 += kAhead) {
      float f[kAhead][kEach], g[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int k = k0 + i;
        g[i] = k < t.k_hi && there ? bs[k] : 0.0f;
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
          const int r = t.r0 + me + 32 * kScaleWarps * e;
          f[i][e] = k < t.k_hi && r < t.r_end ? p.a_scale[(int64_t)k * p.rows + r] : 0.0f;
        }
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (k0 + i >= t.k_hi) break;
        const uint32_t s = n % kScaleStages;
        if (!__all_sync(~0u, bar_wait(bar.scale_empty + 8 * s, ((n / kScaleStages) & 1) ^ 1, gave_up))) return;
#pragma unroll
        for (int e = 0; e < kEach; ++e)
          if (NT >= 32 * kScaleWarps || me < NT) sts1(ring + (s * NT + me + 32 * kScaleWarps * e) * 4, __fmul_rn(f[i][e], g[i]));
        __syncwarp();
        if (threadIdx.x % 32 == 0) bar_arrive(bar.scale_full + 8 * s);
        ++n;
      }
    }
  }
}

// A tile's sums: v[j] is row r0 + part * kMine + j of out, in the column of the thread's lane. n: blocks before.
template <int CTAS, int NT>
__device__ __forceinline__ bool finish(const Tile& t, uint32_t& n, uint32_t scales, const Bars& bar, uint32_t tmem, int quarter, int part,
                                       volatile int* gave_up, float (&v)[Shape<CTAS, NT>::kMine]) {
  using S = Shape<CTAS, NT>;
  constexpr int W = S::kMine < 32 ? S::kMine : 32;
  const uint32_t first_empty = CTAS == 2 ? pair_addr(bar.acc_empty, 0) : bar.acc_empty;
#pragma unroll
  for (int j = 0; j < S::kMine; ++j) v[j] = 0.0f;
  for (int k = t.k_lo; k < t.k_hi; ++k, ++n) {
    const uint32_t acc = n % S::kAcc, s = n % kScaleStages;
    if (!__all_sync(~0u, bar_wait(bar.scale_full + 8 * s, (n / kScaleStages) & 1, gave_up))) return false;
    if (!__all_sync(~0u, bar_wait(bar.acc_full + 8 * acc, (n / S::kAcc) & 1, gave_up))) return false;
    tc_fence_after();
    const uint32_t from = tmem + acc * NT + part * S::kMine + ((uint32_t)(quarter * 32) << 16);
    const uint32_t f = scales + (s * NT + part * S::kMine) * 4;
    float u[2][W];
    tmem_load<W>(from, u[0]);
#pragma unroll
    for (int c = 0; c < S::kMine; c += W) {
      float(&x)[W] = u[c / W % 2];
      tmem_wait<W>(x);
      if (c + W < S::kMine) tmem_load<W>(from + c + W, u[(c / W + 1) % 2]);
#pragma unroll
      for (int j = 0; j < W; j += 4) {
        const float4 g = lds4(f + (c + j) * 4);
        fma2(v[c + j], v[c + j + 1], x[j], x[j + 1], g.x, g.y);
        fma2(v[c + j + 2], v[c + j + 3], x[j + 2], x[j + 3], g.z, g.w);
      }
    }
    tc_fence_before();
    __syncwarp();
    if (threadIdx.x % 32 == 0) {
      bar_arrive(bar.scale_empty + 8 * s);
      if (CTAS == 2) bar_arrive_pair(first_empty + 8 * acc);
      else bar_arrive(first_empty + 8 * acc);
    }
  }
  return true;
}

template <int CTAS, int NT>
__global__ void __launch_bounds__(kProductThreads, 1) fp8_product_kernel(const __grid_constant__ ProductArgs p) {
  using S = Shape<CTAS, NT>;
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t s_bar[2 * S::kStages + 2 * S::kAcc + 2 * kScaleStages + 1];
  __shared__ uint32_t s_tmem;
  __shared__ int s_gave_up;
  const int warp = threadIdx.x / 32, rank = (int)pair_rank();
  dep_launch();
  const uint32_t ring = (smem_addr(smem_raw) + 1023) & ~1023u, scales = ring + S::kRing;
  int* s_first = reinterpret_cast<int*>(smem_raw + (scales - smem_addr(smem_raw)) + S::kScaleBytes);
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
  }
  if (warp == 1) tmem_alloc<CTAS>(smem_addr(&s_tmem), S::kTmem);
  dep_wait();
  const Groups groups{s_first, s_first + p.groups + 1, s_first + 2 * p.groups + 1, (p.cols + S::kM - 1) / S::kM};
  if (warp == 0) read_groups<CTAS, NT>(p, s_first, s_first + p.groups + 1, s_first + 2 * p.groups + 1, groups.nt);
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
    Tile t;
    t.group = -1;
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
    if (threadIdx.x == 0) produce<CTAS, NT>(p, rank, ring, bar, &s_gave_up, next);
    if (threadIdx.x == 32 && (CTAS == 1 || rank == 0)) multiply<CTAS, NT>(ring, bar, tmem, &s_gave_up, next);
    if (warp >= 2) bring_scales<CTAS, NT>(p, rank, scales, bar, &s_gave_up, next);
  } else {
    // warps 4 to 7 finish the accumulator's first half of columns, 8 to 11 the other; a warp reads the quarter of
    // tensor memory's lanes that its number gives it
    const int quarter = warp % 4, part = warp / 4 - 1, lane = threadIdx.x % 32;
    uint32_t n = 0;
    for (Tile t = next(); t.group >= 0; t = next()) {
      float v[S::kMine];
      if (!finish<CTAS, NT>(t, n, scales, bar, tmem, quarter, part, &s_gave_up, v)) break;
      if (CTAS == 1 && p.splits > 1) {
        // the products are done with the ring: it takes the partial sums
#pragma unroll
        for (int j = 0; j < S::kMine; ++j) sts1(ring + ((part * S::kMine + j) * kBM + quarter * 32 + lane) * 4, v[j]);
      } else {
        const int col = t.n0 + (CTAS == 2 ? rank * kBM : 0) + quarter * 32 + lane;
#pragma unroll
        for (int j = 0; j < S::kMine; ++j) {
          const int row = t.r0 + part * S::kMine + j;
          if (row < t.r_end && col < p.cols) store_out(p, t.group, row, col, v[j]);
        }
      }
    }
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
      for (int e = threadIdx.x; e < each * kBM; e += kProductThreads) {
        const int j = rank * each + e / kBM, row = t.r0 + j, col = t.n0 + e % kBM;
        float sum = 0.0f;
        for (int s = 0; s < p.splits; ++s) sum = __fadd_rn(sum, ld_cluster(pair_addr(ring + (j * kBM + e % kBM) * 4, s)));
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

// A matrix [rows][bytes], read in boxes of box_rows by 128 bytes (128-byte swizzle).
bool bytes_map(CUtensorMap* m, const void* p, int64_t rows, int64_t bytes, int64_t ld, int box_rows) {
  const EncodeFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)bytes, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)ld};
  const cuuint32_t box[2] = {(cuuint32_t)kBlock, (cuuint32_t)box_rows}, unit[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(p), dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The most tiles the rows can make, wherever the groups end.
int64_t most_tiles(const relay_fp8_matmul_t& w, int m, int nt) {
  const int64_t cols = (w.cols + m - 1) / m, groups = std::max(w.groups, 1);
  if (w.by_depth) return groups * ((w.rows + nt - 1) / nt) * cols;
  return (w.groups == 0 ? (w.rows + nt - 1) / nt : w.rows / nt + std::min<int64_t>(groups, w.rows)) * cols;
}

template <int CTAS, int NT>
cudaError_t launch(ProductArgs p, const relay_fp8_matmul_t& w, int splits, cudaStream_t s) {
  using S = Shape<CTAS, NT>;
  static thread_local int ready_device = -1;
  constexpr int kFixed = 1024 + S::kRing + S::kScaleBytes;
  constexpr int kMost = kFixed + (3 * RELAY_FP8_MAX_GROUPS + 1) * 4;
  static_assert(kMost <= 227 * 1024 - 1024, "shared memory of a CTA");
  static_assert(S::kRing >= NT * kBM * 4 || CTAS == 2, "the ring takes the partial sums");
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
  if (w.depth > 0 &&
      (!bytes_map(&p.a, w.a, a_rows, w.depth, w.a_stride, S::kShare) || !bytes_map(&p.b, w.b, b_rows, w.depth, w.b_stride, kBM)))
    return cudaErrorInvalidValue;
  const int64_t tiles = most_tiles(w, S::kM, NT);
  if (tiles * 8 > INT_MAX / 2) return cudaErrorInvalidConfiguration;
  p.splits = splits;
  const int blocks = CTAS == 2 ? (int)std::min<int64_t>(2 * tiles, sm_count() / 2 * 2) : (int)(tiles * splits);
  return launch_chained_clusters(kernel, CTAS == 2 ? 2 : splits, blocks, kProductThreads, kFixed + (3 * p.groups + 1) * 4, s, p);
}

cudaError_t run(const ProductArgs& p, const relay_fp8_matmul_t& w, cudaStream_t s) {
  const int64_t per_group = w.by_depth ? w.rows : w.rows / std::max(w.groups, 1);
  if (per_group > 128) return launch<2, 256>(p, w, 1, s);
  if (per_group > 32) return launch<1, 128>(p, w, 1, s);
  return launch<1, 32>(p, w, 4, s);
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
    p.extra = t_extra;
    const cudaError_t e = run(p, *w, stream);
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
