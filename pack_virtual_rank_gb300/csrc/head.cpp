// head.cpp -- relay_linear_xent and relay_linear_distill: validation, workspace layout and
// the order of launches.
//
//   rows      the entries of a row (distill), then the live rows packed to the front; the weight
//             packed too where its rows cannot be read through tensor maps, or are fp32
//   logits    tile maxima and sums, and the logits at the entries
//   combine   log-sum-exp and loss of each row
//   gradient  every piece: gradient of the logits; then, in one launch, d_hidden += its product with
//             the weight and d_weight of the piece's rows = its transposed product with hidden
//
// When all the logits of the batch make one piece, the first pass keeps their exponentials and
// the gradient is a scaling of them; otherwise each piece multiplies its logits again.
#include <limits.h>
#include <string.h>

#include <algorithm>
#include <cmath>
#include <string>
#include <vector>

#include "head.h"
#include "program.h"
#include "spans.h"

namespace relay {
namespace {

int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

bool wants_dw(const relay_head_t& h) {
  for (int a = 0; a < h.A; ++a)
    if (h.d_weight[a] != nullptr) return true;
  return false;
}

relay_status_t bad(const std::string& msg) {
  return report_error(RELAY_ERR_INVALID_ARGUMENT, "relay_head: " + msg);
}

// Sizes and strides only (what the workspace depends on).
relay_status_t check_shape(const relay_head_t* h, int top, HeadGeom* g) {
  if (h == nullptr) return bad("head is NULL");
  if (h->dtype != RELAY_F32 && h->dtype != RELAY_BF16) return bad("dtype must be RELAY_F32 or RELAY_BF16");
  if (h->A < 1 || h->A > RELAY_HEAD_MAX_SHARDS) return bad("A must be 1..8 shards");
  if (top < 0 || top > RELAY_HEAD_MAX_TOP) return bad("top must be 1..128");
  if (h->tokens < 0 || h->tokens > INT32_MAX - kHeadRowTile) return bad("tokens out of range");
  if (h->dim < 1 || h->dim > (1 << 24)) return bad("dim must be 1..2^24");
  if (h->piece_bytes < 0) return bad("piece_bytes is negative");
  memset(g, 0, sizeof *g);
  int64_t vocab = 0, tiles = 0;
  for (int a = 0; a < h->A; ++a) {
    if (h->rows[a] < 0 || h->rows[a] > INT32_MAX) return bad("rows[" + std::to_string(a) + "] out of range");
    g->rows[a] = (int32_t)h->rows[a];
    g->base[a] = (int32_t)std::min<int64_t>(vocab, INT32_MAX);
    g->tile0[a] = (int32_t)tiles;
    vocab += h->rows[a];
    tiles += (h->rows[a] + kHeadTile - 1) / kHeadTile;
    // padded columns are numbered in 32 bits
    if (vocab > INT32_MAX || tiles * kHeadTile > INT32_MAX) return bad("the vocabulary has more than 2^31 - 1 rows");
  }
  if (vocab < 1) return bad("the vocabulary is empty");
  for (int a = h->A; a <= RELAY_HEAD_MAX_SHARDS; ++a) g->tile0[a] = (int32_t)tiles;
  g->A = h->A;
  g->top = std::max(top, 1);
  g->tokens = (int32_t)h->tokens;
  g->dim = (int32_t)h->dim;
  g->vocab = (int32_t)vocab;
  g->mpad = (int32_t)up(h->tokens, kHeadRowTile);
  g->tau = g->inv_tau = 1.0f;
  g->ctas = g->tokens <= kHeadRowTile / 2 ? 1 : 2;  // one CTA's rows: the other would multiply padding
  return RELAY_OK;
}

// Bump allocation over the caller's workspace; base 0 only measures.
struct Layout {
  uintptr_t at;
  uintptr_t take(int64_t bytes) {
    const uintptr_t p = at;
    at += (uintptr_t)up(bytes, 256);
    return p;
  }
};

struct Arrangement {
  HeadWork w;
  int tiles_per_piece;
  bool keep;  // one piece: the first pass keeps its exponentials
  int64_t bytes;
};

Arrangement arrange(const relay_head_t& h, const HeadGeom& g, int top, uintptr_t base) {
  Arrangement ar{};
  const int planes = head_planes(h.dtype);
  const int tiles = g.tile0[RELAY_HEAD_MAX_SHARDS];
  const bool dh = h.d_hidden != nullptr, dw = wants_dw(h);
  // tensor maps want 16-byte aligned rows
  bool pack = h.dtype == RELAY_F32;
  for (int a = 0; a < h.A; ++a)
    pack |= h.rows[a] > 0 && (reinterpret_cast<uintptr_t>(h.weight[a]) % 16 || h.weight_stride % 8);
  Layout l{base};
  HeadWork& w = ar.w;
  w.dim_pad = (int32_t)up(g.dim, 64);  // rows of whole 128-byte lines: a box row is one line, not two
  w.splits = 1;
  w.n_live = reinterpret_cast<int32_t*>(l.take(8));
  w.perm = reinterpret_cast<int32_t*>(l.take(4ll * g.mpad));
  w.wrow = reinterpret_cast<float*>(l.take(4ll * g.mpad));
  w.hid = reinterpret_cast<uint16_t*>(l.take(2ll * planes * g.mpad * w.dim_pad));
  if (pack) w.wpack = reinterpret_cast<uint16_t*>(l.take(2ll * planes * tiles * kHeadTile * w.dim_pad));
  if (top > 0) w.live = reinterpret_cast<uint8_t*>(l.take(g.tokens));
  const int64_t ents = (int64_t)g.tokens * g.top;
  w.ent_col = reinterpret_cast<int32_t*>(l.take(4 * ents));
  w.ent_q = reinterpret_cast<float*>(l.take(4 * ents));
  w.ent_z = reinterpret_cast<float*>(l.take(4 * ents));
  w.part = reinterpret_cast<float2*>(l.take(8ll * tiles * (kHeadTile / kHeadStatTile) * g.mpad));
  w.lse = reinterpret_cast<float2*>(l.take(8ll * g.mpad));
  ar.tiles_per_piece = tiles;
  if ((dh || dw) && g.mpad > 0) {
    const int64_t cap = h.piece_bytes > 0 ? h.piece_bytes : RELAY_HEAD_PIECE_BYTES;
    w.grad_planes = head_grad_planes(h.dtype, g.ctas);
    const int64_t per_tile = 2ll * w.grad_planes * g.mpad * kHeadTile;
    ar.tiles_per_piece = (int)std::min<int64_t>(tiles, std::max<int64_t>(1, cap / per_tile));
    ar.keep = ar.tiles_per_piece == tiles && head_scale_fits(g);
    w.grad_ld = (int64_t)ar.tiles_per_piece * kHeadTile;
    w.grad = reinterpret_cast<uint16_t*>(l.take(per_tile * ar.tiles_per_piece));
    if (dh) {
      // room for the cuts of a batch that keeps few rows, up to 256 MiB of partial sums
      w.dh_ld = (int32_t)up(g.dim, 4);
      const int64_t one = 4ll * g.mpad * w.dh_ld;
      w.tiles_per_piece = ar.tiles_per_piece;
      w.with_dw = dw;
      w.whole = ar.keep && reinterpret_cast<uintptr_t>(h.d_hidden) % 16 == 0 &&
                h.d_hidden_stride * esize_of(h.dtype) % 16 == 0;
      w.splits = (int)std::max<int64_t>(1, std::min<int64_t>(std::min(ar.tiles_per_piece, 64), (256ll << 20) / one));
      w.dh = reinterpret_cast<float*>(l.take(one * w.splits));
    }
  }
  ar.bytes = (int64_t)(l.at - base);
  return ar;
}

struct Named {
  Span span;
  std::string what;
};

relay_status_t check_buffers(const relay_head_t& h, const HeadGeom& g, int top, const void* entries,
                             const void* teacher, int teacher_esize, const float* row_weight,
                             const float* loss, const void* workspace, int64_t workspace_bytes,
                             int64_t need) {
  const int64_t E = esize_of(h.dtype);
  std::vector<Named> in, out;
  auto matrix = [&](std::vector<Named>& v, const void* p, int64_t rows, int64_t ld, const std::string& what) {
    v.push_back(Named{matrix_span(p, rows, g.dim * E, ld * E), what});
  };
  auto put = [&](std::vector<Named>& v, const void* p, int64_t bytes, const std::string& what) {
    v.push_back(Named{array_span(p, bytes), what});
  };
  auto aligned = [](const void* p, int64_t e) { return reinterpret_cast<uintptr_t>(p) % e == 0; };
  const bool dw = wants_dw(h);
  if (h.hidden_stride < g.dim || h.weight_stride < g.dim) return bad("a row stride is less than dim");
  if (h.d_hidden != nullptr && h.d_hidden_stride < g.dim) return bad("d_hidden_stride is less than dim");
  if (dw && h.d_weight_stride < g.dim) return bad("d_weight_stride is less than dim");
  const int64_t ld = std::max(std::max(h.hidden_stride, h.weight_stride),
                              std::max(h.d_hidden ? h.d_hidden_stride : 0, dw ? h.d_weight_stride : 0));
  if (ld > (1ll << 31)) return bad("a row stride is more than 2^31 elements");
  if (g.tokens > 0) {
    if (h.hidden == nullptr) return bad("hidden is NULL");
    if (entries == nullptr) return bad(top > 0 ? "teacher_index is NULL" : "targets is NULL");
    if (top > 0 && teacher == nullptr) return bad("teacher_logits is NULL");
    if (loss == nullptr) return bad("loss is NULL");
  }
  if (!aligned(h.hidden, E) || !aligned(h.d_hidden, E)) return bad("hidden or d_hidden is not element-aligned");
  if (!aligned(entries, 4) || !aligned(loss, 4) || !aligned(row_weight, 4) ||
      (teacher_esize > 0 && !aligned(teacher, teacher_esize)))
    return bad("a per-row array is not element-aligned");
  for (int a = 0; a < h.A; ++a) {
    const std::string n = "[" + std::to_string(a) + "]";
    if (h.rows[a] == 0) continue;
    if (h.weight[a] == nullptr) return bad("weight" + n + " is NULL");
    if (dw && h.d_weight[a] == nullptr) return bad("d_weight" + n + " is NULL, other shards' are not");
    if (!aligned(h.weight[a], E) || !aligned(h.d_weight[a], E)) return bad("weight or d_weight" + n + " is not element-aligned");
    matrix(in, h.weight[a], h.rows[a], h.weight_stride, "weight" + n);
    if (dw) matrix(out, h.d_weight[a], h.rows[a], h.d_weight_stride, "d_weight" + n);
  }
  if (need > 0 && workspace == nullptr) return bad("workspace is NULL");
  if (workspace_bytes < need)
    return bad("the workspace holds " + std::to_string(workspace_bytes) + " bytes, " + std::to_string(need) + " are needed");
  matrix(in, h.hidden, g.tokens, h.hidden_stride, "hidden");
  matrix(out, h.d_hidden, g.tokens, h.d_hidden_stride, "d_hidden");
  const int64_t ents = (int64_t)g.tokens * g.top;
  put(in, entries, 4 * ents, top > 0 ? "teacher_index" : "targets");
  put(in, teacher, teacher_esize * ents, "teacher_logits");
  put(in, row_weight, 4ll * g.tokens, "row_weight");
  put(out, loss, 4ll * g.tokens, "loss");
  put(out, workspace, workspace_bytes, "workspace");
  for (size_t i = 0; i < out.size(); ++i) {
    for (size_t j = i + 1; j < out.size(); ++j)
      if (overlap(out[i].span, out[j].span)) return bad(out[i].what + " overlaps " + out[j].what);
    for (const Named& s : in)
      if (overlap(out[i].span, s.span)) return bad(out[i].what + " overlaps " + s.what);
  }
  return RELAY_OK;
}

#define RELAY_HEAD_TRY(call)                                                             \
  do {                                                                                   \
    const cudaError_t e_ = (call);                                                       \
    if (e_ != cudaSuccess)                                                               \
      return report_error(RELAY_ERR_CUDA, std::string("relay_head: ") + cudaGetErrorString(e_)); \
  } while (0)

relay_status_t run_head(const relay_head_t& h, HeadGeom g, int top, const int32_t* entries,
                        const void* teacher, int teacher_dtype, const float* row_weight, float* loss,
                        void* workspace, cudaStream_t stream) {
  g.sms = sm_count();
  const uintptr_t base = (uintptr_t)up((int64_t)reinterpret_cast<uintptr_t>(workspace), 256);
  const Arrangement ar = arrange(h, g, top, base);
  const HeadWork& w = ar.w;
  const bool distill = top > 0, dh = h.d_hidden != nullptr, dw = wants_dw(h);
  const int tiles = g.tile0[RELAY_HEAD_MAX_SHARDS];
  // rows of every plane are numbered in 32 bits
  const int64_t planes = std::max(head_planes(h.dtype), w.grad_planes);
  if (planes * g.mpad > INT32_MAX || (w.wpack != nullptr && planes * tiles * kHeadTile > INT32_MAX))
    return report_error(RELAY_ERR_UNSUPPORTED, "relay_head: more than 2^31 - 1 rows over all parts of an fp32 value");
  HeadShards sh{};
  for (int a = 0; a < h.A; ++a) {
    sh.w[a] = h.weight[a];
    sh.dw[a] = h.d_weight[a];
  }
  sh.w_ld = h.weight_stride;
  sh.dw_ld = h.d_weight_stride;
  sh.dh = h.d_hidden;
  sh.dh_ld = h.d_hidden_stride;
  if (g.tokens == 0) {
    if (dw)
      for (int a = 0; a < h.A; ++a)
        if (h.rows[a] > 0)
          RELAY_HEAD_TRY(cudaMemset2DAsync(sh.dw[a], sh.dw_ld * esize_of(h.dtype), 0,
                                           (size_t)g.dim * esize_of(h.dtype), (size_t)h.rows[a], stream));
    return RELAY_OK;
  }
  if (distill) RELAY_HEAD_TRY(head_teacher(g, w, teacher, teacher_dtype, entries, stream));
  RELAY_HEAD_TRY(head_pack(g, w, h.dtype, h.hidden, h.hidden_stride, entries, teacher, teacher_dtype, row_weight, loss,
                           h.d_hidden, h.d_hidden_stride, stream));
  if (w.wpack != nullptr) RELAY_HEAD_TRY(head_pack_weight(g, w, sh, h.dtype, stream));
  RELAY_HEAD_TRY(head_logits(g, w, sh, h.dtype, 0, tiles, ar.keep ? kHeadStatsKeep : kHeadStats, stream));
  if (!ar.keep || !head_scale_joins(g)) RELAY_HEAD_TRY(head_combine(g, w, distill, loss, stream));
  if (!dh && !dw) return RELAY_OK;
  for (int t = 0; t < tiles; t += ar.tiles_per_piece) {
    const int hi = std::min(tiles, t + ar.tiles_per_piece);
    if (ar.keep)
      RELAY_HEAD_TRY(head_scale(g, w, h.dtype, distill, loss, stream));
    else
      RELAY_HEAD_TRY(head_logits(g, w, sh, h.dtype, t, hi, kHeadGradient, stream));
    RELAY_HEAD_TRY(head_back(g, w, sh, h.dtype, t, hi, t == 0, dh, dw, stream));
  }
  if (dh) RELAY_HEAD_TRY(head_write_dh(g, w, h.dtype, h.d_hidden, h.d_hidden_stride, stream));
  return RELAY_OK;
}

}  // namespace
}  // namespace relay

extern "C" {

int64_t relay_head_workspace_size(const relay_head_t* head, int top) {
  using namespace relay;
  int64_t bytes = -1;
  guarded([&]() -> relay_status_t {
    HeadGeom g;
    const relay_status_t st = check_shape(head, top, &g);
    if (st == RELAY_OK) bytes = arrange(*head, g, top, 0).bytes + 256;
    return st;
  });
  return bytes;
}

relay_status_t relay_linear_xent(const relay_head_t* head, const int32_t* targets,
                                 const float* row_weight, float* loss, void* workspace,
                                 int64_t workspace_bytes, cudaStream_t stream) {
  using namespace relay;
  return guarded([&]() -> relay_status_t {
    HeadGeom g;
    relay_status_t st = check_shape(head, 0, &g);
    if (st != RELAY_OK) return st;
    st = check_buffers(*head, g, 0, targets, nullptr, 0, row_weight, loss, workspace, workspace_bytes,
                       arrange(*head, g, 0, 0).bytes + 256);
    if (st != RELAY_OK) return st;
    return run_head(*head, g, 0, targets, nullptr, 0, row_weight, loss, workspace, stream);
  });
}

relay_status_t relay_test_head_wait(const relay_head_t* head, const int32_t* targets, float* loss, void* workspace,
                                    int64_t workspace_bytes, int extra_bytes, cudaStream_t stream) {
  using namespace relay;
  return guarded([&]() -> relay_status_t {
    if (extra_bytes < 0 || extra_bytes > 65536) return bad("0 <= extra_bytes <= 65536");
    head_test_extra(extra_bytes);
    const relay_status_t st = relay_linear_xent(head, targets, nullptr, loss, workspace, workspace_bytes, stream);
    head_test_extra(0);
    return st;
  });
}

relay_status_t relay_linear_distill(const relay_head_t* head, const void* teacher_logits,
                                    relay_dtype_t teacher_dtype, const int32_t* teacher_index,
                                    int top, float temperature, const float* row_weight,
                                    float* loss, void* workspace, int64_t workspace_bytes,
                                    cudaStream_t stream) {
  using namespace relay;
  return guarded([&]() -> relay_status_t {
    HeadGeom g;
    if (top < 1) return bad("top must be 1..128");
    relay_status_t st = check_shape(head, top, &g);
    if (st != RELAY_OK) return st;
    if (teacher_dtype != RELAY_F32 && teacher_dtype != RELAY_BF16)
      return bad("teacher_dtype must be RELAY_F32 or RELAY_BF16");
    // its reciprocal is used times log2 e
    if (!(temperature > 0.0f) || !std::isfinite(temperature) || !std::isfinite(1.4426951f / temperature))
      return bad("temperature must be finite and positive");
    g.tau = temperature;
    g.inv_tau = 1.0f / temperature;
    st = check_buffers(*head, g, top, teacher_index, teacher_logits, esize_of(teacher_dtype), row_weight,
                       loss, workspace, workspace_bytes, arrange(*head, g, top, 0).bytes + 256);
    if (st != RELAY_OK) return st;
    return run_head(*head, g, top, teacher_index, teacher_logits, teacher_dtype, row_weight, loss,
                    workspace, stream);
  });
}

}  // extern "C"
