/*
 * relay.h -- C ABI of the GB300 sharded relay collectives.
 *
 * A relay collective runs among A "active" ranks (0..A-1) of an R-rank node and
 * recruits the H = R - A idle ranks (A..R-1, helper h = rank A+h) as relay helpers.
 * Here every virtual rank is a set of buffers in ONE GPU's HBM: a transfer over a
 * (src, dst) "link" is a store from a kernel executed for rank src into memory owned
 * by rank dst, and each serialized group of the schedule is one batched kernel launch
 * on the caller's stream.
 *
 * Sources (page "Link-balance the sharded relay schedules (up to 3.2x vs NCCL)",
 * torchrec pull request #4570, and the commits of its stack, cited by their
 * Differential Revision number):
 *   cost model       -- the paragraph before summary item 1
 *   items 1..7       -- the numbered items of that page's summary
 *   D115998367       -- zero-chunk per-group direct fallback
 *   D115998376       -- reduce-scatter semantics, in-place convention, SUM/AVG only
 *   D115998385       -- all-gather semantics and in-place convention
 *   D115998370       -- all-to-all semantics (out-of-place only), helper sizing
 *   D115998382       -- actives are consecutive local ranks; A in {2, 4}; R > A
 *   D115998394, D115998388 -- helper-buffer size contract and its literals
 *
 * Ownership: the caller allocates and owns every buffer and the stream. The library
 * allocates no device memory and keeps no state between calls. Calls are asynchronous
 * on `stream`; a status reports only validation and launch errors.
 *
 * Element counts are in ELEMENTS of the payload type; byte figures say so.
 */
#ifndef RELAY_H
#define RELAY_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define RELAY_ABI_VERSION 1
#define RELAY_MAX_RANKS 64
#define RELAY_ALIGN_ELEMS 128 /* chunks are aligned down to 128 elements (D115998394) */

typedef enum {
  RELAY_OK = 0,
  RELAY_ERR_INVALID_ARGUMENT = 1, /* bad A/R/dtype/scale/pointer/alias/size */
  RELAY_ERR_UNSUPPORTED = 2,      /* valid request this library does not execute */
  RELAY_ERR_CUDA = 3              /* a CUDA launch or event call failed */
} relay_status_t;

typedef enum { RELAY_F32 = 0, RELAY_BF16 = 1, RELAY_I32 = 2 } relay_dtype_t;

typedef enum {
  RELAY_ALLREDUCE = 0,
  RELAY_REDUCE_SCATTER = 1,
  RELAY_ALL_GATHER = 2,
  RELAY_ALL_TO_ALL = 3
} relay_coll_t;

/* Schedule the planner picked. */
typedef enum {
  RELAY_KIND_RELAY = 0,      /* helpers carry the relay chunks (items 1, 2, 4, 5, 6) */
  RELAY_KIND_ZERO_CHUNK = 1, /* A=2 chunk aligned down to 0: direct halves (D115998367) */
  RELAY_KIND_DIRECT = 2,     /* pure-direct below the crossover (items 3, 4, 7) */
  RELAY_KIND_LEGACY = 3      /* A=2 numChunks = H+1, three groups (item 1, "before") */
} relay_kind_t;

/* Schedule request. */
typedef enum {
  RELAY_SCHEDULE_AUTO = 0,   /* relay iff the per-active-rank input passes the crossover */
  RELAY_SCHEDULE_RELAY = 1,  /* relay whenever the geometry allows it */
  RELAY_SCHEDULE_DIRECT = 2, /* pure-direct */
  RELAY_SCHEDULE_LEGACY = 3  /* A=2 only: the three-group numChunks = H+1 schedule */
} relay_schedule_t;

/* relay_opts_t.flags */
#define RELAY_FLAG_CHECK_HAZARDS 1 /* host checks before launching: every segment lies
                                      inside a declared buffer, and no launch writes what
                                      another segment of it reads or writes (O(segs^2)) */
#define RELAY_FLAG_DRY_RUN 2       /* validate, plan, build and check; launch nothing */
#define RELAY_FLAG_SEPARATE_PASSES 4 /* one launch per pass even for small calls */
#define RELAY_FLAG_FUSED_PASSES 8  /* one cooperative launch for the whole call whenever it
                                      qualifies, whatever its size */
#define RELAY_FLAG_CHAINED 32      /* one chained launch for the whole call whenever its
                                      program allows it (the default does the same; the flag
                                      documents the intent) */
#define RELAY_FLAG_KEEP_SCRATCH 64 /* chained launch: write every scratch line back to
                                      memory. By default a CTA drops from L2, without a
                                      write-back, the whole 128-byte lines of device-memory
                                      scratch that an earlier pass of its chain wrote and that
                                      nothing reads again in the call */
/* Launch policy. A call that records pass events, or sets RELAY_FLAG_SEPARATE_PASSES,
 * launches each pass separately. Any other call runs as ONE chained launch where its
 * program allows: the segments of all passes are cut into pieces so that each dependency
 * between passes links identical element ranges; pieces that touch the same bytes, one of
 * them writing, form a group; one CTA runs tile t of every piece of a group in pass order
 * with a block barrier between passes. No CTA waits for another, and a consumer reads
 * from L2 what its own CTA just wrote. It takes programs whose pieces number at most 384
 * after cutting (fp32 partials of a bf16 payload included). Else a call of at most
 * RELAY_FUSED_MAX_BYTES runs as one cooperative launch (at most 4 passes
 * and 384 segments after alignment splitting, no mixed-width segments; passes separated
 * by grid-wide barriers), and anything else pass by pass.
 * relay_last_launch() names the form the calling thread's last call took. */
#define RELAY_FUSED_MAX_BYTES (256ll << 20)
#define RELAY_FLAG_PAYLOAD_PARTIAL 16 /* 4-active reduce-scatter, bf16 payload. By default
                                      (flag clear) each helper's partial crosses to its owner
                                      in fp32: twice the bytes of that hop and H*chunk + 128
                                      more elements of owner scratch; the owner adds its own
                                      value and the partial, scales once and rounds once, so
                                      results are within one bf16 ulp of the fp32-accumulated
                                      sum (and of the exact sum unless a tiny term needs more
                                      than 24 bits next to large ones). With the flag set the
                                      partial crosses in the payload type, one payload-sized
                                      chunk per return hop as in the link model (item 6): it
                                      is rounded to bf16 at the helper before the owner adds,
                                      a second rounding that can move a result several ulps
                                      off the exact sum on cancelling inputs. fp32 and int32
                                      payloads are unaffected. */

typedef struct relay_opts {
  int32_t offload_permille;      /* A=4 allreduce / reduce-scatter / all-gather offload share;
                                    <0: 500 (item 4) */
  int32_t schedule;              /* relay_schedule_t */
  int64_t relay_threshold_bytes; /* <0: per-collective default crossover (items 3, 4, 7) */
  void* pass_events;             /* NULL, or cudaEvent_t[n_pass_events]: event i is recorded on
                                    the stream before pass i and event n_passes after the last;
                                    needs n_pass_events >= n_passes + 1 */
  int32_t n_pass_events;
  int32_t flags;                 /* RELAY_FLAG_* */
} relay_opts_t;

/* Fill `opts` with the defaults (every field "use the default"). */
void relay_opts_init(relay_opts_t* opts);

/*
 * Schedule geometry (plan). Integer only; identical on every machine.
 *
 * count is the per-group count the collective is called with:
 *   allreduce: elements per rank (input = output = count);
 *   reduce-scatter: recvCount (input = A*count, output = count) (D115998376);
 *   all-gather: sendCount (input = count, output = A*count) (D115998385);
 *   all-to-all: segmentCount (input = output = A*count) (D115998370).
 *
 * A = 2 (item 1): numChunks = H+2, chunk = align_down(count / numChunks, 128); relay
 *   chunk h (offset h*chunk) goes to helper h; the direct region follows the relay
 *   region: dirA = [H*chunk, (H+1)*chunk) rides group 1, dirB = the rest rides group 2.
 *   chunk == 0 -> zero-chunk fallback: dirA = count/2 at offset 0, dirB = the rest.
 *   Legacy (item 1, before): numChunks = H+1, three groups, direct = count - H*chunk.
 *   Below the crossover: one full direct exchange (item 3).
 * A = 4: chunk ("oc") is the offload slice each helper carries; direct_total = pD =
 *   count - H*oc. allreduce, reduce-scatter and all-gather take
 *   oc = align_down(permille*count/(1000*H)) (item 4; 500 permille = equal direct and
 *   offload regions). allreduce: owner slice = align_down(pD/A), the last owner takes
 *   the remainder. reduce-scatter (item 6): direct part split direct_g1 =
 *   align_down((A-1)*pD/A) in group 1 and the rest in group 2. all-gather (item 5):
 *   direct split 1:(A-1), direct_g1 = align_down(pD/A). all-to-all (item 7, coalesced
 *   helper offload): oc = align_down(count/(2(A-1)+H)); group 1 carries (A-1)*oc of
 *   direct, group 2 the rest. Pure-direct (oc = 0): allreduce keeps two groups (direct
 *   reduce-scatter + all-gather); the others take one.
 */
typedef struct relay_plan {
  int32_t coll, dtype, A, R, H, esize;
  int32_t kind;            /* relay_kind_t */
  int32_t num_groups;      /* serialized groups of the schedule (cost model) */
  int32_t offload_permille;
  int32_t wide_partial;    /* 1: 4-active reduce-scatter partials cross in fp32 (bf16
                              payload without RELAY_FLAG_PAYLOAD_PARTIAL) */
  int64_t count;
  int64_t chunk;           /* A=2: relay chunk; A=4: offload slice per helper */
  int64_t relay_total;     /* H * chunk */
  int64_t dirA_offset, dirA_size, dirB_size; /* A=2 direct regions */
  int64_t direct_total;    /* A=4: pD */
  int64_t direct_g1, direct_g2;              /* A=4 RS/AG/A2A direct split */
  int64_t owner_slice, owner_slice_last;     /* A=4 allreduce owner slices */
  int64_t helper_elems;    /* scratch each helper needs (elements) */
  int64_t active_scratch_elems; /* scratch each active needs (elements) */
  int64_t input_elems, output_elems; /* per active rank */
} relay_plan_t;

/* Plan a collective. opts may be NULL. INVALID_ARGUMENT on A not in {2,4}, R <= A,
 * R > RELAY_MAX_RANKS, bad dtype/coll, permille outside [0,1000], byte-size overflow,
 * or LEGACY at A=4 / LEGACY whose chunk aligns down to 0. */
relay_status_t relay_plan(relay_coll_t coll, size_t count, relay_dtype_t dtype, int A, int R,
                          const relay_opts_t* opts, relay_plan_t* out);

/* Link-byte accountant (cost model): out[(g*R + src)*R + dst] = payload BYTES the
 * executed schedule moves from rank src to rank dst in serialized group g, counted
 * from the very segments the kernels execute. cap is the length of `out` in entries
 * and must be >= num_groups*R*R. Returns INVALID_ARGUMENT if it is not. */
relay_status_t relay_plan_link_bytes(const relay_plan_t* plan, uint64_t* out, size_t cap);

/* Cost model: sum over groups of the largest (src, dst) entry, in BYTES. */
uint64_t relay_plan_cost_bytes(const relay_plan_t* plan);

/* Pass descriptions: one entry per kernel pass the executed schedule launches, in
 * launch order. Returns the number of passes (even when cap is smaller), or -1 on a
 * bad plan. in_place selects the in-place variant where it changes the passes. */
typedef enum {
  RELAY_PASS_G1 = 0,            /* group 1: transfers (scatter to helpers + direct) */
  RELAY_PASS_G2 = 1,            /* group 2: helper reduce/forward + direct transfers */
  RELAY_PASS_G3 = 2,            /* legacy group 3: direct exchange */
  RELAY_PASS_ACTIVE_REDUCE = 3, /* actives' own + received, scale, cast */
  RELAY_PASS_PACK = 4,          /* all-to-all: gather strided by segmentCount */
  RELAY_PASS_HELPER_FORWARD = 5,/* all-to-all: helper per-destination coalesced forward */
  RELAY_PASS_UNPACK = 6         /* all-to-all: scatter strided by segmentCount */
} relay_pass_kind_t;

typedef struct relay_pass_info {
  int32_t kind;     /* relay_pass_kind_t */
  int32_t num_segments;
  int64_t bytes_read, bytes_written; /* algorithmic bytes of the pass */
} relay_pass_info_t;

int relay_plan_passes(const relay_plan_t* plan, int in_place, relay_pass_info_t* out, int cap);
const char* relay_pass_name(int kind);

/* Scratch sizes of a plan, in elements (the plan's helper_elems / active_scratch_elems):
 * what each helper and each active must be given for this schedule. */
int64_t relay_helper_size(const relay_plan_t* plan);
int64_t relay_active_scratch_size(const relay_plan_t* plan);

/* The page's helper-buffer contract for one group (what its distributed layer
 * allocates per helper), in elements: the passthrough size with num_chunks = (R-A)+1 at
 * A=2 (D115998370); 2*count for the 4-active allreduce (D115998382) and reduce-scatter
 * (item 6); A*count for the 4-active all-gather (D115998397); 1 for the 4-active
 * all-to-all, which the page runs pure-direct (D115998358). -1 on bad arguments. This
 * library's schedules never need more than the contract, except the coalesced 4-active
 * all-to-all, which the page does not have. */
int64_t relay_helper_contract_size(relay_coll_t coll, int64_t count, int A, int R);

/* Helper-buffer size contract of the page's distributed layer (D115998394, D115998388,
 * D115998370): min(count_g, A * align_down(count_g / num_chunks, 128)); count_g when the
 * aligned chunk is 0 (the page only says the fallback can over-allocate). */
int64_t relay_passthrough_helper_size(int64_t count_g, int A, int num_chunks);

/*
 * The collectives. Pointer arrays hold R entries, entry r for virtual rank r:
 *   send[a], recv[a] (a < A): the actives' input and output buffers;
 *   scratch[a] (a < A):       >= plan.active_scratch_elems elements (may be NULL if 0);
 *   scratch[A+h]:             helper h, >= plan.helper_elems elements (NULL if 0).
 *   send/recv entries of helpers are ignored (may be NULL).
 * All device pointers; element-aligned; any further alignment is optional (16-byte
 * aligned buffers take the vectorized path).
 * Scratch is workspace: every scratch byte a call reads it wrote earlier in the same call,
 * and its contents after the call are unspecified (see RELAY_FLAG_KEEP_SCRATCH).
 * Aliasing: every buffer must be disjoint from every other except the in-place forms:
 *   allreduce      recv[a] == send[a]                          (D115998369)
 *   reduce-scatter recv[a] == send[a] + a*count elements       (D115998376)
 *   all-gather     send[a] == recv[a] + a*count elements       (D115998385)
 *   all-to-all     out-of-place only                           (D115998370)
 * scale multiplies the fp32 sum once before the cast: 1 for SUM, 1/A for AVG
 * (D115998376); int32 accepts only scale == 1 (integer AVG is undefined).
 * Arithmetic: fp32 and bf16 sum in fp32 in ascending source rank, multiply by scale
 * once, round to nearest-even into the payload type; int32 sums wrap modulo 2^32. The
 * one partial sum that crosses a link, the 4-active relay reduce-scatter's helper partial
 * (item 6), is summed over the A-1 non-owner sources in ascending rank; the owner then
 * adds its own value first and the partial second. For a bf16 payload the partial
 * crosses in fp32 unless RELAY_FLAG_PAYLOAD_PARTIAL asks for the payload type (see that
 * flag for the rounding each choice gives).
 * count == 0 returns RELAY_OK without a launch.
 */
relay_status_t relay_allreduce(void* const* send, void* const* recv, void* const* scratch,
                               size_t count, relay_dtype_t dtype, int A, int R, float scale,
                               const relay_opts_t* opts, cudaStream_t stream);
relay_status_t relay_reduce_scatter(void* const* send, void* const* recv, void* const* scratch,
                                    size_t recv_count, relay_dtype_t dtype, int A, int R,
                                    float scale, const relay_opts_t* opts, cudaStream_t stream);
relay_status_t relay_all_gather(void* const* send, void* const* recv, void* const* scratch,
                                size_t send_count, relay_dtype_t dtype, int A, int R,
                                const relay_opts_t* opts, cudaStream_t stream);
relay_status_t relay_all_to_all(void* const* send, void* const* recv, void* const* scratch,
                                size_t segment_count, relay_dtype_t dtype, int A, int R,
                                const relay_opts_t* opts, cudaStream_t stream);

/*
 * Fused multi-group call (D115998367, D115998376, D115998378): the R = num_groups*A
 * ranks form num_groups sparse groups of A consecutive ranks (group g = ranks g*A ..
 * g*A+A-1, D115998382). Every rank is active in its own group and a relay helper in
 * every other group; each group plans its own schedule from counts[g] (a group whose
 * chunk aligns down to zero takes the direct fallback while the others relay). The
 * groups run phase-synchronized: one launch carries every group's group-1 transfers,
 * the next every group's group-2 transfers, and so on, then every group's closing
 * reductions.
 *   send[r], recv[r]   (r < R): rank r's input and output for its own group;
 *   scratch[g*R + r]   rank r's scratch for group g: its active scratch when r is in
 *                      group g (plan.active_scratch_elems), its helper scratch otherwise
 *                      (plan.helper_elems); NULL where the size is 0.
 * Sizes, dtypes, in-place forms and scale are as for the single-group calls; scale is
 * ignored for all-gather and all-to-all. Every buffer must be disjoint from every other
 * except the in-place forms.
 */
relay_status_t relay_multi_group(relay_coll_t coll, int num_groups, const size_t* counts,
                                 void* const* send, void* const* recv, void* const* scratch,
                                 relay_dtype_t dtype, int A, float scale,
                                 const relay_opts_t* opts, cudaStream_t stream);

/* Link-byte accountant of a fused call: out[(p*R + src)*R + dst] = payload BYTES moved
 * from rank src to rank dst in phase p (the groups' serialized group p, summed over
 * groups). *num_phases receives the number of phases; cap >= num_phases*R*R. */
relay_status_t relay_multi_group_link_bytes(relay_coll_t coll, int num_groups,
                                            const size_t* counts, relay_dtype_t dtype, int A,
                                            const relay_opts_t* opts, uint64_t* out, size_t cap,
                                            int* num_phases);

/*
 * Flat packing of a caller's tensor list (D115998366: the distributed layer packs the
 * tensors into the active flat buffer and unpacks the result, one launch each).
 * relay_pack_flat copies tensors srcs[0..n-1] (counts[i] elements each) end to end
 * into `flat`; relay_unpack_flat copies them back out into dsts. One launch for up to
 * 384 non-empty tensors. `flat` must hold sum(counts) elements and overlap no tensor.
 */
relay_status_t relay_pack_flat(const void* const* srcs, const size_t* counts, int n, void* flat,
                               relay_dtype_t dtype, cudaStream_t stream);
relay_status_t relay_unpack_flat(const void* flat, void* const* dsts, const size_t* counts, int n,
                                 relay_dtype_t dtype, cudaStream_t stream);

/*
 * relay_copy -- copies `count` elements of `dtype` from `src` to `dst` with the library's
 * streaming kernel, asynchronously on `stream`. It is how callers stage a collective's
 * inputs into HBM and its results back out when those live in host memory. The page has
 * no counterpart: its buffers always sit in device memory.
 *   - Either pointer may be device memory, pinned or registered host memory, or (only
 *     where the device reports cudaDevAttrPageableMemoryAccess) ordinary pageable host
 *     memory. The SMs load and store across the host link themselves. On GB300 this
 *     reaches the link's rate whether or not the copy engines do.
 *   - max_ctas caps the CTAs of the launch. Each CTA then walks 16 KiB tiles. 0 means
 *     one CTA per tile, the fastest form for device-to-device copies. A copy over the host
 *     link reaches the link's rate with about one CTA per SM, which leaves the other CTA
 *     slots to kernels running at the same time on other streams.
 *   - Pointers must be element-aligned, and the two ranges must not overlap.
 *   - count == 0 returns RELAY_OK without a launch.
 *   - Errors: RELAY_ERR_INVALID_ARGUMENT (NULL, misaligned, overlapping, max_ctas < 0);
 *     RELAY_ERR_UNSUPPORTED (pageable host memory on a device that cannot address it);
 *     RELAY_ERR_CUDA (pointer query or launch failure).
 */
relay_status_t relay_copy(void* dst, const void* src, size_t count, relay_dtype_t dtype,
                          int max_ctas, cudaStream_t stream);

/*
 * relay_allreduce_noalloc -- an allreduce for callers that cannot allocate device
 * memory when they call it (an allocator or memory-pool hook that would recurse into
 * itself, a process that reserved all of HBM at start-up, a path that cannot take the
 * synchronisation an allocation may cause). The page has no counterpart to this entry
 * point.
 *
 * Arguments and results are those of relay_allreduce, without `scratch`: the helpers'
 * relay slots and the actives' receive staging come from one file-scope device array of
 * RELAY_NOALLOC_SCRATCH_BYTES that every GPU loading this library holds until exit.
 * The call allocates nothing (no cudaMalloc, cudaFree or allocating library routine).
 *   - Limit: A*round256(active_scratch_elems*esize) + H*round256(helper_elems*esize)
 *     bytes (relay_plan gives both sizes) must fit the array; larger calls return
 *     RELAY_ERR_INVALID_ARGUMENT with a message. For the 2-active relay that is about
 *     2*count*esize, i.e. up to 32 MiB per rank.
 *   - Set-up: the first call on a device looks up the array's device address
 *     (cudaGetSymbolAddress) with that device current; make that first call before any
 *     stream capture.
 *   - Sharing: every call on a device uses the same array and leaves its contents
 *     there. Nothing in it needs clearing (each call writes every element before it
 *     reads it), but calls whose execution overlaps on the GPU (other streams, other
 *     host threads) race on it: order them.
 */
#define RELAY_NOALLOC_SCRATCH_BYTES (64u << 20)
relay_status_t relay_allreduce_noalloc(void* const* send, void* const* recv, size_t count,
                                       relay_dtype_t dtype, int A, int R, float scale,
                                       const relay_opts_t* opts, cudaStream_t stream);

/*
 * The objective of a training step over virtual ranks. The page has no counterpart: its
 * collectives move and sum what these calls produce (gradients, per-expert counts).
 *
 * ---- Output projection with a vocabulary sharded on the active ranks ----
 *
 * logits z[n][v] = hidden[n] . weight[v]. The vocabulary is the concatenation of A shards;
 * shard a holds rows[a] rows of the weight (and of its gradient) in rank a's memory. The
 * hidden rows are the whole batch's, once (after an all-gather every rank holds the same).
 * The logits of the batch are not held all at once: the gradients work on pieces of the vocabulary of at
 * most piece_bytes, and the workspace holds a value per logit of a piece (2 bytes for a bf16 head, 4 up to 128
 * rows; 6 for an fp32 head). A batch whose logits all fit one piece keeps their exponentials there,
 * and its logits are multiplied once; otherwise they are multiplied a second time, piece by piece. A loss
 * without gradients holds none.
 *
 * The default of piece_bytes is a budget of memory, under 1% of the GPU's 284 GB. What it decides (ms a call with both
 * gradients, bf16 unless said; kept / multiplied again in pieces of 1 GiB or less):
 *   2048 x 4096 x 131072 (0.5 GiB of exponentials)   4.1 / 5.3
 *   4096 x 2048 x 131072 (1 GiB)                     4.4 / 5.4
 *   8192 x 4096 x 131072 (2 GiB, what the default just holds)   18.7 / 22.7
 *   32768 x 2048 x 50000 (3.1 GiB)                   14.9 / 17.3
 *   16384 x 4096 x 128256 (3.9 GiB)                  37.7 / 44.8
 *   2048 x 2048 x 65536 fp32 (0.75 GiB)              5.6 / 7.1
 * Keeping is worth 14 to 23% of a call at every size; the size of a piece that is not kept hardly
 * matters (0.5 to 2 GiB: within 4%). A caller with the memory to spare passes a piece_bytes that its batch
 * fits.
 */
#define RELAY_HEAD_MAX_SHARDS 8
#define RELAY_HEAD_MAX_TOP 128
#define RELAY_HEAD_PIECE_BYTES (2ll << 30)
typedef struct relay_head {
  int32_t dtype;             /* RELAY_F32 or RELAY_BF16: hidden, weight and their gradients */
  int32_t A;                 /* shards, 1..RELAY_HEAD_MAX_SHARDS */
  int64_t tokens, dim;       /* hidden is [tokens][dim]; tokens may be 0, dim >= 1 */
  const void* hidden;
  int64_t hidden_stride;     /* elements between rows, >= dim (all four strides) */
  const void* weight[RELAY_HEAD_MAX_SHARDS]; /* shard a: [rows[a]][dim] */
  int64_t rows[RELAY_HEAD_MAX_SHARDS];       /* >= 0; the sum in [1, 2^31 - 1] */
  int64_t weight_stride;
  void* d_hidden;            /* [tokens][dim], or NULL: not wanted */
  int64_t d_hidden_stride;
  void* d_weight[RELAY_HEAD_MAX_SHARDS];     /* all NULL: not wanted; else one per shard */
  int64_t d_weight_stride;
  int64_t piece_bytes;       /* 0: RELAY_HEAD_PIECE_BYTES. Less memory for a smaller value; a
                                piece is never less than 256 columns */
} relay_head_t;

/* Bytes of workspace (device memory, any alignment, contents unspecified before and after)
 * the two calls below need; it depends on the gradients wanted, the strides and the weights' alignment
 * (rows off a 16-byte boundary, and fp32 rows, are copied). top: 0 for relay_linear_xent, else the K of
 * relay_linear_distill. -1 on an invalid head (relay_last_error says why). */
int64_t relay_head_workspace_size(const relay_head_t* head, int top);

/*
 * relay_linear_xent -- softmax cross entropy against one target per row.
 *   targets[tokens] int32: index into the concatenated vocabulary. Any value outside
 *     [0, sum of rows) ignores the row: loss 0, d_hidden 0, no part in d_weight, and
 *     nothing its hidden row holds (NaN included) reaches any output.
 *   loss[tokens] fp32: log(sum_v exp z[n][v]) - z[n][target].
 *   row_weight[tokens] fp32 (NULL: 1): dL/dloss[n]. The gradients are those of
 *     L = sum_n row_weight[n] * loss[n] and overwrite d_hidden and d_weight.
 * Arithmetic: products of the inputs accumulate in fp32; maxima, sums and the loss are
 * fp32. For a bf16 head the gradient of each logit is rounded to bf16 once before its two
 * products (up to 128 rows d_weight's takes it as two bf16 parts, 16 bits), which accumulate in fp32 and are
 * rounded to bf16 once. Every sum has a fixed
 * order: equal calls give equal bits. A NaN or +infinite logit gives its
 * row NaN; one of -inf has probability 0 (a row of nothing else is NaN). An fp32 head multiplies
 * bf16 parts of its values; it gives such logits as a product of fp32 values does, where the hidden
 * value that meets an infinite weight is 0 or at least 2^-95.
 * All pointers device memory, element-aligned; outputs overlap nothing else.
 * tokens == 0 writes zeros to d_weight.
 */
relay_status_t relay_linear_xent(const relay_head_t* head, const int32_t* targets,
                                 const float* row_weight, float* loss, void* workspace,
                                 int64_t workspace_bytes, cudaStream_t stream);

/*
 * relay_linear_distill -- distillation from the K largest logits of a teacher.
 *   teacher_index[tokens][top] int32: vocabulary ids, in any order. An id outside
 *     [0, sum of rows) is an absent entry, whatever its logit. A row with no entry, or
 *     whose entries are all -inf, is ignored as above. An id given twice counts twice.
 *   teacher_logits[tokens][top], teacher_dtype RELAY_F32 or RELAY_BF16.
 *   q[n] = softmax over the row's entries of teacher_logits / temperature;
 *   loss[n] = temperature^2 * sum_k q log(q / p), p = softmax(z / temperature) over the
 *     whole vocabulary; temperature finite and above 4.3e-39; 1 <= top <= RELAY_HEAD_MAX_TOP.
 * Everything else is as for relay_linear_xent.
 */
relay_status_t relay_linear_distill(const relay_head_t* head, const void* teacher_logits,
                                    relay_dtype_t teacher_dtype, const int32_t* teacher_index,
                                    int top, float temperature, const float* row_weight,
                                    float* loss, void* workspace, int64_t workspace_bytes,
                                    cudaStream_t stream);

/*
 * ---- Expert router: top-k choice, per-expert counts, balance loss ----
 *
 * relay_router_forward: logits[tokens][experts] (RELAY_F32 or RELAY_BF16, row_stride
 *   elements apart). A row is counted unless mask (NULL: all counted) holds 0 for it or
 *   every logit of it is -inf.
 *   index[tokens][top] int32: the top largest logits, largest first, ties to the lower
 *     expert; -1 for a row that is not counted. (A row with fewer than `top` logits above
 *     -inf fills up with the lowest experts left, gate 0.)
 *   gate[tokens][top] fp32: the softmax over all experts at index, or, with normalize != 0,
 *     the softmax over the row's chosen logits; 0 for a row that is not counted.
 *   counts[experts] int32: rows that chose the expert. prob_sum[experts] fp32: the sum of the
 *     rows' softmax. Both in a fixed order of summation, and both sums over ranks: with
 *     relay_allreduce over them between this call and relay_balance_loss, the balance
 *     loss is that of all ranks' tokens.
 *   1 <= top <= experts, top <= RELAY_ROUTER_MAX_TOP, experts <= RELAY_ROUTER_MAX_EXPERTS.
 *   A NaN or +infinite logit makes its row's gates and prob_sum NaN, whatever is beside it;
 *   index stays in range and distinct, with a NaN below -inf.
 *   Two launches at most. workspace: relay_router_workspace_size bytes, any alignment.
 */
#define RELAY_ROUTER_MAX_EXPERTS 1024
#define RELAY_ROUTER_MAX_TOP 32
int64_t relay_router_workspace_size(int64_t tokens, int experts);
relay_status_t relay_router_forward(const void* logits, int64_t row_stride, relay_dtype_t dtype,
                                    int64_t tokens, int experts, int top, int normalize,
                                    const uint8_t* mask, int32_t* index, float* gate,
                                    int32_t* counts, float* prob_sum, void* workspace,
                                    int64_t workspace_bytes, cudaStream_t stream);

/* relay_balance_loss -- with T = sum(counts) / top counted tokens:
 *   loss[0] = coef * experts * sum_e (counts[e] / (top * T)) * (prob_sum[e] / T)
 *   d_prob[e] = coef * experts * counts[e] / (top * T^2), its derivative by one token's
 *     probability of e (the counts are constants). Both 0 when T = 0. */
relay_status_t relay_balance_loss(const int32_t* counts, const float* prob_sum, int experts,
                                  int top, float coef, float* loss, float* d_prob,
                                  cudaStream_t stream);

/* relay_router_backward -- d_logits[tokens][experts] (dtype and strides of logits' own) from
 *   d_gate[tokens][top] (NULL: 0) and d_prob[experts] (NULL: 0, usually relay_balance_loss's).
 *   index is relay_router_forward's; rows whose first index is negative get 0. normalize must
 *   be the forward's. */
relay_status_t relay_router_backward(const void* logits, int64_t row_stride, relay_dtype_t dtype,
                                     int64_t tokens, int experts, int top, int normalize,
                                     const int32_t* index, const float* d_gate,
                                     const float* d_prob, void* d_logits, int64_t d_row_stride,
                                     cudaStream_t stream);

/*
 * ---- Expert router with scores, a bias for balance and groups of experts ----
 *
 * relay_grouped_router_forward: rows as in relay_router_forward, chosen otherwise.
 *   score s: softmax over the row's logits, or 1 / (1 + exp(-x)) of each.
 *   choice value c = s + bias (bias[experts] fp32, NULL: 0); an expert whose logit or bias is -inf cannot be chosen.
 *   With kept < groups: groups of experts / groups neighbours; a group's value is the sum of its group_sum (1 or 2) largest
 *     choice values (of those that can be chosen); the `kept` largest groups stay, ties to the lower.
 *   index[tokens][top]: the top largest choice values of the groups that stay, largest first, ties to the lower expert;
 *     -1 where fewer can be chosen. Both choices are by exact values: what fp32 cannot tell apart is compared in 64 bits.
 *   gate[tokens][top] = scale * s, or with normalize != 0 scale * s / the sum of the row's chosen s (0 where that is 0); 0 at -1. The
 *     bias is in the choice alone.
 *   counts[experts] int32: rows that chose the expert. prob_sum[experts] fp32: the sum over rows of s divided by the row's sum of
 *     s. Both as relay_router_forward's: summed over ranks by relay_allreduce, taken by relay_balance_loss (counts also by
 *     relay_router_bias_update). A row that mask leaves out, or of which no expert can be chosen, has index -1 and gate 0 and is in
 *     neither.
 *   A NaN logit makes its row's gates and prob_sum NaN; index stays in range and distinct, with a NaN below what else can be chosen
 *     (the other scores being those without it). So does a logit of +inf with softmax: the experts of +inf share the row.
 *   Scores are fp32: one below 2^-126 (softmax: of the row's largest score) is 0, in gates and gradients. bias values are finite
 *   or -inf.
 *   1 <= groups <= RELAY_ROUTER_MAX_GROUPS, a divisor of experts; with kept < groups at most RELAY_ROUTER_MAX_GROUPED experts;
 *   top <= RELAY_ROUTER_MAX_TOP and the experts of the kept groups. Two launches at most. workspace: relay_router_workspace_size bytes.
 *
 * relay_grouped_router_backward: d_logits from d_gate (NULL: 0) and d_prob (NULL: 0, the derivative by one token's share of each
 *   expert: relay_balance_loss's). index is the forward's; entries of -1 have no gradient, rows whose first is -1 are 0. Of `how` it
 *   takes score, experts, top, normalize and scale. The choice and the bias have no gradient.
 *
 * relay_router_bias_update: bias_out[e] = bias[e] + rate where counts[e] is below the mean of counts, - rate where it is above,
 *   bias[e] where it is the mean. In place with bias_out = bias.
 */
#define RELAY_ROUTER_MAX_GROUPS 32
#define RELAY_ROUTER_MAX_GROUPED 512
enum { RELAY_SCORE_SOFTMAX = 0, RELAY_SCORE_SIGMOID = 1 };
typedef struct relay_routing {
  int32_t score, experts, groups, kept, top, group_sum, normalize;
  float scale;
} relay_routing_t;
relay_status_t relay_grouped_router_forward(const relay_routing_t* how, const void* logits, int64_t row_stride,
                                            relay_dtype_t dtype, int64_t tokens, const float* bias, const uint8_t* mask,
                                            int32_t* index, float* gate, int32_t* counts, float* prob_sum, void* workspace,
                                            int64_t workspace_bytes, cudaStream_t stream);
relay_status_t relay_grouped_router_backward(const relay_routing_t* how, const void* logits, int64_t row_stride,
                                             relay_dtype_t dtype, int64_t tokens, const int32_t* index, const float* d_gate,
                                             const float* d_prob, void* d_logits, int64_t d_row_stride, cudaStream_t stream);
relay_status_t relay_router_bias_update(const int32_t* counts, const float* bias, int experts, float rate, float* bias_out,
                                        cudaStream_t stream);

/*
 * ---- Products in 8-bit floating point, a scale for each block of 128 ----
 *
 * Values are e4m3 (1 byte, largest 448) times an fp32 scale. A row-scaled matrix [rows][depth] has a scale for each 128
 * neighbours of a row, scale[blocks of depth][rows] (rows contiguous); a tile-scaled one [cols][depth] a scale for each 128 x
 * 128, scale[blocks of cols][blocks of depth]. Blocks start at multiples of 128; the last of a dimension may be short.
 * Row strides are multiples of 16 (bytes), addresses of 8-bit matrices on 16-byte boundaries.
 *
 * Groups (experts): offset[groups + 1] int32 in device memory, ascending; group g holds rows offset[g] .. offset[g + 1] - 1 of
 * the rows, which stand sorted by group. A group may be empty; what rows before offset[0] and from offset[groups] on
 * hold has no effect, and they are not written. Offsets outside [0, rows] or out of order give unspecified results, and no access out of range.
 *
 * relay_quantize_fp8 -- x[batch][rows][cols] (RELAY_F32 or RELAY_BF16; the batch's matrices one behind the other,
 *   rows * x_stride elements apart) to 8 bits, as it lies (q, scale), transposed (qt, scale_t), or both. Scales are powers of two,
 *   the least that bring a block's largest magnitude to 448 or below (2^-126 at least; 1 for a block of zeros), so a value is rounded
 *   once, to nearest-even. A block that holds a NaN or an infinity has scale NaN.
 *   tiles / tiles_t: 0 row-scaled, 1 tile-scaled (of qt: rows are x's columns). A batch other than 1 has tiles only.
 *   With groups, qt's rows (length relay_fp8_depth) hold the groups one behind the other, each filled up with zeros to a
 *   multiple of 128; q is by x's own rows and has no tiles.
 *
 * relay_matmul_fp8 -- by_depth 0: out[r][n] = sum_d a[r][d] b[g(r)][n][d]: a row-scaled [rows][depth], b tile-scaled
 *     [groups][cols][depth] (its matrices one behind the other), g(r) the row's group; groups 0 and offset NULL: one b for all rows.
 *   by_depth 1: out[g][r][n] = sum over group g's part of the depth of a[r][d] b[n][d]: a row-scaled [rows][depth], b
 *     tile-scaled [cols][depth], depth laid out as qt's above (`depth` its whole length); out[groups][rows][cols], zeros for an
 *     empty group; groups 0: one group of any depth. This is a weight's gradient: a = the output's gradient, b = the input, both transposed.
 *   Products of a block of 128 accumulate in the tensor cores (fp32), the blocks in fp32 by fused multiply-adds with the
 *   two scales' product (which has to be in fp32's range); out is rounded once to RELAY_F32 or RELAY_BF16. Equal calls give equal bits.
 *   One launch. Scales may be any fp32 values. depth 0 gives zeros.
 * An input's gradient is the product with the transposed weight: quantize the weight once as it lies and transposed (the tiles'
 * scales and values are the same).
 */
#define RELAY_FP8_MAX_ROWS (1 << 22)
#define RELAY_FP8_MAX_GROUPS 1024
typedef struct relay_fp8_quantize {
  const void* x;
  int64_t x_stride;            /* elements, >= cols */
  int64_t batch, rows, cols;   /* batch 1 .. RELAY_FP8_MAX_GROUPS; rows, cols <= RELAY_FP8_MAX_ROWS; cols >= 1 */
  void* q;                     /* NULL: not wanted */
  int64_t q_stride;            /* bytes */
  float* scale;
  void* qt;                    /* NULL: not wanted */
  int64_t qt_stride;
  float* scale_t;
  const int32_t* offset;       /* NULL: no groups */
  int32_t groups, dtype, tiles, tiles_t;
} relay_fp8_quantize_t;
typedef struct relay_fp8_matmul {
  const void* a;
  int64_t a_stride;            /* bytes */
  const float* a_scale;        /* [blocks of depth][rows] */
  const void* b;
  int64_t b_stride;
  const float* b_scale;
  void* out;
  int64_t out_stride;          /* elements */
  int64_t rows, cols, depth;
  const int32_t* offset;       /* NULL: no groups */
  int32_t groups, out_dtype, by_depth, reserved;
} relay_fp8_matmul_t;
/* Length of the transposed rows: rows, or with groups 128 * (rows / 128 + min(groups, rows)): room for any offsets. */
int64_t relay_fp8_depth(int64_t rows, int groups);
relay_status_t relay_quantize_fp8(const relay_fp8_quantize_t* what, cudaStream_t stream);
relay_status_t relay_matmul_fp8(const relay_fp8_matmul_t* what, cudaStream_t stream);

/*
 * ---- All gradients at once: their norm, and clipping ----
 *
 * A list of n tensors in device memory: grad[i] holds count[i] elements of dtype[i] (RELAY_F32 or RELAY_BF16), contiguous;
 * count 0 is an empty tensor. The arrays are read during the call alone.
 *
 * relay_grad_norm -- norm[0] (fp32) = sqrt of the sum of all elements' squares, 0 for an empty list. It is within 10 x 2^-24 of
 *   its value over the whole range of finite values (2^-149 below 2^-126, +inf where fp32 cannot hold it), summed in a fixed order. A NaN or an infinity
 *   shows in norm. A tensor given twice counts twice. Norms of several lists (ranks) join by the same call over their norms.
 *   Two launches for 512 tensors, one more for each 512 beyond; one for up to four pieces of 32 KiB, which never span two tensors.
 *   workspace: relay_grad_workspace_size bytes, any alignment.
 *
 * relay_grad_clip -- out[i] = grad[i] * min(1, max_norm / (norm[0] + 1e-6)): sum, quotient and product are rounded to fp32 each, and
 *   the product to the tensor's dtype. out NULL, or with grad[i]'s own address: in place. norm[0] is read on the device, after what
 *   precedes the call on the stream. With nothing to clip, or a norm that is NaN or infinite, the values stay as they are (the caller
 *   sees it in norm). max_norm finite and above 0. No tensor that is written may overlap another. The list is walked from its end:
 *   right after relay_grad_norm over the same list its last 100 MB are still in L2.
 */
#define RELAY_GRADS_MAX (1 << 20)
typedef struct relay_grads {
  int32_t n;
  void* const* grad;
  const size_t* count;
  const int32_t* dtype;
} relay_grads_t;
int64_t relay_grad_workspace_size(const relay_grads_t* grads);
relay_status_t relay_grad_norm(const relay_grads_t* grads, float* norm, void* workspace, int64_t workspace_bytes,
                               cudaStream_t stream);
relay_status_t relay_grad_clip(const relay_grads_t* grads, const relay_grads_t* out, const float* norm, float max_norm,
                               cudaStream_t stream);

/*
 * relay_device_status -- reads and clears the device's fault word. Passes whose sources
 * sit off the 16-byte grid stage each tile's source bytes in shared memory with a bulk
 * copy and wait for it on an mbarrier (the schedule's strided pack/unpack, item 7). That
 * wait is bounded (200 ms of the global timer); if it ever runs out, the kernel records a
 * fault, leaves that tile unwritten and returns instead of hanging. Call this after
 * synchronizing the streams that ran collectives: RELAY_ERR_CUDA if a wait gave up since
 * the last call (or a CUDA call failed), RELAY_OK otherwise. Synchronous.
 */
relay_status_t relay_device_status(void);

/*
 * relay_test_staged_wait -- a test of that bounded wait: one staged copy of `count`
 * elements (at most one 16 KiB tile) from `src` to `dst` (device memory, dst 16-byte
 * aligned) whose barrier expects `extra_bytes` more than its copy brings. With
 * extra_bytes > 0 the wait runs out, the copy's destination is left unwritten, and the
 * next relay_device_status() reports RELAY_ERR_CUDA; the context stays usable. With 0 it
 * is an ordinary copy. The page has no counterpart.
 */
relay_status_t relay_test_staged_wait(void* dst, const void* src, size_t count,
                                      relay_dtype_t dtype, int extra_bytes, cudaStream_t stream);

/*
 * relay_test_head_wait -- a test of the bounded waits (500 ms) of the losses' products: a
 * relay_linear_xent whose barriers expect `extra_bytes` more than their loads bring. With
 * extra_bytes > 0 the waits run out, the outputs are unspecified, and the next
 * relay_device_status() reports RELAY_ERR_CUDA; the context stays usable. With 0 it is
 * an ordinary call.
 */
relay_status_t relay_test_head_wait(const relay_head_t* head, const int32_t* targets, float* loss, void* workspace,
                                    int64_t workspace_bytes, int extra_bytes, cudaStream_t stream);

/* relay_test_fp8_wait -- the same for relay_matmul_fp8. */
relay_status_t relay_test_fp8_wait(const relay_fp8_matmul_t* what, int extra_bytes, cudaStream_t stream);

/* Human-readable text of the last error this thread's calls produced. */
const char* relay_last_error(void);
/* How the calling thread's last collective call was launched: "chained: G groups, P
 * pieces, D dropped" (D: scratch sources whose dead lines the launch drops from L2),
 * "cooperative" or "passes" (see the launch policy above); "dry run" for a
 * RELAY_FLAG_DRY_RUN call that would not run chained, "none" before the first call. */
const char* relay_last_launch(void);
int relay_abi_version(void);

#ifdef __cplusplus
}
#endif
#endif /* RELAY_H */
