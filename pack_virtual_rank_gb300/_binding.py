"""ctypes binding of ``librelay.so`` (the C ABI in ``include/relay.h``).

Argument marshalling only: every step of a collective runs in the library's CUDA
kernels. PyTorch is used for device memory and streams. There is no fallback: if the
library is not built the calls raise.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional, Sequence

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "librelay.so")

# enums (relay.h)
OK, ERR_INVALID_ARGUMENT, ERR_UNSUPPORTED, ERR_CUDA = 0, 1, 2, 3
F32, BF16, I32 = 0, 1, 2
ALLREDUCE, REDUCE_SCATTER, ALL_GATHER, ALL_TO_ALL = 0, 1, 2, 3
KIND_RELAY, KIND_ZERO_CHUNK, KIND_DIRECT, KIND_LEGACY = 0, 1, 2, 3
SCHEDULE_AUTO, SCHEDULE_RELAY, SCHEDULE_DIRECT, SCHEDULE_LEGACY = 0, 1, 2, 3
FLAG_CHECK_HAZARDS = 1
FLAG_DRY_RUN = 2
FLAG_SEPARATE_PASSES = 4
FLAG_FUSED_PASSES = 8
FLAG_PAYLOAD_PARTIAL = 16
FLAG_CHAINED = 32
FLAG_KEEP_SCRATCH = 64
ESIZE = {F32: 4, BF16: 2, I32: 4}
PASS_NAMES = ("group1", "group2", "group3", "active_reduce", "pack", "helper_forward", "unpack")


class RelayError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"relay status {status}: {message}")
        self.status = status


class RelayOpts(ctypes.Structure):
    _fields_ = [("offload_permille", ctypes.c_int32), ("schedule", ctypes.c_int32),
                ("relay_threshold_bytes", ctypes.c_int64), ("pass_events", ctypes.c_void_p),
                ("n_pass_events", ctypes.c_int32), ("flags", ctypes.c_int32)]


class RelayPlan(ctypes.Structure):
    _fields_ = ([(f, ctypes.c_int32) for f in ("coll", "dtype", "A", "R", "H", "esize", "kind",
                                               "num_groups", "offload_permille", "wide_partial")]
                + [(f, ctypes.c_int64) for f in ("count", "chunk", "relay_total", "dirA_offset",
                                                 "dirA_size", "dirB_size", "direct_total",
                                                 "direct_g1", "direct_g2", "owner_slice",
                                                 "owner_slice_last", "helper_elems",
                                                 "active_scratch_elems", "input_elems",
                                                 "output_elems")])

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_}


class RelayPassInfo(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("num_segments", ctypes.c_int32),
                ("bytes_read", ctypes.c_int64), ("bytes_written", ctypes.c_int64)]


HEAD_MAX_SHARDS = 8
HEAD_MAX_TOP = 128
ROUTER_MAX_EXPERTS = 1024
ROUTER_MAX_TOP = 32
ROUTER_MAX_GROUPS = 32
ROUTER_MAX_GROUPED = 512
SCORES = {"softmax": 0, "sigmoid": 1}
FP8_BLOCK = 128            # values that share a scale
FP8_MAX_ROWS = 1 << 22
FP8_MAX_GROUPS = 1024


class RelayHead(ctypes.Structure):
    """A sharded output projection (relay_head_t); build it with ``make_head``."""
    _fields_ = [("dtype", ctypes.c_int32), ("A", ctypes.c_int32), ("tokens", ctypes.c_int64),
                ("dim", ctypes.c_int64), ("hidden", ctypes.c_void_p),
                ("hidden_stride", ctypes.c_int64), ("weight", ctypes.c_void_p * HEAD_MAX_SHARDS),
                ("rows", ctypes.c_int64 * HEAD_MAX_SHARDS), ("weight_stride", ctypes.c_int64),
                ("d_hidden", ctypes.c_void_p), ("d_hidden_stride", ctypes.c_int64),
                ("d_weight", ctypes.c_void_p * HEAD_MAX_SHARDS),
                ("d_weight_stride", ctypes.c_int64), ("piece_bytes", ctypes.c_int64)]


class RelayGrads(ctypes.Structure):
    """A list of tensors in device memory (relay_grads_t); build it with ``make_grads``."""
    _fields_ = [("n", ctypes.c_int32), ("grad", ctypes.POINTER(ctypes.c_void_p)),
                ("count", ctypes.POINTER(ctypes.c_size_t)), ("dtype", ctypes.POINTER(ctypes.c_int32))]


_lib = None


def lib():
    """Load librelay.so (build it first with ``pack_virtual_rank_gb300.build.build()``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built: call pack_virtual_rank_gb300.build.build() "
                           "(needs nvcc); there is no fallback implementation")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, sz, f32 = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t,
                             ctypes.c_float)
    P = ctypes.POINTER
    L.relay_opts_init.argtypes = [P(RelayOpts)]
    L.relay_opts_init.restype = None
    L.relay_abi_version.restype = i32
    L.relay_last_error.restype = ctypes.c_char_p
    L.relay_last_launch.restype = ctypes.c_char_p
    L.relay_plan.argtypes = [i32, sz, i32, i32, i32, P(RelayOpts), P(RelayPlan)]
    L.relay_plan.restype = i32
    L.relay_plan_link_bytes.argtypes = [P(RelayPlan), P(ctypes.c_uint64), sz]
    L.relay_plan_link_bytes.restype = i32
    L.relay_plan_cost_bytes.argtypes = [P(RelayPlan)]
    L.relay_plan_cost_bytes.restype = ctypes.c_uint64
    L.relay_plan_passes.argtypes = [P(RelayPlan), i32, P(RelayPassInfo), i32]
    L.relay_plan_passes.restype = i32
    L.relay_pass_name.argtypes = [i32]
    L.relay_pass_name.restype = ctypes.c_char_p
    L.relay_passthrough_helper_size.argtypes = [i64, i32, i32]
    L.relay_passthrough_helper_size.restype = i64
    arr = P(vp)
    for name in ("relay_allreduce", "relay_reduce_scatter"):
        fn = getattr(L, name)
        fn.argtypes = [arr, arr, arr, sz, i32, i32, i32, f32, P(RelayOpts), vp]
        fn.restype = i32
    for name in ("relay_all_gather", "relay_all_to_all"):
        fn = getattr(L, name)
        fn.argtypes = [arr, arr, arr, sz, i32, i32, i32, P(RelayOpts), vp]
        fn.restype = i32
    L.relay_multi_group.argtypes = [i32, i32, P(sz), arr, arr, arr, i32, i32, f32, P(RelayOpts), vp]
    L.relay_multi_group.restype = i32
    L.relay_multi_group_link_bytes.argtypes = [i32, i32, P(sz), i32, i32, P(RelayOpts),
                                               P(ctypes.c_uint64), sz, P(ctypes.c_int)]
    L.relay_multi_group_link_bytes.restype = i32
    L.relay_helper_size.argtypes = [P(RelayPlan)]
    L.relay_helper_size.restype = i64
    L.relay_active_scratch_size.argtypes = [P(RelayPlan)]
    L.relay_active_scratch_size.restype = i64
    L.relay_helper_contract_size.argtypes = [i32, i64, i32, i32]
    L.relay_helper_contract_size.restype = i64
    L.relay_allreduce_noalloc.argtypes = [arr, arr, sz, i32, i32, i32, f32, P(RelayOpts), vp]
    L.relay_allreduce_noalloc.restype = i32
    L.relay_pack_flat.argtypes = [arr, P(sz), i32, vp, i32, vp]
    L.relay_pack_flat.restype = i32
    L.relay_unpack_flat.argtypes = [vp, arr, P(sz), i32, i32, vp]
    L.relay_unpack_flat.restype = i32
    L.relay_copy.argtypes = [vp, vp, sz, i32, i32, vp]
    L.relay_copy.restype = i32
    L.relay_device_status.argtypes = []
    L.relay_device_status.restype = i32
    L.relay_test_staged_wait.argtypes = [vp, vp, sz, i32, i32, vp]
    L.relay_test_staged_wait.restype = i32
    L.relay_head_workspace_size.argtypes = [P(RelayHead), i32]
    L.relay_head_workspace_size.restype = i64
    L.relay_linear_xent.argtypes = [P(RelayHead), vp, vp, vp, vp, i64, vp]
    L.relay_linear_xent.restype = i32
    L.relay_linear_distill.argtypes = [P(RelayHead), vp, i32, vp, i32, f32, vp, vp, vp, i64, vp]
    L.relay_linear_distill.restype = i32
    L.relay_test_head_wait.argtypes = [P(RelayHead), vp, vp, vp, i64, i32, vp]
    L.relay_test_head_wait.restype = i32
    L.relay_router_workspace_size.argtypes = [i64, i32]
    L.relay_router_workspace_size.restype = i64
    L.relay_router_forward.argtypes = [vp, i64, i32, i64, i32, i32, i32, vp, vp, vp, vp, vp, vp, i64, vp]
    L.relay_router_forward.restype = i32
    L.relay_balance_loss.argtypes = [vp, vp, i32, i32, f32, vp, vp, vp]
    L.relay_balance_loss.restype = i32
    L.relay_router_backward.argtypes = [vp, i64, i32, i64, i32, i32, i32, vp, vp, vp, vp, i64, vp]
    L.relay_router_backward.restype = i32
    for name in ("forward", "backward", "balance"):
        fn = getattr(L, f"relay_packed_router_{name}")
        fn.argtypes = [ctypes.c_char_p]
        fn.restype = i32
    L.relay_grad_workspace_size.argtypes = [P(RelayGrads)]
    L.relay_grad_workspace_size.restype = i64
    L.relay_grad_norm.argtypes = [P(RelayGrads), vp, vp, i64, vp]
    L.relay_grad_norm.restype = i32
    L.relay_grad_clip.argtypes = [P(RelayGrads), P(RelayGrads), vp, f32, vp]
    L.relay_grad_clip.restype = i32
    for name in ("forward", "backward"):
        fn = getattr(L, f"relay_packed_grouped_{name}")
        fn.argtypes = [ctypes.c_char_p, ctypes.c_char_p]
        fn.restype = i32
    L.relay_router_bias_update.argtypes = [vp, vp, i32, f32, vp, vp]
    L.relay_router_bias_update.restype = i32
    L.relay_fp8_depth.argtypes = [i64, i32]
    L.relay_fp8_depth.restype = i64
    for name in ("relay_quantize_fp8", "relay_matmul_fp8"):
        fn = getattr(L, name)
        fn.argtypes = [ctypes.c_char_p, vp]
        fn.restype = i32
    L.relay_test_fp8_wait.argtypes = [ctypes.c_char_p, i32, vp]
    L.relay_test_fp8_wait.restype = i32
    if L.relay_abi_version() != 1:
        raise RuntimeError("librelay.so ABI version mismatch")
    _lib = L
    return L


def _check(status: int):
    if status != OK:
        raise RelayError(status, lib().relay_last_error().decode(errors="replace"))


def device_status() -> None:
    """Raise if a bounded wait in a relay kernel gave up since the last check (reads and
    clears the device's fault word; synchronous)."""
    _check(lib().relay_device_status())


def last_launch() -> str:
    """How this thread's last collective call was launched: "chained", "cooperative" or
    "passes" ("dry run" for a dry run that would not run chained)."""
    return lib().relay_last_launch().decode()


def dtype_code(dtype) -> int:
    """Accept a relay dtype code, "f32"/"bf16"/"i32", or a torch dtype."""
    if isinstance(dtype, int):
        return dtype
    if isinstance(dtype, str):
        return {"f32": F32, "bf16": BF16, "i32": I32}[dtype]
    import torch
    return {torch.float32: F32, torch.bfloat16: BF16, torch.int32: I32}[dtype]


def make_opts(offload_permille: int = -1, schedule: int = SCHEDULE_AUTO,
              relay_threshold_bytes: int = -1, flags: int = 0, pass_events=None) -> RelayOpts:
    o = RelayOpts()
    lib().relay_opts_init(ctypes.byref(o))
    o.offload_permille = offload_permille
    o.schedule = schedule
    o.relay_threshold_bytes = relay_threshold_bytes
    o.flags = flags
    if pass_events is not None:
        for e in pass_events:
            # torch creates the CUDA event lazily, on its first record
            if hasattr(e, "cuda_event") and int(e.cuda_event) == 0:
                e.record()
        handles = (ctypes.c_void_p * len(pass_events))(*[int(e.cuda_event) if hasattr(e, "cuda_event")
                                                          else int(e) for e in pass_events])
        o._events_keepalive = handles
        o.pass_events = ctypes.cast(handles, ctypes.c_void_p)
        o.n_pass_events = len(pass_events)
    return o


# ------------------------------------------------------------------------ planning --

def relay_plan(coll: int, count: int, dtype, A: int, R: int,
               opts: Optional[RelayOpts] = None) -> RelayPlan:
    p = RelayPlan()
    _check(lib().relay_plan(coll, count, dtype_code(dtype), A, R,
                            ctypes.byref(opts) if opts is not None else None, ctypes.byref(p)))
    return p


def relay_plan_link_bytes(plan: RelayPlan) -> np.ndarray:
    G, R = plan.num_groups, plan.R
    out = np.zeros(max(G, 1) * R * R, np.uint64)
    _check(lib().relay_plan_link_bytes(ctypes.byref(plan),
                                       out.ctypes.data_as(ctypes.POINTER(ctypes.c_uint64)),
                                       out.size))
    return out[: G * R * R].reshape(G, R, R)


def relay_plan_cost_bytes(plan: RelayPlan) -> int:
    return int(lib().relay_plan_cost_bytes(ctypes.byref(plan)))


def relay_plan_passes(plan: RelayPlan, in_place: bool = False) -> list:
    n = lib().relay_plan_passes(ctypes.byref(plan), int(in_place), None, 0)
    if n < 0:
        raise RelayError(ERR_INVALID_ARGUMENT, "not a plan")
    buf = (RelayPassInfo * max(n, 1))()
    lib().relay_plan_passes(ctypes.byref(plan), int(in_place), buf, n)
    return [{"kind": buf[i].kind, "name": PASS_NAMES[buf[i].kind],
             "num_segments": buf[i].num_segments, "bytes_read": buf[i].bytes_read,
             "bytes_written": buf[i].bytes_written} for i in range(n)]


def relay_passthrough_helper_size(count_g: int, A: int, num_chunks: int) -> int:
    return int(lib().relay_passthrough_helper_size(count_g, A, num_chunks))


def relay_helper_size(plan: RelayPlan) -> int:
    return int(lib().relay_helper_size(ctypes.byref(plan)))


def relay_active_scratch_size(plan: RelayPlan) -> int:
    return int(lib().relay_active_scratch_size(ctypes.byref(plan)))


def relay_helper_contract_size(coll: int, count: int, A: int, R: int) -> int:
    return int(lib().relay_helper_contract_size(coll, count, A, R))


def relay_pass_name(kind: int) -> str:
    return lib().relay_pass_name(kind).decode()


# --------------------------------------------------------------------- collectives --

def _ptr(x) -> Optional[int]:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if not x.is_cuda:
        raise ValueError("relay buffers must be CUDA tensors (device memory)")
    if not x.is_contiguous():
        raise ValueError("relay buffers must be contiguous")
    return x.data_ptr()


def _ptr_array(xs: Sequence, R: int):
    if len(xs) != R:
        raise ValueError(f"expected {R} entries (one per virtual rank), got {len(xs)}")
    return (ctypes.c_void_p * R)(*[_ptr(x) for x in xs])


def _stream(stream) -> int:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _pad(xs, R):
    xs = list(xs) if xs is not None else []
    return xs + [None] * (R - len(xs))


def relay_allreduce(send, recv, scratch, count: int, dtype, A: int, R: int, scale: float = 1.0,
                    opts: Optional[RelayOpts] = None, stream=None) -> None:
    _check(lib().relay_allreduce(_ptr_array(_pad(send, R), R), _ptr_array(_pad(recv, R), R),
                                 _ptr_array(_pad(scratch, R), R), count, dtype_code(dtype), A, R,
                                 scale, ctypes.byref(opts) if opts is not None else None,
                                 _stream(stream)))


def relay_reduce_scatter(send, recv, scratch, recv_count: int, dtype, A: int, R: int,
                         scale: float = 1.0, opts: Optional[RelayOpts] = None, stream=None) -> None:
    _check(lib().relay_reduce_scatter(_ptr_array(_pad(send, R), R), _ptr_array(_pad(recv, R), R),
                                      _ptr_array(_pad(scratch, R), R), recv_count,
                                      dtype_code(dtype), A, R, scale,
                                      ctypes.byref(opts) if opts is not None else None,
                                      _stream(stream)))


def relay_all_gather(send, recv, scratch, send_count: int, dtype, A: int, R: int,
                     opts: Optional[RelayOpts] = None, stream=None) -> None:
    _check(lib().relay_all_gather(_ptr_array(_pad(send, R), R), _ptr_array(_pad(recv, R), R),
                                  _ptr_array(_pad(scratch, R), R), send_count, dtype_code(dtype),
                                  A, R, ctypes.byref(opts) if opts is not None else None,
                                  _stream(stream)))


def relay_all_to_all(send, recv, scratch, segment_count: int, dtype, A: int, R: int,
                     opts: Optional[RelayOpts] = None, stream=None) -> None:
    _check(lib().relay_all_to_all(_ptr_array(_pad(send, R), R), _ptr_array(_pad(recv, R), R),
                                  _ptr_array(_pad(scratch, R), R), segment_count,
                                  dtype_code(dtype), A, R,
                                  ctypes.byref(opts) if opts is not None else None,
                                  _stream(stream)))


def relay_allreduce_noalloc(send, recv, count: int, dtype, A: int, R: int, scale: float = 1.0,
                            opts: Optional[RelayOpts] = None, stream=None) -> None:
    """Allreduce whose scratch is the library's built-in device array (see relay.h)."""
    _check(lib().relay_allreduce_noalloc(_ptr_array(_pad(send, R), R), _ptr_array(_pad(recv, R), R),
                                         count, dtype_code(dtype), A, R, scale,
                                         ctypes.byref(opts) if opts is not None else None,
                                         _stream(stream)))


COLLECTIVES = {ALLREDUCE: relay_allreduce, REDUCE_SCATTER: relay_reduce_scatter,
               ALL_GATHER: relay_all_gather, ALL_TO_ALL: relay_all_to_all}


def alloc_scratch(plan: RelayPlan, device, torch_dtype=None):
    """R scratch buffers sized by the plan (None where a rank needs none)."""
    import torch
    td = torch_dtype or {F32: torch.float32, BF16: torch.bfloat16, I32: torch.int32}[plan.dtype]
    out = []
    for r in range(plan.R):
        n = plan.active_scratch_elems if r < plan.A else plan.helper_elems
        out.append(torch.empty(n, dtype=td, device=device) if n > 0 else None)
    return out


# -------------------------------------------------------------- fused multi-group --

def group_ranks(g: int, A: int, R: int) -> list:
    """Global ranks of group g's local ranks: its A actives, then its helpers."""
    return [g * A + a for a in range(A)] + [r for r in range(R) if r // A != g]


def relay_multi_group(coll: int, counts: Sequence[int], send, recv, scratch, dtype, A: int,
                      scale: float = 1.0, opts: Optional[RelayOpts] = None, stream=None) -> None:
    """Fused call over len(counts) groups of A consecutive ranks (R = groups * A).
    send/recv: R entries (rank r's buffers for its own group); scratch: one list of R
    entries per group (rank r's scratch for that group)."""
    G = len(counts)
    R = G * A
    flat = [x for per_group in scratch for x in _pad(per_group, R)]
    if len(flat) != G * R:
        raise ValueError("scratch needs one list of R entries per group")
    c = (ctypes.c_size_t * G)(*counts)
    _check(lib().relay_multi_group(coll, G, c, _ptr_array(send, R), _ptr_array(recv, R),
                                   (ctypes.c_void_p * (G * R))(*[_ptr(x) for x in flat]),
                                   dtype_code(dtype), A, scale,
                                   ctypes.byref(opts) if opts is not None else None,
                                   _stream(stream)))


def relay_multi_group_link_bytes(coll: int, counts: Sequence[int], dtype, A: int,
                                 opts: Optional[RelayOpts] = None) -> np.ndarray:
    G = len(counts)
    R = G * A
    out = np.zeros(3 * R * R, np.uint64)
    phases = ctypes.c_int(0)
    c = (ctypes.c_size_t * G)(*counts)
    _check(lib().relay_multi_group_link_bytes(
        coll, G, c, dtype_code(dtype), A, ctypes.byref(opts) if opts is not None else None,
        out.ctypes.data_as(ctypes.POINTER(ctypes.c_uint64)), out.size, ctypes.byref(phases)))
    return out[: phases.value * R * R].reshape(phases.value, R, R)


def alloc_multi_scratch(coll: int, counts: Sequence[int], dtype, A: int, device,
                        opts: Optional[RelayOpts] = None):
    """Per group, R scratch buffers sized by that group's plan (None where not needed)."""
    import torch
    G = len(counts)
    R = G * A
    td = {F32: torch.float32, BF16: torch.bfloat16, I32: torch.int32}[dtype_code(dtype)]
    out = []
    for g in range(G):
        p = relay_plan(coll, counts[g], dtype, A, R, opts)
        row = [None] * R
        for l, r in enumerate(group_ranks(g, A, R)):
            n = p.active_scratch_elems if l < A else p.helper_elems
            if n > 0:
                row[r] = torch.empty(n, dtype=td, device=device)
        out.append(row)
    return out


# ------------------------------------------------------------ flat pack / unpack --

def relay_pack_flat(tensors: Sequence, flat, dtype=None, stream=None) -> None:
    """Copy `tensors` end to end into `flat` (one launch)."""
    n = len(tensors)
    dt = dtype_code(dtype if dtype is not None else flat.dtype)
    counts = (ctypes.c_size_t * max(n, 1))(*[t.numel() for t in tensors])
    _check(lib().relay_pack_flat((ctypes.c_void_p * max(n, 1))(*[_ptr(t) for t in tensors]),
                                 counts, n, _ptr(flat), dt, _stream(stream)))


def relay_unpack_flat(flat, tensors: Sequence, dtype=None, stream=None) -> None:
    """Copy consecutive pieces of `flat` back into `tensors` (one launch)."""
    n = len(tensors)
    dt = dtype_code(dtype if dtype is not None else flat.dtype)
    counts = (ctypes.c_size_t * max(n, 1))(*[t.numel() for t in tensors])
    _check(lib().relay_unpack_flat(_ptr(flat), (ctypes.c_void_p * max(n, 1))(*[_ptr(t) for t in tensors]),
                                   counts, n, dt, _stream(stream)))


# ---------------------------------------------------------------------- host link --

def _any_ptr(x) -> int:
    """Address of a contiguous tensor in device memory or host memory (pinned or not)."""
    if isinstance(x, int):
        return x
    if not x.is_contiguous():
        raise ValueError("relay_copy tensors must be contiguous")
    return x.data_ptr()


def relay_copy(dst, src, max_ctas: int = 0, stream=None) -> None:
    """Copy `src` into `dst` (same dtype and numel) with the library's streaming kernel.
    Either may be a CUDA tensor or a host tensor (pinned, or pageable where the device
    reads host page tables); max_ctas caps the launch's CTAs (0: one per 16 KiB tile)."""
    if dst.dtype != src.dtype or dst.numel() != src.numel():
        raise ValueError("relay_copy: dst and src must have the same dtype and size")
    _check(lib().relay_copy(_any_ptr(dst), _any_ptr(src), src.numel(), dtype_code(src.dtype),
                            max_ctas, _stream(stream)))


# ------------------------------------------- training objective: losses and router --

# What these calls ask torch for on every call, looked up once: small calls cost more host time
# than kernel time.
_torch = None
_float32 = _int32 = _e4m3 = _raw_stream = _device = None
_code: dict = {}


def _bind_torch() -> None:
    global _torch, _float32, _int32, _e4m3, _raw_stream, _device
    import torch
    _torch, _float32, _int32, _e4m3 = torch, torch.float32, torch.int32, torch.float8_e4m3fn
    _code.update({torch.float32: F32, torch.bfloat16: BF16})
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    _device = getattr(torch._C, "_cuda_getDevice", None)


def _handle(stream) -> int:
    """The stream's handle; the current stream's for None."""
    if stream is None and _raw_stream is not None and _device is not None:
        return _raw_stream(_device())
    return _stream(stream) or 0


def _dtype(x, name: str) -> int:
    try:
        return _code[x.dtype]
    except KeyError:
        raise ValueError(f"{name} must be float32 or bfloat16, got {x.dtype}") from None


def _array(x, name: str, dtype, shape) -> Optional[int]:
    """Address of a contiguous CUDA tensor of the given dtype and shape."""
    if x.dtype is not dtype or x.shape != shape:
        raise ValueError(f"{name} must be {dtype} of shape {tuple(shape)}, got {x.dtype} of {tuple(x.shape)}")
    if not x.is_cuda or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor (device memory)")
    return x.data_ptr()


def _matrix(x, name: str) -> int:
    """Address of a CUDA matrix whose rows are contiguous (any row stride)."""
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (device memory)")
    if x.dim() != 2 or (x.shape[1] > 1 and x.stride(1) != 1):
        raise ValueError(f"{name} must be a matrix with contiguous rows")
    return x.data_ptr()


def _row_stride(x) -> int:
    return x.stride(0) if x.shape[0] > 1 else max(x.stride(0), x.shape[1])


def _common_stride(xs, name: str) -> int:
    strides = {x.stride(0) for x in xs if x.shape[0] > 1}
    if len(strides) > 1:
        raise ValueError(f"the {name} shards must have one row stride")
    return strides.pop() if strides else max(x.shape[1] for x in xs)


def _own_workspace(alloc, stream):
    """A workspace for one call, allocated (and freed) in the order of the call's stream."""
    if stream is None:
        return alloc()
    if not hasattr(stream, "cuda_stream"):
        raise ValueError("pass a workspace with a raw stream handle")
    import torch
    with torch.cuda.stream(stream):
        return alloc()


def _space(x):
    """Address and bytes of a workspace (any type)."""
    if not x.is_cuda or not x.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor (device memory)")
    return x.data_ptr(), x.numel() * x.element_size()


def _columns(x, name: str) -> int:
    if x.dim() != 2:
        raise ValueError(f"{name} must be a matrix, a row of choices for each token, got {tuple(x.shape)}")
    return x.shape[1]


def make_head(hidden, weights: Sequence, d_hidden=None, d_weights: Optional[Sequence] = None,
              piece_bytes: int = 0) -> RelayHead:
    """Describe an output projection for relay_linear_xent and relay_linear_distill:
    hidden [tokens, dim], one weight shard [rows, dim] per active rank (their concatenation is
    the vocabulary), and the gradients to write, if any. The tensors must outlive the head (it
    keeps references) and it can be used for any number of calls."""
    weights = list(weights)
    if not 1 <= len(weights) <= HEAD_MAX_SHARDS:
        raise ValueError(f"1 to {HEAD_MAX_SHARDS} weight shards, got {len(weights)}")
    if _torch is None:
        _bind_torch()
    h = RelayHead()
    h.dtype, h.A = _dtype(hidden, "hidden"), len(weights)
    h.hidden = _matrix(hidden, "hidden")
    h.tokens, h.dim = hidden.shape
    h.hidden_stride = _row_stride(hidden)
    h.piece_bytes = piece_bytes
    for a, x in enumerate(weights):
        h.weight[a] = _matrix(x, f"weights[{a}]")
        h.rows[a] = x.shape[0]
        if x.dtype != hidden.dtype or x.shape[1] != h.dim:
            raise ValueError(f"weights[{a}] must be {hidden.dtype} with rows of {h.dim}")
    h.weight_stride = _common_stride(weights, "weight")
    if d_hidden is not None:
        if d_hidden.dtype != hidden.dtype or d_hidden.shape != hidden.shape:
            raise ValueError("d_hidden must have hidden's dtype and shape")
        h.d_hidden = _matrix(d_hidden, "d_hidden")
        h.d_hidden_stride = _row_stride(d_hidden)
    if d_weights is not None:
        d_weights = list(d_weights)
        if [tuple(x.shape) for x in d_weights] != [tuple(x.shape) for x in weights]:
            raise ValueError("d_weights must have the weights' shapes")
        for a, x in enumerate(d_weights):
            if x.dtype != hidden.dtype:
                raise ValueError(f"d_weights[{a}] must be {hidden.dtype}")
            h.d_weight[a] = _matrix(x, f"d_weights[{a}]")
        h.d_weight_stride = _common_stride(d_weights, "d_weight")
    h._tensors = (hidden, weights, d_hidden, d_weights)
    return h


def relay_head_workspace_size(head: RelayHead, top: int = 0) -> int:
    n = int(lib().relay_head_workspace_size(ctypes.byref(head), top))
    if n < 0:
        raise RelayError(ERR_INVALID_ARGUMENT, lib().relay_last_error().decode(errors="replace"))
    return n


def alloc_head_workspace(head: RelayHead, device, top: int = 0):
    """Workspace of relay_linear_xent (top = 0) or of relay_linear_distill with `top` entries."""
    import torch
    return torch.empty(relay_head_workspace_size(head, top), dtype=torch.uint8, device=device)


def relay_linear_xent(head: RelayHead, targets, loss, row_weight=None, workspace=None,
                      stream=None) -> None:
    """Cross entropy of the projection's logits against int32 targets (outside the vocabulary:
    the row is ignored), with the gradients the head asks for (see relay.h)."""
    if _torch is None:
        _bind_torch()
    t = (head.tokens,)
    if workspace is None:
        workspace = _own_workspace(lambda: alloc_head_workspace(head, loss.device), stream)
    _check(lib().relay_linear_xent(
        ctypes.byref(head), _array(targets, "targets", _int32, t),
        None if row_weight is None else _array(row_weight, "row_weight", _float32, t),
        _array(loss, "loss", _float32, t), *_space(workspace), _handle(stream)))


def relay_linear_distill(head: RelayHead, teacher_logits, teacher_index, temperature: float, loss,
                         row_weight=None, workspace=None, stream=None) -> None:
    """Distillation from a teacher's top logits [tokens, top] (fp32 or bf16) at the int32 ids
    teacher_index (outside the vocabulary: no entry), with the gradients the head asks for."""
    if _torch is None:
        _bind_torch()
    t, top = (head.tokens,), _columns(teacher_index, "teacher_index")
    if workspace is None:
        workspace = _own_workspace(lambda: alloc_head_workspace(head, loss.device, top), stream)
    code = _dtype(teacher_logits, "teacher_logits")
    _check(lib().relay_linear_distill(
        ctypes.byref(head), _array(teacher_logits, "teacher_logits", teacher_logits.dtype, t + (top,)),
        code, _array(teacher_index, "teacher_index", _int32, t + (top,)), top, temperature,
        None if row_weight is None else _array(row_weight, "row_weight", _float32, t),
        _array(loss, "loss", _float32, t), *_space(workspace), _handle(stream)))


def alloc_router_workspace(tokens: int, experts: int, device):
    """Workspace of relay_router_forward."""
    import torch
    n = int(lib().relay_router_workspace_size(tokens, experts))
    if n < 0:
        raise RelayError(ERR_INVALID_ARGUMENT, lib().relay_last_error().decode(errors="replace"))
    return torch.empty(n, dtype=torch.uint8, device=device)


# The router's calls pass their arguments as one block of 8-byte words: ctypes converts an argument
# in 0.2 us, so that fifteen of them took as long as the kernel of a small call.
_pack8, _pack13, _pack15 = (struct.Struct(f"{n}q").pack for n in (8, 13, 15))
_double_bits = struct.Struct("d")
_int64 = struct.Struct("q")


def _rows(x, name: str):
    """Address, rows, columns and row stride of a CUDA matrix whose rows are contiguous."""
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (device memory)")
    if x.dim() != 2:
        raise ValueError(f"{name} must be a matrix with contiguous rows")
    t, e = x.shape
    s0, s1 = x.stride()
    if s1 != 1 and e > 1:
        raise ValueError(f"{name} must be a matrix with contiguous rows")
    return x.data_ptr(), t, e, s0 if t > 1 else max(s0, e)


def relay_router_forward(logits, index, gate, counts, prob_sum, mask=None, normalize: bool = False,
                         workspace=None, stream=None) -> None:
    """Top-k experts of each row of logits [tokens, experts] (k = index.shape[1]), their gates, and
    the per-expert counts and probability sums (see relay.h). mask: bool or uint8 per row."""
    if _torch is None:
        _bind_torch()
    ptr, t, e, stride = _rows(logits, "logits")
    tk = (t, _columns(index, "index"))
    # `mask` stays the tensor: when nothing but the call holds it, the workspace below would take its memory
    mask_ptr = 0 if mask is None else _array(mask, "mask", _torch.bool if mask.dtype is _torch.bool else _torch.uint8, (t,))
    if workspace is None:
        workspace = _own_workspace(lambda: alloc_router_workspace(t, e, logits.device), stream)
    _check(lib().relay_packed_router_forward(_pack15(
        ptr, stride, _dtype(logits, "logits"), t, e, tk[1], bool(normalize), mask_ptr,
        _array(index, "index", _int32, tk), _array(gate, "gate", _float32, tk),
        _array(counts, "counts", _int32, (e,)), _array(prob_sum, "prob_sum", _float32, (e,)),
        *_space(workspace), _handle(stream))))


def relay_balance_loss(counts, prob_sum, top: int, coef: float, loss, d_prob, stream=None) -> None:
    """Balance loss of (possibly all-reduced) counts and probability sums, and its derivative by
    one token's probability of each expert."""
    if _torch is None:
        _bind_torch()
    e = counts.shape
    _check(lib().relay_packed_router_balance(_pack8(
        _array(counts, "counts", _int32, e), _array(prob_sum, "prob_sum", _float32, e), counts.numel(),
        top, _int64.unpack(_double_bits.pack(coef))[0], _array(loss, "loss", _float32, (1,)),
        _array(d_prob, "d_prob", _float32, e), _handle(stream))))


def relay_router_backward(logits, index, d_logits, d_gate=None, d_prob=None, normalize: bool = False,
                          stream=None) -> None:
    """Gradient of the router's logits from the gates' and the probabilities' (see relay.h)."""
    if _torch is None:
        _bind_torch()
    ptr, t, e, stride = _rows(logits, "logits")
    d_ptr, d_t, d_e, d_stride = _rows(d_logits, "d_logits")
    tk = (t, _columns(index, "index"))
    if d_logits.dtype is not logits.dtype or d_t != t or d_e != e:
        raise ValueError("d_logits must have the logits' dtype and shape")
    _check(lib().relay_packed_router_backward(_pack13(
        ptr, stride, _dtype(logits, "logits"), t, e, tk[1], bool(normalize), _array(index, "index", _int32, tk),
        0 if d_gate is None else _array(d_gate, "d_gate", _float32, tk),
        0 if d_prob is None else _array(d_prob, "d_prob", _float32, (e,)), d_ptr, d_stride, _handle(stream))))


# ------------------------------------------------- router with scores, bias and groups --

_pack_routing = struct.Struct("7if").pack
_pack10 = struct.Struct("10q").pack


def _routing(score, experts, groups, kept, top, group_sum, normalize, scale) -> bytes:
    if score not in SCORES:
        raise ValueError(f"score must be 'softmax' or 'sigmoid', got {score!r}")
    return _pack_routing(SCORES[score], experts, groups, groups if kept is None else kept, top, group_sum, bool(normalize), scale)


def relay_grouped_router_forward(logits, index, gate, counts, prob_sum, bias=None, mask=None, groups: int = 1,
                                 kept: Optional[int] = None, group_sum: int = 2, score: str = "sigmoid",
                                 normalize: bool = True, scale: float = 1.0, workspace=None, stream=None) -> None:
    """Top-k experts of each row of logits [tokens, experts] (k = index.shape[1]) by score + bias among the `kept` (None:
    all) best of `groups` groups, their gates (scores alone, renormalized and scaled), the per-expert counts and
    the sums of the scores' shares (see relay.h). workspace: alloc_router_workspace. mask: bool or uint8 per row."""
    if _torch is None:
        _bind_torch()
    ptr, t, e, stride = _rows(logits, "logits")
    tk = (t, _columns(index, "index"))
    how = _routing(score, e, groups, kept, tk[1], group_sum, normalize, scale)
    # `mask` stays the tensor: when nothing but the call holds it, the workspace below would take its memory
    mask_ptr = 0 if mask is None else _array(mask, "mask", _torch.bool if mask.dtype is _torch.bool else _torch.uint8, (t,))
    if workspace is None:
        workspace = _own_workspace(lambda: alloc_router_workspace(t, e, logits.device), stream)
    _check(lib().relay_packed_grouped_forward(how, _pack13(
        ptr, stride, _dtype(logits, "logits"), t, 0 if bias is None else _array(bias, "bias", _float32, (e,)), mask_ptr,
        _array(index, "index", _int32, tk), _array(gate, "gate", _float32, tk), _array(counts, "counts", _int32, (e,)),
        _array(prob_sum, "prob_sum", _float32, (e,)), *_space(workspace), _handle(stream))))


def relay_grouped_router_backward(logits, index, d_logits, d_gate=None, d_prob=None, score: str = "sigmoid",
                                  normalize: bool = True, scale: float = 1.0, stream=None) -> None:
    """Gradient of the logits of relay_grouped_router_forward from the gates' and the shares' (see relay.h)."""
    if _torch is None:
        _bind_torch()
    ptr, t, e, stride = _rows(logits, "logits")
    d_ptr, d_t, d_e, d_stride = _rows(d_logits, "d_logits")
    tk = (t, _columns(index, "index"))
    if d_logits.dtype is not logits.dtype or d_t != t or d_e != e:
        raise ValueError("d_logits must have the logits' dtype and shape")
    _check(lib().relay_packed_grouped_backward(_routing(score, e, 1, 1, tk[1], 1, normalize, scale), _pack10(
        ptr, stride, _dtype(logits, "logits"), t, _array(index, "index", _int32, tk),
        0 if d_gate is None else _array(d_gate, "d_gate", _float32, tk),
        0 if d_prob is None else _array(d_prob, "d_prob", _float32, (e,)), d_ptr, d_stride, _handle(stream))))


def relay_router_bias_update(counts, bias, rate: float, out=None, stream=None) -> None:
    """Raise the bias of experts chosen less often than the mean by `rate`, lower that of those chosen more often; in
    place, or into `out`."""
    if _torch is None:
        _bind_torch()
    e = counts.shape
    b = _array(bias, "bias", _float32, e)
    _check(lib().relay_router_bias_update(_array(counts, "counts", _int32, e), b, counts.numel(), rate,
                                          b if out is None else _array(out, "out", _float32, e), _handle(stream)))


# --------------------------------------------------------------- products in 8 bits --

def fp8_depth(rows: int, groups: int = 0) -> int:
    """Length of the transposed rows of relay_quantize_fp8: rows, or with groups room for each of them to start a
    block of 128."""
    n = int(lib().relay_fp8_depth(rows, groups))
    if n < 0:
        raise RelayError(ERR_INVALID_ARGUMENT, lib().relay_last_error().decode(errors="replace"))
    return n


def alloc_fp8(rows: int, cols: int, device, tiles: bool = False, batch: Optional[int] = None):
    """An 8-bit matrix [rows, cols] (or a batch of them) whose row stride the products accept, and its scales:
    [blocks of cols, rows], or with tiles [blocks of rows, blocks of cols] (with a batch in front)."""
    import torch
    lead = () if batch is None else (batch,)
    if batch is not None and not tiles:
        raise ValueError("a batch of matrices has tiles")
    kb = -(-cols // FP8_BLOCK)
    q = torch.empty(lead + (rows, max(-(-cols // 16) * 16, 16)), dtype=torch.float8_e4m3fn, device=device)[..., :cols]
    shape = lead + (-(-rows // FP8_BLOCK), kb) if tiles else (kb, rows)
    return q, torch.empty(shape, dtype=torch.float32, device=device)


def _batched(x, name: str):
    """Address, batch, rows, columns and row stride of a CUDA matrix, or of matrices one behind the other."""
    shape, strides = x.shape, x.stride()
    if not x.is_cuda or not 2 <= len(shape) <= 3:
        raise ValueError(f"{name} must be a CUDA matrix, or a batch of them (device memory)")
    r, c = shape[-2:]
    n, sn = (1, 0) if len(shape) == 2 else (shape[0], strides[0])
    ld = strides[-2] if r > 1 else max(sn, c) if n > 1 else max(strides[-2], c)
    if (c > 1 and strides[-1] != 1) or (n > 1 and sn != r * ld):
        raise ValueError(f"{name} must have contiguous rows, its matrices one behind the other")
    return x.data_ptr(), n, r, c, ld


def _fp8(x, name: str):
    if x.dtype is not _e4m3:
        raise ValueError(f"{name} must be float8_e4m3fn, got {x.dtype}")
    return _batched(x, name)


def _scales(x, name: str, shape) -> int:
    """A leading dimension of 1 may be there or not."""
    if x.shape != shape:
        if x.dim() == len(shape) + 1 and x.shape[0] == 1:
            x = x[0]
        elif len(shape) == x.dim() + 1 and shape[0] == 1:
            shape = shape[1:]
    return _array(x, name, _float32, shape)


def _offset(offset):
    if offset is None:
        return 0, 0
    if offset.dim() != 1 or offset.shape[0] < 2:
        raise ValueError(f"offset must be int32 [groups + 1], got {tuple(offset.shape)}")
    return _array(offset, "offset", _int32, offset.shape), offset.shape[0] - 1


_pack_fp8 = struct.Struct("12q4i").pack


def relay_quantize_fp8(x, q=None, scale=None, qt=None, scale_t=None, tiles: bool = False, tiles_t: bool = False,
                       offset=None, stream=None) -> None:
    """x [rows, cols] (or a batch of matrices) to 8 bits with a power of two for each block of 128: as it lies (q,
    scale), transposed (qt, scale_t), or both; allocate them with alloc_fp8. offset (int32, device memory): the rows
    belong to groups, each of which starts a block of qt's rows of length fp8_depth(rows, groups) (see relay.h)."""
    if _torch is None:
        _bind_torch()
    ptr, n, r, c, ld = _batched(x, "x")
    off, groups = _offset(offset)
    rb, cb = -(-r // FP8_BLOCK), -(-c // FP8_BLOCK)
    if q is None and qt is None:
        raise ValueError("neither q nor qt is given")
    q_ptr = s_ptr = q_ld = qt_ptr = st_ptr = qt_ld = 0
    if q is not None:
        q_ptr, q_n, q_r, q_c, q_ld = _fp8(q, "q")
        if (q_n, q_r, q_c) != (n, r, c) or scale is None:
            raise ValueError(f"q must have x's shape, and come with scale: got {tuple(q.shape)}")
        s_ptr = _scales(scale, "scale", (n, rb, cb) if tiles else (cb, r))
    if qt is not None:
        qt_ptr, q_n, q_r, q_c, qt_ld = _fp8(qt, "qt")
        depth = r if groups == 0 else fp8_depth(r, groups)
        if (q_n, q_r, q_c) != (n, c, depth) or scale_t is None:
            raise ValueError(f"qt must be {(n, c, depth)}, and come with scale_t: got {tuple(qt.shape)}")
        db = -(-depth // FP8_BLOCK)
        st_ptr = _scales(scale_t, "scale_t", (n, cb, db) if tiles_t else (db, c))
    _check(lib().relay_quantize_fp8(_pack_fp8(ptr, ld, n, r, c, q_ptr, q_ld, s_ptr, qt_ptr, qt_ld, st_ptr, off, groups,
                                              _dtype(x, "x"), bool(tiles), bool(tiles_t)), _handle(stream)))


def _matmul_fp8_words(a, a_scale, b, b_scale, out, offset, by_depth) -> bytes:
    if _torch is None:
        _bind_torch()
    a_ptr, a_n, r, d, a_ld = _fp8(a, "a")
    b_ptr, b_n, n, b_d, b_ld = _fp8(b, "b")
    off, groups = _offset(offset)
    kb, nb, many = -(-d // FP8_BLOCK), -(-n // FP8_BLOCK), max(groups, 1)
    if a_n != 1 or b_d != d or b_n != (1 if by_depth else many):
        raise ValueError(f"a must be [rows, depth] and b [{'' if by_depth or not groups else 'groups, '}cols, depth]: "
                         f"got {tuple(a.shape)} and {tuple(b.shape)} for {groups} groups")
    out_ptr, o_n, o_r, o_c, o_ld = _batched(out, "out")
    if (o_n, o_r, o_c) != (many if by_depth else 1, r, n):
        raise ValueError(f"out must be {(many, r, n) if by_depth else (r, n)}, got {tuple(out.shape)}")
    return _pack_fp8(a_ptr, a_ld, _scales(a_scale, "a_scale", (kb, r)), b_ptr, b_ld,
                     _scales(b_scale, "b_scale", (b_n, nb, kb)), out_ptr, o_ld, r, n, d, off, groups, _dtype(out, "out"),
                     bool(by_depth), 0)


def relay_matmul_fp8(a, a_scale, b, b_scale, out, offset=None, by_depth: bool = False, stream=None) -> None:
    """out[r, n] = sum_d a[r, d] b[n, d] of 8-bit matrices: a row-scaled, b tile-scaled (see relay_quantize_fp8). With
    offset, rows belong to groups and meet their group's b [groups, cols, depth]; with by_depth the groups are
    stretches of the depth, and out is [groups, rows, cols] (see relay.h)."""
    _check(lib().relay_matmul_fp8(_matmul_fp8_words(a, a_scale, b, b_scale, out, offset, by_depth), _handle(stream)))


# ------------------------------------------------------------- all gradients at once --

def make_grads(tensors: Sequence) -> RelayGrads:
    """Describe a list of contiguous CUDA tensors (fp32 and bf16, any shapes) for relay_grad_norm and
    relay_grad_clip. The tensors must outlive the list (it keeps references), and it can be used for any
    number of calls."""
    if _torch is None:
        _bind_torch()
    tensors = list(tensors)
    for i, x in enumerate(tensors):
        if not x.is_cuda or not x.is_contiguous():
            raise ValueError(f"tensors[{i}] must be a contiguous CUDA tensor (device memory)")
    n = len(tensors)
    g = RelayGrads()
    g.n = n
    # assigned, the arrays live as long as the list; nothing here refers back to it (a cycle would hold the tensors until a
    # garbage collection, which device memory does not bring about)
    g.grad = (ctypes.c_void_p * max(n, 1))(*[x.data_ptr() for x in tensors])
    g.count = (ctypes.c_size_t * max(n, 1))(*[x.numel() for x in tensors])
    g.dtype = (ctypes.c_int32 * max(n, 1))(*[_dtype(x, f"tensors[{i}]") for i, x in enumerate(tensors)])
    g._tensors = tensors
    return g


def alloc_grad_workspace(grads: RelayGrads, device):
    """Workspace of relay_grad_norm."""
    import torch
    n = int(lib().relay_grad_workspace_size(ctypes.byref(grads)))
    if n < 0:
        raise RelayError(ERR_INVALID_ARGUMENT, lib().relay_last_error().decode(errors="replace"))
    return torch.empty(n, dtype=torch.uint8, device=device)


def relay_grad_norm(grads: RelayGrads, norm, workspace=None, stream=None) -> None:
    """norm[0] = the 2-norm over all tensors of the list (see relay.h)."""
    if _torch is None:
        _bind_torch()
    if workspace is None:
        workspace = _own_workspace(lambda: alloc_grad_workspace(grads, norm.device), stream)
    _check(lib().relay_grad_norm(ctypes.byref(grads), _array(norm, "norm", _float32, (1,)), *_space(workspace),
                                 _handle(stream)))


def relay_grad_clip(grads: RelayGrads, norm, max_norm: float, out: Optional[RelayGrads] = None, stream=None) -> None:
    """Scale every tensor by min(1, max_norm / (norm[0] + 1e-6)), in place or into the tensors of `out`."""
    if _torch is None:
        _bind_torch()
    _check(lib().relay_grad_clip(ctypes.byref(grads), None if out is None else ctypes.byref(out),
                                 _array(norm, "norm", _float32, (1,)), max_norm, _handle(stream)))
