"""Refusals of the losses and the router, and the sizes they ask for: host-side checks that launch
nothing (device addresses are made up and never read)."""
import ctypes

import pytest

import pack_virtual_rank_gb300 as rv

BASE = 1 << 40


def head(tokens=100, dim=64, rows=(300, 200), dtype=rv.BF16, grads=True):
    h = rv.RelayHead()
    h.dtype, h.A, h.tokens, h.dim = dtype, len(rows), tokens, dim
    h.hidden, h.hidden_stride = BASE, dim
    h.weight_stride = h.d_weight_stride = dim
    for a, r in enumerate(rows):
        h.rows[a] = r
        h.weight[a] = BASE + ((a + 1) << 32)
        if grads:
            h.d_weight[a] = BASE + ((a + 17) << 32)
    if grads:
        h.d_hidden, h.d_hidden_stride = BASE + (40 << 32), dim
    return h


def xent(h, targets=BASE + (50 << 32), loss=BASE + (51 << 32), workspace=BASE + (52 << 32), size=None):
    L = rv.lib()
    if size is None:
        size = L.relay_head_workspace_size(ctypes.byref(h), 0) if h is not None else 0
    st = L.relay_linear_xent(ctypes.byref(h) if h is not None else None, targets, None, loss, workspace,
                             size, None)
    return st, L.relay_last_error().decode()


def refused(answer, words):
    st, text = answer
    assert st == rv.ERR_INVALID_ARGUMENT, text
    assert words in text, text


def test_head_struct_matches_header(relay_lib):
    assert ctypes.sizeof(rv.RelayHead) == 8 + 2 * 8 + 2 * 8 + 8 * 8 + 8 * 8 + 8 + 2 * 8 + 8 * 8 + 2 * 8


@pytest.mark.parametrize("field,value,words", [
    ("dtype", rv.I32, "dtype"), ("A", 0, "shards"), ("A", 9, "shards"), ("tokens", -1, "tokens"),
    ("tokens", 2 ** 31, "tokens"), ("dim", 0, "dim"), ("piece_bytes", -1, "piece_bytes"),
    ("hidden", 0, "hidden is NULL"), ("hidden", BASE + 1, "element-aligned"),
    ("hidden_stride", 63, "stride"), ("weight_stride", 63, "stride"), ("d_hidden_stride", 63, "d_hidden_stride"),
    ("d_weight_stride", 1, "d_weight_stride"), ("d_hidden", BASE + 64, "overlaps"),
    ("d_hidden", BASE + (51 << 32), "overlaps"), ("hidden_stride", 2 ** 32, "stride"),
])
def test_head_refusals(relay_lib, field, value, words):
    h = head()
    size = rv.relay_head_workspace_size(h)
    setattr(h, field, value)
    refused(xent(h, size=size), words)


def test_head_refusals_of_shards_and_arrays(relay_lib):
    refused(xent(None), "head is NULL")
    for rows, words in (((-1, 5), "rows[0]"), ((0, 0), "empty"), ((2 ** 31 - 1, 1), "more than")):
        refused(xent(head(rows=rows), size=1 << 40), words)
    h = head()
    h.weight[1] = None
    refused(xent(h), "weight[1] is NULL")
    h = head()
    h.d_weight[0] = None
    refused(xent(h), "d_weight[0] is NULL")
    h = head()
    h.d_weight[1] = h.weight[0]
    refused(xent(h), "overlaps")
    refused(xent(head(), targets=None), "targets is NULL")
    refused(xent(head(), loss=None), "loss is NULL")
    refused(xent(head(), loss=BASE + 2), "element-aligned")
    refused(xent(head(), workspace=None), "workspace is NULL")
    n = rv.relay_head_workspace_size(head())
    refused(xent(head(), size=n - 1), "are needed")
    refused(xent(head(), workspace=BASE - 100), "overlaps")


def test_distill_refusals(relay_lib):
    L, far = rv.lib(), BASE + (60 << 32)

    def call(top=4, tau=1.0, dtype=rv.F32, logits=far, index=far + (1 << 32)):
        h = head()
        st = L.relay_linear_distill(ctypes.byref(h), logits, dtype, index, top, tau, None, far + (2 << 32),
                                    far + (3 << 32), 1 << 40, None)
        return st, L.relay_last_error().decode()
    for top in (0, -1, 129):
        refused(call(top=top), "top")
    for tau in (0.0, -1.0, float("inf"), float("nan"), 1e-42):
        refused(call(tau=tau), "temperature")
    refused(call(dtype=rv.I32), "teacher_dtype")
    refused(call(logits=None), "teacher_logits is NULL")
    refused(call(index=None), "teacher_index is NULL")
    refused(call(logits=far + 1), "element-aligned")


def test_workspace_size_is_bounded(relay_lib):
    """The logits are never kept: the workspace grows with the piece, not with the vocabulary."""
    small = rv.relay_head_workspace_size(head(8192, 1024, (200000,)))
    big = rv.relay_head_workspace_size(head(8192, 1024, (1600000,)))
    logits = 8192 * 1600000 * 2
    assert big - small < logits // 20 and big < logits // 8
    h = head(8192, 1024, (200000,))
    h.piece_bytes = 64 << 20
    assert rv.relay_head_workspace_size(h) < small - (900 << 20)
    assert rv.lib().relay_head_workspace_size(None, 0) == -1


def test_router_refusals(relay_lib):
    L, far = rv.lib(), BASE

    def fwd(dtype=rv.F32, tokens=10, experts=8, top=2, stride=None, logits=far, index=far + (1 << 32),
            counts=far + (3 << 32), ws=far + (5 << 32), size=1 << 20):
        st = L.relay_router_forward(logits, experts if stride is None else stride, dtype, tokens, experts, top, 0,
                                    None, index, far + (2 << 32), counts, far + (4 << 32), ws, size, None)
        return st, L.relay_last_error().decode()
    refused(fwd(dtype=rv.I32), "dtype")
    refused(fwd(tokens=-1), "tokens")
    for experts in (0, 1025):
        refused(fwd(experts=experts, top=1), "experts")
    for top in (0, 9, 33):
        refused(fwd(top=top), "top")
    refused(fwd(stride=7), "row_stride")
    refused(fwd(logits=None), "NULL")
    refused(fwd(counts=None), "NULL")
    refused(fwd(ws=None), "workspace is NULL")
    refused(fwd(size=3), "are needed")
    refused(fwd(index=far + 8), "overlaps")
    refused(fwd(logits=far + 2), "element-aligned")

    def bwd(d=far + (8 << 32), d_stride=8, top=2):
        st = L.relay_router_backward(far, 8, rv.F32, 10, 8, top, 0, far + (1 << 32), None, None, d, d_stride, None)
        return st, L.relay_last_error().decode()
    refused(bwd(d=None), "NULL")
    refused(bwd(d=far), "overlaps")
    refused(bwd(d_stride=7), "stride")
    refused(bwd(top=9), "top")
    st = L.relay_balance_loss(far, far + (1 << 32), 8, 2, 1.0, far + 4, far + (2 << 32), None)
    refused((st, L.relay_last_error().decode()), "overlaps")
    st = L.relay_balance_loss(None, far, 8, 2, 1.0, far + (1 << 32), far + (2 << 32), None)
    refused((st, L.relay_last_error().decode()), "NULL")


def test_binding_refuses_host_and_wrong_tensors(relay_lib):
    import torch
    h, w = torch.zeros(4, 8), torch.zeros(10, 8)
    with pytest.raises(ValueError, match="device memory"):
        rv.make_head(h, [w])
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        rv.make_head(h.half(), [w.half()])
    with pytest.raises(ValueError, match="shards"):
        rv.make_head(h, [])
    with pytest.raises(ValueError, match="device memory"):
        rv.relay_router_backward(h, torch.zeros(4, 2), h)
