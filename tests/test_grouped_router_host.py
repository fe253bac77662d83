"""Refusals of the router with scores, bias and groups: host-side checks that launch nothing (device addresses are made
up), and what the Python calls refuse before them."""
import math
import struct

import pytest
import torch

import pack_virtual_rank_gb300 as rv

BASE = 1 << 40
far = [BASE + (i << 36) for i in range(10)]
HOW = dict(score=1, experts=64, groups=8, kept=4, top=6, group_sum=2, normalize=1, scale=1.0)
FWD = dict(logits=far[0], stride=64, dtype=rv.F32, tokens=100, bias=far[1], mask=0, index=far[2], gate=far[3], counts=far[4],
           prob_sum=far[5], ws=far[6], size=1 << 24, stream=0)
BWD = dict(logits=far[0], stride=64, dtype=rv.F32, tokens=100, index=far[2], d_gate=far[3], d_prob=far[4], d_logits=far[5], d_stride=64,
           stream=0)


def call(name, base, **change):
    how = dict(HOW, **{k: v for k, v in change.items() if k in HOW})
    d = dict(base, **{k: v for k, v in change.items() if k not in HOW})
    st = getattr(rv.lib(), "relay_packed_grouped_" + name)(struct.pack("7if", *how.values()), struct.pack(f"{len(d)}q", *d.values()))
    return st, rv.lib().relay_last_error().decode()


def refused(answer, words):
    st, text = answer
    assert st == rv.ERR_INVALID_ARGUMENT and words in text, (st, text)


SHARED = [
    (dict(score=2), "score"), (dict(experts=0), "experts"), (dict(experts=1025), "experts"), (dict(groups=0), "groups"),
    (dict(groups=33), "groups"), (dict(groups=7), "divide"), (dict(kept=0), "kept"), (dict(kept=9), "kept"),
    (dict(experts=520, stride=520, d_stride=520), "up to 512"), (dict(group_sum=0), "group_sum"), (dict(group_sum=3), "group_sum"),
    (dict(top=0), "top"), (dict(top=33), "top"), (dict(top=9, kept=1), "top"), (dict(scale=math.inf), "scale"),
    (dict(scale=math.nan), "scale"), (dict(dtype=rv.I32), "dtype"), (dict(tokens=-1), "tokens"), (dict(tokens=2 ** 31), "tokens"),
    (dict(stride=63), "stride"), (dict(stride=2 ** 32), "stride"), (dict(logits=0), "NULL"), (dict(index=0), "NULL"),
    (dict(logits=far[0] + 2), "element-aligned"), (dict(index=far[2] + 1), "element-aligned")]


@pytest.mark.parametrize("change,words", SHARED + [
    (dict(gate=0), "NULL"), (dict(counts=0), "NULL"), (dict(ws=0), "workspace is NULL"), (dict(size=64), "are needed"),
    (dict(bias=far[1] + 2), "element-aligned"), (dict(index=far[0] + 64), "overlaps"), (dict(bias=far[4]), "overlaps"),
    (dict(prob_sum=far[1] + 4), "overlaps"), (dict(ws=far[3]), "overlaps"), (dict(mask=far[2]), "overlaps")])
def test_forward_refusals(relay_lib, change, words):
    change = {k: v for k, v in change.items() if k in HOW or k in FWD}
    refused(call("forward", FWD, **change), words)


@pytest.mark.parametrize("change,words", SHARED + [
    (dict(d_logits=0), "NULL"), (dict(d_stride=63), "stride"), (dict(d_logits=far[0]), "overlaps"), (dict(d_logits=far[3]), "overlaps"),
    (dict(d_gate=far[3] + 1), "element-aligned")])
def test_backward_refusals(relay_lib, change, words):
    refused(call("backward", BWD, **change), words)


def test_bias_update_refusals(relay_lib):
    def update(counts=far[0], bias=far[1], experts=8, rate=0.1, out=far[2]):
        st = rv.lib().relay_router_bias_update(counts, bias, experts, rate, out, None)
        return st, rv.lib().relay_last_error().decode()
    refused(update(counts=None), "NULL")
    refused(update(out=None), "NULL")
    refused(update(experts=0), "experts")
    refused(update(rate=math.nan), "rate")
    refused(update(out=far[1] + 4), "overlaps")
    refused(update(out=far[0]), "overlaps")
    refused(update(bias=far[1] + 2), "element-aligned")


def test_nothing_to_do(relay_lib):
    assert call("backward", BWD, tokens=0)[0] == rv.OK


class Device:
    """A host tensor that says it is device memory."""
    is_cuda = True

    def __init__(self, x):
        self._x = x

    def __getattr__(self, name):
        return getattr(self._x, name)


def dev(*shape, dtype=torch.float32):
    return Device(torch.zeros(*shape, dtype=dtype))


def test_binding_refusals(relay_lib):
    x, index, gate = dev(6, 8), dev(6, 2, dtype=torch.int32), dev(6, 2)
    counts, prob = dev(8, dtype=torch.int32), dev(8)
    with pytest.raises(ValueError, match="score must be"):
        rv.relay_grouped_router_forward(x, index, gate, counts, prob, score="tanh", stream=0)
    with pytest.raises(ValueError, match="index must be a matrix"):
        rv.relay_grouped_router_forward(x, dev(6, dtype=torch.int32), gate, counts, prob, stream=0)
    with pytest.raises(ValueError, match="bias must be"):
        rv.relay_grouped_router_forward(x, index, gate, counts, prob, bias=dev(7), workspace=dev(1000), stream=0)
    with pytest.raises(ValueError, match="workspace must be"):
        rv.relay_grouped_router_forward(x, index, gate, counts, prob, workspace=torch.zeros(10), stream=0)
    with pytest.raises(ValueError, match="d_logits must have"):
        rv.relay_grouped_router_backward(x, index, dev(6, 7), stream=0)
    with pytest.raises(ValueError, match="out must be"):
        rv.relay_router_bias_update(counts, prob, 0.1, dev(7), stream=0)
    with pytest.raises(ValueError, match="counts must be"):
        rv.relay_router_bias_update(prob, prob, 0.1, stream=0)
