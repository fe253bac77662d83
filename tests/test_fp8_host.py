"""Refusals of the 8-bit quantization and product: host-side checks that launch nothing (device addresses are made
up), and what the Python calls refuse before them."""
import struct

import pytest
import torch

import pack_virtual_rank_gb300 as rv

BASE = 1 << 40
far = [BASE + (i << 36) for i in range(8)]
QUANT = dict(x=far[0], x_stride=300, batch=1, rows=200, cols=300, q=far[1], q_stride=304, scale=far[2], qt=far[3], qt_stride=208,
             scale_t=far[4], offset=0, groups=0, dtype=rv.BF16, tiles=0, tiles_t=0)
PROD = dict(a=far[0], a_stride=304, a_scale=far[1], b=far[2], b_stride=304, b_scale=far[3], out=far[4], out_stride=100, rows=200, cols=100,
            depth=300, offset=0, groups=0, out_dtype=rv.BF16, by_depth=0, reserved=0)


def call(name, base, **change):
    d = dict(base, **change)
    st = getattr(rv.lib(), name)(struct.pack("12q4i", *d.values()), None)
    return st, rv.lib().relay_last_error().decode()


def refused(answer, words):
    st, text = answer
    assert st == rv.ERR_INVALID_ARGUMENT and words in text, (st, text)


@pytest.mark.parametrize("change,words", [
    (dict(dtype=rv.I32), "dtype"), (dict(rows=-1), "rows or cols"), (dict(rows=2 ** 22 + 1), "rows or cols"), (dict(cols=0), "rows or cols"),
    (dict(batch=-1), "batch"), (dict(batch=1025), "batch"), (dict(groups=1025, offset=far[5]), "groups out of range"),
    (dict(groups=2), "go together"), (dict(offset=far[5]), "go together"), (dict(q=0, qt=0), "neither q nor qt"),
    (dict(scale=0), "a scale is NULL"), (dict(scale_t=0), "a scale is NULL"), (dict(batch=2), "a batch of matrices"),
    (dict(batch=2, tiles=1), "a batch of matrices"), (dict(offset=far[5], groups=2, tiles=1), "tiles of rows in groups"),
    (dict(x=0), "x is NULL"), (dict(x_stride=299), "x_stride"), (dict(q_stride=296), "q_stride"), (dict(q_stride=310), "q_stride"),
    (dict(qt_stride=192), "qt_stride"), (dict(x=far[0] + 1), "element-aligned"), (dict(scale=far[2] + 2), "element-aligned"),
    (dict(q=far[1] + 8), "16-byte"), (dict(qt=far[3] + 4), "16-byte"), (dict(q=far[0] + 16), "overlaps"), (dict(qt=far[1]), "overlaps"),
    (dict(scale_t=far[2]), "overlaps"), (dict(offset=far[5], groups=2, qt_stride=272), "qt_stride"),
])
def test_quantize_refusals(relay_lib, change, words):
    refused(call("relay_quantize_fp8", QUANT, **change), words)


@pytest.mark.parametrize("change,words", [
    (dict(out_dtype=rv.I32), "out_dtype"), (dict(rows=-1), "rows or cols"), (dict(cols=0), "rows or cols"), (dict(depth=-1), "depth"),
    (dict(groups=-1), "groups out of range"), (dict(groups=2), "go together"), (dict(offset=far[5]), "go together"),
    (dict(by_depth=1, offset=far[5], groups=2), "whole blocks"), (dict(out=0), "out is NULL"), (dict(a=0), "a scale is NULL"),
    (dict(b_scale=0), "a scale is NULL"), (dict(a=far[0] + 8), "16-byte"), (dict(b=far[2] + 1), "16-byte"), (dict(a_stride=300), "a_stride"),
    (dict(b_stride=288), "b_stride"), (dict(out_stride=99), "out_stride"), (dict(out=far[4] + 1), "element-aligned"),
    (dict(a_scale=far[1] + 2), "element-aligned"), (dict(out=far[0] + 64), "out overlaps a"), (dict(out=far[2]), "out overlaps b"),
    (dict(out=far[1]), "out overlaps a_scale"), (dict(out=far[3] + 4), "out overlaps b_scale"),
    (dict(cols=2 ** 22, out_stride=2 ** 22, groups=1024, offset=far[5]), "2^31"),
])
def test_product_refusals(relay_lib, change, words):
    refused(call("relay_matmul_fp8", PROD, **change), words)


def test_more_tiles_than_are_numbered(relay_lib):
    n = 2 ** 22
    st, text = call("relay_matmul_fp8", PROD, rows=n, cols=n, out_stride=n, a=1 << 50, b=1 << 51, a_scale=1 << 52, b_scale=1 << 53,
                    out=1 << 54)
    assert st == rv.ERR_UNSUPPORTED and "2^28 tiles" in text


def test_nothing_to_do(relay_lib):
    assert call("relay_quantize_fp8", QUANT, rows=0)[0] == rv.OK
    assert call("relay_quantize_fp8", QUANT, batch=0, tiles=1, tiles_t=1)[0] == rv.OK
    assert call("relay_matmul_fp8", PROD, rows=0)[0] == rv.OK


def test_depth(relay_lib):
    assert rv.fp8_depth(1000) == 1000
    assert rv.fp8_depth(1000, 4) == 128 * (7 + 4) and rv.fp8_depth(3, 8) == 128 * 3 and rv.fp8_depth(0, 8) == 0
    for rows, groups in ((-1, 0), (5, -1), (5, 1025), (2 ** 22 + 1, 0)):
        with pytest.raises(rv.RelayError, match="out of range"):
            rv.fp8_depth(rows, groups)
    # no offsets need more: every group a short last block
    for rows, groups in ((1000, 4), (127, 3), (129, 2), (4096, 32), (5, 9)):
        worst = max(sum(-(-n // 128) for n in [1] * k + [rows - k]) for k in range(min(groups, rows)))
        assert 128 * worst <= rv.fp8_depth(rows, groups)


class Device:
    """A host tensor that says it is device memory."""
    is_cuda = True

    def __init__(self, x):
        self._x = x

    def __getattr__(self, name):
        return getattr(self._x, name)


def dev(*shape, dtype=torch.float32):
    return Device(torch.zeros(*shape, dtype=dtype))


E = torch.float8_e4m3fn


def test_binding_refusals(relay_lib):
    x = dev(6, 40)
    with pytest.raises(ValueError, match="neither q nor qt"):
        rv.relay_quantize_fp8(x, stream=0)
    with pytest.raises(ValueError, match="q must be float8_e4m3fn"):
        rv.relay_quantize_fp8(x, dev(6, 40), dev(1, 6), stream=0)
    with pytest.raises(ValueError, match="q must have x's shape"):
        rv.relay_quantize_fp8(x, dev(6, 41, dtype=E), dev(1, 6), stream=0)
    with pytest.raises(ValueError, match="come with scale"):
        rv.relay_quantize_fp8(x, dev(6, 40, dtype=E), stream=0)
    with pytest.raises(ValueError, match="scale must be"):
        rv.relay_quantize_fp8(x, dev(6, 40, dtype=E), dev(6, 1), stream=0)
    with pytest.raises(ValueError, match="qt must be"):
        rv.relay_quantize_fp8(x, qt=dev(40, 6, dtype=E), scale_t=dev(1, 40), offset=dev(3, dtype=torch.int32), stream=0)
    with pytest.raises(ValueError, match="offset must be"):
        rv.relay_quantize_fp8(x, qt=dev(40, 6, dtype=E), scale_t=dev(1, 40), offset=dev(1, dtype=torch.int32), stream=0)
    with pytest.raises(ValueError, match="device memory"):
        rv.relay_quantize_fp8(torch.zeros(6, 40), dev(6, 40, dtype=E), dev(1, 6), stream=0)
    a, b, out = dev(6, 48, dtype=E), dev(10, 48, dtype=E), dev(6, 10)
    with pytest.raises(ValueError, match="a must be"):
        rv.relay_matmul_fp8(a, dev(1, 6), dev(10, 32, dtype=E), dev(1, 1), out, stream=0)
    with pytest.raises(ValueError, match="a must be"):
        rv.relay_matmul_fp8(a, dev(1, 6), b, dev(1, 1), out, offset=dev(4, dtype=torch.int32), stream=0)
    with pytest.raises(ValueError, match="out must be"):
        rv.relay_matmul_fp8(a, dev(1, 6), b, dev(1, 1), dev(6, 11), stream=0)
    with pytest.raises(ValueError, match="a_scale must be"):
        rv.relay_matmul_fp8(a, dev(6, 1), b, dev(1, 1), out, stream=0)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        rv.relay_matmul_fp8(a, dev(1, 6), b, dev(1, 1), dev(6, 10, dtype=torch.float16), stream=0)
    with pytest.raises(ValueError, match="a batch of matrices has tiles"):
        rv.alloc_fp8(4, 4, "cpu", batch=2)
