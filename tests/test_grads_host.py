"""Refusals of the gradient norm and clipping: host-side checks that launch nothing (device addresses are made up)."""
import ctypes

import pytest
import torch

import pack_virtual_rank_gb300 as rv

BASE = 1 << 40
NORM, WS = BASE + (90 << 32), BASE + (91 << 32)


def grads(ptrs=(BASE, BASE + 4096), counts=(100, 50), dtypes=(rv.F32, rv.BF16), n=None):
    g = rv.RelayGrads()
    k = len(ptrs)
    g.n = k if n is None else n
    g._keep = ((ctypes.c_void_p * k)(*ptrs), (ctypes.c_size_t * k)(*counts), (ctypes.c_int32 * k)(*dtypes))
    g.grad = ctypes.cast(g._keep[0], ctypes.POINTER(ctypes.c_void_p))
    g.count = ctypes.cast(g._keep[1], ctypes.POINTER(ctypes.c_size_t))
    g.dtype = ctypes.cast(g._keep[2], ctypes.POINTER(ctypes.c_int32))
    return g


def refused(st, words):
    text = rv.lib().relay_last_error().decode()
    assert st == rv.ERR_INVALID_ARGUMENT and words in text, (st, text)


def norm(g, out=NORM, ws=WS, size=1 << 20):
    return rv.lib().relay_grad_norm(None if g is None else ctypes.byref(g), out, ws, size, None)


def clip(g, out=None, n=NORM, most=1.0):
    return rv.lib().relay_grad_clip(None if g is None else ctypes.byref(g), None if out is None else ctypes.byref(out), n, most, None)


@pytest.mark.parametrize("call", [norm, clip])
def test_lists_that_are_refused(relay_lib, call):
    refused(call(None), "grads is NULL")
    refused(call(grads(n=-1)), "number of tensors")
    refused(call(grads(n=(1 << 20) + 1)), "number of tensors")
    refused(call(grads(dtypes=(rv.F32, rv.I32))), "grads[1]: dtype")
    refused(call(grads(ptrs=(None, BASE))), "grads[0] is NULL")
    refused(call(grads(ptrs=(BASE + 2, BASE + 4096))), "element-aligned")
    refused(call(grads(counts=(1 << 43, 1))), "2^42")
    g = rv.RelayGrads()
    g.n = 1
    refused(call(g), "an array is NULL")
    assert rv.lib().relay_grad_workspace_size(ctypes.byref(g)) == -1
    assert rv.lib().relay_grad_workspace_size(None) == -1


def test_norm_refusals(relay_lib):
    refused(norm(grads(), out=None), "norm is NULL")
    refused(norm(grads(), out=NORM + 2), "element-aligned")
    refused(norm(grads(), ws=None), "workspace is NULL")
    refused(norm(grads(), size=8), "are needed")
    refused(norm(grads(), out=BASE + 396), "overlap")
    refused(norm(grads(), ws=BASE - 4), "overlap")
    refused(norm(grads(), out=WS), "overlap")


def test_clip_refusals(relay_lib):
    for most in (0.0, -1.0, float("inf"), float("nan")):
        refused(clip(grads(), most=most), "max_norm")
    refused(clip(grads(), n=None), "norm is NULL")
    refused(clip(grads(), n=BASE + 8), "overlaps")
    refused(clip(grads(ptrs=(BASE, BASE + 396))), "overlaps")
    far = BASE + (1 << 36)
    refused(clip(grads(), grads(ptrs=(far,), counts=(100,), dtypes=(rv.F32,))), "as many tensors")
    refused(clip(grads(), grads(ptrs=(far, far + 4096), counts=(100, 51))), "out[1]")
    refused(clip(grads(), grads(ptrs=(far, far + 4096), dtypes=(rv.F32, rv.F32))), "out[1]")
    refused(clip(grads(), grads(ptrs=(far, far + 4))), "overlaps")
    refused(clip(grads(), grads(ptrs=(BASE + 4, far))), "overlaps")            # shifted onto its own input
    refused(clip(grads(), grads(ptrs=(BASE + 4096, BASE))), "overlaps")        # onto each other's


def test_binding_refuses_other_tensors(relay_lib):
    with pytest.raises(ValueError, match=r"tensors\[0\] must be a contiguous CUDA tensor"):
        rv.make_grads([torch.zeros(3)])
