"""A list of gradients holds its tensors as long as it lives itself, and no longer: without the cyclic collector."""
import ctypes
import gc
import weakref

import torch

import pack_virtual_rank_gb300 as rv


class Device:
    """A host tensor that says it is device memory."""
    is_cuda = True

    def __init__(self, x):
        self._x = x

    def __getattr__(self, name):
        return getattr(self._x, name)


def test_a_dropped_list_frees_its_tensors(relay_lib):
    types = [t * 2 for t in (ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32)]   # the tables' types are cycles themselves
    gc.collect()
    gc.disable()
    try:
        xs = [Device(torch.zeros(5)), Device(torch.zeros(3, dtype=torch.bfloat16))]
        held = [weakref.ref(x) for x in xs]
        grads = rv.make_grads(xs)
        del xs
        assert all(h() is not None for h in held)
        assert (grads.n, grads.count[0], grads.count[1], grads.dtype[0], grads.dtype[1]) == (2, 5, 3, rv.F32, rv.BF16)
        assert grads.grad[0] == held[0]().data_ptr() and grads.grad[1] == held[1]().data_ptr()
        assert rv.lib().relay_grad_workspace_size(ctypes.byref(grads)) > 0
        of_list = weakref.ref(grads)
        del grads
        assert of_list() is None
        assert all(h() is None for h in held)
        assert gc.collect() == 0 and len(types) == 3       # nor do the list's tables wait for it
    finally:
        gc.enable()


def test_a_list_of_none(relay_lib):
    grads = rv.make_grads([])
    assert grads.n == 0 and rv.lib().relay_grad_workspace_size(ctypes.byref(grads)) == 8
