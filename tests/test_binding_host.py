"""What the Python calls of the losses and the router refuse before they reach the library. Tensors that claim to
be on a device stand for the arguments that are right: no GPU is needed, and nothing may be launched on them."""
import pytest
import torch

import pack_virtual_rank_gb300 as rv


class Device:
    """A host tensor that says it is device memory."""
    is_cuda = True

    def __init__(self, x):
        self._x = x

    def __getattr__(self, name):
        return getattr(self._x, name)


def dev(*shape, dtype=torch.float32):
    return Device(torch.zeros(*shape, dtype=dtype))


def head():
    return rv.make_head(dev(6, 8), [dev(10, 8)])


def xent(workspace):
    rv.relay_linear_xent(head(), dev(6, dtype=torch.int32), dev(6), workspace=workspace, stream=0)


def distill(workspace):
    rv.relay_linear_distill(head(), dev(6, 3), dev(6, 3, dtype=torch.int32), 1.0, dev(6), workspace=workspace, stream=0)


def router(workspace):
    rv.relay_router_forward(dev(6, 8), dev(6, 2, dtype=torch.int32), dev(6, 2), dev(8, dtype=torch.int32), dev(8),
                            workspace=workspace, stream=0)


@pytest.mark.parametrize("call", [xent, distill, router])
def test_workspace_has_to_be_device_memory(relay_lib, call):
    with pytest.raises(ValueError, match="workspace must be a contiguous CUDA tensor"):
        call(torch.zeros(1 << 20, dtype=torch.uint8))
    with pytest.raises(ValueError, match="workspace must be a contiguous CUDA tensor"):
        call(Device(torch.zeros(1 << 20, 2, dtype=torch.uint8)[:, 0]))


@pytest.mark.parametrize("call", [xent, distill, router])
def test_workspace_is_measured_in_bytes(relay_lib, call):
    """One that is too small is refused by the library with its size in bytes, whatever its type."""
    with pytest.raises(rv.RelayError, match="the workspace holds 24 bytes"):
        call(dev(3, dtype=torch.float64))


def test_choices_have_to_be_a_matrix(relay_lib):
    """One index per row, or none, is no matrix of choices: refused by name, like every other shape."""
    flat = dev(6, dtype=torch.int32)
    with pytest.raises(ValueError, match="teacher_index must be a matrix"):
        rv.relay_linear_distill(head(), dev(6), flat, 1.0, dev(6), stream=0)
    with pytest.raises(ValueError, match="index must be a matrix"):
        rv.relay_router_forward(dev(6, 8), flat, dev(6), dev(8, dtype=torch.int32), dev(8), stream=0)
    with pytest.raises(ValueError, match="index must be a matrix"):
        rv.relay_router_backward(dev(6, 8), flat, dev(6, 8), stream=0)
    with pytest.raises(ValueError, match="d_logits must have the logits' dtype and shape"):
        rv.relay_router_backward(dev(6, 8), dev(6, 2, dtype=torch.int32), dev(6, 7), stream=0)
