"""What the Python calls of the losses and the router do with their arguments besides passing them on."""
import pytest
import torch

import pack_virtual_rank_gb300 as rv

pytestmark = pytest.mark.gpu


def test_mask_made_for_the_call():
    """A mask that nothing but the call holds lives as long as the call needs it: its memory must not become the
    call's own workspace."""
    x = torch.randn(10, 8, device="cuda")
    f = dict(device="cuda")
    keep = torch.tensor([True, False] * 5)
    held = keep.cuda()
    got = []
    for temporary in (False, True):
        index, gate = torch.empty(10, 2, dtype=torch.int32, **f), torch.empty(10, 2, **f)
        counts, probs = torch.empty(8, dtype=torch.int32, **f), torch.empty(8, **f)
        torch.cuda.synchronize()
        for _ in range(20):
            rv.relay_router_forward(x, index, gate, counts, probs, mask=keep.cuda() if temporary else held)
        torch.cuda.synchronize()
        got.append([index, gate, counts, probs])
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert bool((got[0][0][1::2] == -1).all()) and bool((got[0][0][::2] >= 0).all())
