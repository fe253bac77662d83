"""The norm over lists of which a thread sums many chunks, at magnitudes whose sums come near fp32's end."""
import math

import pytest
import torch

import pack_virtual_rank_gb300 as rv

pytestmark = pytest.mark.gpu
F, U = 2.0 ** -24, 2.0 ** -8
# a chain of 16 squares and two additions of four chains, halved by the root, and the root's own rounding
NORM = 10 * F


# 456 blocks at most take chunks of 32 KiB in turn: 17 chunks a block and more, 2 to 64 values of it a thread
@pytest.mark.parametrize("dtype,count", [(torch.bfloat16, 130_000_000), (torch.float32, 65_000_000)])
@pytest.mark.parametrize("power", [40, 49, 50, 56, 57, 58, 59, 60, 61, 100])
def test_sums_of_many_chunks(dtype, count, power):
    x = torch.full((count,), 2.0 ** power, dtype=dtype, device="cuda")
    x[::3] = -(2.0 ** power)
    norm = torch.empty(1, device="cuda")
    grads = rv.make_grads([x])
    rv.relay_grad_norm(grads, norm)
    want = math.sqrt(count) * 2.0 ** power               # every square is 2^(2 power)
    assert abs(norm.item() - want) <= NORM * want
    rv.relay_grad_clip(grads, norm, 1.0)
    unit = F if dtype is torch.float32 else U
    part = torch.cat([x[:3000], x[-3000:]]).double().abs()
    each = 2.0 ** power / want                            # the norm, its addition, the division, the product; the result's rounding
    assert bool(((part - each).abs() <= (NORM + 3 * F + unit) * each).all())


def test_both_sides_of_the_limit_in_one_list():
    """Chunks that are summed as they are beside chunks that are summed scaled, many of each."""
    n = 16_000_000
    xs = [torch.full((n,), 2.0 ** p, dtype=torch.bfloat16, device="cuda") for p in (45, 48, 52, 59, 30)]
    norm = torch.empty(1, device="cuda")
    for some in (xs, xs[::-1], xs[:3]):
        rv.relay_grad_norm(rv.make_grads(some), norm)
        want = math.sqrt(sum(n * float(x[0]) ** 2 for x in some))
        assert abs(norm.item() - want) <= NORM * want
