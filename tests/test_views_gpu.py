"""Inputs and outputs that lie side by side in the rows of one buffer overlap nowhere, although the ranges of
their addresses do: the losses and the router take them, and refuse what really overlaps."""
import pytest
import torch

import pack_virtual_rank_gb300 as rv

pytestmark = pytest.mark.gpu


def views(rows, widths, dtype, gap=0):
    """Column views of one buffer, `gap` columns between them, every element 7."""
    buf = torch.full((rows, sum(widths) + gap * len(widths)), 7.0, dtype=dtype, device="cuda")
    out, at = [], 0
    for n in widths:
        out.append(buf[:, at:at + n])
        at += n + gap
    return buf, out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gap", [0, 3])
def test_losses_of_column_views(gap, dtype):
    g = torch.Generator().manual_seed(1)
    h, w = torch.randn(50, 40, generator=g).to(dtype), (torch.randn(90, 40, generator=g) * 0.3).to(dtype)
    target = torch.randint(-3, 90, (50,), generator=g, dtype=torch.int32).cuda()

    def run(hidden, d_hidden, weight, d_weight):
        hidden.copy_(h)
        weight.copy_(w)
        loss = torch.zeros(50, device="cuda")
        rv.relay_linear_xent(rv.make_head(hidden, [weight], d_hidden, [d_weight]), target, loss)
        return [loss, d_hidden.clone(), d_weight.clone()]
    e = lambda n: torch.empty(n, 40, dtype=dtype, device="cuda")  # noqa: E731
    alone = run(e(50), e(50), e(90), e(90))
    hb, (hv, dhv) = views(50, [40, 40], dtype, gap)
    wb, (wv, dwv) = views(90, [40, 40], dtype, gap)
    for a, b in zip(alone, run(hv, dhv, wv, dwv)):
        assert torch.equal(a, b)
    if gap:
        for buf in (hb, wb):
            assert bool((buf[:, 40:43] == 7).all()) and bool((buf[:, 83:] == 7).all())
    # one column shared is an overlap
    wide = torch.zeros(50, 90, dtype=dtype, device="cuda")
    for a, b in ((wide[:, :40], wide[:, 39:79]), (wide[:, 39:79], wide[:, :40])):
        with pytest.raises(rv.RelayError, match="overlaps"):
            rv.relay_linear_xent(rv.make_head(a, [e(90)], b), target, torch.zeros(50, device="cuda"))
    # a view that ends in the next row's columns
    flat = torch.zeros(51 * 80, dtype=dtype, device="cuda")
    a, b = flat[:4000].view(50, 80)[:, :40], flat[41:4041].view(50, 80)[:, :40]
    with pytest.raises(rv.RelayError, match="overlaps"):
        rv.relay_linear_xent(rv.make_head(a, [e(90)], b), target, torch.zeros(50, device="cuda"))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_router_of_column_views(dtype):
    g = torch.Generator().manual_seed(2)
    x = torch.randn(100, 24, generator=g).to(dtype)
    buf, (xv, dv) = views(100, [24, 24], dtype, 2)
    xv.copy_(x)
    f = dict(device="cuda")
    index, gate = torch.zeros(100, 3, dtype=torch.int32, **f), torch.zeros(100, 3, **f)
    counts, probs = torch.zeros(24, dtype=torch.int32, **f), torch.zeros(24, **f)
    rv.relay_router_forward(xv, index, gate, counts, probs)
    dx = torch.empty(100, 24, dtype=dtype, **f)
    rv.relay_router_backward(x.cuda(), index, dx, d_gate=gate)
    rv.relay_router_backward(xv, index, dv, d_gate=gate)
    assert torch.equal(dv, dx) and torch.equal(xv.cpu(), x)
    assert bool((buf[:, 24:26] == 7).all()) and bool((buf[:, 50:] == 7).all())
    with pytest.raises(rv.RelayError, match="overlaps"):
        rv.relay_router_backward(xv, index, buf[:, 23:47], d_gate=gate)
