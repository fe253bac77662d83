"""Long sums of one sign in the gradients. The tensor cores cut when they add, always towards 0, so a sum kept in
them loses a share that grows with its length, without limit; sums that move to registers after a fixed number
of products lose no more than that many do.

The bound on the mean relative error: 1.1e-5 for the cutting (512 products that each cut half a unit of 24 bits, 4.3e-8, from a sum
that is half of its end on average), whatever the length; and four standard deviations of the mean of n results rounded to
bf16 (at most 2^-9 each, 1.2e-3 rms). The other roundings are per term and average over the terms too."""
import math

import pytest
import torch

import pack_virtual_rank_gb300 as rv

pytestmark = pytest.mark.gpu


def bound(n):
    return 512 * 2.1e-8 + 4 * 1.2e-3 / math.sqrt(n)


def mean_error(got, want):
    return ((got.double() - want) / want).mean().item()


def test_weight_gradient_over_many_tokens():
    """131072 tokens: 8192 products of 16 tokens each into a row of d_weight."""
    T, D, V = 131072, 256, 256
    g = torch.Generator(device="cuda").manual_seed(1)
    h = (torch.randn(T, D, generator=g, device="cuda").abs() + 0.1).bfloat16()
    w = (torch.randn(V, D, generator=g, device="cuda") * 0.1).bfloat16()
    target = torch.zeros(T, dtype=torch.int32, device="cuda")
    dw, loss = torch.empty_like(w), torch.empty(T, device="cuda")
    rv.relay_linear_xent(rv.make_head(h, [w], None, [dw]), target, loss)
    p = torch.softmax(h.double() @ w.double().t(), dim=1)
    want = (p.t() @ h.double())[1:]                        # column 0 is every row's target
    e = mean_error(dw[1:], want)
    assert abs(e) <= bound(want.numel()), e
    rv.device_status()


def test_hidden_gradient_over_a_large_vocabulary():
    """131072 columns in one piece and one cut: 8192 products of 16 columns each into a row of d_hidden."""
    T, D, V = 8192, 4096, 131072
    g = torch.Generator(device="cuda").manual_seed(2)
    h = (torch.randn(T, D, generator=g, device="cuda") * 2).bfloat16()
    w = (torch.rand(V, D, generator=g, device="cuda") * 0.03 + 0.002).bfloat16()
    w[0] = 0.0                                             # the targets' own row adds nothing
    target = torch.zeros(T, dtype=torch.int32, device="cuda")
    dh, loss = torch.empty_like(h), torch.empty(T, device="cuda")
    head = rv.make_head(h, [w], dh, None, 4 << 30)
    rv.relay_linear_xent(head, target, loss)
    rows = torch.arange(5, T, T // 16, device="cuda")
    want = torch.zeros(len(rows), D, dtype=torch.float64, device="cuda")
    z = torch.cat([h[rows].double() @ x.double().t() for x in w.split(16384)], dim=1)
    p = torch.softmax(z, dim=1)
    for at in range(0, V, 16384):
        want += p[:, at:at + 16384] @ w[at:at + 16384].double()
    e = mean_error(dh[rows], want)
    assert abs(e) <= bound(want.numel()), e
    rv.device_status()
