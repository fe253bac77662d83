"""Clipping by factors below fp32's normal range: a norm near the range's end, or a small max_norm."""
import pytest
import torch

import pack_virtual_rank_gb300 as rv

pytestmark = pytest.mark.gpu
F, U = 2.0 ** -24, 2.0 ** -8


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("skew", [0, 1])
@pytest.mark.parametrize("total,most", [(2.0 ** 127, 1.0), (3e38, 1e-3), (1e38, 1e-7), (1e38, 3e-30), (1e-3, 2e-42), (1e25, 1e-5), (1e30, 0.7),
                                        (3e38, 1e38), (1e36, 7e-35), (6e37, 8e-38), (6e36, 7e-42), (2e38, 4e-34), (3e38, 1e-44), (5e37, 2e38)])
def test_small_factors(total, most, skew, dtype):
    g = torch.Generator().manual_seed(3)
    x = (torch.randn(40000, generator=g, dtype=torch.float64) * (total / 200)).to(dtype).cuda()
    x[7] = 0.0
    norm = torch.full((1,), total, device="cuda")
    buf = torch.full((40010,), 7.0, dtype=dtype, device="cuda")
    y = buf[skew:skew + 40000]                            # with skew, the two lie differently on the 16-byte grid
    rv.relay_grad_clip(rv.make_grads([x]), norm, most, out=rv.make_grads([y]))
    c = min(1.0, float(torch.tensor(most)) / (norm.double().item() + 1e-6))
    want = x.double() * c
    unit = F if dtype is torch.float32 else U
    # the factor: its addition, division and the product; the result's rounding, below the normal range half its
    # smallest step (of the product in fp32, and of the result)
    step = 2.0 ** -150 + (0.0 if dtype is torch.float32 else 2.0 ** -134)
    assert bool(((y.double() - want).abs() <= (3 * F + unit) * want.abs() + step).all())
    assert bool((buf[:skew] == 7.0).all()) and bool((buf[skew + 40000:] == 7.0).all())
    rv.relay_grad_clip(rv.make_grads([x]), norm, most)
    assert torch.equal(x, y)
