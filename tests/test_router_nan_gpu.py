"""Rows of the router without a finite logit: one that holds a NaN is counted, with NaN gates and NaN
probabilities (a diverged token shows), one of -inf alone is not counted, and neither changes the rows beside
it."""
import math

import pytest
import torch

import pack_virtual_rank_gb300 as rv

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def route(x, top, normalize, mask, d_gate):
    t, e = x.shape
    f = dict(device="cuda")
    index, gate = torch.full((t, top), -7, dtype=torch.int32, **f), torch.full((t, top), 7.0, **f)
    counts, probs = torch.full((e,), -7, dtype=torch.int32, **f), torch.full((e,), 7.0, **f)
    dx = torch.full_like(x, 7.0, **f)
    rv.relay_router_forward(x.cuda(), index, gate, counts, probs, mask=mask.cuda(), normalize=normalize)
    rv.relay_router_backward(x.cuda(), index, dx, d_gate=d_gate.cuda(), normalize=normalize)
    torch.cuda.synchronize()
    return [v.cpu() for v in (index, gate, counts, probs, dx)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("experts,top", [(1, 1), (8, 2), (20, 20), (60, 4), (100, 5), (256, 8), (384, 8), (1000, 3)])
def test_rows_without_a_finite_logit(experts, top, normalize, dtype):
    g = torch.Generator().manual_seed(experts)
    x = torch.randn(70, experts, generator=g).to(DT[dtype])
    mask = torch.ones(70, dtype=torch.bool)
    nans = [0, 3, 10, 11, 12, 33, 69]
    x[0] = math.nan
    x[3] = math.nan
    x[3, 0] = -math.inf
    x[10] = -math.inf
    x[10, experts - 1] = math.nan
    x[11] = -torch.full((), math.nan)                       # the sign bit set
    x[12, experts // 2] = math.nan                          # beside finite logits
    x[33] = -math.inf
    x[33, experts // 3] = -torch.full((), math.nan)
    x[69] = math.nan
    if experts == 1:
        x[3] = math.nan
    x[20] = x[40] = -math.inf                               # nothing above -inf
    x[21] = x[41] = math.nan                                # masked out
    mask[[21, 41]] = False
    gone = [20, 21, 40, 41]
    d = torch.randn(70, top, generator=g)
    index, gate, counts, probs, dx = route(x, top, normalize, mask, d)
    for r in nans:
        assert sorted(set(index[r].tolist())) == sorted(index[r].tolist()), r
        assert bool(((index[r] >= 0) & (index[r] < experts)).all()), r
        assert bool(torch.isnan(gate[r]).all()), r
        assert bool(torch.isnan(dx[r]).all()), r
    for r in gone:
        assert bool((index[r] == -1).all()) and bool((gate[r] == 0).all()) and bool((dx[r] == 0).all()), r
    assert bool(torch.isnan(probs).all())
    assert counts.sum().item() == top * (70 - len(gone))
    assert torch.equal(counts, torch.bincount(index[index >= 0], minlength=experts).int())
    # the others as they are without those rows
    mask[nans] = False
    index2, gate2, _, probs2, dx2 = route(x, top, normalize, mask, d)
    rest = [r for r in range(70) if r not in nans]
    assert torch.equal(index[rest], index2[rest]) and torch.equal(gate[rest], gate2[rest])
    assert torch.equal(dx[rest], dx2[rest]) and not bool(torch.isnan(probs2).any())
