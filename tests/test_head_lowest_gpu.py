"""Finite logits at the ends of the type's range. A vocabulary row is banned by the lowest value of the type
(through a column of ones in hidden): probability 0, also where a whole tile of columns is banned, where a row
of hidden has nothing else, and below temperature 1. Logits near the largest value are as good as any."""
import pytest
import torch

import objective_ref as ref
from test_head_special_gpu import DIM, DT, ROWS, V, call

pytestmark = pytest.mark.gpu


def inputs(tokens, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    h = torch.randn(tokens, DIM, generator=g)
    h[:, -1] = 1.0
    w = torch.randn(V, DIM, generator=g) * 0.25
    w[:, -1] = 0.0
    banned = torch.rand(V, generator=g) < 0.3
    banned[0:256] = True
    banned[301:301 + 384] = True
    banned[299:301] = torch.tensor([False, True])
    return g, h.to(DT[dtype]), w.to(DT[dtype]), banned, (~banned).nonzero()[:, 0], torch.rand(tokens, generator=g) + 0.25


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens", [1, 40, 300])
@pytest.mark.parametrize("piece_bytes", [0, 1])
@pytest.mark.parametrize("tau", [0.25, 1.0, 3.0])
def test_banned_by_the_lowest_value(tau, piece_bytes, tokens, dtype):
    g, h, w, banned, free, rw = inputs(tokens, dtype, 3)
    w[banned, -1] = torch.finfo(DT[dtype]).min
    at = torch.randint(0, len(free), (tokens, 6), generator=g)
    logits = torch.randn(tokens, 6, generator=g)
    if tau == 1.0:
        want = ref.head(h, [w[free]], at[:, :1].int(), None, rw, 1.0)
        loss, dh, dw = call(h, w, rw, free[at[:, 0]].int(), None, piece_bytes)
    else:
        want = ref.head(h, [w[free]], at.int(), logits, rw, tau)
        loss, dh, dw = call(h, w, rw, None, (free[at].int(), logits, tau), piece_bytes)
    ref.close("loss", loss, want["loss"], want["loss_b"])
    ref.close("d_hidden", dh, want["d_hidden"], want["d_hidden_b"])
    ref.close("d_weight", dw[free], want["d_weight"], want["d_weight_b"])
    assert bool((dw[banned] == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens", [3, 200])
@pytest.mark.parametrize("piece_bytes", [0, 1])
@pytest.mark.parametrize("sign", [-1.0, 1.0])
def test_rows_of_one_extreme_value(sign, piece_bytes, tokens, dtype):
    """hidden is 0 but for its last column, and so is the weight: every logit is the same value at the end of
    the range. The softmax is uniform: loss log V, gradients of 1/V and 1/V - 1."""
    g = torch.Generator().manual_seed(4)
    h = torch.zeros(tokens, DIM, dtype=DT[dtype])
    h[:, -1] = 1.0
    w = torch.zeros(V, DIM, dtype=DT[dtype])
    w[:, -1] = sign * torch.finfo(DT[dtype]).max
    target = torch.randint(0, V, (tokens,), generator=g, dtype=torch.int32)
    loss, _, dw = call(h, w, torch.ones(tokens), target, None, piece_bytes)
    assert bool(((loss - torch.log(torch.tensor(float(V)))).abs() < 1e-5).all())
    want = torch.full((V,), tokens / V, dtype=torch.float64)
    want -= torch.bincount(target.long(), minlength=V)
    # each term of a row of d_weight is rounded to bf16 at most twice (bf16 heads), the sum once
    slack = ref.U if dtype == "bf16" else 2.0 ** -19
    bound = 3 * slack * (tokens / V + torch.bincount(target.long(), minlength=V).double())
    assert bool(((dw[:, -1].double() - want).abs() <= bound).all())
    assert bool((dw[:, :-1] == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("piece_bytes", [0, 1])
def test_one_logit_near_the_largest_value(piece_bytes, dtype):
    """A row whose largest logit is near the type's largest has all its probability there."""
    g, h, w, _, _, rw = inputs(50, dtype, 5)
    hot = 333
    w[hot, -1] = 3.0e38
    target = torch.randint(0, V, (50,), generator=g, dtype=torch.int32)
    target[::2] = hot
    other = target != hot
    loss, dh, dw = call(h, w, rw, target, None, piece_bytes)
    assert bool((loss[~other] == 0).all())
    z = w[hot].double() @ h.double().t()
    assert bool(((loss.double() - z)[other].abs() <= 2.0 ** -20 * z[other]).all())
    # p is 1 at `hot`, 0 elsewhere: only rows with another target have a gradient, +w there and -w at the target
    assert bool((dh[~other] == 0).all())
    want = torch.zeros(V, DIM, dtype=torch.float64)
    size = torch.zeros(V, DIM, dtype=torch.float64)
    for n in other.nonzero()[:, 0].tolist():
        row = rw[n].double() * h[n].double()
        want[hot] += row
        want[target[n].long()] -= row
        size[hot] += row.abs()
        size[target[n].long()] += row.abs()
    unit = ref.U if dtype == "bf16" else 2.0 ** -19
    assert bool(((dw.double() - want).abs() <= 3 * unit * size).all())
