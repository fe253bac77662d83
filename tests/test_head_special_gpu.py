"""Logits that are not finite, or as low or high as the type goes, in rows that take part: a vocabulary
row banned through a column of ones in hidden and an infinite (or lowest) value in the weight has probability
0, a NaN or +infinite logit makes its own row NaN, and the rest stays what the definition gives without
the banned rows."""
import math

import pytest
import torch

import objective_ref as ref
import pack_virtual_rank_gb300 as rv

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
DIM, ROWS = 72, [300, 1, 511]
V = sum(ROWS)


def inputs(tokens, dtype, seed):
    """hidden's last column is positive (its first rows 1), so that the weight's last column is a bias."""
    g = torch.Generator().manual_seed(seed)
    h = torch.randn(tokens, DIM, generator=g)
    h[:, -1] = torch.rand(tokens, generator=g) * 3 + 0.01
    h[::3, -1] = 1.0
    w = torch.randn(V, DIM, generator=g) * 0.25
    banned = torch.rand(V, generator=g) < 0.3
    banned[0:256] = True                                   # whole tiles of columns
    banned[301:301 + 384] = True
    banned[299:301] = torch.tensor([False, True])          # a shard of nothing else
    free = (~banned).nonzero()[:, 0]
    rw = torch.rand(tokens, generator=g) + 0.25
    return g, h.to(DT[dtype]), w.to(DT[dtype]), banned, free, rw


def call(h, w, rw, target=None, teacher=None, piece_bytes=0):
    """loss, d_hidden and d_weight on the CPU."""
    hc, wc = h.cuda(), [x.contiguous() for x in w.cuda().split(ROWS)]
    dh, dw, loss = torch.full_like(hc, 7.0), [torch.full_like(x, 7.0) for x in wc], torch.full((h.shape[0],), 7.0, device="cuda")
    head = rv.make_head(hc, wc, dh, dw, piece_bytes)
    if teacher is None:
        rv.relay_linear_xent(head, target.cuda(), loss, row_weight=rw.cuda())
    else:
        index, logits, tau = teacher
        rv.relay_linear_distill(head, logits.cuda(), index.cuda(), tau, loss, row_weight=rw.cuda())
    torch.cuda.synchronize()
    rv.device_status()
    return loss.cpu(), dh.cpu(), torch.cat(dw).cpu()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens", [1, 40, 300])
@pytest.mark.parametrize("piece_bytes", [0, 1])
@pytest.mark.parametrize("bias", ["-inf", "overflow"])
def test_banned_by_minus_infinity(bias, piece_bytes, tokens, dtype):
    """-inf in the weight, or products that leave fp32's range: probability 0."""
    g, h, w, banned, free, rw = inputs(tokens, dtype, 1)
    if bias == "overflow":
        h[:, -1] = (h[:, -1].float() * 1e5).to(h.dtype)
        w[~banned, -1] = (w[~banned, -1].float() * 1e-5).to(w.dtype)
        w[banned, -1] = (-(torch.rand(V, generator=g) + 1) * 1e38).to(w.dtype)[banned]
    else:
        w[banned, -1] = -math.inf
    at = torch.randint(0, len(free), (tokens,), generator=g, dtype=torch.int32)
    target = free[at.long()].int()
    idx = torch.randint(0, len(free), (tokens, 5), generator=g)
    logits = torch.randn(tokens, 5, generator=g)
    for teacher in (None, (free[idx].int(), logits, 2.0)):
        if teacher is None:
            want = ref.head(h, [w[free]], at[:, None], None, rw, 1.0)
        else:
            want = ref.head(h, [w[free]], idx.int(), logits, rw, 2.0)
        loss, dh, dw = call(h, w, rw, target, teacher, piece_bytes)
        ref.close("loss", loss, want["loss"], want["loss_b"])
        ref.close("d_weight", dw[free], want["d_weight"], want["d_weight_b"])
        assert bool((dw[banned] == 0).all())
        if bias == "overflow":
            ref.close("d_hidden", dh, want["d_hidden"], want["d_hidden_b"])
        else:
            ref.close("d_hidden", dh[:, :-1], want["d_hidden"][:, :-1], want["d_hidden_b"][:, :-1])
            assert bool(torch.isnan(dh[:, -1]).all())       # 0 * -inf, as in the definition


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("piece_bytes", [0, 1])
@pytest.mark.parametrize("tokens", [40, 300])
def test_nan_and_infinite_logits_stay_in_their_rows(tokens, piece_bytes, dtype):
    """A NaN in hidden, and hidden of the sign that makes the banned rows +inf: those rows are NaN, the others
    what they are without them."""
    g, h, w, banned, free, rw = inputs(tokens, dtype, 2)
    w[banned, -1] = -math.inf
    bad = torch.zeros(tokens, dtype=torch.bool)
    bad[[2, 7, 39]] = True
    h[2, 5] = math.nan
    h[7, -1] = -1.0                                         # +inf logits
    h[39, -1] = 0.0                                         # 0 * -inf
    at = torch.randint(0, len(free), (tokens,), generator=g, dtype=torch.int32)
    clean = h.clone()
    clean[bad] = 1.0
    want = ref.head(clean, [w[free]], at[:, None], None, rw, 1.0)
    loss, dh, dw = call(h, w, rw, free[at.long()].int(), None, piece_bytes)
    assert bool(torch.isnan(loss[bad]).all()) and bool(torch.isnan(dh[bad]).all())
    assert bool(torch.isnan(dw).all())                      # every row of d_weight sums over every row of hidden
    ref.close("loss", loss[~bad], want["loss"][~bad], want["loss_b"][~bad])
    ref.close("d_hidden", dh[~bad][:, :-1], want["d_hidden"][~bad][:, :-1], want["d_hidden_b"][~bad][:, :-1])
