"""The training-objective example: the collectives and the losses together, against plain torch on one
step, and a few steps of it going down."""
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


def test_one_step_against_plain_torch():
    import training_objective as ex

    import objective_ref as ref
    import pack_virtual_rank_gb300 as rv
    o = ex.Objective(tokens=130, dim=64, vocab=901)
    logits, d_logits = o.route()
    o.project(tau=2.0)
    torch.cuda.synchronize()
    rv.device_status()
    hidden = torch.cat([h.cpu() for h in o.hidden])
    for full in o.full:
        assert torch.equal(full.cpu(), hidden)            # the gather is exact
    weight, rw = [w.cpu() for w in o.weight], o.row_weight.cpu()
    for args, loss, grads in (((o.target.cpu()[:, None], None, rw, 1.0), o.loss_hard, o.hard),
                              ((o.teacher_index.cpu(), o.teacher_logits.cpu(), rw, 2.0), o.loss_soft, o.soft)):
        want = ref.head(hidden, weight, *args)
        ref.close("loss", loss, want["loss"], want["loss_b"])
        ref.close("d_hidden", grads[0], want["d_hidden"], want["d_hidden_b"])
        ref.close("d_weight", torch.cat([g for g in grads[1]]), want["d_weight"], want["d_weight_b"])
    want = ref.router(torch.cat([x.cpu() for x in logits]), o.top_k, True, None, o.coef, None)
    for a in range(o.A):
        assert torch.equal(o.counts[a].cpu(), want["counts"])
    assert abs(o.balance.item() - want["loss"].item()) <= 1e-5 * want["loss"].item()
    got = torch.cat([d.cpu() for d in d_logits]).double()
    assert bool(((got - want["d_logits"]).abs() <= 1e-5 * want["d_logits_size"] + 1e-37).all())


def test_steps_go_down():
    import training_objective as ex
    losses = ex.main(12)
    assert losses[-1][0] < losses[0][0] - 0.5
    assert losses[-1][1] < losses[0][1]
    assert losses[-1][2] <= losses[0][2] * 1.001
