"""One training step's objective over virtual ranks, end to end.

A active ranks of an R-rank node train a token classifier whose vocabulary is sharded on them:

  * each rank routes its own tokens (relay_router_forward); the per-expert counts and probability
    sums are summed over the ranks (relay_allreduce, int32 and fp32), so that the balance
    loss is the whole batch's (relay_balance_loss), and go back to each rank's router logits
    (relay_router_backward);
  * the ranks' hidden rows are gathered (relay_all_gather) and meet the sharded output projection:
    cross entropy against the labels (relay_linear_xent) and distillation from the few largest
    logits of a teacher (relay_linear_distill), each with its gradients;
  * every rank updates its vocabulary shard, its hidden rows and its router.

Run it: ``python examples/training_objective.py`` (needs the built library and a GB300).
"""
from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import pack_virtual_rank_gb300 as rv  # noqa: E402


class Objective:
    """The state of the ranks and the buffers their calls write, allocated once."""

    def __init__(self, tokens=512, dim=256, vocab=4099, experts=32, top_k=4, teacher_top=16, A=2, R=8,
                 dtype=torch.bfloat16, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        f32 = dict(dtype=torch.float32, device=device)
        self.A, self.R, self.tokens, self.top_k, self.coef = A, R, tokens, top_k, 0.01
        total = A * tokens
        # parameters: hidden rows stand for the model below, shards of the output projection, routers
        self.hidden = [torch.randn(tokens, dim, generator=g, device=device).to(dtype) for _ in range(A)]
        rows = [vocab // A + (1 if a < vocab % A else 0) for a in range(A)]
        self.weight = [(torch.randn(r, dim, generator=g, device=device) * dim ** -0.5).to(dtype) for r in rows]
        self.router = torch.randn(dim, experts, generator=g, device=device) * dim ** -0.5
        # data: labels (every seventh row is a prompt: ignored) and a teacher that favours them
        self.label = torch.randint(0, vocab, (total,), generator=g, device=device, dtype=torch.int32)
        self.target = torch.where(torch.arange(total, device=device) % 7 == 0, -100, self.label).to(torch.int32)
        others = torch.randint(0, vocab, (total, teacher_top - 1), generator=g, device=device, dtype=torch.int32)
        self.teacher_index = torch.cat([self.label[:, None], others], dim=1).contiguous()
        self.teacher_logits = torch.randn(total, teacher_top, generator=g, device=device)
        self.teacher_logits[:, 0] += 6.0
        self.row_weight = torch.full((total,), 1.0 / total, **f32)
        # what the calls write
        self.full = [torch.empty(total, dim, dtype=dtype, device=device) for _ in range(A)]
        grads = lambda: (torch.empty(total, dim, dtype=dtype, device=device), [torch.empty_like(w) for w in self.weight])  # noqa: E731
        self.hard, self.soft = grads(), grads()
        self.loss_hard, self.loss_soft = torch.empty(total, **f32), torch.empty(total, **f32)
        self.index = [torch.empty(tokens, top_k, dtype=torch.int32, device=device) for _ in range(A)]
        self.gate = [torch.empty(tokens, top_k, **f32) for _ in range(A)]
        self.counts = [torch.empty(experts, dtype=torch.int32, device=device) for _ in range(A)]
        self.prob_sum = [torch.empty(experts, **f32) for _ in range(A)]
        self.balance, self.d_prob = torch.empty(1, **f32), torch.empty(experts, **f32)
        # plans, scratch and workspaces
        self.gather_scratch = rv.alloc_scratch(rv.relay_plan(rv.ALL_GATHER, tokens * dim, dtype, A, R), device)
        self.sum_scratch = {d: rv.alloc_scratch(rv.relay_plan(rv.ALLREDUCE, experts, d, A, R), device) for d in (rv.I32, rv.F32)}
        self.router_workspace = rv.alloc_router_workspace(tokens, experts, device)
        # every rank gathers the same rows; one copy is the projection's input
        self.head_hard = rv.make_head(self.full[0], self.weight, *self.hard)
        self.head_soft = rv.make_head(self.full[0], self.weight, *self.soft)
        self.workspace = torch.empty(max(rv.relay_head_workspace_size(self.head_hard),
                                         rv.relay_head_workspace_size(self.head_soft, teacher_top)),
                                     dtype=torch.uint8, device=device)

    def route(self):
        """The routers of all ranks; returns each rank's logits and their gradient."""
        logits = [h.float() @ self.router for h in self.hidden]
        for a in range(self.A):
            rv.relay_router_forward(logits[a], self.index[a], self.gate[a], self.counts[a], self.prob_sum[a],
                                    normalize=True, workspace=self.router_workspace)
        for bufs, dt in ((self.counts, rv.I32), (self.prob_sum, rv.F32)):
            rv.relay_allreduce(bufs, bufs, self.sum_scratch[dt], bufs[0].numel(), dt, self.A, self.R)
        # every rank holds the same sums now
        rv.relay_balance_loss(self.counts[0], self.prob_sum[0], self.top_k, self.coef, self.balance, self.d_prob)
        d_logits = [torch.empty_like(x) for x in logits]
        for a in range(self.A):
            rv.relay_router_backward(logits[a], self.index[a], d_logits[a], d_prob=self.d_prob, normalize=True)
        return logits, d_logits

    def project(self, tau=2.0):
        """Losses over the gathered rows and the sharded vocabulary, and their gradients."""
        rv.relay_all_gather(self.hidden, self.full, self.gather_scratch, self.hidden[0].numel(),
                            self.hidden[0].dtype, self.A, self.R)
        rv.relay_linear_xent(self.head_hard, self.target, self.loss_hard, row_weight=self.row_weight,
                             workspace=self.workspace)
        rv.relay_linear_distill(self.head_soft, self.teacher_logits, self.teacher_index, tau, self.loss_soft,
                                row_weight=self.row_weight, workspace=self.workspace)

    def step(self, lr=400.0):
        """One step; returns the mean cross entropy, distillation and balance losses before it."""
        _, d_logits = self.route()
        self.project()
        for a in range(self.A):
            rows = slice(a * self.tokens, (a + 1) * self.tokens)
            self.weight[a].sub_(lr / 40 * (self.hard[1][a].float() + self.soft[1][a].float()))
            self.router.sub_(lr * (self.hidden[a].float().t() @ d_logits[a]) / self.A)
            self.hidden[a].sub_(lr / 4 * (self.hard[0][rows].float() + self.soft[0][rows].float()))
        kept = (self.target >= 0).sum()
        return (self.loss_hard.sum() / kept).item(), self.loss_soft.mean().item(), self.balance.item()


def main(steps: int = 20):
    objective = Objective()
    losses = [objective.step() for _ in range(steps)]
    for i, (hard, soft, balance) in enumerate(losses):
        if i % 5 == 0 or i == steps - 1:
            print(f"step {i:3d}: cross entropy {hard:.4f}, distillation {soft:.4f}, balance {balance:.5f}")
    return losses


if __name__ == "__main__":
    main()
