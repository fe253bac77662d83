"""Calls queued one behind the other without waiting: kernels of a chain start before the one in front has
ended, so every one must wait for it before it touches memory. Losses of different inputs through one
workspace, and router calls between them, give the bits that each gives alone."""
import pytest
import torch

import pack_virtual_rank_gb300 as rv

pytestmark = pytest.mark.gpu


class Loss:
    def __init__(self, seed, tokens, dim, rows, dtype, top=0, offset=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        def mat(r):
            buf = torch.randn(offset + r * dim, generator=g, device="cuda").to(dtype)
            return buf[offset:].view(r, dim)
        self.h, self.ws = mat(tokens), [mat(r) for r in rows]
        V = sum(rows)
        self.loss = torch.zeros(tokens, device="cuda")
        self.dh, self.dw = torch.zeros_like(self.h), [torch.zeros_like(w) for w in self.ws]
        self.head = rv.make_head(self.h, self.ws, self.dh, self.dw)
        self.top = top
        self.target = torch.randint(-20, V, (tokens,), generator=g, device="cuda", dtype=torch.int32)
        if top:
            self.index = torch.randint(0, V, (tokens, top), generator=g, device="cuda", dtype=torch.int32)
            self.logits = torch.randn(tokens, top, generator=g, device="cuda")

    def run(self, work):
        if self.top:
            rv.relay_linear_distill(self.head, self.logits, self.index, 2.0, self.loss, workspace=work)
        else:
            rv.relay_linear_xent(self.head, self.target, self.loss, workspace=work)

    def results(self):
        return [self.loss, self.dh] + self.dw


class Route:
    def __init__(self, seed, tokens, experts, top):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.x = torch.randn(tokens, experts, generator=g, device="cuda")
        f = dict(device="cuda")
        self.index, self.gate = torch.zeros(tokens, top, dtype=torch.int32, **f), torch.zeros(tokens, top, **f)
        self.counts, self.probs = torch.zeros(experts, dtype=torch.int32, **f), torch.zeros(experts, **f)
        self.loss, self.d_prob, self.dx, self.k = torch.zeros(1, **f), torch.zeros(experts, **f), torch.zeros_like(self.x), top

    def run(self, work):
        rv.relay_router_forward(self.x, self.index, self.gate, self.counts, self.probs, workspace=work)
        rv.relay_balance_loss(self.counts, self.probs, self.k, 0.1, self.loss, self.d_prob)
        rv.relay_router_backward(self.x, self.index, self.dx, d_gate=self.gate, d_prob=self.d_prob)

    def results(self):
        return [self.index, self.gate, self.counts, self.probs, self.loss, self.dx]


def test_queued_calls_give_the_bits_of_single_ones():
    calls = [Loss(1, 130, 64, [500, 300], torch.bfloat16), Route(2, 3000, 64, 4), Loss(3, 40, 72, [900], torch.float32),
             Loss(4, 700, 200, [3000], torch.bfloat16, top=9), Route(5, 20000, 256, 8),
             Loss(6, 90, 33, [400, 77], torch.bfloat16, offset=1), Loss(7, 300, 128, [20000], torch.bfloat16),
             Loss(8, 257, 40, [600], torch.float32, top=3)]
    size = max([rv.relay_head_workspace_size(c.head, c.top) for c in calls if isinstance(c, Loss)] + [608 * 256 * 8 + 16])
    work = torch.empty(size, dtype=torch.uint8, device="cuda")
    want = []
    for c in calls:
        work.fill_(0xFF)
        c.run(work)
        torch.cuda.synchronize()
        want.append([x.clone() for x in c.results()])
    for _ in range(20):
        for c in calls:
            for x in c.results():
                x.zero_()
        torch.cuda.synchronize()
        for c in calls:
            c.run(work)
        torch.cuda.synchronize()
        for c, w in zip(calls, want):
            for a, b in zip(c.results(), w):
                assert torch.equal(a, b)
    rv.device_status()
