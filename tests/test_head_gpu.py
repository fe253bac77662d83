"""Cross entropy and distillation over a sharded vocabulary against their 64-bit definitions, with
elementwise bounds derived in objective_ref.py: sizes from one row and one column up, ragged
shards and strides, misaligned rows, ignored rows that hold NaN, every row ignored, pieces of
the vocabulary, gradients against differences, other streams, repeatability."""
import math

import pytest
import torch

import objective_ref as ref
import pack_virtual_rank_gb300 as rv

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
PAD = 7.0


def strided(rows, cols, dtype, offset=0, extra=0):
    """A [rows, cols] view with a row stride of cols + extra, `offset` elements into its memory,
    every byte around it PAD."""
    buf = torch.full((offset + rows * (cols + extra) + 8,), PAD, dtype=dtype, device="cuda")
    return buf, buf[offset:offset + rows * (cols + extra)].view(rows, cols + extra)[:, :cols]


def inputs(tokens, dim, rows, dtype, seed, scale=2.0):
    g = torch.Generator().manual_seed(seed)
    h = torch.randn(tokens, dim, generator=g).to(DT[dtype])
    ws = [(torch.randn(r, dim, generator=g) * (scale / math.sqrt(dim))).to(DT[dtype]) for r in rows]
    rw = torch.rand(tokens, generator=g) + 0.25
    return g, h, ws, rw


def place(x, offset=0, extra=0):
    buf, v = strided(x.shape[0], x.shape[1], x.dtype, offset, extra)
    v.copy_(x)
    return v


class Call:
    """One call on the GPU: poisoned outputs with canaries around them, results on the CPU."""

    def __init__(self, h, ws, rw, grads=True, piece_bytes=0, offset=0, extra=0, only=None):
        self.tokens = h.shape[0]
        self.hidden = place(h, offset, extra)
        self.weights = [place(w, offset, extra) for w in ws]
        self.dh_buf, self.dh = strided(*h.shape, h.dtype, offset, extra)
        self.dw = [strided(*w.shape, w.dtype, offset, extra) for w in ws]
        self.rw = None if rw is None else rw.cuda()
        self.loss = torch.full((self.tokens + 8,), PAD, device="cuda")
        want_h, want_w = grads and only != "weight", grads and only != "hidden"
        self.head = rv.make_head(self.hidden, self.weights, self.dh if want_h else None,
                                 [d for _, d in self.dw] if want_w else None, piece_bytes)
        self.want_h, self.want_w = want_h, want_w

    def finish(self):
        torch.cuda.synchronize()
        rv.device_status()
        assert bool((self.loss[self.tokens:] == PAD).all())
        for buf, view in [(self.dh_buf, self.dh)] + list(self.dw):
            outside = torch.ones_like(buf, dtype=torch.bool)
            torch.as_strided(outside, view.shape, view.stride(), view.storage_offset()).fill_(False)
            assert bool((buf[outside] == PAD).all()), "wrote outside an output"
        out = {"loss": self.loss[:self.tokens].cpu()}
        if self.want_h:
            out["d_hidden"] = self.dh.cpu()
        if self.want_w:
            out["d_weight"] = torch.cat([d.cpu() for _, d in self.dw])
        return out

    def xent(self, target, stream=None):
        rv.relay_linear_xent(self.head, target.cuda(), self.loss[:self.tokens], row_weight=self.rw, stream=stream)
        return self.finish()

    def distill(self, logits, index, tau):
        ws = rv.alloc_head_workspace(self.head, "cuda", index.shape[1])
        ws.fill_(0xA5)
        rv.relay_linear_distill(self.head, logits.cuda(), index.cuda(), tau, self.loss[:self.tokens],
                                row_weight=self.rw, workspace=ws)
        return self.finish()


def check(out, want):
    for name in out:
        ref.close(name, out[name], want[name], want[name + "_b"])


def targets(g, tokens, vocab, ignored=0.3):
    t = torch.randint(0, vocab, (tokens,), generator=g, dtype=torch.int32)
    out = torch.rand(tokens, generator=g) < ignored
    return torch.where(out, torch.tensor([-100, -1, vocab, 2 ** 31 - 1], dtype=torch.int32)[torch.arange(tokens) % 4], t)


SIZES = [  # tokens, dim, rows per shard
    (1, 1, [1]), (1, 64, [257]), (2, 8, [3, 1]), (5, 16, [0, 9, 0]), (17, 33, [100, 7]),
    (127, 64, [256]), (128, 128, [255, 257]), (129, 72, [300, 1, 511]), (130, 200, [64] * 8),
    (257, 96, [1000]), (300, 264, [513, 700]), (64, 1000, [129]), (33, 520, [2000, 31]),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: f"{s[0]}x{s[1]}x{'+'.join(map(str, s[2]))}")
def test_xent_matches_definition(size, dtype):
    tokens, dim, rows = size
    g, h, ws, rw = inputs(tokens, dim, rows, dtype, 1)
    t = targets(g, tokens, sum(rows), 0.3 if tokens > 2 else 0.0)
    want = ref.head(h, ws, t[:, None], None, rw, 1.0)
    check(Call(h, ws, rw).xent(t), want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size,top,tau", [((1, 8, [5]), 1, 1.0), ((3, 24, [40, 1]), 7, 2.0), ((65, 64, [300]), 31, 0.5),
                                          ((130, 136, [256, 100]), 32, 4.0), ((97, 40, [77, 600]), 33, 1.5),
                                          ((200, 256, [1025]), 128, 2.0)])
def test_distill_matches_definition(size, top, tau, dtype):
    tokens, dim, rows = size
    V = sum(rows)
    g, h, ws, rw = inputs(tokens, dim, rows, dtype, 2)
    index = torch.randint(0, V, (tokens, top), generator=g, dtype=torch.int32)   # ids may repeat
    logits = torch.randn(tokens, top, generator=g) * 3
    gone = torch.rand(tokens, top, generator=g) < 0.2
    index[gone] = torch.tensor([-1, V], dtype=torch.int32)[torch.arange(int(gone.sum())) % 2]
    logits[gone] = math.nan                      # an absent entry's logit is not looked at
    low = torch.rand(tokens, top, generator=g) < 0.1
    logits[low & ~gone] = -math.inf
    index[::5] = -1                              # rows without a teacher
    if tokens > 6:
        logits[6] = -math.inf                    # and one whose entries hold nothing
        logits[7 % tokens] = torch.finfo(torch.float32).min
    for teacher in (torch.float32, torch.bfloat16):
        lg = logits.to(teacher)
        want = ref.head(h, ws, index, lg.float(), rw, tau)
        check(Call(h, ws, rw).distill(lg, index, tau), want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("offset,extra", [(1, 0), (0, 1), (3, 5), (8, 8), (0, 24)])
def test_strides_and_misaligned_rows(dtype, offset, extra):
    g, h, ws, rw = inputs(140, 72, [200, 301], dtype, 3)
    t = targets(g, 140, 501)
    want = ref.head(h, ws, t[:, None], None, rw, 1.0)
    check(Call(h, ws, rw, offset=offset, extra=extra).xent(t), want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("piece_bytes", [1, 300 * 256 * 2, 1 << 20])
def test_pieces_of_the_vocabulary(dtype, piece_bytes):
    g, h, ws, rw = inputs(300, 104, [700, 513], dtype, 4)
    t = targets(g, 300, 1213)
    want = ref.head(h, ws, t[:, None], None, rw, 1.0)
    check(Call(h, ws, rw, piece_bytes=piece_bytes).xent(t), want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_gradient_or_none(dtype):
    g, h, ws, rw = inputs(150, 88, [400], dtype, 5)
    t = targets(g, 150, 400)
    want = ref.head(h, ws, t[:, None], None, None, 1.0)
    check(Call(h, ws, None, only="hidden").xent(t), want)
    check(Call(h, ws, None, only="weight").xent(t), want)
    check(Call(h, ws, None, grads=False).xent(t), want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ignored_rows_reach_nothing(dtype):
    g, h, ws, rw = inputs(200, 64, [300], dtype, 6)
    t = targets(g, 200, 300, 0.5)
    dead = (t < 0) | (t >= 300)
    want = ref.head(h, ws, t[:, None], None, rw, 1.0)
    h[dead] = torch.tensor([math.nan, math.inf, -math.inf, torch.finfo(h.dtype).min])[
        torch.arange(int(dead.sum())) % 4][:, None].to(h.dtype)
    rw[dead] = math.nan
    out = Call(h, ws, rw).xent(t)
    check(out, want)
    assert bool((out["loss"][dead] == 0).all()) and bool((out["d_hidden"][dead] == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_row_ignored_and_no_rows(dtype):
    for tokens in (1, 130, 0):
        g, h, ws, rw = inputs(tokens, 40, [70, 5], dtype, 7)
        out = Call(h, ws, rw).xent(torch.full((tokens,), -100, dtype=torch.int32))
        for x in out.values():
            assert bool((x == 0).all())
        out = Call(h, ws, rw).distill(torch.zeros(tokens, 3), torch.full((tokens, 3), -1, dtype=torch.int32), 1.0)
        for x in out.values():
            assert bool((x == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_confident_rows(dtype):
    """Targets whose probability is within 1e-4 of 1: their gradient must not be the rounding error of
    a probability near 1."""
    g, h, ws, rw = inputs(100, 128, [300], dtype, 8, scale=1.0)
    t = torch.randint(0, 300, (100,), generator=g, dtype=torch.int32)
    h = (h.float() + 18.0 * ws[0][t.long()].float()).to(h.dtype)
    want = ref.head(h, ws, t[:, None], None, rw, 1.0)
    assert want["loss"].median() < 1e-3
    out = Call(h, ws, rw).xent(t)
    check(out, want)


def test_gradient_against_differences():
    """Directional differences of the fp32 loss itself: step 2^-6, loss errors below 1e-5 a row."""
    tokens, dim, rows = 40, 48, [60, 37]
    g, h, ws, rw = inputs(tokens, dim, rows, "f32", 9)
    t = targets(g, tokens, 97)
    out = Call(h, ws, rw).xent(t)
    dh, dw = torch.randn(h.shape, generator=g), [torch.randn(w.shape, generator=g) for w in ws]
    norm = math.sqrt((dh ** 2).sum() + sum((d ** 2).sum() for d in dw))
    step = 2.0 ** -4

    def total(sign):
        hh = h + sign * step / norm * dh
        ww = [w + sign * step / norm * d for w, d in zip(ws, dw)]
        o = Call(hh, ww, rw, grads=False).xent(t)
        return (o["loss"].double() * rw.double()).sum().item()
    slope = (total(1) - total(-1)) / (2 * step)
    want = ((out["d_hidden"].double() * dh).sum() + (out["d_weight"].double() * torch.cat(dw)).sum()).item() / norm
    # third derivatives of a row's loss along a unit direction are below 1 here: step^2 / 6 * weight
    assert abs(slope - want) <= rw.sum().item() * (step * step / 6) * 0.05 + 2e-5 * tokens / step


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_other_stream_and_equal_bits(dtype):
    g, h, ws, rw = inputs(260, 136, [600, 90], dtype, 10)
    t = targets(g, 260, 690)
    a = Call(h, ws, rw).xent(t)
    c = Call(h, ws, rw)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    b = c.xent(t, stream=s)
    for name in a:
        assert torch.equal(a[name], b[name]), name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_captures_into_a_graph(dtype):
    g, h, ws, rw = inputs(100, 64, [300], dtype, 11)
    t = targets(g, 100, 300)
    want = Call(h, ws, rw).xent(t)
    c = Call(h, ws, rw)
    tc, work = t.cuda(), rv.alloc_head_workspace(c.head, "cuda")
    rv.relay_linear_xent(c.head, tc, c.loss[:100], row_weight=c.rw, workspace=work)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rv.relay_linear_xent(c.head, tc, c.loss[:100], row_weight=c.rw, workspace=work)
    c.loss[:100].fill_(PAD)
    graph.replay()
    out = c.finish()
    for name in want:
        assert torch.equal(out[name], want[name]), name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens", [1, 7, 128, 129])
@pytest.mark.parametrize("offset,extra", [(0, 0), (0, 8), (1, 0)])
def test_loss_alone(tokens, offset, extra, dtype):
    """Scoring without gradients, ignored rows full of NaN among the scored ones."""
    g, h, ws, rw = inputs(tokens, 136, [300, 0, 41], dtype, 12)
    t = targets(g, tokens, 341, 0.4 if tokens > 1 else 0.0)
    index = torch.randint(-1, 341, (tokens, 9), generator=g, dtype=torch.int32)
    index[::4] = -1 if tokens > 1 else 5
    logits = torch.randn(tokens, 9, generator=g)
    hard, soft = ref.head(h, ws, t[:, None], None, rw, 1.0), ref.head(h, ws, index, logits, rw, 3.0)
    dead = (t < 0) | (t >= 341)
    h1, h2 = h.clone(), h.clone()
    h1[dead] = math.nan
    h2[(index < 0).all(dim=1)] = math.inf
    out = Call(h1, ws, rw, grads=False, offset=offset, extra=extra).xent(t)
    check(out, hard)
    assert bool((out["loss"][dead] == 0).all())
    check(Call(h2, ws, rw, grads=False, offset=offset, extra=extra).distill(logits, index, 3.0), soft)


@pytest.mark.parametrize("tokens,top", [(512, 16), (513, 16), (512, 17), (30, 2)])
def test_distill_row_sources(tokens, top):
    """Small batches of few entries read their entries in the packing kernel, others a kernel before: the
    same rows take part on both sides of the limit."""
    g, h, ws, rw = inputs(tokens, 64, [70, 200], "bf16", 13)
    index = torch.randint(-40, 270, (tokens, top), generator=g, dtype=torch.int32)
    logits = torch.randn(tokens, top, generator=g)
    index[5] = -1
    logits[7] = -math.inf
    index[8, 1:], logits[8, 0] = 400, -math.inf
    logits[9, 1:] = -math.inf
    h2 = h.clone()
    live = ((index >= 0) & (index < 270) & (logits > -math.inf)).any(dim=1)
    h2[~live] = math.nan
    want = ref.head(h, ws, index, logits, rw, 2.0)
    out = Call(h2, ws, rw).distill(logits, index, 2.0)
    check(out, want)
    assert bool((out["loss"][~live] == 0).all())
