"""The expert router and its balance loss against their 64-bit definitions: every width of the
kernel, ties, masked and empty rows, lowest values and infinities, strides, the gradient against
differences, and statistics summed over ranks with relay_allreduce."""
import math

import pytest
import torch

import objective_ref as ref
import pack_virtual_rank_gb300 as rv

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
F = 2.0 ** -24
# a softmax of up to 1024 fp32 terms: exp within 2 ulp, the sum within 10 rounding steps of a
# tree, one division and one product
SOFT = 32 * F


def run(logits, top, normalize=False, mask=None, coef=0.5, d_gate=None, extra=0):
    t, e = logits.shape
    buf = torch.full((t, e + extra), 9.0, dtype=logits.dtype, device="cuda")
    x = buf[:, :e]
    x.copy_(logits)
    out = dict(index=torch.full((t, top), -7, dtype=torch.int32, device="cuda"),
               gate=torch.full((t, top), 7.0, device="cuda"),
               counts=torch.full((e,), -7, dtype=torch.int32, device="cuda"),
               prob_sum=torch.full((e,), 7.0, device="cuda"), loss=torch.full((1,), 7.0, device="cuda"),
               d_prob=torch.full((e,), 7.0, device="cuda"))
    m = None if mask is None else mask.cuda()
    rv.relay_router_forward(x, out["index"], out["gate"], out["counts"], out["prob_sum"], mask=m,
                            normalize=normalize)
    rv.relay_balance_loss(out["counts"], out["prob_sum"], top, coef, out["loss"], out["d_prob"])
    dbuf = torch.full((t, e + extra), 9.0, dtype=logits.dtype, device="cuda")
    rv.relay_router_backward(x, out["index"], dbuf[:, :e], d_gate=None if d_gate is None else d_gate.cuda(),
                             d_prob=out["d_prob"], normalize=normalize)
    torch.cuda.synchronize()
    assert bool((dbuf[:, e:] == 9.0).all())
    out["d_logits"] = dbuf[:, :e]
    return {k: v.cpu() for k, v in out.items()}


def check(out, want, dtype, tokens):
    assert torch.equal(out["index"], want["index"])
    assert torch.equal(out["counts"], want["counts"])
    assert bool(((out["gate"].double() - want["gate"]).abs() <= SOFT * want["gate"] + 1e-37).all())
    # a sum of `tokens` fp32 terms in pieces: at most tokens/16 + 64 steps in one chain
    steps = (tokens / 16 + 64) * F + SOFT
    assert bool(((out["prob_sum"].double() - want["prob_sum"]).abs() <= steps * want["prob_sum"] + 1e-37).all())
    assert abs(out["loss"].item() - want["loss"].item()) <= (steps + 64 * F) * abs(want["loss"].item())
    assert bool(((out["d_prob"].double() - want["d_prob"]).abs() <= 8 * F * want["d_prob"]).all())
    unit = ref.U if dtype == "bf16" else F
    bound = 2 * SOFT * want["d_logits_size"] + unit * want["d_logits"].abs() + 1e-37
    assert bool(((out["d_logits"].double() - want["d_logits"]).abs() <= bound).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("tokens,experts,top", [
    (1, 1, 1), (1, 8, 2), (3, 5, 5), (16, 64, 2), (33, 32, 32), (100, 60, 4), (257, 128, 8), (1000, 200, 6),
    (5000, 256, 8), (300, 384, 8), (77, 513, 3), (129, 1024, 16), (20000, 33, 1)])
def test_router_matches_definition(tokens, experts, top, normalize, dtype):
    g = torch.Generator().manual_seed(tokens + experts)
    x = (torch.randn(tokens, experts, generator=g) * 2).to(DT[dtype])
    d = torch.randn(tokens, top, generator=g)
    mask = torch.rand(tokens, generator=g) < 0.8 if tokens > 2 else None
    want = ref.router(x, top, normalize, mask, 0.5, d)
    check(run(x, top, normalize, mask, 0.5, d), want, dtype, tokens)
    check(run(x, top, normalize, mask, 0.5, d, extra=3), want, dtype, tokens)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("experts", [7, 48, 256, 1000])
def test_ties_lowest_values_and_empty_rows(experts, dtype):
    g = torch.Generator().manual_seed(5)
    x = torch.randint(-2, 3, (400, experts), generator=g).to(DT[dtype])   # ties everywhere, -0 among them
    x[x == 0] = torch.where(torch.rand(int((x == 0).sum()), generator=g) < 0.5, -0.0, 0.0).to(DT[dtype])
    x[3] = 1.0
    x[4] = torch.finfo(DT[dtype]).min
    x[5] = -math.inf                       # no logit above -inf: the row is not counted
    x[6, 1:] = -math.inf                   # one finite logit
    x[7, :] = torch.finfo(DT[dtype]).min
    x[7, 2] = 0.5
    mask = torch.ones(400, dtype=torch.uint8)
    mask[10:20] = 0
    x[12] = math.nan                       # masked rows are not looked at
    d = torch.randn(400, 4, generator=g)
    for normalize in (False, True):
        clean = x.clone()
        clean[12] = 0.0
        want = ref.router(clean, 4, normalize, mask, 2.0, d)
        check(run(x, 4, normalize, mask, 2.0, d), want, dtype, 400)


def test_nothing_counted():
    x = torch.randn(50, 24)
    out = run(x, 3, mask=torch.zeros(50, dtype=torch.bool), d_gate=torch.ones(50, 3))
    assert bool((out["index"] == -1).all())
    for name in ("gate", "counts", "prob_sum", "loss", "d_prob", "d_logits"):
        assert bool((out[name] == 0).all()), name
    out = run(torch.randn(0, 24), 3)
    for name in ("counts", "prob_sum", "loss", "d_prob"):
        assert bool((out[name] == 0).all()), name


def test_nan_logits_stay_in_range():
    x = torch.randn(64, 40)
    x[::3, ::4] = math.nan
    x[1, 5] = math.inf
    out = run(x, 8)
    assert bool(((out["index"] >= 0) & (out["index"] < 40)).all())
    assert all(len(set(r.tolist())) == 8 for r in out["index"])
    assert bool(torch.isnan(out["gate"][::3]).all())


@pytest.mark.parametrize("normalize", [False, True])
def test_gradient_against_differences(normalize):
    """L = sum(gate * c) + balance loss, along a random direction that changes no choice; the counts are
    constants. Differences in float64 of the definition, at a step of 1e-5."""
    g = torch.Generator().manual_seed(11)
    x = torch.randn(30, 20, generator=g)
    c, d = torch.randn(30, 4, generator=g), torch.randn(30, 20, generator=g)
    out = run(x, 4, normalize, coef=3.0, d_gate=c)
    counts = out["counts"]

    def total(s):
        r = ref.router(x.double() + s * d.double(), 4, normalize, None, 3.0, None, counts)
        assert torch.equal(r["index"], out["index"])
        return ((r["gate"] * c.double()).sum() + r["loss"]).item()
    slope = (total(1e-5) - total(-1e-5)) / 2e-5
    got = (out["d_logits"].double() * d.double()).sum().item()
    size = (out["d_logits"].double().abs() * d.double().abs()).sum().item()
    assert abs(slope - got) <= 1e-6 * size + 1e-8


def test_statistics_summed_over_ranks():
    """Two active ranks: counts (int32) and probability sums (fp32) through relay_allreduce give the
    statistics and the gradient of the whole batch."""
    A, R, t, e, k = 2, 8, 700, 64, 4
    g = torch.Generator().manual_seed(13)
    xs = [torch.randn(t, e, generator=g) for _ in range(A)]
    want = ref.router(torch.cat(xs), k, False, None, 0.1, None)
    logits = [x.cuda() for x in xs]
    index = [torch.empty(t, k, dtype=torch.int32, device="cuda") for _ in range(A)]
    gate = [torch.empty(t, k, device="cuda") for _ in range(A)]
    counts = [torch.empty(e, dtype=torch.int32, device="cuda") for _ in range(A)]
    prob = [torch.empty(e, device="cuda") for _ in range(A)]
    for a in range(A):
        rv.relay_router_forward(logits[a], index[a], gate[a], counts[a], prob[a])
    for bufs, dt in ((counts, rv.I32), (prob, rv.F32)):
        plan = rv.relay_plan(rv.ALLREDUCE, e, dt, A, R)
        rv.relay_allreduce(bufs, bufs, rv.alloc_scratch(plan, "cuda"), e, dt, A, R)
    for a in range(A):
        loss, d_prob = torch.empty(1, device="cuda"), torch.empty(e, device="cuda")
        rv.relay_balance_loss(counts[a], prob[a], k, 0.1, loss, d_prob)
        dx = torch.empty(t, e, device="cuda")
        rv.relay_router_backward(logits[a], index[a], dx, d_prob=d_prob)
        assert torch.equal(counts[a].cpu(), want["counts"])
        assert abs(loss.item() - want["loss"].item()) <= 1e-5 * want["loss"].item()
        part = slice(a * t, (a + 1) * t)
        bound = 2 * SOFT * want["d_logits_size"][part] + F * want["d_logits"][part].abs() + 1e-37
        assert bool(((dx.cpu().double() - want["d_logits"][part]).abs() <= 2 * bound).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_equal_calls_equal_bits(dtype):
    x = torch.randn(9000, 96, generator=torch.Generator().manual_seed(3)).to(DT[dtype])
    a, b = run(x, 6), run(x, 6)
    for name in a:
        assert torch.equal(a[name], b[name]), name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("experts,top", [(8, 3), (60, 4), (128, 8), (256, 8), (600, 5)])
def test_large_offsets_and_near_equal_logits(experts, top, dtype):
    """Rows far from 0 (an additive mask over all experts), rows whose values differ in their last bits
    only, and NaN beside them: the choice is by whole values."""
    g = torch.Generator().manual_seed(17)
    x = torch.randn(300, experts, generator=g)
    x[0:50] = x[0:50] * 100 - 1e9
    x[50:100] = x[50:100] * 1e30
    x[100:200] = 1.0 + torch.randint(0, 40, (100, experts), generator=g) * 2.0 ** -23
    x[200:250] = -3.0 - torch.randint(0, 5, (50, experts), generator=g) * 2.0 ** -22
    x = x.to(DT[dtype])
    for normalize in (False, True):
        want = ref.router(x, top, normalize, None, 1.0, None)
        out = run(x, top, normalize, coef=1.0)
        assert torch.equal(out["index"], want["index"])
        assert torch.equal(out["counts"], want["counts"])
        # exp of a difference d is off by |d| f: 2^-9 covers d up to 88 in bf16's and fp32's arithmetic
        small = want["gate"] > 1e-30
        assert bool(((out["gate"].double() - want["gate"]).abs() <= 2.0 ** -15 * want["gate"] + 1e-30).all()), small.sum()
