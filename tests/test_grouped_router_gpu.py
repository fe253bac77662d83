"""The router with scores, bias and groups against its 64-bit definition: every width of the kernel, ties, near ties, experts
that cannot be chosen, masked and special rows, strides, the gradient against differences, captured calls."""
import math

import pytest
import torch

import grouped_router_ref as ref
import pack_virtual_rank_gb300 as rv

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
F, U = 2.0 ** -24, 2.0 ** -8
# a share of a sum of up to 1024 fp32 scores: exp of x within (2 |x| + 6) F for |x| up to 16, the sum within 10
# steps of a tree, a reciprocal and a product
SOFT = 64 * F


def run(x, top, bias=None, mask=None, d_gate=None, d_prob=None, extra=0, **how):
    t, e = x.shape
    buf = torch.full((t, e + extra), 9.0, dtype=x.dtype, device="cuda")
    xc = buf[:, :e]
    xc.copy_(x)
    out = dict(index=torch.full((t, top), -7, dtype=torch.int32, device="cuda"), gate=torch.full((t, top), 7.0, device="cuda"),
               counts=torch.full((e,), -7, dtype=torch.int32, device="cuda"), prob_sum=torch.full((e,), 7.0, device="cuda"))
    rv.relay_grouped_router_forward(xc, out["index"], out["gate"], out["counts"], out["prob_sum"],
                                    bias=None if bias is None else bias.cuda(), mask=None if mask is None else mask.cuda(), **how)
    dbuf = torch.full((t, e + extra), 9.0, dtype=x.dtype, device="cuda")
    back = {k: how[k] for k in ("score", "normalize", "scale") if k in how}
    rv.relay_grouped_router_backward(xc, out["index"], dbuf[:, :e], d_gate=None if d_gate is None else d_gate.cuda(),
                                     d_prob=None if d_prob is None else d_prob.cuda(), **back)
    torch.cuda.synchronize()
    assert bool((dbuf[:, e:] == 9.0).all())
    out["d_logits"] = dbuf[:, :e]
    return {k: v.cpu() for k, v in out.items()}


def check(out, want, dtype, tokens):
    assert torch.equal(out["index"], want["index"])
    assert torch.equal(out["counts"], want["counts"])
    assert bool(((out["gate"].double() - want["gate"]).abs() <= SOFT * want["gate"].abs() + 1e-36).all())
    steps = (tokens / 16 + 64) * F + SOFT
    assert bool(((out["prob_sum"].double() - want["prob_sum"]).abs() <= steps * want["prob_sum"] + 1e-36).all())
    unit = U if dtype == "bf16" else F
    bound = 2 * SOFT * want["size"] + unit * want["d_logits"].abs() + 1e-36
    assert bool(((out["d_logits"].double() - want["d_logits"]).abs() <= bound).all())


SHAPES = [  # tokens, experts, groups, kept, top
    (1, 1, 1, 1, 1), (1, 8, 2, 1, 2), (3, 6, 3, 2, 4), (5, 64, 8, 4, 8), (33, 32, 32, 5, 5), (100, 60, 4, 2, 6), (64, 256, 8, 4, 8),
    (300, 256, 1, 1, 8), (70, 160, 8, 3, 6), (40, 512, 16, 7, 32), (50, 272, 17, 3, 9), (33, 510, 6, 2, 8), (20, 1024, 4, 4, 16),
    (77, 600, 1, 1, 3), (9, 448, 2, 1, 20), (400, 15, 5, 2, 3), (2000, 24, 3, 2, 4), (60, 384, 12, 12, 8)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("score,normalize,group_sum,biased", [
    ("sigmoid", True, 2, True), ("sigmoid", False, 1, False), ("softmax", False, 1, False), ("softmax", True, 2, True),
    ("sigmoid", True, 2, False), ("softmax", False, 2, False), ("sigmoid", False, 1, True)])
@pytest.mark.parametrize("tokens,experts,groups,kept,top", SHAPES)
def test_matches_definition(tokens, experts, groups, kept, top, score, normalize, group_sum, biased, dtype):
    g = torch.Generator().manual_seed(tokens + experts + top)
    x = (torch.randn(tokens, experts, generator=g) * 2).to(DT[dtype])
    bias = torch.randn(experts, generator=g) * (0.1 if score == "sigmoid" else 0.01) if biased else None
    mask = torch.rand(tokens, generator=g) < 0.8 if tokens > 4 else None
    d, dp = torch.randn(tokens, top, generator=g), torch.rand(experts, generator=g)
    how = dict(groups=groups, kept=kept, group_sum=group_sum, score=score, normalize=normalize, scale=2.5)
    want = ref.route(x, top, bias, mask, d_gate=d, d_prob=dp, **how)
    for extra in (0, 3):
        check(run(x, top, bias, mask, d, dp, extra, **how), want, dtype, tokens)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bias", ["none", "zero", "steps"])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("experts,groups,kept", [(24, 1, 1), (64, 8, 3), (256, 8, 4), (300, 3, 2)])
def test_ties(experts, groups, kept, score, bias, dtype):
    """Equal choice values everywhere: of experts, and of groups."""
    g = torch.Generator().manual_seed(7)
    x = torch.randint(-2, 3, (120, experts), generator=g).to(DT[dtype])
    x[x == 0] = torch.where(torch.rand(int((x == 0).sum()), generator=g) < 0.5, -0.0, 0.0).to(DT[dtype])
    x[3] = 1.0
    x[4] = torch.finfo(DT[dtype]).min
    x[6, 1:] = -math.inf
    b = {"none": None, "zero": torch.zeros(experts), "steps": torch.randint(0, 2, (experts,), generator=g) * 0.25}[bias]
    for group_sum in (1, 2):
        how = dict(groups=groups, kept=kept, group_sum=group_sum, score=score, scale=1.0)
        want = ref.route(x, 8, b, **how)
        check(run(x, 8, b, **how), want, dtype, 120)


@pytest.mark.parametrize("groups,kept", [(1, 1), (8, 4)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_choice_values_nearer_than_fp32_tells(groups, kept, score):
    """Logits and biases a few units in the last place apart: the choice is by exact values."""
    g = torch.Generator().manual_seed(3)
    x = 1.0 + torch.randint(0, 30, (200, 64), generator=g) * 2.0 ** -23
    x[100:] = torch.randn(100, 64, generator=g)
    s = torch.sigmoid(x[100:].double()) if score == "sigmoid" else torch.softmax(x[100:].double(), 1)
    bias = torch.randint(0, 9, (64,), generator=g) * 2.0 ** -26
    bias[:32] = (0.7 - s[0, :32]).float() if score == "sigmoid" else (0.05 - s[0, :32]).float()   # row 100: all but equal
    how = dict(groups=groups, kept=kept, score=score, group_sum=2)
    want = ref.route(x, 8, bias, **how)
    out = run(x, 8, bias, **how)
    assert torch.equal(out["index"], want["index"])
    assert torch.equal(out["counts"], want["counts"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("experts,groups,kept,top", [(8, 1, 1, 2), (93, 1, 1, 1), (64, 8, 4, 8), (256, 8, 8, 3), (512, 1, 1, 32)])
def test_the_best_stand_behind_equal_ones(experts, groups, kept, top, score, dtype):
    """The choice ends among equal ones; a few nearer to them than fp32 or a key's upper bits tell, and larger, come later."""
    g = torch.Generator().manual_seed(13)
    x, bias = torch.ones(90, experts), torch.zeros(experts)
    for r in range(1, 90):                                # row 0: all equal
        some = torch.randperm(experts, generator=g)[:1 + r % 6]
        if dtype == "f32":
            x[r, some] += 2.0 ** -23 * (1 + r % 5)
        x[r, torch.randperm(experts, generator=g)[:r % 3]] = 0.5
    ends = torch.arange(max(0, experts - 3), experts)
    x[5] = 1.0
    if dtype == "f32":
        x[5, ends] += 2.0 ** -22
    raised = bias.clone()
    raised[ends] = 2.0 ** -30
    for b in (None, bias, raised):
        how = dict(groups=groups, kept=kept, score=score, group_sum=2)
        xt = x.to(DT[dtype])
        want = ref.route(xt, top, b, **how)
        out = run(xt, top, b, **how)
        assert torch.equal(out["index"], want["index"])
        assert torch.equal(out["counts"], want["counts"])


def test_experts_that_cannot_be_chosen():
    g = torch.Generator().manual_seed(5)
    x = torch.randn(90, 32, generator=g)
    x[:30, ::3] = -math.inf
    x[40] = -math.inf
    x[41, 4:] = -math.inf
    bias = torch.randn(32, generator=g) * 0.1
    bias[16:24] = -math.inf                    # a group of its own
    bias[0:6] = -math.inf
    d, dp = torch.randn(90, 8, generator=g), torch.rand(32, generator=g)
    for how in (dict(groups=4, kept=2), dict(groups=8, kept=8), dict(groups=1), dict(groups=4, kept=2, group_sum=1)):
        for score in ("sigmoid", "softmax"):
            want = ref.route(x, 8, bias, d_gate=d, d_prob=dp, score=score, **how)
            assert int((want["index"] < 0).sum()) > 0
            check(run(x, 8, bias, None, d, dp, score=score, **how), want, "f32", 90)
    dead = torch.full((32,), -math.inf)
    out = run(x, 4, dead, d_gate=d[:, :4].contiguous(), d_prob=dp)
    assert bool((out["index"] == -1).all())
    for name in ("gate", "counts", "prob_sum", "d_logits"):
        assert bool((out[name] == 0).all()), name


def test_wide_biases_and_large_logits():
    """Biases that outweigh the scores by far, logits that saturate them."""
    g = torch.Generator().manual_seed(9)
    x = torch.randn(100, 48, generator=g) * 4
    x[50:] *= 5
    for bias in (torch.randn(48, generator=g) * 100, torch.where(torch.rand(48, generator=g) < 0.3, -1e30, 0.0), torch.full((48,), 3e38)):
        for groups, kept in ((1, 1), (6, 2)):
            how = dict(groups=groups, kept=kept)
            want = ref.route(x, 6, bias.float(), **how)
            out = run(x, 6, bias.float(), **how)
            assert torch.equal(out["index"], want["index"])


def test_special_logits():
    x = torch.randn(64, 40)
    x[::3, ::4] = math.nan
    x[1, 5] = math.inf
    bias = torch.randn(40) * 0.1
    for score in ("sigmoid", "softmax"):
        for b in (None, bias):
            for groups, kept in ((1, 1), (4, 2)):
                out = run(x, 8, b, score=score, groups=groups, kept=kept)
                assert bool(((out["index"] >= 0) & (out["index"] < 40)).all())
                assert all(len(set(r.tolist())) == 8 for r in out["index"])
                assert bool(torch.isnan(out["gate"][::3]).all()) and bool(torch.isnan(out["prob_sum"]).all())
                assert bool(torch.isnan(out["d_logits"][::3]).any(dim=1).all()) or score == "sigmoid"
    out = run(x[1:2], 8, None, score="sigmoid", normalize=False)
    assert out["index"][0, 0] == 5 and out["gate"][0, 0] == 1.0       # a score of +inf is 1


def test_nothing_counted():
    out = run(torch.randn(50, 24), 3, mask=torch.zeros(50, dtype=torch.bool), d_gate=torch.ones(50, 3))
    assert bool((out["index"] == -1).all())
    for name in ("gate", "counts", "prob_sum", "d_logits"):
        assert bool((out[name] == 0).all()), name
    out = run(torch.randn(0, 24), 3)
    assert bool((out["counts"] == 0).all()) and bool((out["prob_sum"] == 0).all())


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("normalize", [False, True])
def test_gradient_against_differences(score, normalize):
    """L = sum(gate * c) + sum(prob_sum * dp), along a random direction that changes no choice; differences in 64 bits of the
    definition at a step of 1e-5."""
    g = torch.Generator().manual_seed(11)
    x = torch.randn(30, 24, generator=g)
    bias = torch.randn(24, generator=g) * 0.05
    c, dp, d = torch.randn(30, 4, generator=g), torch.rand(24, generator=g), torch.randn(30, 24, generator=g)
    how = dict(groups=6, kept=3, score=score, normalize=normalize, scale=1.5)
    out = run(x, 4, bias, None, c, dp, **how)

    def total(h):
        r = ref.route(x.double() + h * d.double(), 4, bias, **how)
        assert torch.equal(r["index"], out["index"])
        return ((r["gate"] * c.double()).sum() + (r["prob_sum"] * dp.double()).sum()).item()
    slope = (total(1e-5) - total(-1e-5)) / 2e-5
    got = (out["d_logits"].double() * d.double()).sum().item()
    size = (out["d_logits"].double().abs() * d.double().abs()).sum().item()
    # the differences' own error: a third of the third derivative, at most 1e-10 of the size, and 1e-16 / 1e-5 of the total
    assert abs(slope - got) <= 2 * SOFT * size + 1e-9 * size + 1e-9


@pytest.mark.parametrize("experts", [1, 7, 256, 1000])
def test_bias_update(experts):
    g = torch.Generator().manual_seed(experts)
    counts = torch.randint(0, 50, (experts,), generator=g, dtype=torch.int32)
    counts[experts // 2] = 2 ** 31 - 1 if experts == 256 else 25
    bias = torch.randn(experts, generator=g)
    less = counts.to(torch.int64).sum() - experts * counts.to(torch.int64)
    want = bias + torch.sign(less).float() * 0.001
    c, b, out = counts.cuda(), bias.cuda(), torch.empty(experts, device="cuda")
    rv.relay_router_bias_update(c, b, 0.001, out)
    assert torch.equal(out.cpu(), want) and torch.equal(b.cpu(), bias)
    rv.relay_router_bias_update(c, b, 0.001)
    assert torch.equal(b.cpu(), want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_equal_calls_equal_bits_captured_and_on_another_stream(dtype):
    g = torch.Generator().manual_seed(3)
    x = torch.randn(9000, 96, generator=g).to(DT[dtype]).cuda()
    bias = (torch.randn(96, generator=g) * 0.1).cuda()
    d = torch.randn(9000, 6, device="cuda")
    ws = rv.alloc_router_workspace(9000, 96, "cuda")
    out = dict(index=torch.empty(9000, 6, dtype=torch.int32, device="cuda"), gate=torch.empty(9000, 6, device="cuda"),
               counts=torch.empty(96, dtype=torch.int32, device="cuda"), prob_sum=torch.empty(96, device="cuda"))
    loss, d_prob, dx = torch.empty(1, device="cuda"), torch.empty(96, device="cuda"), torch.empty_like(x)
    kept = torch.empty_like(bias)

    def step(stream=None):
        rv.relay_grouped_router_forward(x, out["index"], out["gate"], out["counts"], out["prob_sum"], bias=bias, groups=8, kept=3,
                                        workspace=ws, stream=stream)
        rv.relay_balance_loss(out["counts"], out["prob_sum"], 6, 0.01, loss, d_prob, stream=stream)
        rv.relay_grouped_router_backward(x, out["index"], dx, d_gate=d, d_prob=d_prob, stream=stream)
        rv.relay_router_bias_update(out["counts"], bias, 0.001, kept, stream=stream)
    written = list(out.values()) + [loss, d_prob, dx, kept]
    step()
    first = [v.clone() for v in written]
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    step(stream)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(written, first))
    with torch.cuda.graph(graph):
        step()
    for v in written:
        v.zero_()
    ws.fill_(255)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(written, first))


def test_statistics_summed_over_ranks_balance_the_next_step():
    """Two ranks: counts and shares through relay_allreduce, the balance loss and the bias update of the whole batch."""
    A, R, t, e, k = 2, 8, 500, 64, 4
    g = torch.Generator().manual_seed(13)
    xs = [torch.randn(t, e, generator=g) + torch.linspace(-1, 1, e) for _ in range(A)]
    bias = torch.randn(e, generator=g) * 0.1
    how = dict(groups=8, kept=4)
    want = ref.route(torch.cat(xs), k, bias, **how)
    outs = [run_rank(x, k, bias, how) for x in xs]
    for i, dt in ((2, rv.I32), (3, rv.F32)):
        plan = rv.relay_plan(rv.ALLREDUCE, e, dt, A, R)
        bufs = [o[i] for o in outs]
        rv.relay_allreduce(bufs, bufs, rv.alloc_scratch(plan, "cuda"), e, dt, A, R)
    less = want["counts"].to(torch.int64).sum() - e * want["counts"].to(torch.int64)
    n, per = A * t, 0.1 * e * want["counts"].double() / (k * (A * t) ** 2)
    for o in outs:
        loss, d_prob, b = torch.empty(1, device="cuda"), torch.empty(e, device="cuda"), bias.cuda()
        rv.relay_balance_loss(o[2], o[3], k, 0.1, loss, d_prob)
        rv.relay_router_bias_update(o[2], b, 0.01)
        assert torch.equal(o[2].cpu(), want["counts"])
        assert torch.equal(b.cpu(), bias + torch.sign(less).float() * 0.01)
        assert abs(loss.item() - (per * want["prob_sum"]).sum().item()) <= ((n / 16 + 128) * F + SOFT) * abs(loss.item())


def run_rank(x, k, bias, how):
    t, e = x.shape
    out = (torch.empty(t, k, dtype=torch.int32, device="cuda"), torch.empty(t, k, device="cuda"),
           torch.empty(e, dtype=torch.int32, device="cuda"), torch.empty(e, device="cuda"))
    rv.relay_grouped_router_forward(x.cuda(), *out, bias=bias.cuda(), **how)
    return out


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_a_single_renormalized_gate_has_no_gradient(score):
    """Its gate is the scale, whatever the logits: the gradient is 0, not what rounding leaves of a difference."""
    x, d = torch.randn(300, 24), torch.randn(300, 1)
    out = run(x, 1, torch.randn(24) * 0.1, d_gate=d, score=score, normalize=True, scale=2.5)
    assert bool((out["gate"] == 2.5).all()) and bool((out["d_logits"] == 0).all())
