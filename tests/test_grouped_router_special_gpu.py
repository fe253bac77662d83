"""The router with scores, bias and groups on rows at the ends: NaN and infinite logits in the choice and in the
gradients, scores next to the end of fp32's range."""
import math

import pytest
import torch

import grouped_router_ref as ref
from test_grouped_router_gpu import F, SOFT, run

pytestmark = pytest.mark.gpu

GROUPINGS = [(1, 1), (4, 2), (8, 8)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("group_sum", [1, 2])
@pytest.mark.parametrize("groups,kept", GROUPINGS)
def test_a_nan_logit_stands_below_the_others(groups, kept, group_sum, biased, score, dtype):
    """Where enough others can be chosen, the choice is the one without the NaN experts; and the rows beside stay."""
    g = torch.Generator().manual_seed(5)
    x = (torch.randn(64, 40, generator=g) * 2).to(dtype)
    bad = torch.zeros(64, dtype=torch.bool)
    bad[::3] = True
    x[::3, ::4] = math.nan
    x[3, 0], x[3, 8] = math.nan, math.nan
    x[6, 1] = -math.inf
    bias = torch.randn(40, generator=g) * 0.02 if biased else None
    how = dict(groups=groups, kept=kept, group_sum=group_sum, score=score)
    want = ref.route(torch.where(torch.isnan(x), -math.inf, x.double()), 8, bias, **how)
    out = run(x, 8, bias, **how)
    assert torch.equal(out["index"], want["index"])
    assert torch.equal(out["counts"], want["counts"])
    assert bool(torch.isnan(out["gate"][bad]).all()) and bool(torch.isfinite(out["gate"][~bad]).all())
    assert bool(((out["gate"][~bad].double() - want["gate"][~bad]).abs() <= SOFT * want["gate"][~bad]).all())
    assert bool(torch.isnan(out["prob_sum"]).all())


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("group_sum", [1, 2])
def test_more_chosen_than_there_are_numbers(group_sum, biased, score):
    """The NaN experts fill what is left, by their numbers; groups of nothing else stand behind all others, and before
    one of which nothing can be chosen."""
    x = torch.full((3, 12), math.nan)
    x[0, [3, 7]] = torch.tensor([1.0, 2.0])
    x[1, 4:8] = torch.tensor([0.5, -3.0, 0.5, 0.25])
    x[2, :4] = -math.inf
    bias = torch.zeros(12) if biased else None
    how = dict(score=score, group_sum=group_sum)
    out = run(x, 6, bias, **how)
    assert out["index"][0].tolist() == [7, 3, 0, 1, 2, 4]
    assert out["index"][1].tolist() == [4, 6, 7, 5, 0, 1]
    assert out["index"][2].tolist() == [4, 5, 6, 7, 8, 9]
    out = run(x, 6, bias, groups=3, kept=2, **how)
    assert out["index"][1].tolist() == [4, 6, 7, 5, 0, 1]
    assert out["index"][2].tolist() == [4, 5, 6, 7, 8, 9]


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("group_sum", [1, 2])
@pytest.mark.parametrize("groups,kept", GROUPINGS)
def test_infinite_logits_are_the_largest(groups, kept, group_sum, biased):
    """Softmax: experts of +inf share the row, the others' scores are 0 (as with a logit far above the rest). The
    row's gates show it as NaN."""
    g = torch.Generator().manual_seed(6)
    x = torch.randn(30, 40, generator=g)
    x[::2, 17] = math.inf
    x[4, 3], x[8, 39], x[8, 0] = math.inf, math.inf, -math.inf
    bias = torch.randn(40, generator=g) * 0.02 if biased else None
    how = dict(groups=groups, kept=kept, group_sum=group_sum, score="softmax")
    want = ref.route(torch.where(x == math.inf, 1e4, x.double()), 8, bias, **how)
    out = run(x, 8, bias, **how)
    assert torch.equal(out["index"], want["index"])
    assert bool(torch.isnan(out["gate"][::2]).all()) and bool(torch.isfinite(out["gate"][1::2]).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("normalize", [False, True])
def test_a_nan_logit_shows_in_its_row_of_the_gradient(normalize, score, dtype):
    """In counted rows alone, whichever gradient comes in; masked rows are 0 and the others as they were."""
    g = torch.Generator().manual_seed(8)
    clean = (torch.randn(60, 40, generator=g)).to(dtype)
    x, mask = clean.clone(), torch.ones(60, dtype=torch.bool)
    x[::3, 5::7] = math.nan
    mask[::6] = False
    d, dp = torch.randn(60, 8, generator=g), torch.rand(40, generator=g)
    how = dict(groups=4, kept=2, score=score, normalize=normalize)
    bad = torch.zeros(60, dtype=torch.bool)
    bad[::3] = True
    for dg, ds in ((d, dp), (d, None), (None, dp)):
        out = run(x, 8, None, mask, dg, ds, **how)["d_logits"]
        base = run(clean, 8, None, mask, dg, ds, **how)["d_logits"]
        shown = torch.isnan(out).any(dim=1)
        assert torch.equal(shown, bad & mask)
        assert bool((out[~mask] == 0).all()) and torch.equal(out[~bad], base[~bad])
        if score == "softmax" or ds is not None or normalize:
            assert bool(torch.isnan(out[bad & mask]).all(dim=1).any())


@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_chosen_scores_of_zero(dtype, normalize):
    """Softmax: the experts that can be chosen lie so far below drained ones that their scores are 0. Gates are 0 and have no
    gradient; the shares' gradient is the usual one."""
    g = torch.Generator().manual_seed(9)
    x = torch.randn(50, 24, generator=g)
    x[:40, :4] += 150.0
    x = x.to(dtype)
    bias = torch.zeros(24)
    bias[:4] = -math.inf
    d, dp = torch.randn(50, 3, generator=g), torch.rand(24, generator=g)
    how = dict(score="softmax", normalize=normalize, scale=2.5)
    out = run(x, 3, bias, None, d, dp, **how)
    want = ref.route(x, 3, bias, d_gate=torch.where(torch.arange(50)[:, None] < 40, 0.0, d), d_prob=dp, **how)
    assert torch.equal(out["index"], want["index"])
    assert bool((out["gate"][:40] == 0).all()) and bool((out["gate"][40:] > 0).all())
    unit = 2.0 ** -24 if dtype is torch.float32 else 2.0 ** -8
    bound = 2 * SOFT * want["size"] + unit * want["d_logits"].abs() + 1e-36
    assert bool(((out["d_logits"].double() - want["d_logits"]).abs() <= bound).all())


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("top", [1, 4])
@pytest.mark.parametrize("normalize", [False, True])
def test_gates_and_gradients_agree_on_what_is_zero(normalize, top, score):
    """Scores from 2^-110 to 2^-160 (softmax: of the row's largest): what is below fp32's normal range is 0, in the gates and
    in their gradients, and what is above it is right to its rounding."""
    x = -torch.linspace(110, 160, 401)[:, None] * math.log(2.0) + torch.linspace(-0.2, 0.2, 16)
    bias = torch.zeros(16)
    if score == "softmax":
        x[:, 0] = 0.0
        bias[0] = -math.inf
    d = torch.ones(401, top) + torch.arange(top)
    out = run(x, top, bias, None, d, None, score=score, normalize=normalize)
    index = out["index"].long()
    # the scores' logarithms to the base 2; the two sides' exponentials may differ next to the border
    power = x.double().gather(1, index) / math.log(2.0)
    below, above = power < -126.01, power > -125.99
    assert bool((out["gate"][below] == 0).all()) and bool((out["gate"][above] > 0).all())
    assert bool(torch.isfinite(out["d_logits"]).all())
    chosen = out["d_logits"].gather(1, index)
    assert bool((chosen[below] == 0).all())
    rows = above.all(dim=1)
    want = ref.route(x[rows], top, bias, d_gate=d[rows], score=score, normalize=normalize)
    # exp of x within (2 |x| + 6) F for the fast exponential, |x| <= 88, both of a quotient's sides; gates by the exact one
    off = (out["gate"][rows].double() - want["gate"]).abs()
    assert bool((off <= 16 * F * want["gate"] + 2.0 ** -150).all())
    off = (out["d_logits"][rows].double() - want["d_logits"]).abs()
    assert bool((off <= 4 * (2 * 88 + 6) * F * want["size"] + 2.0 ** -126).all())


@pytest.mark.parametrize("size", [1e-7, 1.0, 1000.0, 1e15])
@pytest.mark.parametrize("normalize", [False, True])
def test_gradients_of_small_sigmoids(normalize, size):
    """All scores of a row near the end of fp32's range: shares and renormalized gates are ordinary numbers, and so are their
    gradients, for small and for large ones coming in."""
    g = torch.Generator().manual_seed(10)
    x = -86.0 + torch.randn(64, 24, generator=g) * 0.3
    x[5, 7], x[6, :20] = -math.inf, -math.inf
    x[7, 3] = 2.0
    d, dp = torch.randn(64, 4, generator=g) * size, torch.randn(24, generator=g) * size
    for dg, ds in ((d, dp), (d, None), (None, dp)):
        how = dict(score="sigmoid", normalize=normalize)
        out = run(x, 4, None, None, dg, ds, **how)
        want = ref.route(x, 4, d_gate=dg, d_prob=ds, **how)
        assert torch.equal(out["index"], want["index"])
        # exp of x within (2 |x| + 6) F, in the score, the sum and the slope
        bound = 4 * (2 * 88 + 6) * F * want["size"] + 2.0 ** -126
        assert bool(((out["d_logits"].double() - want["d_logits"]).abs() <= bound).all())
