"""The norm of all gradients and their clipping against 64 bits: types, odd sizes and addresses, lists longer than a
launch, values at the ends of the range, captured calls, other streams."""
import math

import pytest
import torch

import pack_virtual_rank_gb300 as rv

pytestmark = pytest.mark.gpu
F, U = 2.0 ** -24, 2.0 ** -8
# a chain of 16 squares and two additions of four chains, halved by the root, and the root's own rounding
NORM = 10 * F
# the norm, its addition, the division, the product
CLIP = NORM + 3 * F
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def norm_of(xs):
    return math.sqrt(sum(float(x.double().square().sum()) for x in xs))


def views(sizes, dtypes, skips, seed=0, scale=1.0):
    """Tensors at odd places of larger buffers, and the buffers."""
    g = torch.Generator().manual_seed(seed)
    bufs = [torch.full((n + 40,), 7.0, dtype=d, device="cuda") for n, d in zip(sizes, dtypes)]
    xs = [b[8 + s:8 + s + n] for b, n, s in zip(bufs, sizes, skips)]
    for x in xs:
        x.copy_((torch.randn(x.shape, generator=g) * scale).to(x.dtype))
    return xs, bufs


def check_clip(xs, outs, norm, max_norm):
    c = min(1.0, max_norm / (norm + 1e-6))
    for x, y in zip(xs, outs):
        want = x.double() * c
        unit = F if x.dtype is torch.float32 else U
        # values below the normal range round by half its smallest step
        assert bool(((y.double() - want).abs() <= (CLIP + unit) * want.abs() + 2.0 ** -134).all())


SIZES = [1, 0, 3, 7, 8, 255, 2048, 8191, 8192, 8193, 16384, 16391, 70001]


@pytest.mark.parametrize("kind", ["f32", "bf16", "mixed"])
@pytest.mark.parametrize("skew", [0, 1, 5])
def test_norm_and_clip(kind, skew):
    dtypes = [DT[kind] if kind != "mixed" else (torch.float32, torch.bfloat16)[i % 2] for i in range(len(SIZES))]
    xs, bufs = views(SIZES, dtypes, [skew * i % 8 for i in range(len(SIZES))], seed=skew)
    grads, norm = rv.make_grads(xs), torch.full((1,), 7.0, device="cuda")
    rv.relay_grad_norm(grads, norm)
    want = norm_of(xs)
    assert abs(norm.item() - want) <= NORM * want
    before = [x.clone() for x in xs]
    for out_skew in (0, 1):
        outs, obufs = views(SIZES, dtypes, [(skew * i + out_skew) % 8 for i in range(len(SIZES))], seed=9)
        rv.relay_grad_clip(grads, norm, 0.5, out=rv.make_grads(outs))
        check_clip(before, outs, want, 0.5)
        for b, y in zip(obufs, outs):
            assert int((b == 7.0).sum()) >= 40                      # nothing beside the tensors is written
    rv.relay_grad_clip(grads, norm, 0.5)
    check_clip(before, xs, want, 0.5)
    for b in bufs:
        assert int((b == 7.0).sum()) >= 40


def test_nothing_to_clip_leaves_every_bit():
    xs, _ = views([1000, 77], [torch.bfloat16, torch.float32], [1, 2])
    before = [x.clone() for x in xs]
    grads, norm = rv.make_grads(xs), torch.empty(1, device="cuda")
    rv.relay_grad_norm(grads, norm)
    rv.relay_grad_clip(grads, norm, 1e9)
    outs = [torch.zeros_like(x) for x in xs]
    rv.relay_grad_clip(grads, norm, 1e9, out=rv.make_grads(outs))
    for x, b, y in zip(xs, before, outs):
        assert torch.equal(x, b) and torch.equal(y, b)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_what_is_not_finite_shows_and_is_left(kind, bad):
    xs, _ = views([5000, 30], [DT[kind]] * 2, [0, 0])
    xs[0][4321] = bad
    before = [x.clone() for x in xs]
    grads, norm = rv.make_grads(xs), torch.empty(1, device="cuda")
    rv.relay_grad_norm(grads, norm)
    assert math.isnan(norm.item()) if math.isnan(bad) else norm.item() == math.inf
    rv.relay_grad_clip(grads, norm, 1.0)
    for x, b in zip(xs, before):
        assert torch.equal(x.nan_to_num(3.0, 4.0, 5.0), b.nan_to_num(3.0, 4.0, 5.0))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [1e-38, 1e-30, 3e-20, 1e-14, 1e15, 3e18, 1e25, 1e33])
def test_whole_range(kind, scale):
    xs, _ = views([40000, 3], [DT[kind]] * 2, [1, 0], scale=scale)
    xs[1].fill_(0.0)
    norm = torch.empty(1, device="cuda")
    rv.relay_grad_norm(rv.make_grads(xs), norm)
    want = norm_of(xs)
    assert abs(norm.item() - want) <= NORM * want + 2.0 ** -149


def test_large_beside_small():
    x = torch.full((100000,), 1e-20, device="cuda")
    y = torch.full((50000,), 1e20, device="cuda")
    norm = torch.empty(1, device="cuda")
    for xs in ([x, y], [y, x], [x], [y]):
        rv.relay_grad_norm(rv.make_grads(xs), norm)
        assert abs(norm.item() - norm_of(xs)) <= NORM * norm_of(xs)


@pytest.mark.parametrize("n", [0, 1, 48, 49, 512, 513, 1500])
def test_lists_of_any_length(n):
    g = torch.Generator().manual_seed(n)
    sizes = [int(s) for s in torch.randint(0, 300, (n,), generator=g)]
    xs, _ = views(sizes, [(torch.bfloat16, torch.float32)[i % 3 == 0] for i in range(n)], [i % 8 for i in range(n)])
    grads, norm = rv.make_grads(xs), torch.full((1,), 7.0, device="cuda")
    rv.relay_grad_norm(grads, norm)
    want = norm_of(xs)
    assert abs(norm.item() - want) <= NORM * want
    before = [x.clone() for x in xs]
    rv.relay_grad_clip(grads, norm, 0.01)
    check_clip(before, xs, want, 0.01)


def test_norms_of_ranks_join():
    xs, _ = views([3000, 4000], [torch.float32] * 2, [0, 0])
    norms = torch.empty(2, device="cuda")
    for a in range(2):
        rv.relay_grad_norm(rv.make_grads([xs[a]]), norms[a:a + 1])
    norm = torch.empty(1, device="cuda")
    rv.relay_grad_norm(rv.make_grads([norms]), norm)
    assert abs(norm.item() - norm_of(xs)) <= 2 * NORM * norm_of(xs)


def test_a_tensor_twice_counts_twice():
    x = torch.randn(1000, device="cuda")
    norm = torch.empty(1, device="cuda")
    rv.relay_grad_norm(rv.make_grads([x, x]), norm)
    assert abs(norm.item() - norm_of([x, x])) <= NORM * norm_of([x, x])
    with pytest.raises(rv.RelayError, match="overlaps another"):
        rv.relay_grad_clip(rv.make_grads([x, x]), norm, 1.0)


def test_captured_replayed_and_on_another_stream():
    xs, _ = views([70000, 9, 5], [torch.float32, torch.bfloat16, torch.float32], [0, 1, 3])
    outs = [torch.zeros_like(x) for x in xs]
    grads, to, norm = rv.make_grads(xs), rv.make_grads(outs), torch.empty(1, device="cuda")
    ws = rv.alloc_grad_workspace(grads, "cuda")
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    rv.relay_grad_norm(grads, norm, workspace=ws, stream=stream)
    rv.relay_grad_clip(grads, norm, 2.0, out=to, stream=stream)
    torch.cuda.synchronize()
    eager = [norm.clone()] + [y.clone() for y in outs]
    with torch.cuda.graph(graph):
        rv.relay_grad_norm(grads, norm, workspace=ws)
        rv.relay_grad_clip(grads, norm, 2.0, out=to)
    for y in outs:
        y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(eager, [norm] + outs):
        assert torch.equal(a, b)                      # the same bits, captured or not
    for x in xs:
        x.mul_(3.0)
    ws.fill_(255)                                     # whatever the workspace holds
    graph.replay()
    torch.cuda.synchronize()
    want = norm_of(xs)
    assert abs(norm.item() - want) <= NORM * want
    check_clip(xs, outs, want, 2.0)


def test_more_bytes_than_32_bits_number():
    x = torch.ones((1 << 32) // 2 + 12345, dtype=torch.bfloat16, device="cuda")
    x[-3:] = 100.0
    norm = torch.empty(1, device="cuda")
    rv.relay_grad_norm(rv.make_grads([x]), norm)
    want = math.sqrt(x.numel() - 3 + 3 * 10000.0)
    assert abs(norm.item() - want) <= NORM * want
    rv.relay_grad_clip(rv.make_grads([x]), norm, want / 2)
    half = torch.tensor(0.5, dtype=torch.bfloat16).item()
    assert bool((x[:-3] == half).all()) and bool((x[-3:] == 50.0).all())


def test_many_empty_tensors_between_others():
    full = [torch.randn(40000, device="cuda"), torch.randn(9, device="cuda").bfloat16()]
    empty = [torch.empty(0, device="cuda")] * 600
    for xs in (empty + full, full[:1] + empty + full[1:] + empty, empty + full[:1] + empty + full[1:] + empty):
        norm = torch.full((1,), 7.0, device="cuda")
        rv.relay_grad_norm(rv.make_grads(xs), norm)
        assert abs(norm.item() - norm_of(full)) <= NORM * norm_of(full)
        outs = [torch.zeros_like(x) for x in xs]
        rv.relay_grad_clip(rv.make_grads(xs), norm, 0.5, out=rv.make_grads(outs))
        check_clip(xs, outs, norm_of(full), 0.5)
