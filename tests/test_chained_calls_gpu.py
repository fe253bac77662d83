"""Calls that read what the call before them wrote, queued without a pause: each may start before the one before has ended, and
sees all of it. Tensors and rows off the 16-byte grid among them, whose ends are read value by value."""
import math

import pytest
import torch

import fp8_ref
import pack_virtual_rank_gb300 as rv

pytestmark = pytest.mark.gpu
F = 2.0 ** -24


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("count", [700, 70_001, 3_000_001])
def test_norm_and_clipping_in_turn(count, dtype):
    """Each round clips to about half of the norm, until the 1e-6 that is added to it takes over."""
    buf = torch.ones(count + 9, dtype=dtype, device="cuda")
    xs = [buf[1:1 + count], torch.ones(5, dtype=dtype, device="cuda")]
    grads, n = rv.make_grads(xs), 40
    norms = torch.zeros(n + 1, device="cuda")
    ws = rv.alloc_grad_workspace(grads, "cuda")
    rv.relay_grad_norm(grads, norms[:1], workspace=ws)
    first = math.sqrt(count + 5)
    limits = [first / 2.0 ** (i + 1) for i in range(n)]
    for i in range(n):
        rv.relay_grad_clip(grads, norms[i:i + 1], limits[i])
        rv.relay_grad_norm(grads, norms[i + 1:i + 2], workspace=ws)
    torch.cuda.synchronize()
    got = norms.double().cpu()
    unit = 2.0 ** -24 if dtype is torch.float32 else 2.0 ** -8
    # once the norm is far below 1e-6 the values leave the type's normal range: each is off by half its smallest step at most (and by
    # one of the product in fp32), and the norm by no more than the norm of these errors, root of the count times one; and by its own
    step = math.sqrt(count + 5) * (2.0 ** -150 + (0.0 if dtype is torch.float32 else 2.0 ** -134)) + 2.0 ** -150
    for i in range(n):
        # the limit over the norm before, with 1e-6 added to it; the factor's roundings, the value's, the norm's
        want = got[i] * min(1.0, limits[i] / (got[i].item() + 1e-6))
        assert abs(got[i + 1] - want) <= (13 * F + unit) * want + step, i
    assert got[n] < 2.0 ** (1 - n) * first


@pytest.mark.parametrize("rows,cols", [(300, 256), (300, 250), (37, 1001), (1000, 1000)])
def test_products_and_quantizations_in_turn(rows, cols):
    """y is quantized behind the product that writes it, over and over with another input."""
    g = torch.Generator().manual_seed(rows)
    xs = [torch.randn(rows, cols, generator=g).bfloat16().cuda() for _ in range(12)]
    w = rv.alloc_fp8(cols, cols, "cuda", tiles=True)
    rv.relay_quantize_fp8(torch.randn(cols, cols, generator=g).cuda(), *w, tiles=True)
    xq, y = rv.alloc_fp8(rows, cols, "cuda"), torch.empty(rows, cols, device="cuda", dtype=torch.bfloat16)
    out = [rv.alloc_fp8(rows, cols, "cuda") + rv.alloc_fp8(cols, rows, "cuda") for _ in xs]
    for x, (q, s, qt, st) in zip(xs, out):
        rv.relay_quantize_fp8(x, *xq)
        rv.relay_matmul_fp8(*xq, *w, y)
        rv.relay_quantize_fp8(y, q, s, qt, st)
    torch.cuda.synchronize()
    for x, (q, s, qt, st) in zip(xs, out):
        one = rv.alloc_fp8(rows, cols, "cuda")
        rv.relay_quantize_fp8(x, *one)
        torch.cuda.synchronize()
        rv.relay_matmul_fp8(*one, *w, y)
        torch.cuda.synchronize()
        want, want_s = fp8_ref.quantize(y.cpu(), False)
        assert torch.equal(q.float().cpu().double(), want) and torch.equal(s.cpu().double(), want_s)
        want, want_s = fp8_ref.quantize(y.cpu().t(), False)
        assert torch.equal(qt.float().cpu().double(), want) and torch.equal(st.cpu().double(), want_s)
