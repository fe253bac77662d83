"""One training step of a layer of experts, as the calls are used together: the ranks' tokens are routed, their counts summed
over the ranks, rows sorted by expert, quantized and multiplied, the gates' and rows' gradients taken back, all gradients
clipped by their global norm. Against the same step in 64 bits on the same choices and quantized operands."""
import pytest
import torch

import fp8_ref
import grouped_router_ref
import pack_virtual_rank_gb300 as rv

pytestmark = pytest.mark.gpu
U = 2.0 ** -8


@pytest.mark.parametrize("captured", [False, True])
def test_a_step(captured):
    A, R, t, dim, wide, experts, k = 2, 8, 150, 200, 264, 8, 3
    g = torch.Generator().manual_seed(4)
    x = [torch.randn(t, dim, generator=g).bfloat16() for _ in range(A)]
    logits = [torch.randn(t, experts, generator=g) * 1.5 for _ in range(A)]
    bias = torch.randn(experts, generator=g) * 0.1
    w = (torch.randn(experts, wide, dim, generator=g) * 0.1).bfloat16()
    dout = [(torch.randn(t, wide, generator=g) * 0.01).bfloat16() for _ in range(A)]
    how = dict(groups=4, kept=2, scale=1.5)
    rows = A * t * k
    cuda = dict(device="cuda")
    xc, lc, wc, dc, bc = [v.cuda() for v in x], [v.cuda() for v in logits], w.cuda(), [v.cuda() for v in dout], bias.cuda()
    f32, i32 = dict(dtype=torch.float32, **cuda), dict(dtype=torch.int32, **cuda)
    index, gate = [torch.empty(t, k, **i32) for _ in range(A)], [torch.empty(t, k, **f32) for _ in range(A)]
    counts, prob = [torch.empty(experts, **i32) for _ in range(A)], [torch.empty(experts, **f32) for _ in range(A)]
    scratch = {d: rv.alloc_scratch(rv.relay_plan(rv.ALLREDUCE, experts, d, A, R), "cuda") for d in (rv.I32, rv.F32)}
    ws = rv.alloc_router_workspace(t, experts, "cuda")
    deep = rv.fp8_depth(rows, experts)
    wq, wt = rv.alloc_fp8(wide, dim, "cuda", tiles=True, batch=experts), rv.alloc_fp8(dim, wide, "cuda", tiles=True, batch=experts)
    xq, xt = rv.alloc_fp8(rows, dim, "cuda"), rv.alloc_fp8(dim, deep, "cuda", tiles=True)
    gq, gt = rv.alloc_fp8(rows, wide, "cuda"), rv.alloc_fp8(wide, deep, "cuda")
    y, dx = torch.empty(rows, wide, **f32), torch.empty(rows, dim, **f32)
    dw = torch.empty(experts, wide, dim, dtype=torch.bfloat16, **cuda)
    loss, d_prob = torch.empty(1, **f32), torch.empty(experts, **f32)
    d_logits, next_bias = [torch.empty(t, experts, **f32) for _ in range(A)], torch.empty(experts, **f32)
    grads = rv.make_grads([dw] + d_logits)
    norm, gws = torch.empty(1, **f32), rv.alloc_grad_workspace(grads, "cuda")
    clipped = [torch.empty_like(v) for v in [dw] + d_logits]
    to = rv.make_grads(clipped)
    out = {}

    def step():
        for a in range(A):
            rv.relay_grouped_router_forward(lc[a], index[a], gate[a], counts[a], prob[a], bias=bc, workspace=ws, **how)
        # rows by expert; every row of these inputs has k experts
        order = torch.sort(torch.cat(index).flatten(), stable=True).indices
        for bufs, d in ((counts, rv.I32), (prob, rv.F32)):
            rv.relay_allreduce(bufs, bufs, scratch[d], experts, d, A, R)
        offset = torch.nn.functional.pad(counts[0].cumsum(0), (1, 0)).to(torch.int32)
        sent = torch.cat(xc)[order // k]
        rv.relay_quantize_fp8(wc, *wq, *wt, tiles=True, tiles_t=True)
        rv.relay_quantize_fp8(sent, *xq, *xt, tiles_t=True, offset=offset)
        rv.relay_matmul_fp8(*xq, *wq, y, offset=offset)
        dy = torch.cat(dc)[order // k].float() * torch.cat(gate).flatten()[order, None]
        d_gate = torch.empty(rows, **f32)
        d_gate[order] = (y * torch.cat(dc)[order // k].float()).sum(dim=1)
        rv.relay_quantize_fp8(dy, *gq, *gt, offset=offset)
        rv.relay_matmul_fp8(*gq, *wt, dx, offset=offset)
        rv.relay_matmul_fp8(*gt, *xt, dw, offset=offset, by_depth=True)
        rv.relay_balance_loss(counts[0], prob[0], k, 0.01, loss, d_prob)
        for a in range(A):
            rv.relay_grouped_router_backward(lc[a], index[a], d_logits[a], d_gate=d_gate[a * t * k:(a + 1) * t * k].view(t, k),
                                             d_prob=d_prob, scale=how["scale"])
        rv.relay_router_bias_update(counts[0], bc, 0.001, next_bias)
        rv.relay_grad_norm(grads, norm, workspace=gws)
        rv.relay_grad_clip(grads, norm, 0.05, out=to)
        out.update(order=order, offset=offset, dy=dy, d_gate=d_gate)
    step()
    if captured:
        torch.cuda.synchronize()
        eager = [v.clone() for v in clipped + [y, dx, norm, next_bias]]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for v in clipped + [y, dx, norm, next_bias, dw]:
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, clipped + [y, dx, norm, next_bias]))
    torch.cuda.synchronize()
    rv.device_status()

    want = [grouped_router_ref.route(v, k, bias, **how) for v in logits]
    total = sum(r["counts"].to(torch.int64) for r in want)
    for a in range(A):
        assert torch.equal(index[a].cpu(), want[a]["index"])
        assert torch.equal(counts[a].cpu().to(torch.int64), total)
    order, off = out["order"].cpu(), out["offset"].cpu()
    assert torch.equal(next_bias.cpu(), bias + torch.sign(total.sum() - experts * total).float() * 0.001)
    sent, dy = torch.cat(x)[order // k], out["dy"].cpu()
    for e in range(experts):
        part = slice(int(off[e]), int(off[e + 1]))
        for got, a, b in ((y[part], sent[part], w[e]), (dx[part], dy[part], w[e].t())):
            ref, bound = fp8_ref.matmul(*fp8_ref.quantize(a, False), *fp8_ref.quantize(b, True), True)
            assert bool(((got.double().cpu() - ref).abs() <= bound).all())
        ref, bound = fp8_ref.matmul(*fp8_ref.quantize(dy[part].t(), False), *fp8_ref.quantize(sent[part].t(), True), False)
        assert bool(((dw[e].double().cpu() - ref).abs() <= bound).all())
    # the gates' gradient comes from y (fp32), the balance loss's from the counts of both ranks
    dg, dp = out["d_gate"].cpu(), d_prob.cpu()
    per = 0.01 * experts * total.double() / (k * (A * t) ** 2)
    assert bool(((dp.double() - per).abs() <= 1e-6 * per).all())
    for a in range(A):
        r = grouped_router_ref.route(logits[a], k, bias, d_gate=dg[a * t * k:(a + 1) * t * k].view(t, k), d_prob=dp, **how)
        assert bool(((d_logits[a].double().cpu() - r["d_logits"]).abs() <= 2.0 ** -16 * r["size"] + 1e-30).all())
    all_grads = [dw] + d_logits
    size = sum(float(v.double().square().sum()) for v in all_grads) ** 0.5
    assert size > 0.05 and abs(norm.item() - size) <= 1e-6 * size
    for got, v in zip(clipped, all_grads):
        unit = U if v.dtype is torch.bfloat16 else 2.0 ** -24
        want_v = v.double() * 0.05 / (size + 1e-6)
        assert bool(((got.double() - want_v).abs() <= (unit + 2e-6) * want_v.abs() + 1e-38).all())
