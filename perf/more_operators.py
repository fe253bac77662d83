"""What a training step of a model with experts needs beside its collectives and its objective, as measured:
routing by scores, a bias for balance and groups of experts; the experts' products in 8-bit floating point with
a scale for each block of 128; the norm of all gradients and their clipping.

``run`` has two sides on the same inputs: the plain form (elementary torch operations in 32 bits, the choice of
experts and long sums in 64) and the library's operators. ``exact`` is the definition in 64 bits.
"""
import math
import random

import torch

own = False

DEV = "cuda"
BLOCK = 128
E4M3_MAX = 448.0


def _dt(case):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[case["dtype"]]


# ------------------------------------------------------------------------------ cases --

def listed():
    route = dict(op="route", score="sigmoid", bias=True, group_sum=2, normalize=True, scale=2.5, masked=0.0,
                 drained=0, grad=True)
    linear = dict(op="linear", dtype="bf16", groups=0, grad=True, out="bf16")
    return [
        # routing one token of each of a few sequences: one launch, latency counts
        dict(route, name="route_decode_4", tokens=4, experts=256, groups=8, kept=4, top=8, dtype="f32", grad=False),
        # scores by softmax, the group's best expert speaks for it, padded rows, an odd number of rows
        dict(route, name="route_train_10007", tokens=10007, experts=160, groups=8, kept=3, top=6, dtype="f32",
             score="softmax", bias=False, group_sum=1, normalize=False, scale=16.0, masked=0.25),
        # a training batch over many experts, with the bias for balance and a node that is drained
        dict(route, name="route_train_65536", tokens=65536, experts=256, groups=8, kept=4, top=8, dtype="bf16",
             drained=32),
        # serving: a few rows through one projection, the weight quantized once
        dict(linear, name="linear_decode_8", rows=8, dim=4096, cols=4096, grad=False),
        # serving experts: a few rows to each of many experts, ragged
        dict(linear, name="experts_decode_96", rows=96, dim=2048, cols=1408, groups=32, grad=False),
        # fine-tuning a projection of odd sizes, results in full precision
        dict(linear, name="linear_train_1003", rows=1003, dim=1000, cols=1544, dtype="f32", out="f32"),
        # a prompt through one projection
        dict(linear, name="linear_prompt_4096", rows=4096, dim=4096, cols=4096, grad=False),
        # training experts: rows sorted by expert, ragged, some experts without rows
        dict(linear, name="experts_train_16384", rows=16384, dim=2048, cols=2816, groups=16),
        # training a large projection
        dict(linear, name="linear_train_8192", rows=8192, dim=4096, cols=8192),
        # clipping a small model's gradients: few tensors, latency counts
        dict(op="clip", name="clip_small", layers=2, dim=256, hidden=1024, vocab=2048, dtype="f32", odd=False),
        # mixed types, odd sizes, tensors anywhere in a flat buffer
        dict(op="clip", name="clip_mixed", layers=12, dim=1023, hidden=2731, vocab=5003, dtype="mixed", odd=True),
        # a model's gradients, far more than the caches hold
        dict(op="clip", name="clip_large", layers=24, dim=2048, hidden=8192, vocab=32000, dtype="bf16", odd=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "linear", "linear", "clip"])
    if op == "route":
        groups = rng.choice([1, 2, 4, 6, 8, 16])
        size = max(1, _log(rng, 2, 512) // groups)
        experts = groups * size
        kept = rng.randint(1, groups)
        top = rng.randint(1, min(8, kept * size))
        return dict(op=op, tokens=_log(rng, 1, 65536 * 256 // max(experts, 256)), experts=experts, groups=groups,
                    kept=kept, top=top, dtype=rng.choice(["bf16", "f32"]), score=rng.choice(["sigmoid", "sigmoid", "softmax"]),
                    bias=rng.random() < 0.7, group_sum=rng.choice([1, 2]), normalize=rng.random() < 0.6,
                    scale=rng.choice([1.0, 2.5, 16.0]), masked=rng.choice([0.0, 0.0, 0.25]),
                    drained=rng.choice([0, 0, size // 2]), grad=rng.random() < 0.75)
    if op == "linear":
        rows, dim, cols = _log(rng, 1, 16384), _log(rng, 32, 4096), _log(rng, 32, 8192)
        if rng.random() < 0.7:
            dim, cols = (dim + 15) // 16 * 16, (cols + 15) // 16 * 16
        groups = rng.choice([0, 0, 2, 5, 8, 32])
        if groups:
            dim, cols = min(dim, 2048), min(cols, 2816)
        while rows * dim * cols > 8192 * 4096 * 8192:
            rows //= 2
        return dict(op=op, rows=rows, dim=dim, cols=cols, groups=groups, dtype=rng.choice(["bf16", "bf16", "f32"]),
                    out=rng.choice(["bf16", "bf16", "f32"]), grad=rng.random() < 0.6)
    return dict(op=op, layers=rng.randint(1, 24), dim=_log(rng, 32, 2048), hidden=_log(rng, 64, 8192), vocab=_log(rng, 200, 32000),
                dtype=rng.choice(["bf16", "f32", "mixed"]) if rng.random() < 0.7 else "bf16", odd=rng.random() < 0.5)


# Sizes of a clip case's tensors, in the order of a model's parameters.
def _sizes(case):
    d, h = case["dim"], case["hidden"]
    layer = [d, d * d, d * d, d * d, d * d, d, d * h, d * h, h * d]
    sizes = [case["vocab"] * d] + layer * case["layers"] + [d]
    if case["odd"]:
        sizes = [max(1, n - i % 7) for i, n in enumerate(sizes)] + [1, 0, 3]
    return sizes


def _types(case, n):
    if case["dtype"] == "mixed":   # vectors and scalars are kept in full precision
        return [torch.float32 if s < 100000 else torch.bfloat16 for s in n]
    return [_dt(case)] * len(n)


# Rows of each expert: known on the host when the inputs are made, in device memory for the call. A few
# experts are much in demand, some get no row.
def _lengths(case, seed):
    r, g = random.Random(seed), case["groups"]
    want = [r.random() ** 2 * (0.0 if r.random() < 0.1 else 1.0) for _ in range(g)]
    want[r.randrange(g)] += 0.5
    total = sum(want)
    n = [int(case["rows"] * w / total) for w in want]
    n[max(range(g), key=lambda i: want[i])] += case["rows"] - sum(n)
    return n


def work(case):
    if case["op"] == "route":
        e = 2 if case["dtype"] == "bf16" else 4
        t, x, k = case["tokens"], case["tokens"] * case["experts"], case["top"]
        b, f = x * e + 8 * t * k + 16 * case["experts"], 10 * x
        if case["grad"]:
            b, f = b + x * e + 4 * t * k, f + 10 * x
        return {"bytes": b, "flops": f}
    if case["op"] == "linear":
        e, o = 2 if case["dtype"] == "bf16" else 4, 2 if case["out"] == "bf16" else 4
        r, d, n, g = case["rows"], case["dim"], case["cols"], max(case["groups"], 1)
        live = sum(1 for x in _lengths(case, 0) if x) if case["groups"] else 1
        if not case["grad"]:
            return {"bytes": r * d * e + live * n * d + r * n * o, "flops": 2 * r * d * n}
        return {"bytes": r * (d + n) * e + live * n * d * e + r * (d + n) * o + g * n * d * o, "flops": 6 * r * d * n}
    n = _sizes(case)
    return {"bytes": sum(2 * s * (4 if t == torch.float32 else 2) for s, t in zip(n, _types(case, n))), "flops": 3 * sum(n)}


# ---------------------------------------------------------------------------- inputs --

def _route_inputs(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    t, e, k = case["tokens"], case["experts"], case["top"]
    lean = torch.randn(e, generator=g, device=DEV) * 0.5          # some experts are favoured
    logits = (torch.randn(t, e, generator=g, device=DEV) * 1.5 + lean).to(_dt(case))
    bias = None
    if case["bias"] or case["drained"]:
        bias = torch.randn(e, generator=g, device=DEV) * (0.05 if case["score"] == "sigmoid" else 0.002)
        if case["drained"]:
            bias[e - case["drained"]:] = -math.inf
    mask = None
    if case["masked"]:
        mask = torch.ones(t, dtype=torch.bool, device=DEV)
        mask[torch.randperm(t, generator=g, device=DEV)[:int(t * case["masked"])]] = False
    return dict(logits=logits, bias=bias, mask=mask, coef=0.001, rate=0.001,
                d_gate=torch.randn(t, k, generator=g, device=DEV) / t)


def _linear_inputs(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r, d, n, groups, dt = case["rows"], case["dim"], case["cols"], case["groups"], _dt(case)
    x = torch.randn(r, d, generator=g, device=DEV)
    # a few channels are far larger than the rest, as activations' are
    loud = torch.rand(d, generator=g, device=DEV) < 0.01
    x = (x * torch.where(loud, 20.0, 1.0)).to(dt)
    w = torch.randn(max(groups, 1), n, d, generator=g, device=DEV) / math.sqrt(d)
    st = dict(x=x, weight=w.to(dt))
    if groups:
        st["lengths"] = _lengths(case, seed)
        st["most"] = max(st["lengths"])
        st["offset"] = torch.tensor([0] + st["lengths"]).cumsum(0).to(torch.int32).to(DEV)
    if case["grad"]:
        # a row's gradient is of its own size: tokens differ in how wrong they are
        size = torch.exp(torch.randn(r, 1, generator=g, device=DEV) * 2.0) / r
        st["dy"] = (torch.randn(r, n, generator=g, device=DEV) * size).to(dt)
    return st


def _clip_inputs(case, seed):
    """Gradients as views of one flat buffer for each type, zeros in the gaps."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    sizes = _sizes(case)
    types = _types(case, sizes)
    at = {torch.float32: 0, torch.bfloat16: 0}
    place, gaps = [], {torch.float32: [], torch.bfloat16: []}
    for i, (n, t) in enumerate(zip(sizes, types)):
        place.append(at[t])
        gap = i % 3 if case["odd"] else -n % 128
        gaps[t].append((at[t] + n, gap))
        at[t] += n + gap
    flat = {}
    for t, n in at.items():
        if n == 0:
            continue
        flat[t] = torch.empty(n, dtype=t, device=DEV)
        for lo in range(0, n, 1 << 26):
            part = flat[t][lo:lo + (1 << 26)]
            part.copy_(torch.randn(part.numel(), generator=g, device=DEV) * 0.01)
        for end, gap in gaps[t]:
            flat[t][end:end + gap] = 0.0
    grads = [flat[t][p:p + n] for n, t, p in zip(sizes, types, place)]
    return dict(flat=flat, grads=grads, place=place, max_norm=1.0)


def prepare(case, seed):
    st = {"route": _route_inputs, "linear": _linear_inputs, "clip": _clip_inputs}[case["op"]](case, seed)
    st["case"] = dict(case)
    f32, i32 = dict(dtype=torch.float32, device=DEV), dict(dtype=torch.int32, device=DEV)
    if case["op"] == "route":
        if own:
            import pack_virtual_rank_gb300 as rv
            t, e, k = case["tokens"], case["experts"], case["top"]
            st["index"], st["gate"] = torch.empty(t, k, **i32), torch.empty(t, k, **f32)
            st["counts"], st["prob_sum"] = torch.empty(e, **i32), torch.empty(e, **f32)
            st["loss"], st["d_prob"] = torch.empty(1, **f32), torch.empty(e, **f32)
            st["d_logits"] = torch.empty_like(st["logits"])
            st["new_bias"] = torch.empty(e, **f32)
            st["workspace"] = rv.alloc_router_workspace(t, e, DEV)
    elif case["op"] == "linear":
        r, d, n, groups = case["rows"], case["dim"], case["cols"], max(case["groups"], 1)
        out = {"bf16": torch.bfloat16, "f32": torch.float32}[case["out"]]
        if not case["grad"]:   # weights of a serving program are quantized once
            q, s = _quantize_tiles(st.pop("weight").float())
            st["wq"], st["ws"] = torch.zeros(groups, n, (d + 15) // 16 * 16, dtype=torch.float8_e4m3fn, device=DEV)[:, :, :d], s
            st["wq"].copy_(q.to(torch.float8_e4m3fn))
        if own:
            import pack_virtual_rank_gb300 as rv
            st["y"] = torch.empty(r, n, dtype=out, device=DEV)
            st["xq"], st["xs"] = rv.alloc_fp8(r, d, DEV)
            if case["grad"]:
                deep = rv.fp8_depth(r, case["groups"])
                st["wq"], st["ws"] = rv.alloc_fp8(n, d, DEV, tiles=True, batch=groups)
                st["wt"], st["wts"] = rv.alloc_fp8(d, n, DEV, tiles=True, batch=groups)
                st["xt"], st["xts"] = rv.alloc_fp8(d, deep, DEV, tiles=True)
                st["gq"], st["gs"] = rv.alloc_fp8(r, n, DEV)
                st["gt"], st["gts"] = rv.alloc_fp8(n, deep, DEV)
                st["dx"] = torch.empty(r, d, dtype=out, device=DEV)
                st["dw"] = torch.empty(groups, n, d, dtype=out, device=DEV)
    elif own:
        import pack_virtual_rank_gb300 as rv
        st["out"] = {t: torch.zeros_like(x) for t, x in st["flat"].items()}
        clipped = [st["out"][x.dtype][p:p + x.numel()] for x, p in zip(st["grads"], st["place"])]
        st["list"], st["list_out"] = rv.make_grads(st["grads"]), rv.make_grads(clipped)
        st["norm"] = torch.empty(1, **f32)
        st["workspace"] = rv.alloc_grad_workspace(st["list"], DEV)
    return st


# ------------------------------------------------------------------------------- run --

def run(state):
    case = state["case"]
    if case["op"] == "route":
        return _run_route_own(state, case) if own else _run_route_plain(state, case)
    if case["op"] == "linear":
        return _run_linear_own(state, case) if own else _run_linear_plain(state, case)
    return _run_clip_own(state) if own else _run_clip_plain(state)


def _run_route_own(st, case):
    import pack_virtual_rank_gb300 as rv
    how = dict(groups=case["groups"], kept=case["kept"], score=case["score"], normalize=case["normalize"], scale=case["scale"])
    rv.relay_grouped_router_forward(st["logits"], st["index"], st["gate"], st["counts"], st["prob_sum"], bias=st["bias"],
                                    mask=st["mask"], group_sum=case["group_sum"], workspace=st["workspace"], **how)
    out = {n: st[n] for n in ("index", "gate", "counts", "prob_sum")}
    if case["grad"]:
        rv.relay_balance_loss(st["counts"], st["prob_sum"], case["top"], st["coef"], st["loss"], st["d_prob"])
        rv.relay_grouped_router_backward(st["logits"], st["index"], st["d_logits"], d_gate=st["d_gate"], d_prob=st["d_prob"],
                                         score=case["score"], normalize=case["normalize"], scale=case["scale"])
        out["d_logits"] = st["d_logits"]
        if case["bias"]:
            rv.relay_router_bias_update(st["counts"], st["bias"], st["rate"], st["new_bias"])
            out["bias"] = st["new_bias"]
    return out


def _run_linear_own(st, case):
    import pack_virtual_rank_gb300 as rv
    offset = st.get("offset")
    if not case["grad"]:
        rv.relay_quantize_fp8(st["x"], st["xq"], st["xs"])
        rv.relay_matmul_fp8(st["xq"], st["xs"], st["wq"], st["ws"], st["y"], offset=offset)
        return {"y": st["y"]}
    rv.relay_quantize_fp8(st["weight"], st["wq"], st["ws"], st["wt"], st["wts"], tiles=True, tiles_t=True)
    rv.relay_quantize_fp8(st["x"], st["xq"], st["xs"], st["xt"], st["xts"], tiles_t=True, offset=offset)
    rv.relay_matmul_fp8(st["xq"], st["xs"], st["wq"], st["ws"], st["y"], offset=offset)
    rv.relay_quantize_fp8(st["dy"], st["gq"], st["gs"], st["gt"], st["gts"], offset=offset)
    rv.relay_matmul_fp8(st["gq"], st["gs"], st["wt"], st["wts"], st["dx"], offset=offset)
    rv.relay_matmul_fp8(st["gt"], st["gts"], st["xt"], st["xts"], st["dw"], offset=offset, by_depth=True)
    return {"y": st["y"], "dx": st["dx"], "dw": st["dw"]}


def _run_clip_own(st):
    import pack_virtual_rank_gb300 as rv
    rv.relay_grad_norm(st["list"], st["norm"], workspace=st["workspace"])
    rv.relay_grad_clip(st["list"], st["norm"], st["max_norm"], out=st["list_out"])
    return dict({"norm": st["norm"]}, **{str(t): x for t, x in st["out"].items()})


def _run_route_plain(st, case):
    t, e, k, g = case["tokens"], case["experts"], case["top"], case["groups"]
    x = st["logits"].double()          # which of two near values is larger is decided in 64 bits
    if case["score"] == "sigmoid":
        s = 1.0 / (1.0 + (-x).exp())
    else:
        s = (x - x.max(dim=1, keepdim=True).values).exp()
        s = s / s.sum(dim=1, keepdim=True)
    c = s if st["bias"] is None else s + st["bias"].double()
    c = torch.where(x == -math.inf, torch.full_like(c, -math.inf), c)
    if case["kept"] < g:
        best = torch.sort(c.view(t, g, e // g), dim=2, descending=True).values[:, :, :case["group_sum"]]
        value = torch.where(best == -math.inf, torch.zeros_like(best), best).sum(dim=2)
        value = torch.where(best[:, :, 0] == -math.inf, torch.full_like(value, -math.inf), value)
        stay = torch.sort(value, dim=1, descending=True, stable=True).indices[:, :case["kept"]]
        keep = torch.zeros(t, g, dtype=torch.bool, device=DEV).scatter_(1, stay, True)
        c = torch.where(keep.repeat_interleave(e // g, dim=1), c, torch.full_like(c, -math.inf))
    order = torch.sort(c, dim=1, descending=True, stable=True)
    index = order.indices[:, :k]
    live = order.values[:, 0] > -math.inf
    if st["mask"] is not None:
        live = live & st["mask"]
    ok = live[:, None] & (order.values[:, :k] > -math.inf)
    s = s.float()
    chosen = torch.where(ok, s.gather(1, index), torch.zeros(t, k, device=DEV))
    z = chosen.sum(dim=1, keepdim=True) if case["normalize"] else torch.ones(t, 1, device=DEV)
    z = torch.where(z > 0, z, torch.ones_like(z))
    gate = chosen / z * case["scale"]
    total = s.sum(dim=1, keepdim=True)
    p = torch.where(live[:, None], s / total, torch.zeros_like(s))
    hot = torch.zeros(t, e, device=DEV).scatter_(1, index, ok.float())
    counts, prob_sum = hot.sum(dim=0).to(torch.int32), p.sum(dim=0)
    out = dict(index=torch.where(ok, index, torch.full_like(index, -1)).to(torch.int32), gate=gate, counts=counts,
               prob_sum=prob_sum)
    if case["grad"]:
        n = (counts.sum() / k).clamp(min=1)
        per = st["coef"] * e * counts.float() / (k * n * n)
        dg = torch.where(ok, st["d_gate"], torch.zeros_like(st["d_gate"])) * case["scale"]
        if case["normalize"]:
            dg = (dg - (dg * chosen).sum(dim=1, keepdim=True) / z) / z
        ds = (per - (p * per).sum(dim=1, keepdim=True)) / total * live[:, None]
        ds = ds.scatter_add(1, index, torch.where(ok, dg, torch.zeros_like(dg)))
        if case["score"] == "sigmoid":
            # 1 - s of a large logit is lost in 32 bits
            dx = ds * s * (1.0 / (1.0 + x.exp())).float()
        else:
            dx = s * (ds - (s * ds).sum(dim=1, keepdim=True))
        out["d_logits"] = dx.to(st["logits"].dtype)
        if case["bias"]:
            more = counts.sum(dtype=torch.int64) - e * counts.to(torch.int64)
            out["bias"] = st["bias"] + st["rate"] * torch.sign(more).float()
    return out


def _scale(top):
    """The least power of two that brings `top` to 448 or less (1 for a block of zeros)."""
    m, e = torch.frexp(top)
    e = torch.where(m > E4M3_MAX / 512, e - 8, e - 9).clamp(min=-126)
    return torch.where(top > 0, torch.ldexp(torch.ones_like(top), e), torch.ones_like(top))


def _quantize_rows(x):
    """Values of x in 8 bits, a scale for each 128 neighbours of a row, and the scales."""
    r, d = x.shape[-2:]
    pad = torch.nn.functional.pad(x, (0, -d % BLOCK)).unflatten(-1, (-1, BLOCK))
    s = _scale(pad.abs().amax(dim=-1, keepdim=True))
    q = (pad / s).to(torch.float8_e4m3fn).float()
    return q.flatten(-2)[..., :d], s[..., 0]


def _quantize_tiles(x):
    """The same with a scale for each 128 x 128."""
    n, d = x.shape[-2:]
    pad = torch.nn.functional.pad(x, (0, -d % BLOCK, 0, -n % BLOCK))
    pad = pad.unflatten(-1, (-1, BLOCK)).unflatten(-3, (-1, BLOCK))            # [.., nb, 128, db, 128]
    s = _scale(pad.abs().amax(dim=(-3, -1), keepdim=True))
    q = (pad / s).to(torch.float8_e4m3fn).float()
    return q.flatten(-2).flatten(-3, -2)[..., :n, :d], s[..., :, 0, :, 0]


def _rows_back(q, s):
    return q * s.repeat_interleave(BLOCK, dim=-1)[..., :q.shape[-1]]


def _tiles_back(q, s):
    s = s.repeat_interleave(BLOCK, dim=-1)[..., :q.shape[-1]]
    return q * s.repeat_interleave(BLOCK, dim=-2)[..., :q.shape[-2], :]


def _spread(st, case, x, deep):
    """Rows by group, [groups, most (up to a multiple of `deep`), width], zeros behind a group's last."""
    if not case["groups"]:
        return torch.nn.functional.pad(x[None], (0, 0, 0, -x.shape[0] % deep)), None
    row = torch.arange(x.shape[0], device=DEV)
    group = torch.searchsorted(st["offset"][1:].long(), row, right=True)
    most = max(deep, -(-st["most"] // deep) * deep)
    at = group * most + row - st["offset"].long()[group]
    buf = torch.zeros(case["groups"] * most, x.shape[1], device=DEV, dtype=x.dtype)
    buf[at] = x
    return buf.view(case["groups"], most, -1), at


def _gather_rows(y, at, rows):
    return y[0, :rows] if at is None else y.flatten(0, 1)[at]


def _run_linear_plain(st, case):
    out = {"bf16": torch.bfloat16, "f32": torch.float32}[case["out"]]
    r = case["rows"]
    x = st["x"].float()
    if case["grad"]:
        wide = st["weight"].float()
        w = _tiles_back(*_quantize_tiles(wide))
    else:
        w = _tiles_back(st["wq"].float(), st["ws"])
    xs, at = _spread(st, case, _rows_back(*_quantize_rows(x)), 1)
    res = {"y": _gather_rows(xs @ w.transpose(1, 2), at, r).to(out)}
    if not case["grad"]:
        return res
    dy = st["dy"].float()
    wt = _tiles_back(*_quantize_tiles(wide.transpose(1, 2)))
    gs, at = _spread(st, case, _rows_back(*_quantize_rows(dy)), 1)
    res["dx"] = _gather_rows(gs @ wt.transpose(1, 2), at, r).to(out)
    # along the rows: blocks of 128 rows of one group
    xt, _ = _spread(st, case, x, BLOCK)
    gt, _ = _spread(st, case, dy, BLOCK)
    xt = _tiles_back(*_quantize_tiles(xt.transpose(1, 2)))
    gt = _rows_back(*_quantize_rows(gt.transpose(1, 2)))
    res["dw"] = (gt @ xt.transpose(1, 2)).to(out)
    return res


def _run_clip_plain(st):
    norm = torch.stack([x.float().square().sum(dtype=torch.float64) for x in st["grads"]]).sum().sqrt()
    factor = (st["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
    # the tensors lie in flat buffers, with zeros between them
    return dict({"norm": norm.float().reshape(1)}, **{str(t): (x.float() * factor).to(t) for t, x in st["flat"].items()})


# ----------------------------------------------------------------------------- exact --

def exact(case, seed):
    if case["op"] == "route":
        return _exact_route(case, _route_inputs(case, seed))
    if case["op"] == "linear":
        return _exact_linear(case, _linear_inputs(case, seed))
    return _exact_clip(_clip_inputs(case, seed))


def _first_largest(left, k):
    """Positions of the k largest of each row, one after the other, the first of equal ones."""
    picks, n = [], left.shape[1]
    left = left.clone()
    place = torch.arange(n, device=DEV)
    for _ in range(k):
        best = left.amax(dim=1, keepdim=True)
        at = torch.where(left == best, place, n).amin(dim=1, keepdim=True)
        picks.append(at)
        left.scatter_(1, at, math.nan)
        left = torch.where(left.isnan(), torch.full_like(left, -math.inf), left)
    return torch.cat(picks, dim=1)


def _exact_route(case, st):
    t, e, k, g = case["tokens"], case["experts"], case["top"], case["groups"]
    x = st["logits"].double()
    s = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.softmax(x, dim=1)
    c = s + (0.0 if st["bias"] is None else st["bias"].double())
    if case["kept"] < g:
        by = c.reshape(t * g, e // g)
        two = by.topk(min(case["group_sum"], e // g), dim=1).values
        value = torch.where(two > -math.inf, two, 0.0).sum(dim=1)
        value = value.masked_fill(two[:, 0] == -math.inf, -math.inf).view(t, g)
        stay = torch.zeros(t, g, dtype=torch.bool, device=DEV)
        stay.scatter_(1, _first_largest(value, case["kept"]), True)
        c = c.masked_fill(~stay[:, torch.arange(e, device=DEV) // (e // g)], -math.inf)
    index = _first_largest(c, k)
    ok = c.gather(1, index) > -math.inf
    live = ok.any(dim=1) if st["mask"] is None else ok.any(dim=1) & st["mask"]
    ok &= live[:, None]
    hot = torch.zeros(t, e, dtype=torch.float64, device=DEV).scatter_add_(1, index, ok.double())
    share = s / s.sum(dim=1, keepdim=True) * live[:, None]
    counts = hot.sum(dim=0)
    norm = (s * hot).sum(dim=1, keepdim=True) if case["normalize"] else torch.ones(t, 1, dtype=torch.float64, device=DEV)
    norm = norm.masked_fill(norm == 0, 1.0)
    full = case["scale"] * s * hot / norm
    out = dict(index=index.masked_fill(~ok, -1).to(torch.int32), gate=full.gather(1, index) * ok, counts=counts.to(torch.int32),
               prob_sum=share.sum(dim=0))
    if case["grad"]:
        n = max(float(counts.sum()) / k, 1.0)
        per = case["experts"] * st["coef"] * counts / (k * n * n)
        dg = torch.zeros(t, e, dtype=torch.float64, device=DEV).scatter_add_(1, index, st["d_gate"].double() * ok)
        # by the scores' logarithms: d gate_i / d log s_j = gate_i (1[i = j] - share of j, where renormalized)
        log_s = full * dg
        if case["normalize"]:
            log_s = log_s - hot * s / norm * log_s.sum(dim=1, keepdim=True)
        spread = share * per
        log_s = log_s + spread - share * spread.sum(dim=1, keepdim=True)
        if case["score"] == "sigmoid":
            out["d_logits"] = log_s * torch.sigmoid(-x)
        else:
            out["d_logits"] = log_s - s * log_s.sum(dim=1, keepdim=True)
        if case["bias"]:
            out["bias"] = st["bias"].double() + st["rate"] * torch.sign(counts.mean() - counts)
    return out


def _round_e4m3(v):
    """Nearest value of 8 bits with a 3-bit fraction, ties to even, down to steps of 2^-9."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return torch.round(v / step) * step


def _exact_quantized(x, tile):
    """[rows, depth] with a power of two for each 128 of the depth (and each 128 rows where `tile`)."""
    r, d = x.shape
    x = x.double()
    top = torch.nn.functional.pad(x.abs(), (0, -d % BLOCK)).view(r, -1, BLOCK).amax(dim=2)
    if tile:
        top = torch.nn.functional.pad(top, (0, 0, 0, -r % BLOCK)).view(-1, BLOCK, top.shape[1]).amax(dim=1)
        top = top.repeat_interleave(BLOCK, dim=0)[:r]
    k = torch.ceil(torch.log2((top / E4M3_MAX).clamp(min=2.0 ** -126)))
    k = torch.where(top > E4M3_MAX * torch.exp2(k), k + 1, k)        # log2 next to a power of two
    k = torch.where((top <= E4M3_MAX * torch.exp2(k - 1)) & (k > -126), k - 1, k)
    s = torch.where(top > 0, torch.exp2(k), 1.0).repeat_interleave(BLOCK, dim=1)[:, :d]
    return _round_e4m3(x / s) * s


def _exact_linear(case, st):
    if work(case)["flops"] > 8e12:
        return None
    r = case["rows"]
    lengths = st["lengths"] if case["groups"] else [r]
    x, w = st["x"], st["weight"]
    y = torch.zeros(r, case["cols"], dtype=torch.float64, device=DEV)
    dx = torch.zeros(r, case["dim"], dtype=torch.float64, device=DEV)
    dw = torch.zeros(w.shape, dtype=torch.float64, device=DEV)
    lo = 0
    for i, n in enumerate(lengths):
        part = slice(lo, lo + n)
        lo += n
        if n == 0:
            continue
        y[part] = _exact_quantized(x[part], False) @ _exact_quantized(w[i], True).t()
        if case["grad"]:
            dy = st["dy"][part]
            dx[part] = _exact_quantized(dy, False) @ _exact_quantized(w[i].t(), True).t()
            dw[i] = _exact_quantized(dy.t(), False) @ _exact_quantized(x[part].t(), True).t()
    return {"y": y, "dx": dx, "dw": dw} if case["grad"] else {"y": y}


def _exact_clip(st):
    total = 0.0
    for x in st["grads"]:
        for part in x.split(1 << 26):
            total += float(part.double().square().sum())
    norm = math.sqrt(total)
    factor = min(1.0, st["max_norm"] / (norm + 1e-6))
    out = {"norm": torch.tensor([norm], dtype=torch.float64, device=DEV)}
    for t, flat in st["flat"].items():
        full = torch.zeros(flat.shape, dtype=torch.float64, device=DEV)
        for x, p in zip(st["grads"], st["place"]):
            if x.dtype == t:
                torch.mul(x.double(), factor, out=full[p:p + x.numel()])
        out[str(t)] = full
    return out
