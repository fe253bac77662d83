"""The objective of a training step, as measured: cross entropy and distillation over a vocabulary
sharded on the active virtual ranks (projection included), and the expert router with its balance loss.

``run`` has two sides on the same inputs: the plain form (elementary torch operations in 32 bits) and
the library's operators. ``exact`` is the definition in 64 bits.
"""
import math

import torch

own = False

IGNORE = -100
DEV = "cuda"


def _dt(case):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[case["dtype"]]


# ------------------------------------------------------------------------------ cases --

def listed():
    xent = dict(op="xent", dtype="bf16", ignored=0.0, grad=True)
    distill = dict(op="distill", dtype="bf16", ignored=0.0, grad=True, tau=2.0)
    router = dict(op="router", normalize=False, masked=0.0, grad=True)
    return [
        # scoring the next token of a few sequences: the weight is read once, latency counts
        dict(xent, name="xent_score_8", tokens=8, dim=1024, vocab=32768, shards=2, grad=False),
        # one sequence on a small model: few tiles, launches count
        dict(xent, name="xent_train_129", tokens=129, dim=512, vocab=8192, shards=1),
        # fine-tuning: prompt rows ignored, ragged vocabulary over four ranks
        dict(xent, name="xent_train_2047", tokens=2047, dim=2048, vocab=50001, shards=4, ignored=0.3),
        # pre-training: a full batch of a rank over a large vocabulary on eight ranks
        dict(xent, name="xent_train_8192", tokens=8192, dim=4096, vocab=131072, shards=8),
        # full-precision training
        dict(xent, name="xent_train_f32", tokens=1024, dim=1024, vocab=32000, shards=2, dtype="f32",
             ignored=0.1),
        # distilling a small student on short sequences
        dict(distill, name="distill_train_64", tokens=64, dim=512, vocab=8192, shards=1, top=8),
        # distilling with stored teacher logits, ragged sizes, padded teacher entries
        dict(distill, name="distill_train_1999", tokens=1999, dim=2048, vocab=32768, shards=2, top=64,
             ignored=0.2),
        # a large batch, sharp temperature
        dict(distill, name="distill_train_4096", tokens=4096, dim=4096, vocab=65537, shards=8, top=32,
             tau=1.0),
        # routing one token of each of a few sequences
        dict(router, name="router_decode_16", tokens=16, experts=64, top=2, dtype="f32", grad=False,
             normalize=True),
        # a sequence with padded rows over an odd number of experts
        dict(router, name="router_train_10007", tokens=10007, experts=60, top=4, dtype="bf16",
             masked=0.25, normalize=True),
        # a large batch over many experts
        dict(router, name="router_train_131072", tokens=131072, experts=256, top=8, dtype="f32"),
        dict(router, name="router_train_65536", tokens=65536, experts=128, top=8, dtype="bf16",
             normalize=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["xent", "xent", "distill", "router"])
    if op == "router":
        experts = _log(rng, 8, 384)
        return dict(op=op, tokens=_log(rng, 1, 131072 * 256 // max(experts, 256)), experts=experts,
                    top=rng.randint(1, min(8, experts)), dtype=rng.choice(["bf16", "f32"]),
                    normalize=rng.random() < 0.5, masked=rng.choice([0.0, 0.25]),
                    grad=rng.random() < 0.75)
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    top = 1 if dtype == "bf16" else 2      # full precision stands for smaller models
    tokens, vocab = _log(rng, 1, 8192 // top), _log(rng, 500, 131072 // top)
    dim = _log(rng, 64, 4096 // top)
    if rng.random() < 0.8:
        dim = (dim + 15) // 16 * 16
    case = dict(op=op, tokens=tokens, dim=dim, vocab=vocab, shards=rng.choice([1, 2, 4, 8]),
                dtype=dtype, ignored=rng.choice([0.0, 0.1, 0.5]), grad=rng.random() < 0.8)
    if op == "distill":
        case.update(top=_log(rng, 1, 128), tau=rng.choice([1.0, 2.0, 4.0]))
    return case


def _valid_rows(case):
    return case["tokens"] - int(case["tokens"] * case["ignored"])


def _counted_rows(case):
    return case["tokens"] - int(case["tokens"] * case["masked"])


def _shard_rows(case):
    n, a = case["vocab"], case["shards"]
    return [n // a + (1 if i < n % a else 0) for i in range(a)]


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    t = case["tokens"]
    if case["op"] == "router":
        x, k, c = t * case["experts"], case["top"], _counted_rows(case)
        live = c * case["experts"]
        b = live * e + 8 * t * k + 8 * case["experts"]
        f = 6 * live
        if case["grad"]:
            # the gradient of every logit, the incoming gradient of every gate
            b += x * e + 4 * t * k + 4
            f += 6 * live
        return {"bytes": b, "flops": f}
    d, v, r = case["dim"], case["vocab"], _valid_rows(case)
    b = (r * d + v * d) * e + 8 * t
    f = 2 * r * v * d
    if case["op"] == "distill":
        b += r * case["top"] * (4 + e)
    if case["grad"]:
        b += (t * d + v * d) * e + 4 * t
        f *= 3
    return {"bytes": b, "flops": f}


# ---------------------------------------------------------------------------- inputs --

def _rows_out(case, frac, g):
    """A truth value per row: round(frac * tokens) of them, spread at random, are set."""
    out = torch.zeros(case["tokens"], dtype=torch.bool, device=DEV)
    n = int(case["tokens"] * frac)
    out[torch.randperm(case["tokens"], generator=g, device=DEV)[:n]] = True
    return out


def _head_inputs(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    t, d, v, dt = case["tokens"], case["dim"], case["vocab"], _dt(case)
    weight = torch.empty(v, d, dtype=dt, device=DEV)
    for i in range(0, v, 16384):
        n = min(16384, v - i)
        weight[i:i + n] = (torch.randn(n, d, generator=g, device=DEV) * (2.0 / math.sqrt(d))).to(dt)
    out = _rows_out(case, case["ignored"], g)
    target = torch.randint(0, v, (t,), generator=g, device=DEV, dtype=torch.int32)
    # hidden rows lean towards their target by different amounts: p(target) from 1/V to nearly 1
    lean = torch.rand(t, 1, generator=g, device=DEV) * 4.0
    hidden = torch.randn(t, d, generator=g, device=DEV) + lean * weight[target.long()].float()
    hidden = hidden.to(dt)
    valid = max(_valid_rows(case), 1)
    row_weight = (torch.rand(t, generator=g, device=DEV) + 0.5) / valid
    st = dict(hidden=hidden, weight=list(weight.split(_shard_rows(case))), row_weight=row_weight)
    if case["op"] == "xent":
        st["target"] = torch.where(out, torch.full_like(target, IGNORE), target)
        return st
    k = min(case["top"], v)
    # distinct ids: one from each of k equal stretches of the vocabulary, in order of the teacher's logits
    j = torch.arange(k, device=DEV)
    lo, hi = j * v // k, (j + 1) * v // k
    index = lo + (torch.rand(t, k, generator=g, device=DEV) * (hi - lo)).long()
    index = torch.minimum(index, hi - 1)
    # the row's own target is the teacher's favourite in its stretch
    pos = (target.long()[:, None] >= lo) & (target.long()[:, None] < hi)
    index = torch.where(pos, target.long()[:, None], index)
    logit = torch.randn(t, k, generator=g, device=DEV) * 2.0 + torch.where(pos, 6.0, 0.0)
    logit, order = torch.sort(logit, dim=1, descending=True)
    index = index.gather(1, order).to(torch.int32)
    # rows without a teacher, and rows whose last entries are padding
    keep = torch.randint(1, k + 1, (t, 1), generator=g, device=DEV)
    ragged = torch.rand(t, 1, generator=g, device=DEV) < 0.25
    index = torch.where(ragged & (j >= keep), torch.full_like(index, -1), index)
    st["teacher_index"] = torch.where(out[:, None], torch.full_like(index, -1), index).contiguous()
    st["teacher_logits"] = logit.to(_dt(case)).contiguous()
    return st


def _router_inputs(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    t, e, k = case["tokens"], case["experts"], case["top"]
    bias = torch.randn(e, generator=g, device=DEV) * 0.5     # some experts are favoured
    logits = (torch.randn(t, e, generator=g, device=DEV) * 1.5 + bias).to(_dt(case))
    mask = None
    if case["masked"]:
        mask = ~_rows_out(case, case["masked"], g)
    return dict(logits=logits, mask=mask, coef=0.01,
                d_gate=torch.randn(t, k, generator=g, device=DEV) / t)


def prepare(case, seed):
    st = _router_inputs(case, seed) if case["op"] == "router" else _head_inputs(case, seed)
    st["case"] = dict(case)
    if not own:
        return st
    import pack_virtual_rank_gb300 as rv
    t = case["tokens"]
    f32 = dict(dtype=torch.float32, device=DEV)
    if case["op"] == "router":
        e, k = case["experts"], case["top"]
        st["index"] = torch.empty(t, k, dtype=torch.int32, device=DEV)
        st["gate"] = torch.empty(t, k, **f32)
        st["counts"] = torch.empty(e, dtype=torch.int32, device=DEV)
        st["prob_sum"] = torch.empty(e, **f32)
        st["loss"] = torch.empty(1, **f32)
        st["d_prob"] = torch.empty(e, **f32)
        st["d_logits"] = torch.empty_like(st["logits"])
        st["workspace"] = rv.alloc_router_workspace(t, e, DEV)
        return st
    st["loss"] = torch.empty(t, **f32)
    if case["grad"]:
        st["d_hidden"] = torch.empty_like(st["hidden"])
        st["d_weight"] = [torch.empty_like(w) for w in st["weight"]]
    st["head"] = rv.make_head(st["hidden"], st["weight"], st.get("d_hidden"), st.get("d_weight"))
    top = st["teacher_index"].shape[1] if case["op"] == "distill" else 0
    st["workspace"] = rv.alloc_head_workspace(st["head"], DEV, top=top)
    return st


# ------------------------------------------------------------------------------- run --

def run(state):
    case = state["case"]
    if case["op"] == "router":
        return _run_router_own(state, case) if own else _run_router_plain(state, case)
    return _run_head_own(state, case) if own else _run_head_plain(state, case)


def _run_head_own(st, case):
    import pack_virtual_rank_gb300 as rv
    if case["op"] == "xent":
        rv.relay_linear_xent(st["head"], st["target"], st["loss"], row_weight=st["row_weight"],
                             workspace=st["workspace"])
    else:
        rv.relay_linear_distill(st["head"], st["teacher_logits"], st["teacher_index"], case["tau"],
                                st["loss"], row_weight=st["row_weight"], workspace=st["workspace"])
    out = {"loss": st["loss"]}
    if case["grad"]:
        out["d_hidden"], out["d_weight"] = st["d_hidden"], st["d_weight"]
    return out


def _run_router_own(st, case):
    import pack_virtual_rank_gb300 as rv
    rv.relay_router_forward(st["logits"], st["index"], st["gate"], st["counts"], st["prob_sum"],
                            mask=st["mask"], normalize=case["normalize"], workspace=st["workspace"])
    out = {n: st[n] for n in ("index", "gate", "counts", "prob_sum")}
    if case["grad"]:
        rv.relay_balance_loss(st["counts"], st["prob_sum"], case["top"], st["coef"], st["loss"],
                              st["d_prob"])
        rv.relay_router_backward(st["logits"], st["index"], st["d_logits"], d_gate=st["d_gate"],
                                 d_prob=st["d_prob"], normalize=case["normalize"])
        out["loss"], out["d_logits"] = st["loss"], st["d_logits"]
    return out


def _run_head_plain(st, case):
    hidden = st["hidden"].float()
    weight = torch.cat([w.float() for w in st["weight"]])
    inv = 1.0 if case["op"] == "xent" else 1.0 / case["tau"]
    z = (hidden @ weight.t()) * inv
    top = z.max(dim=1, keepdim=True).values
    lse = top + (z - top).exp().sum(dim=1, keepdim=True).log()
    rows = torch.arange(case["tokens"], device=DEV)
    if case["op"] == "xent":
        live = (st["target"] >= 0) & (st["target"] < case["vocab"])
        index = torch.where(live, st["target"], torch.zeros_like(st["target"])).long()[:, None]
        q = live.float()[:, None]
        loss = torch.where(live, lse[:, 0] - z[rows, index[:, 0]], torch.zeros_like(lse[:, 0]))
        back = 1.0
    else:
        ok = (st["teacher_index"] >= 0) & (st["teacher_index"] < case["vocab"])
        live = ok.any(dim=1)
        index = torch.where(ok, st["teacher_index"], torch.zeros_like(st["teacher_index"])).long()
        s = torch.where(ok, st["teacher_logits"].float() * inv, torch.full_like(z[:, :1], -math.inf))
        s = torch.where(live[:, None], s, torch.zeros_like(s))
        s = s - s.max(dim=1, keepdim=True).values
        logq = s - s.exp().sum(dim=1, keepdim=True).log()
        q = torch.where(ok, logq.exp(), torch.zeros_like(s))
        term = torch.where(ok, q * (logq - (z.gather(1, index) - lse)), torch.zeros_like(q))
        loss = term.sum(dim=1) * (case["tau"] * case["tau"])
        back = case["tau"]
    out = {"loss": loss}
    if case["grad"]:
        g = (z - lse).exp_()
        g.scatter_add_(1, index, -q)
        g *= torch.where(live, st["row_weight"] * back, torch.zeros_like(loss))[:, None]
        dt = st["hidden"].dtype
        out["d_hidden"] = (g @ weight).to(dt)
        hidden = torch.where(live[:, None], hidden, torch.zeros_like(hidden))
        out["d_weight"] = [d.contiguous() for d in (g.t() @ hidden).to(dt).split(_shard_rows(case))]
    return out


def _run_router_plain(st, case):
    t, e, k = case["tokens"], case["experts"], case["top"]
    x = st["logits"].float()
    live = torch.ones(t, dtype=torch.bool, device=DEV) if st["mask"] is None else st["mask"]
    order = torch.sort(x, dim=1, descending=True, stable=True)
    chosen, index = order.values[:, :k], order.indices[:, :k]
    p = (x - order.values[:, :1]).exp()
    p = p / p.sum(dim=1, keepdim=True)
    p = torch.where(live[:, None], p, torch.zeros_like(p))
    if case["normalize"]:
        gate = (chosen - chosen[:, :1]).exp()
        gate = gate / gate.sum(dim=1, keepdim=True)
        gate = torch.where(live[:, None], gate, torch.zeros_like(gate))
    else:
        gate = p.gather(1, index)
    hot = torch.zeros(t, e, device=DEV).scatter_(1, index, 1.0) * live[:, None]
    counts, prob_sum = hot.sum(dim=0).to(torch.int32), p.sum(dim=0)
    out = dict(index=torch.where(live[:, None], index, torch.full_like(index, -1)).to(torch.int32),
               gate=gate, counts=counts, prob_sum=prob_sum)
    if case["grad"]:
        n = (counts.sum() / k).clamp(min=1)
        per = st["coef"] * e * counts.float() / (k * n * n)
        out["loss"] = (per * prob_sum).sum().reshape(1)
        a = per.expand(t, e)
        if not case["normalize"]:
            a = a.scatter_add(1, index, st["d_gate"])
        dx = p * (a - (p * a).sum(dim=1, keepdim=True))
        if case["normalize"]:
            d = gate * (st["d_gate"] - (gate * st["d_gate"]).sum(dim=1, keepdim=True))
            dx = dx.scatter_add(1, index, d)
        out["d_logits"] = dx.to(st["logits"].dtype)
    return out


# ----------------------------------------------------------------------------- exact --

def exact(case, seed):
    if case["op"] == "router":
        return _exact_router(case, _router_inputs(case, seed))
    if work(case)["flops"] > 8e12:
        return None
    return _exact_head(case, _head_inputs(case, seed))


def _exact_head(case, st):
    """Row weights of the log-probabilities (one-hot or the teacher's) as a dense matrix, built and
    multiplied in blocks of live rows."""
    weight = torch.cat(st["weight"]).double()
    t, v, d = case["tokens"], case["vocab"], case["dim"]
    dt = st["hidden"].dtype
    tau = 1.0 if case["op"] == "xent" else float(case["tau"])
    loss = torch.zeros(t, dtype=torch.float64, device=DEV)
    dh = torch.zeros(t, d, dtype=torch.float64, device=DEV)
    dw = torch.zeros(v, d, dtype=torch.float64, device=DEV)
    if case["op"] == "xent":
        index = st["target"].long()[:, None]
        score = torch.zeros(t, 1, dtype=torch.float64, device=DEV)
    else:
        index = st["teacher_index"].long()
        score = st["teacher_logits"].double() / tau
    ok = (index >= 0) & (index < v)
    rows = ok.any(dim=1).nonzero()[:, 0]
    for part in rows.split(1024):
        h, good = st["hidden"][part].double(), ok[part]
        logp = torch.log_softmax(h @ weight.t() / tau, dim=1)
        logq = torch.log_softmax(score[part].masked_fill(~good, -math.inf), dim=1)
        q = logq.exp()
        at = index[part].clamp(0, v - 1)
        pair = q * (logq - logp.gather(1, at))
        loss[part] = tau * tau * pair.masked_fill(~good, 0.0).sum(dim=1)
        if case["grad"]:
            dense = torch.zeros_like(logp).scatter_add_(1, at, q.masked_fill(~good, 0.0))
            g = (logp.exp() - dense) * (tau * st["row_weight"][part].double())[:, None]
            dh[part] = g @ weight
            dw += g.t() @ h
    out = {"loss": loss}
    if case["grad"]:
        out["d_hidden"] = dh
        out["d_weight"] = [x.contiguous() for x in dw.split(_shard_rows(case))]
    return out


def _exact_router(case, st):
    t, e, k = case["tokens"], case["experts"], case["top"]
    x = st["logits"].double()
    live = torch.ones(t, dtype=torch.bool, device=DEV) if st["mask"] is None else st["mask"]
    left, picks = x.clone(), []
    for _ in range(k):
        best = left.amax(dim=1, keepdim=True)
        first = torch.where(left == best, torch.arange(e, device=DEV), e).amin(dim=1, keepdim=True)
        picks.append(first)
        left.scatter_(1, first, -math.inf)
    index = torch.cat(picks, dim=1)
    keep = live.double()[:, None]
    p = torch.softmax(x, dim=1) * keep
    chosen = x.gather(1, index)
    gate = torch.softmax(chosen, dim=1) * keep if case["normalize"] else p.gather(1, index)
    counts = torch.bincount(index[live].flatten(), minlength=e)
    out = dict(index=torch.where(live[:, None], index, -1).to(torch.int32), gate=gate,
               counts=counts.to(torch.int32), prob_sum=p.sum(dim=0))
    if case["grad"]:
        n = max(int(live.sum()), 1)
        per = st["coef"] * e * counts.double() / (k * n * n)
        out["loss"] = (per * p.sum(dim=0)).sum().reshape(1)
        dg = st["d_gate"].double() * keep
        inner = p * per
        dx = inner - p * inner.sum(dim=1, keepdim=True)
        pick = gate * dg - gate * (gate * dg).sum(dim=1, keepdim=True)
        if case["normalize"]:
            dx = dx.scatter_add(1, index, pick)
        else:
            dx = dx.scatter_add(1, index, gate * dg) - p * (gate * dg).sum(dim=1, keepdim=True)
        out["d_logits"] = dx
    return out
