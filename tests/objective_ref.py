"""64-bit definitions of the training objective's operators, and the error bounds the tests hold
them to. Everything here is torch in float64 on the CPU.

Bounds, elementwise, with u = 2^-8 (half an ulp of bf16: 8 significant bits, so values in [1, 2)
are 2^-7 apart) and f = 2^-24 (of fp32):
  logits     fp32 sums of exact products, in any order and with truncation at each of the at
             most dim steps: |dz| <= ez = 2 dim f (|h| . |W|) / tau
  loss       log-sum-exp moves by at most max ez plus the fp32 rounding of a sum of
             positive terms (2^-19 covers sums in any order here) and of z and lse themselves
  gradient   exp(z - lse) is off by a factor exp(2 max ez) and a few f. A bf16 head may round
             the probability to bf16 (u of it), and rounds the gradient of the logit (u of that);
             the products sum |g||W| and |g||h| carry both, and the result is rounded once (u).
             An fp32 head has f-sized terms in the same places; its three-part products drop
             terms below 2^-22.
"""
import math

import torch

U, F = 2.0 ** -8, 2.0 ** -24


def head(hidden, weights, index, score, row_weight, tau):
    """loss, d_hidden, d_weight (concatenated) and their bounds. index/score: [tokens, k]; an index
    outside the vocabulary is no entry; score None: cross entropy (k = 1)."""
    bf16 = hidden.dtype == torch.bfloat16
    W = torch.cat([w.double() for w in weights])
    V, D = W.shape
    T = hidden.shape[0]
    idx = index.long()
    ok = (idx >= 0) & (idx < V)
    if score is None:
        score = torch.zeros(T, 1)
    s = torch.where(ok, score.double() / tau, torch.full((), -math.inf, dtype=torch.float64))
    live = (s > -math.inf).any(dim=1) | torch.isnan(s).any(dim=1)
    h = torch.where(live[:, None], hidden.double(), torch.zeros((), dtype=torch.float64))
    z = h @ W.t() / tau
    lse = torch.logsumexp(z, dim=1, keepdim=True)
    q = torch.softmax(torch.where(live[:, None], s, torch.zeros_like(s)), dim=1)
    q = torch.where(ok & live[:, None], q, torch.zeros_like(q))
    at = idx.clamp(0, V - 1)
    pair = torch.where(q > 0, q * (q.clamp_min(1e-300).log() - z.gather(1, at) + lse), torch.zeros_like(q))
    loss = tau * tau * pair.sum(dim=1)
    dense = torch.zeros_like(z).scatter_add_(1, at, q)
    w = torch.ones(T, dtype=torch.float64) if row_weight is None else row_weight.double()
    w = torch.where(live, w * tau, torch.zeros_like(w))
    p = (z - lse).exp()
    g = w[:, None] * (p - dense)
    dh, dw = g @ W, g.t() @ h
    # bounds
    ez = 2 * D * F * (h.abs() @ W.abs().t()) / tau + 4 * F * z.abs()
    rowez = ez.max(dim=1, keepdim=True).values
    at_z = z.gather(1, at).abs().max(dim=1, keepdim=True).values
    loss_b = tau * tau * (2 * rowez + 2.0 ** -19 + 8 * F * (lse.abs() + at_z))[:, 0] \
        + 2.0 ** -18 * loss.abs()
    grow = p * (2 * rowez + 2.0 ** -19) * w.abs()[:, None] + 2.0 ** -19 * dense * w.abs()[:, None]
    unit = (U if bf16 else 2.0 ** -20)
    gb = grow + unit * g.abs() + (U * p * w.abs()[:, None] if bf16 else 0.0)
    out = U if bf16 else F
    steps = 2.0 ** -24 * 2
    dh_b = gb @ W.abs() + steps * V * (g.abs() @ W.abs()) / 16 + out * dh.abs() + 1e-30
    dw_b = gb.t() @ h.abs() + steps * (T + 256) * (g.abs().t() @ h.abs()) / 16 + out * dw.abs() + 1e-30
    return dict(loss=loss, d_hidden=dh, d_weight=dw, loss_b=loss_b, d_hidden_b=dh_b, d_weight_b=dw_b)


def close(name, got, want, bound):
    got = got.double().cpu()
    assert got.shape == want.shape, name
    assert not torch.isnan(got).any(), f"{name}: NaN"
    over = (got - want).abs() / bound
    assert bool((over <= 1).all()), f"{name}: {over.max().item():.3g} of its bound at {over.argmax().item()}"


def router(logits, top, normalize, mask, coef, d_gate, counts=None):
    """index, gate, counts, prob_sum, loss, d_prob, d_logits in float64 (index and counts exact)."""
    x = logits.double()
    T, E = x.shape
    live = torch.ones(T, dtype=torch.bool) if mask is None else mask.bool()
    live = live & (x > -math.inf).any(dim=1)
    order = torch.sort(torch.where(torch.isnan(x), torch.full_like(x, -math.inf), x), dim=1,
                       descending=True, stable=True).indices
    index = order[:, :top]
    safe = torch.where(live[:, None], x, torch.zeros_like(x))
    p = torch.softmax(safe, dim=1) * live[:, None]
    chosen = safe.gather(1, index)
    gate = torch.softmax(chosen, dim=1) * live[:, None] if normalize else p.gather(1, index)
    n = torch.bincount(index[live].flatten(), minlength=E)
    prob_sum = p.sum(dim=0)
    c = n if counts is None else counts
    tokens = c.sum().item() / top
    d_prob = coef * E * c.double() / (top * tokens * tokens) if tokens else torch.zeros(E, dtype=torch.float64)
    loss = (d_prob * prob_sum).sum()
    dg = torch.zeros(T, top, dtype=torch.float64) if d_gate is None else d_gate.double()
    a = d_prob.expand(T, E).clone()
    if not normalize:
        a.scatter_add_(1, index, dg)
    dx = p * (a - (p * a).sum(dim=1, keepdim=True))
    if normalize:
        dx.scatter_add_(1, index, gate * (dg - (gate * dg).sum(dim=1, keepdim=True)))
    dx = dx * live[:, None]
    index = torch.where(live[:, None], index, -1).int()
    size = (p * (a.abs() + (p * a.abs()).sum(dim=1, keepdim=True)))
    if normalize:
        size.scatter_add_(1, index.clamp_min(0).long(), gate * (dg.abs() + (gate * dg.abs()).sum(dim=1, keepdim=True)))
    return dict(index=index, gate=gate, counts=n.int(), prob_sum=prob_sum, loss=loss, d_prob=d_prob,
                d_logits=dx, d_logits_size=size)
