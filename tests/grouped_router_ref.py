"""The router with scores, bias and groups in 64 bits, written from its definition row by row in numpy."""
import math

import numpy as np
import torch


def route(x, top, bias=None, mask=None, groups=1, kept=None, group_sum=2, score="sigmoid", normalize=True, scale=1.0, d_gate=None,
          d_prob=None):
    """x [tokens, experts]. Returns index, gate, counts, prob_sum, and with d_gate or d_prob the gradient d_logits and
    the size of what it is summed from (for bounds on rounding)."""
    x = x.double().numpy()
    t, e = x.shape
    kept = groups if kept is None else kept
    b = np.zeros(e) if bias is None else bias.double().numpy()
    size = e // groups
    index = np.full((t, top), -1, np.int32)
    gate, share = np.zeros((t, top)), np.zeros((t, e))
    grad, big = np.zeros((t, e)), np.zeros((t, e))
    dp = np.zeros(e) if d_prob is None else d_prob.double().numpy()
    for r in range(t):
        if mask is not None and not bool(mask[r]):
            continue
        row = x[r]
        can = (row > -math.inf) & (b > -math.inf)
        if not can.any():
            continue
        if score == "sigmoid":
            s = np.array([1.0 / (1.0 + math.exp(-v)) if v > -700 else 0.0 for v in row])
        else:
            s = np.exp(row - row.max())
            s = s / s.sum()
        # a logit is as large as its score, and does not saturate: it decides where there is no bias
        c = [(s[i] + b[i] if bias is not None else row[i]) if can[i] else -math.inf for i in range(e)]
        if kept < groups:
            value = []
            for g in range(groups):
                part = sorted((i for i in range(g * size, (g + 1) * size) if can[i]), key=lambda i: (-c[i], i))[:group_sum]
                if group_sum == 1 and bias is None:
                    value.append(c[part[0]] if part else -math.inf)
                else:
                    value.append(sum(s[i] + b[i] for i in part) if part else -math.inf)
            stay = sorted(range(groups), key=lambda g: (-value[g], g))[:kept]
            can = can & np.isin(np.arange(e) // size, stay)
        pick = sorted((i for i in range(e) if can[i]), key=lambda i: (-c[i], i))[:top]
        if not pick:
            continue
        k = len(pick)
        index[r, :k] = pick
        chosen = s[pick]
        z = chosen.sum() if normalize else 1.0
        gate[r, :k] = scale * chosen / z if z > 0 else 0.0
        total = s.sum()
        share[r] = s / total if total > 0 else 0.0
        if d_gate is None and d_prob is None:
            continue
        dg = np.zeros(k) if d_gate is None else scale * d_gate[r, :k].double().numpy()
        q, qb = np.zeros(e), np.zeros(e)
        if total > 0:
            q += (dp - (share[r] * dp).sum()) / total
            qb += (np.abs(dp) + (share[r] * np.abs(dp)).sum()) / total
        if normalize and z > 0:
            inner = (dg * chosen).sum() / z
            q[pick] += (dg - inner) / z
            qb[pick] += (np.abs(dg) + (np.abs(dg) * chosen).sum() / z) / z
        elif not normalize:
            q[pick] += dg
            qb[pick] += np.abs(dg)
        if score == "sigmoid":
            slope = np.array([math.exp(-abs(v)) / (1.0 + math.exp(-abs(v))) ** 2 if abs(v) < 700 else 0.0 for v in row])
            grad[r], big[r] = q * slope, qb * slope
        else:
            grad[r] = s * (q - (s * q).sum())
            big[r] = s * (qb + (s * qb).sum())
    counts = np.bincount(index[index >= 0], minlength=e).astype(np.int32)
    out = dict(index=index, gate=gate, counts=counts, prob_sum=share.sum(axis=0), d_logits=grad, size=big)
    return {n: torch.from_numpy(v) for n, v in out.items()}
