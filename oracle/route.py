"""Routing by scores with a bias and groups: float64 oracle (test infrastructure only).

    s = fl32(sigmoid(l)) or fl32(softmax(l)),  key = fl32(s + bias)
    the group_topk groups of largest sum of group_best keys, then the topk largest keys;
    w = s, over the chosen ones' sum if renormalised, times scale

The roundings to float32 belong to the definition: they decide which of two close
experts comes first.  One token at a time, in plain Python over float64 rows.
"""
from __future__ import annotations

import math

import torch

# Weights: a score is off by a rounding to fp32; the sum of up to 64 of them, the quotient and the product with
# the factor add 66 roundings at most
WEIGHT = 70 * 2.0 ** -24


def route(logits, topk, bias=None, scoring="sigmoid", groups=1, group_topk=1, group_best=2, renormalize=True, scale=1.0):
    """(ids int32 [t, topk], weights float64 [t, topk]) on the CPU."""
    x = logits.double().cpu()
    live = x > -math.inf                                       # (false for NaN)
    e = torch.where(live, x, -math.inf)
    if scoring == "sigmoid":
        s = 1 / (1 + torch.exp(-e))
    else:
        p = torch.exp(e - e.amax(-1, keepdim=True).clamp_min(-1e300))
        s = p / p.sum(-1, keepdim=True).clamp_min(1e-300)
    s = s.float()
    key = s if bias is None else s + bias.float().cpu()
    key = torch.where(live & ~key.isnan(), key, -math.inf)
    t, experts = x.shape
    size = experts // groups
    ids = torch.full((t, topk), -1, dtype=torch.int32)
    w = torch.zeros(t, topk, dtype=torch.float64)
    for r in range(t):
        k = key[r].tolist()
        of = []
        for g in range(groups):
            best = sorted((v for v in k[g * size:(g + 1) * size] if v > -math.inf), reverse=True)[:group_best]
            of.append(float(torch.tensor(best, dtype=torch.float64).sum().float()) if best else -math.inf)
        kept = sorted(range(groups), key=lambda g: (-of[g], g))[:group_topk]
        may = [i for g in kept for i in range(g * size, (g + 1) * size) if k[i] > -math.inf]
        may.sort(key=lambda i: (-k[i], i))
        for j, i in enumerate(may[:topk]):
            ids[r, j], w[r, j] = i, float(s[r, i])
        total = float(w[r].sum())
        if renormalize and total > 0:
            w[r] /= total
    return ids, w * scale
