"""fp8 with 128-block scales, routing, and the experts' layer: float64 oracle
(test infrastructure only).

The definitions (include/hq.h states the same in prose):

    quantise   over each 128 consecutive values of a row, s = fl32(max|v| / 448)
               (1 where that is zero), code = RNE_e4m3(fl32(v / s))
    gemm       C[m, n] = sum_k a[m, k] sa[k/128, m] * w[n, k] sw[n/128, k/128]
    route      the topk largest logits, ties to the lowest index, weights
               softmax, -inf never chosen (id -1, weight 0)
    layer      h = quant(x) W1[e]^T, act = SiLU(h[:I]) h[I:],
               y = sum_j w_j quant(act_j) W2[e_j]^T

fl32 marks the two roundings to float32 that belong to the definition: they
decide codes, since 16-bit values over their block's largest fall on the
midpoints of e4m3 often.  torch float64 on the device of the inputs; shares no
code with the library.

Bounds.  A dot product that the kernels form in float32 (exact products of
e4m3 values, 128 of them a group, one scale factor a group, then the groups,
then up to 16 partial sums) is off by at most gamma * sum |a w| with
gamma = (128 + K/128 + 24) 2^-23: each addition and each product with a scale
rounds by 2^-24 of a partial sum that sum |a w| bounds, doubled for adders
that truncate.  A stored value adds half a step of its type.
"""
from __future__ import annotations

import torch

BLOCK = 128
TOP = 448.0


def f32(v: torch.Tensor) -> torch.Tensor:
    return v.to(torch.float32).to(torch.float64)


def e4m3(v: torch.Tensor) -> torch.Tensor:
    """The nearest e4m3 value, ties to even, at most 448 in size."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-TOP, TOP)


def e4m3_half_step(v: torch.Tensor) -> torch.Tensor:
    """Half the e4m3 spacing around |v| (2^-10 below the normals)."""
    return torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 4)


def block_scale(v: torch.Tensor) -> torch.Tensor:
    """[.., k] -> [.., k/128]."""
    s = f32(v.unflatten(-1, (-1, BLOCK)).abs().amax(-1) / TOP)
    return torch.where(s > 0, s, torch.ones_like(s))


def quantize(v: torch.Tensor):
    """float64 [m, k] -> (e4m3 values [m, k], scales [m, k/128])."""
    s = block_scale(v)
    return e4m3(f32(v / s.repeat_interleave(BLOCK, -1))), s


def silu_mul(h: torch.Tensor) -> torch.Tensor:
    g, u = h.chunk(2, -1)
    return g / (1 + torch.exp(-g)) * u


def weight(codes: torch.Tensor, scales: torch.Tensor) -> torch.Tensor:
    """e4m3 values [n, k] and scales [ceil(n/128), k/128] -> float64 [n, k]."""
    n, k = codes.shape
    row = torch.arange(n, device=codes.device) // BLOCK
    return codes.double() * scales.double()[row].repeat_interleave(BLOCK, 1)[:, :k]


def rows(codes: torch.Tensor, scales: torch.Tensor) -> torch.Tensor:
    """e4m3 values [m, k] and scales [m, k/128] -> float64 [m, k]."""
    return codes.double() * scales.double().repeat_interleave(BLOCK, -1)


def gamma(k: int) -> float:
    return (128 + k // 128 + 24) * 2.0 ** -23


def half_step(y: torch.Tensor, dtype) -> torch.Tensor:
    info = torch.finfo(dtype)
    return (y.abs() * info.eps / 2).clamp_min(info.smallest_normal * info.eps / 2)


def gemm(a: torch.Tensor, w: torch.Tensor):
    """Values a [m, k], w [n, k] -> (a w^T, how far the card's sum may be off).

    Two parts.  Adding in float32 in any order: gamma(k) sum |a w|.  And what
    the fp8 matrix instruction itself drops: it adds eight neighbouring
    products in fixed point and cuts each, towards zero, at 2^-13 of the power
    of two of the largest (256 - 256 + v, for v = 1.75 * 2^-6 and less, is 0; for
    v = 1.5 * 2^-5 it is 2^-5; the same v sixteen places on is kept whole).
    Each of the eight is so off by less than 2^-13 max |a w|, together by less
    than 2^-10 max |a| max |w| over the eight."""
    cut = _max8(a) @ _max8(w).t() * 2.0 ** -10
    return a @ w.t(), gamma(a.shape[1]) * (a.abs() @ w.abs().t()) + cut


def _max8(v: torch.Tensor) -> torch.Tensor:
    return v.abs().unflatten(1, (-1, 8)).amax(2)


def route(logits: torch.Tensor, topk: int, renormalize: bool):
    x = logits.double()
    x = torch.where(torch.isnan(x), torch.full_like(x, -torch.inf), x)
    ids = torch.empty(x.shape[0], topk, dtype=torch.int64)
    w = torch.zeros(x.shape[0], topk, dtype=torch.float64)
    for t, row in enumerate(x.tolist()):
        best = sorted(range(len(row)), key=lambda e: (-row[e], e))[:topk]
        best = [e for e in best if row[e] > -float("inf")]
        for j in range(topk):
            ids[t, j] = best[j] if j < len(best) else -1
        if best:
            over = torch.tensor([row[e] for e in best] if renormalize else row, dtype=torch.float64)
            w[t, :len(best)] = torch.exp(torch.tensor([row[e] for e in best], dtype=torch.float64) - torch.logsumexp(over, 0))
    return ids, w


def act_bound(h: torch.Tensor, tau: torch.Tensor) -> torch.Tensor:
    """How far SiLU(g) u may be off where g and u are off by tau, plus the
    float32 steps of forming it (exp to 2 ulp, division, two products):
    |silu'| <= 1.1 and |silu(g)| <= |g|."""
    g, u = h.chunk(2, -1)
    tg, tu = tau.chunk(2, -1)
    # exp(-g) is off by its argument's rounding, |g| 2^-24, besides its own ulps
    return 1.1 * tg * (u.abs() + tu) + (g.abs() + tg) * tu + silu_mul(h).abs() * (10 + g.abs()) * 2.0 ** -23


def requant_range(act: torch.Tensor, tau: torch.Tensor):
    """The values quantising act may give where act is off by up to tau: the
    middle one, and how far another admissible one may be from it (its scale and
    its code moving within tau)."""
    codes, s = quantize(act)
    mid = rows(codes, s)
    b = tau.unflatten(-1, (-1, BLOCK)).amax(-1)
    lo_s, hi_s = (s - b / TOP) * (1 - 2.0 ** -23), (s + b / TOP) * (1 + 2.0 ** -23)
    scales = [sc.repeat_interleave(BLOCK, -1) for sc in (lo_s.clamp_min(torch.finfo(torch.float32).tiny), hi_s)]
    # the quotients within reach, the codes they round to (rounding is monotone),
    # and each of those codes with each scale
    q = torch.stack([(act + d) / e * (1 + r) for d in (-tau, tau) for e in scales for r in (-(2.0 ** -22), 2.0 ** -22)])
    far = torch.zeros_like(mid)
    for c in (e4m3(q.amin(0)), e4m3(q.amax(0))):
        for e in scales:
            far = torch.maximum(far, (c * e - mid).abs())
    return mid, far


def layer(x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, w1, s1, w2, s2, row_err: float = 0.0):
    """(y, bound): the experts' layer on x (float64 values of 16-bit rows), and
    how far a float32 evaluation may be from it before the output's rounding.
    row_err: error of a slot's stored row relative to its 64 columns' largest."""
    xq = rows(*quantize(x))
    y = torch.zeros(x.shape[0], w2.shape[1], dtype=torch.float64, device=x.device)
    tol = torch.zeros_like(y)
    for e in torch.unique(ids).tolist():
        if e < 0 or e >= w1.shape[0]:
            continue
        tok, slot = torch.nonzero(ids == e, as_tuple=True)
        h, th = gemm(xq[tok], weight(w1[e], s1[e]))
        act = silu_mul(h)
        mid, far = requant_range(act, act_bound(h, th))
        d = weight(w2[e], s2[e])
        o, to = gemm(mid, d)
        to = to + far @ d.abs().t() * (1 + gamma(mid.shape[1]))
        p = weights[tok, slot].double().unsqueeze(-1)
        strip = o.unflatten(-1, (-1, 64)).abs().amax(-1).repeat_interleave(64, -1)
        y.index_add_(0, tok, o * p)
        tol.index_add_(0, tok, (to + row_err * strip) * p.abs() + 2.0 ** -21 * (o * p).abs())
    return y, tol
