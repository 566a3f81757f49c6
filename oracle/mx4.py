"""MXFP4 experts' layers: float64 oracle (test infrastructure only).

    quantise   over each 32 consecutive values of a row, X = floor(log2 max|v|) - 2,
               clamped to [-127, 127] (0 for a block of zeros), elements E2M1 nearest to
               v / 2^X, ties to even, at most 6
    layer      h = quant(x) W1[e]^T, act = SiLU(h[:I]) h[I:],
               y = sum_j w_j quant(act_j) W2[e_j]^T

torch float64 on the device of the inputs; shares no code with the library.

Bounds.  Products of two E2M1 values are multiples of 1/4 up to 36, so the fixed-point
sums of eight neighbours inside the matrix instruction keep them whole (they cut at
2^-13 of the largest's power of two).  What remains are fp32 additions: 128 products
and K / 128 groups in any order, each off by 2^-24 of a partial sum that sum |a w|
bounds, doubled for adders that truncate: gamma(K) sum |a w|.
"""
from __future__ import annotations

import torch

BLOCK = 32
TOP = 6.0
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)

# A slot's row on its way into the sum (fp16 with a power of two per 64 columns): each
# value is off by at most 2^-11 of itself down to 2^-29 of the 64 columns' largest, and
# below by 2^-39 of that one.
ROW_SELF, ROW_TOP = 2.0 ** -11, 2.0 ** -39
# The same on its way to outputs of fp16: 24 bits a value, 16 of them significant.
ROW_24 = 2.0 ** -16


def values(codes: torch.Tensor) -> torch.Tensor:
    """Bytes [.., k/2], the lower k in the low half -> E2M1 values [.., k]."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=codes.device)
    return torch.stack([table[(codes & 15).long()], table[(codes >> 4).long()]], -1).flatten(-2)


def pack(v: torch.Tensor) -> torch.Tensor:
    """E2M1 values [.., k] -> bytes [.., k/2]."""
    table = torch.tensor(E2M1, dtype=v.dtype, device=v.device)
    c = (torch.searchsorted(table, v.abs().contiguous()) + 8 * (v < 0)).to(torch.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4)


def e2m1(v: torch.Tensor) -> torch.Tensor:
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(1.0))) - 1)
    return (torch.round(v / step) * step).clamp(-TOP, TOP)


def power(top: torch.Tensor) -> torch.Tensor:
    """X + 127 of blocks by their largest magnitude."""
    x = (torch.floor(torch.log2(top.clamp_min(2.0 ** -400))) - 2).clamp(-127, 127)
    return torch.where(top > 0, x, 0.0) + 127


def _tops(v: torch.Tensor) -> torch.Tensor:
    return v.unflatten(-1, (-1, BLOCK)).abs().amax(-1)


def quantize(v: torch.Tensor):
    """float64 [.., k] -> (E2M1 values [.., k], E8M0 [.., k/32] as float64)."""
    e = power(_tops(v))
    return e2m1(v / torch.exp2(e - 127).repeat_interleave(BLOCK, -1)), e


def rows(vals: torch.Tensor, e8m0: torch.Tensor) -> torch.Tensor:
    return vals.double() * torch.exp2(e8m0.double() - 127).repeat_interleave(BLOCK, -1)


def group_major(e8m0: torch.Tensor) -> torch.Tensor:
    """[m, k/32] -> [k/128, m, 4]."""
    return e8m0.unflatten(-1, (-1, 4)).transpose(0, 1).contiguous()


def row_major(e8m0: torch.Tensor) -> torch.Tensor:
    return e8m0.transpose(0, 1).flatten(-2)


def gamma(k: int) -> float:
    return (128 + k // 128 + 24) * 2.0 ** -23


def gemm(a: torch.Tensor, w: torch.Tensor):
    """(a w^T, how far a float32 sum of it may be off)."""
    return a @ w.t(), gamma(a.shape[1]) * (a.abs() @ w.abs().t())


def silu_mul(h: torch.Tensor) -> torch.Tensor:
    g, u = h.chunk(2, -1)
    return g / (1 + torch.exp(-g)) * u


def act_bound(h: torch.Tensor, tau: torch.Tensor) -> torch.Tensor:
    """How far SiLU(g) u may be off where g and u are off by tau, plus the float32 steps
    of forming it (exp to 2 ulp and its argument's rounding, division, two products):
    |silu'| <= 1.1 and |silu(g)| <= |g|."""
    g, u = h.chunk(2, -1)
    tg, tu = tau.chunk(2, -1)
    return 1.1 * tg * (u.abs() + tu) + (g.abs() + tg) * tu + silu_mul(h).abs() * (10 + g.abs()) * 2.0 ** -23


def requant_range(act: torch.Tensor, tau: torch.Tensor):
    """The values quantising act may give where act is off by up to tau: the middle one,
    and how far another admissible one may be from it."""
    mid = rows(*quantize(act))
    top = _tops(act)
    b = tau.unflatten(-1, (-1, BLOCK)).amax(-1)
    far = torch.zeros_like(mid)
    for t in ((top - b).clamp_min(0.0), top + b):
        p = torch.exp2(power(t) - 127).repeat_interleave(BLOCK, -1)
        for d in (-tau, tau):
            far = torch.maximum(far, (e2m1((act + d) / p) * p - mid).abs())
    return mid, far


def half_step(y: torch.Tensor, dtype) -> torch.Tensor:
    info = torch.finfo(dtype)
    return (y.abs() * info.eps / 2).clamp_min(info.smallest_normal * info.eps / 2)


def weight(codes: torch.Tensor, e8m0: torch.Tensor) -> torch.Tensor:
    return rows(values(codes), e8m0)


def slot_rows_bound(o: torch.Tensor) -> torch.Tensor:
    """How far a stored slot row may be from o."""
    strip = o.unflatten(-1, (-1, 64)).abs().amax(-1).repeat_interleave(64, -1)
    return ROW_SELF * o.abs() + ROW_TOP * strip


def layer(xq: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, w1, e1, w2, e2):
    """(y, bound): the experts' layer on quantised rows xq (float64 values), and how far a
    float32 evaluation with slot rows as above may be from it before the output's rounding."""
    y = torch.zeros(xq.shape[0], w2.shape[1], dtype=torch.float64, device=xq.device)
    tol = torch.zeros_like(y)
    for e in torch.unique(ids).tolist():
        if e < 0 or e >= w1.shape[0]:
            continue
        tok, slot = torch.nonzero(ids == e, as_tuple=True)
        h, th = gemm(xq[tok], weight(w1[e], e1[e]))
        act = silu_mul(h)
        mid, far = requant_range(act, act_bound(h, th))
        d = weight(w2[e], e2[e])
        o, to = gemm(mid, d)
        to = to + far @ d.abs().t() * (1 + gamma(mid.shape[1]))
        p = weights[tok, slot].double().unsqueeze(-1)
        y.index_add_(0, tok, o * p)
        tol.index_add_(0, tok, (to + slot_rows_bound(o)) * p.abs() + 2.0 ** -20 * (o * p).abs())
    return y, tol
