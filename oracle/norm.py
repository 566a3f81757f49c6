"""Root-mean-square norm with the residual's addition and a quantised output: float64
oracle (test infrastructure only).

    h = x + r, rounded to x's type          y = h w / sqrt(mean(h^2) + eps)

Bounds.  The kernel's factor 1 / sqrt(..) is off by at most half of its sum's relative
error plus three roundings: the sum of k squares runs over at most 64 terms a thread
and then over a tree of 10 levels with up to 16 partial sums, each addition off by 2^-24
of a partial sum that the whole bounds (squares do not cancel), so under 90 * 2^-24
for the sum and under 48 * 2^-24 for the factor.  h w rounds once if the weight
is fp32, its product with the factor once: FACTOR covers both.  Codes add half a
step of their type at the scale that is stored, which is itself off by FACTOR and a
division's rounding.
"""
from __future__ import annotations

import torch

FACTOR = 50 * 2.0 ** -24
TOP8, TOP4 = 448.0, 6.0


def norm(x, weight, eps, residual=None):
    """(h in x's type, y float64)."""
    h = x if residual is None else (x.double() + residual.double()).to(x.dtype)
    v = h.double()
    return h, v * weight.double() / torch.sqrt(v.square().mean(-1, keepdim=True) + eps)


def half_step8(v):
    """Half the e4m3 spacing at |v|."""
    return torch.exp2(torch.floor(torch.log2(v.abs().clamp(2.0 ** -6, TOP8))) - 4)


def half_step4(v):
    """Half the E2M1 spacing at |v|."""
    return torch.exp2(torch.floor(torch.log2(v.abs().clamp(1.0, 4.0))) - 2)


def block_top(y, block):
    return y.unflatten(-1, (-1, block)).abs().amax(-1)


def off_scaled(values, scales, y, block, top, half_step):
    """How far codes (their values, [m, k]) and scales [m, k/block] are from y over what they
    may be off, elementwise: at most 1."""
    s = scales.double().repeat_interleave(block, -1)
    v = y / s
    slack = 2 * FACTOR * v.abs()
    bound = half_step(v.abs() + slack) + slack
    return (values.double() - v.clamp(-top, top)).abs() / bound


def off_scale(scales, y, block, top):
    """Relative error of scales [m, k/block] from max|y| / top over what it may be."""
    want = block_top(y, block) / top
    return ((scales.double() - want).abs() / (want * (FACTOR + 2.0 ** -23) + 2.0 ** -149)).masked_fill(want == 0, 0.0)


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def values4(codes):
    """Bytes [m, k/2] -> E2M1 values [m, k] in float64."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=codes.device)
    return torch.stack([table[(codes & 15).long()], table[(codes >> 4).long()]], -1).flatten(-2)


def rows_of(e8m0):
    """Group-major E8M0 [k/128, m, 4] -> [m, k/32]."""
    return e8m0.transpose(0, 1).flatten(-2)


def e8m0_may_be(y):
    """The lowest and highest E8M0 byte of each 32 values' power of two (one where no rounding can decide)."""
    top = block_top(y, 32)

    def byte(t):
        return torch.where(t > 0, (torch.floor(torch.log2(t.clamp_min(2.0 ** -400))) - 2).clamp(-127, 127), 0.0) + 127

    return byte(top * (1 - 2 * FACTOR)), byte(top * (1 + 2 * FACTOR))
