"""The rows that the aligned down product leaves for the sum over a token's
experts: each value keeps its own precision, whatever lies beside it, and what
is not finite stays in its column."""
import pytest
import torch

import bit_quantized_gemm_repack_amd as hq
from oracle import block8 as o8

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E4 = torch.float8_e4m3fn
DT = {"bf16": torch.bfloat16, "f16": torch.float16}

# A row between the two kernels: fp16 with a power of two per 64 columns (half a
# step, 2^-11 of the value; below fp16's normals 2^-25, where the 64 columns'
# largest is at 2^14 or more: 2^-39 of that).
PER_VALUE, PER_STRIP = 2.0 ** -11, 2.0 ** -39


class Down:
    """The down product alone, on quantised rows, with a few columns far larger than the rest."""

    def __init__(self, bm, i, dt, t=40, topk=3, e=4, h=512, size=0.05):
        g = self.g = torch.Generator(DEV)
        g.manual_seed(bm + i)
        self.t, self.topk, self.e, self.dt = t, topk, e, dt
        w = torch.randn(e, h, i, generator=g, device=DEV) * size
        self.large = torch.zeros(h, dtype=torch.bool, device=DEV)
        self.large[[5, 64, 191, 300, 511]] = True
        w[:, self.large] *= 400 / size
        self.w, self.s = w.clamp_(-448, 448).to(E4), (0.5 + torch.rand(e, h // 128, i // 128, generator=g, device=DEV)) / i ** 0.5
        self.plan = hq.MoePlan(h, i, hq.w8a8_block(dt), e, t, "topk_combine", tuning=dict(tile_m=bm))
        self.ids, self.p = hq.route_topk(torch.randn(t, e, generator=g, device=DEV), topk)
        self.ids = self.ids.clone()
        self.ids[2, 1] = -1
        self.al = hq.moe_align(self.ids, e, bm)
        rows = torch.randn(t * topk, i, generator=g, device=DEV, dtype=torch.bfloat16)
        self.sid = self.al[0].long().clamp_max(t * topk - 1)
        used = torch.arange(len(self.sid), device=DEV) < self.al[2]
        self.sid = torch.where(used, self.sid, 0)
        self.codes, self.scale = hq.quantize_blocks(rows[self.sid])
        self.rows = o8.rows(*o8.quantize(rows.double()))

    def run(self):
        wm = self.plan.repack(self.w.view(torch.uint8), self.s)
        y = self.plan.moe_gemm(self.codes, self.t, self.topk, *self.al, *wm, a_scale=self.scale, topk_w=self.p)
        torch.cuda.synchronize()
        return y

    def want(self):
        """y, and how far it may be off before its own rounding."""
        y = torch.zeros(self.t, self.w.shape[1], dtype=torch.float64, device=DEV)
        tol = torch.zeros_like(y)
        for j in range(self.topk):
            for ex in range(self.e):
                tok = torch.nonzero(self.ids[:, j] == ex).squeeze(1)
                o, to = o8.gemm(self.rows[tok * self.topk + j], o8.weight(self.w[ex], self.s[ex]))
                p = self.p[tok, j].double().unsqueeze(1)
                strip = o.unflatten(1, (-1, 64)).abs().amax(2).repeat_interleave(64, 1)
                y.index_add_(0, tok, o * p)
                tol.index_add_(0, tok, (to * (1 + PER_VALUE) + PER_VALUE * o.abs() + PER_STRIP * strip + 2.0 ** -21 * o.abs()) * p)
        return y, tol + o8.half_step(y.abs() + tol, DT[self.dt]) + 1e-30


def _near(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float(((got.double() - want).abs() / tol).max()):.3g} of the bound"


SHAPES = [(16, 256), (64, 256), (128, 256), (128, 768), (64, 1280), (16, 4608)]  # whole rows in LDS, and the tiled product


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("bm,i", SHAPES)
def test_small_columns_beside_large_ones(bm, i, dt):
    """Columns of a 10000th of their neighbours' size are as precise as those."""
    d = Down(bm, i, dt)
    y, (want, tol) = d.run(), d.want()
    assert want[:, d.large].abs().median() > 1000 * want[:, ~d.large].abs().median()
    _near(y, want, tol, "down")


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("bm,i", SHAPES)
def test_nan_stays_in_its_column(bm, i, dt):
    d = Down(bm, i, dt, size=1.0)
    d.w = d.w.clone()
    d.w[1, 70, 3] = float("nan")
    y = d.run()
    hit = (d.ids == 1).any(1)
    d.w[1, 70, 3] = 0.0
    want, tol = d.want()
    assert hit.any() and torch.equal(torch.isnan(y[:, 70]), hit)
    keep = torch.arange(512, device=DEV) != 70
    _near(y[:, keep], want[:, keep], tol[:, keep], "the other columns")


@pytest.mark.parametrize("bm,i", SHAPES)
def test_overflow_stays_in_its_column(bm, i):
    """Large columns beyond fp32's range: infinite (or NaN, where signs meet), the others right."""
    d = Down(bm, i, "bf16")
    d.s = d.s * 3e35
    d.w[:, 64] = 448.0                                # and its rows all of one sign
    d.codes, d.scale = d.codes & 0x7F, d.scale
    d.rows = d.rows.abs()
    y, (want, tol) = d.run(), d.want()
    # a slot's value beyond fp32's range is infinite, and so is its token's sum
    assert (want[:, 64].abs() > torch.finfo(torch.float32).max).all() and torch.isinf(y[:, 64]).all()
    keep = ~d.large
    assert torch.isfinite(want[:, keep].float()).all()
    _near(y[:, keep], want[:, keep], tol[:, keep], "the other columns")


@pytest.mark.parametrize("t", [13, 40, 500])
def test_layer_keeps_small_columns(t):
    """A layer with a few large output columns: the ordinary ones' root mean square
    error stays below half a step of fp16, where no code of the intermediate
    differs, on both sides of the few-token switch."""
    g = torch.Generator(DEV)
    g.manual_seed(t)
    e, h, i = 8, 1024, 512
    w1 = (torch.randn(e, 2 * i, h, generator=g, device=DEV) * 96).clamp_(-448, 448).to(E4)
    s1 = (0.5 + torch.rand(e, 2 * i // 128, h // 128, generator=g, device=DEV)) / (96 * h ** 0.5)
    w2 = torch.randn(e, h, i, generator=g, device=DEV) * 0.05
    large = torch.zeros(h, dtype=torch.bool, device=DEV)
    large[::97] = True
    w2[:, large] *= 8000
    w2 = w2.clamp_(-448, 448).to(E4)
    s2 = (0.5 + torch.rand(e, h // 128, i // 128, generator=g, device=DEV)) / i ** 0.5
    q = hq.w8a8_block("f16")
    gu, dn = hq.MoePlan(2 * i, h, q, e, t, "silu_mul_qfp8"), hq.MoePlan(h, i, q, e, t, "topk_combine")
    wm = (*gu.repack(w1.view(torch.uint8), s1), *dn.repack(w2.view(torch.uint8), s2))
    x = torch.randn(t, h, generator=g, device=DEV, dtype=torch.float16)
    ids, p = hq.route_topk(torch.randn(t, e, generator=g, device=DEV), 2)
    y = hq.moe_layer(gu, dn, x, ids, p, *wm).double()
    torch.cuda.synchronize()
    want = o8.layer(x.double(), ids.long(), p, w1, s1, w2, s2)[0]
    err, ref = (y - want)[:, ~large], want[:, ~large]
    assert (err.pow(2).mean() / ref.pow(2).mean()).sqrt() < torch.finfo(torch.float16).eps / 2
