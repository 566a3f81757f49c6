"""The down product of MXFP4 experts by itself, on codes given: every block height with short and
long K (up to 1024 the weights stay in registers, beyond they come through a ring), odd numbers
of 128-k groups, widths that end inside a tile, blocks partly filled, slots without an expert;
outputs of fp16, to which the slots' rows add next to nothing; NaN weights."""
import pytest
import torch

import bit_quantized_gemm_repack_amd as hq
from oracle import mx4 as om

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f16": torch.float16}

# (tokens, experts, slots a token, n, k)
SHORT = [(90, 5, 3, 640, 128), (300, 7, 2, 448, 384), (33, 40, 4, 256, 768), (700, 3, 2, 320, 1024)]
LONG = [(1, 8, 2, 256, 1152), (90, 5, 3, 640, 1152), (300, 7, 2, 448, 1408), (37, 3, 1, 2048, 2048), (700, 4, 2, 320, 1536), (150, 30, 8, 192, 2176)]


class Down:
    def __init__(self, t, e, topk, n, k, dt, bm):
        self.g = g = torch.Generator(DEV)
        g.manual_seed(t + k)
        self.t, self.e, self.topk, self.n, self.k, self.dt = t, e, topk, n, k, DT[dt]
        self.plan = hq.MoePlan(n, k, hq.w4a4_mxfp4(dt), e, t, "topk_combine", tuning=None if bm is None else dict(tile_m=bm))
        self.codes = self._bytes(e, n, k // 2)
        self.e8 = self._powers(e, n, k // 32, mid=122)
        ids = torch.randint(0, e, (t, topk), generator=g, device=DEV, dtype=torch.int32)
        ids.view(-1)[::11] = -1
        if t > 4:
            ids[3] = e + 5
        self.ids = ids
        self.b = self.plan.block_m(t, topk)
        self.al = hq.moe_align(ids, e, self.b)
        mp = self.al[0].numel()
        self.a, self.s = self._bytes(mp, k // 2), self._powers(k // 128, mp, 4, mid=127)
        self.w = torch.rand(t, topk, generator=g, device=DEV) + 0.1

    def _bytes(self, *shape):
        return torch.randint(0, 256, shape, generator=self.g, dtype=torch.uint8, device=DEV)

    def _powers(self, *shape, mid):
        return torch.randint(mid - 3, mid + 4, shape, generator=self.g, dtype=torch.uint8, device=DEV)

    def run(self, e8=None):
        y = self.plan.moe_gemm(self.a, self.t, self.topk, *self.al, *self.plan.repack(self.codes, e8m0=self.e8 if e8 is None else e8), a_scale=self.s,
                               topk_w=self.w)
        torch.cuda.synchronize()
        return y

    def want(self, rows16):
        """(y, bound before the output's rounding): the products' fp32 sums, the slots' rows, and topk weighted
        additions of fp32."""
        used = int(self.al[2])
        sid = self.al[0][:used].long()
        of = self.al[1].long()[torch.arange(used, device=DEV) // self.b]
        y = torch.zeros(self.t, self.n, dtype=torch.float64, device=DEV)
        tol = torch.zeros_like(y)
        for ex in range(self.e):
            pos = torch.nonzero((sid < self.t * self.topk) & (of == ex)).squeeze(1)
            if not len(pos):
                continue
            o, to = om.gemm(om.rows(om.values(self.a[pos]), om.row_major(self.s[:, pos])), om.weight(self.codes[ex], self.e8[ex]))
            p = self.w.view(-1)[sid[pos]].double().unsqueeze(1)
            y.index_add_(0, sid[pos] // self.topk, o * p)
            tol.index_add_(0, sid[pos] // self.topk, (to + (om.slot_rows_bound(o) if rows16 else om.ROW_24 * o.abs()) + self.topk * 2.0 ** -23 * o.abs()) * p)
        return y, tol


@pytest.mark.parametrize("t,e,topk,n,k", SHORT + LONG)
@pytest.mark.parametrize("bm", [None, 16, 64, 128])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_down(t, e, topk, n, k, bm, dt):
    print(f"[gpu case] down {t} {e} {topk} {n} {k} {bm} {dt}", flush=True)
    d = Down(t, e, topk, n, k, dt, bm)
    y = d.run()
    want, tol = d.want(rows16=dt == "bf16")            # rows to outputs of fp16 are finer
    tol = tol + om.half_step(want.abs() + tol, d.dt) + 1e-30
    off = (y.double() - want).abs()
    assert (off <= tol).all(), f"{int((off > tol).sum())} of {off.numel()} off, worst {float((off / tol).max()):.3g} of the bound"
    if t > 4:
        assert (y[3] == 0).all()


@pytest.mark.parametrize("t,e,topk,n,k", [SHORT[1], LONG[2], LONG[4]])
@pytest.mark.parametrize("bm", [16, 128])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_nan_column(t, e, topk, n, k, bm, dt):
    """A NaN column of one expert: there its tokens are NaN, everything else keeps its bits."""
    print(f"[gpu case] NaN column {t} {e} {topk} {n} {k} {bm} {dt}", flush=True)
    d = Down(t, e, topk, n, k, dt, bm)
    y = d.run()
    e8 = d.e8.clone()
    e8[1, n - 3, 2] = 255
    z = d.run(e8)
    hit = (d.ids == 1).any(-1)
    assert hit.any() and z[hit][:, n - 3].isnan().all()
    z[hit, n - 3] = y[hit, n - 3]
    assert torch.equal(z, y)


@pytest.mark.parametrize("t,n", [(33000, 4096), (9000, 7232)])
def test_windows_of_finer_rows(t, n):
    """Several column windows of a product with rows of 24 bits, the last one narrower."""
    topk, k, e = 4, 256, 6
    print(f"[gpu case] windows {t} {n}", flush=True)
    d = Down(t, e, topk, n, k, "f16", None)
    y = d.run()
    want, tol = d.want(rows16=False)
    tol = tol + om.half_step(want.abs() + tol, d.dt) + 1e-30
    assert ((y.double() - want).abs() <= tol).all()


def test_fp16_outputs_are_off_by_their_rounding():
    """Root mean square over all outputs: what rounding to fp16 once leaves and a hundredth more at most (rows of 11 bits
    had a third more).  The products' bounds are far below: sums of 768 products of whole quarters in fp32."""
    d = Down(1000, 16, 8, 1024, 768, "f16", None)
    y = d.run().double()
    want, _ = d.want(rows16=False)
    once = (want.half().double() - want).pow(2).mean().sqrt()
    assert (y - want).pow(2).mean().sqrt() < 1.01 * once


def test_infinite_rows():
    """fp32's largest numbers, infinities and NaN in the rows to outputs of fp16."""
    t, e, n, k = 64, 2, 256, 256
    d = Down(t, e, 1, n, k, "f16", None)
    d.ids = torch.arange(t, device=DEV, dtype=torch.int32).view(t, 1) % e
    d.al = hq.moe_align(d.ids, e, d.b)
    d.a, d.s = d._bytes(d.al[0].numel(), k // 2), torch.full((k // 128, d.al[0].numel(), 4), 254, dtype=torch.uint8, device=DEV)
    d.codes = torch.full_like(d.codes, 0x77)           # 6 each: sums far beyond fp32
    d.codes[0] = 0x07                                  # 6 and 0
    d.e8 = torch.full_like(d.e8, 130)
    d.w = torch.full((t, 1), 2.0 ** -126, device=DEV)
    y = d.run()
    used = int(d.al[2])
    sid = d.al[0][:used].long()
    pos = torch.nonzero(sid < t).squeeze(1)
    o = torch.zeros(t, n, dtype=torch.float64, device=DEV)
    for ex in range(e):
        mine = pos[d.ids[sid[pos], 0] == ex]
        o[sid[mine]] = om.rows(om.values(d.a[mine]), om.row_major(d.s[:, mine])) @ om.weight(d.codes[ex], d.e8[ex]).t()
    big = o.abs() > 2.0 ** 130
    assert big.any() and not y[big].isfinite().any()
