"""Layers of a few tokens where a tile has many units, a batch many slots, or an
expert more rows than a workgroup holds at a time."""
import pytest
import torch

import bit_quantized_gemm_repack_amd as hq
from oracle import block8 as o8

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E4 = torch.float8_e4m3fn


def _layer(seed, e, h, i, max_t=64):
    g = torch.Generator(DEV)
    g.manual_seed(seed)
    def weight(n, k):
        codes = (torch.randn(e, n, k, generator=g, device=DEV) * 96).clamp_(-448, 448).to(E4)
        return codes, (0.5 + torch.rand(e, n // 128, k // 128, generator=g, device=DEV)) / (96 * k ** 0.5)
    w1, w2 = weight(2 * i, h), weight(h, i)
    gu, dn = (hq.MoePlan(n, k, hq.w8a8_block(), e, max_t, epi) for n, k, epi in ((2 * i, h, "silu_mul_qfp8"), (h, i, "topk_combine")))
    wm = (*gu.repack(w1[0].view(torch.uint8), w1[1]), *dn.repack(w2[0].view(torch.uint8), w2[1]))
    return g, gu, dn, w1, w2, wm


def _check(y, x, ids, p, w1, w2):
    want, tol = o8.layer(x.double(), ids.long(), p, *w1, *w2)
    tol = tol + o8.half_step(want.abs() + tol, torch.bfloat16) + 1e-30
    bad = ~((y.double() - want).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off"


@pytest.mark.parametrize("t", [10, 16, 33, 64])
def test_many_units(monkeypatch, t):
    """16 experts a token of 300: up to 256 units a tile, up to 1024 slots a batch."""
    monkeypatch.setattr(hq, "MOE_FEW_MAX_TOKENS", 64)
    print(f"[gpu case] few units {t}", flush=True)
    e, h, i = 300, 256, 128
    g, gu, dn, w1, w2, wm = _layer(t, e, h, i)
    x = torch.randn(t, h, generator=g, device=DEV, dtype=torch.bfloat16)
    spread = (torch.arange(t * 16, device=DEV) * 7 % e).view(t, 16).int()    # all of a tile's experts differ
    p = torch.rand(t, 16, generator=g, device=DEV)
    for ids in (spread, torch.randint(0, e, (t, 16), generator=g, device=DEV, dtype=torch.int32)):
        y = hq.moe_layer(gu, dn, x, ids, p, *wm)
        torch.cuda.synchronize()
        _check(y, x, ids, p, w1, w2)
    y, ids, p = hq.moe_layer_routed(gu, dn, x, torch.randn(t, e, generator=g, device=DEV), 16, *wm)
    torch.cuda.synchronize()
    _check(y, x, ids, p, w1, w2)


@pytest.mark.parametrize("e,topk,h,i", [(3, 2, 7168, 256), (4, 4, 4096, 384), (2, 2, 12288, 128), (5, 2, 20480, 128)])
@pytest.mark.parametrize("t", [3, 8, 9, 16])
def test_few_experts_many_rows(t, e, topk, h, i):
    """Large rows of few experts: more of an expert's rows than are held at a time, whose weights are then read again."""
    print(f"[gpu case] few rows {t} {e} {topk} {h} {i}", flush=True)
    g, gu, dn, w1, w2, wm = _layer(t + h, e, h, i)
    x = torch.randn(t, h, generator=g, device=DEV, dtype=torch.bfloat16)
    y, ids, p = hq.moe_layer_routed(gu, dn, x, torch.randn(t, e, generator=g, device=DEV), topk, *wm)
    torch.cuda.synchronize()
    _check(y, x, ids, p, w1, w2)
    ids = torch.full((t, topk), e - 1, dtype=torch.int32, device=DEV)        # one expert for all, more than once each
    y = hq.moe_layer(gu, dn, x, ids, p, *wm)
    torch.cuda.synchronize()
    _check(y, x, ids, p, w1, w2)
