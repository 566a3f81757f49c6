"""Routing on every kernel that the sizes choose: sixteen lanes a token (up to
64 experts, or up to 256 and many tokens) and a wave a token, at the borders of
their key counts, with ties, NaN, shut-off experts and rows without any."""
import math

import pytest
import torch

import bit_quantized_gemm_repack_amd as hq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _gen(seed):
    g = torch.Generator(DEV)
    g.manual_seed(seed)
    return g


def _want(x, topk, renorm):
    """ids, weights and, per weight, how far its logit is from the largest."""
    x = x.double()
    x = torch.where(torch.isnan(x), torch.full_like(x, -math.inf), x)
    best, ids = torch.sort(x, dim=1, descending=True, stable=True)  # ties: the lowest index first
    best, ids = best[:, :topk], ids[:, :topk]
    none = best == -math.inf
    over = torch.logsumexp(best if renorm else x, 1, keepdim=True)
    w = torch.exp(best - over).masked_fill(none, 0.0)
    far = (best[:, :1] - best).masked_fill(none, 0.0)
    return ids.masked_fill(none, -1), w, far


def _bound(w, far, e):
    """exp to 1 ulp (2^-23) of a difference that fp32 rounds by 2^-24 of itself;
    the sum's terms likewise, on average over e^-d at differences of log(e) + 1 at
    most; their sum in a tree of up to 26 additions of 2^-24 each; one quotient."""
    return w * ((1 + 1 + 13 + 0.5) * 2.0 ** -23 + (far + math.log(e) + 1) * 2.0 ** -24) * 1.01 + 2.0 ** -126


def _odd_rows(x, e):
    x[1] = -math.inf                                  # no expert
    x[2] = -math.inf
    x[2, e - 1] = -3.0                                # one
    x[3] = 0.25                                       # all equal
    x[4, : e // 2] = math.nan
    x[5] = -x[5].abs()
    x[5, 0], x[5, e - 1] = -0.0, 0.0
    x[6] = math.nan
    return x


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("e,topk", [(17, 16), (64, 16), (65, 8), (128, 1), (129, 16), (160, 6), (192, 8), (193, 3), (256, 8), (257, 8)])
@pytest.mark.parametrize("t", [9, 6143, 6144, 6161])
def test_route_every_kernel(t, e, topk, dt):
    print(f"[gpu case] route {t} {e} {topk} {dt}", flush=True)
    g = _gen(t + e)
    x = torch.randn(t, e, generator=g, device=DEV) * 3
    x[torch.rand(t, e, generator=g, device=DEV) < 0.1] = -math.inf
    x = _odd_rows(x.to(dt), e)
    if t > 9:
        x[-1] = x[3]
        x[7:1000] = torch.round(x[7:1000])            # many ties
    for renorm in (True, False):
        ids, w = hq.route_topk(x, topk, renormalize=renorm)
        torch.cuda.synchronize()
        wi, ww, far = _want(x, topk, renorm)
        assert torch.equal(ids.long(), wi)
        assert ((w.double() - ww).abs() <= _bound(ww, far, e)).all()


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("t,e", [(1, 64), (5, 64), (5, 256), (6200, 256), (6200, 130)])
def test_far_logits(t, e, dt):
    """Differences that are exact in fp32, up to 80: the exponential's own rounding is all there is."""
    x = -(torch.arange(e, device=DEV) * 0.5).clamp_max(80).repeat(t, 1)
    x[:, 0] = 0
    x = x[:, torch.randperm(e, generator=_gen(e), device=DEV)].to(dt).contiguous()
    for renorm in (True, False):
        ids, w = hq.route_topk(x, 16, renormalize=renorm)
        torch.cuda.synchronize()
        wi, ww, far = _want(x, 16, renorm)
        assert torch.equal(ids.long(), wi)
        assert ((w.double() - ww).abs() <= ww * (1 + 1 + 13 + 0.5) * 2.0 ** -23 * 1.01).all()
    far = torch.full((t, e), -60.0, device=DEV, dtype=dt)
    far[:, 3], far[:, 5] = 0.0, -40.0
    ids, w = hq.route_topk(far, 3, renormalize=False)
    torch.cuda.synchronize()
    assert ids[:, 0].eq(3).all() and ids[:, 1].eq(5).all()
    wi, ww, _ = _want(far, 3, False)
    assert ((w.double() - ww).abs() <= ww * (1 + 1 + 13 + 0.5) * 2.0 ** -23 * 1.01).all()


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("e,topk", [(8, 2), (40, 6), (64, 8), (65, 4), (128, 8), (200, 8), (256, 16), (300, 3), (700, 8)])
def test_layer_writes_the_weights_of_routing(e, topk, dt, renorm):
    """ids and weights of a layer from its logits are hq_route_topk's, bit for bit."""
    g = _gen(e)
    q = hq.w8a8_block()
    gu, dn = hq.MoePlan(256, 128, q, e, 64, "silu_mul_qfp8"), hq.MoePlan(128, 128, q, e, 64, "topk_combine")
    ones = lambda n, k: (torch.full((e, n, k), 0x38, dtype=torch.uint8, device=DEV), torch.full((e, n // 128, k // 128), 0.01, device=DEV))
    wm = (*gu.repack(*ones(256, 128)), *dn.repack(*ones(128, 128)))
    for t in (1, 2, 16, 24):
        x = torch.randn(t, 128, generator=g, device=DEV, dtype=torch.bfloat16)
        lg = (torch.randn(t, e, generator=g, device=DEV) * 4).to(dt)
        lg[0, 1] = -math.inf
        y, ids, w = hq.moe_layer_routed(gu, dn, x, lg, topk, *wm, renormalize=renorm)
        ri, rw = hq.route_topk(lg, topk, renormalize=renorm)
        torch.cuda.synchronize()
        assert torch.equal(ids, ri) and torch.equal(w, rw)
