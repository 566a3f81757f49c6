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
