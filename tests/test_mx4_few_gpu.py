"""MXFP4 layers in the two kernels with two tiles of tokens, and at the limits of what takes them:
random routing with slots without an expert, every slot on one expert, rows of NaN."""
import pytest
import torch

import bit_quantized_gemm_repack_amd as hq
from test_mx4_gpu import DEV, DT, Layer, _x
from test_mx4_few_rule import _few

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("e,h,i,topk,t", [(40, 7168, 256, 2, 17), (64, 7168, 256, 2, 32), (30, 7168, 512, 1, 31), (8, 4096, 512, 2, 10), (7, 7168, 256, 1, 17),
                                          (1, 7168, 128, 16, 4), (3, 2176, 640, 5, 4), (2, 6144, 384, 1, 5)])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_layer(e, h, i, topk, t, dt):
    print(f"[gpu case] few {t} {e} {topk} {h} {i} {dt}", flush=True)
    assert _few(e, h, i, topk, t)
    L = Layer(t + e, e, h, i, t, dt)
    x = _x(L.g, t, h, DT[dt])
    ids = torch.randint(-1, e + 1, (t, topk), generator=L.g, device=DEV).to(torch.int32)
    w = torch.randn(t, topk, generator=L.g, device=DEV)
    y = L.run(x, ids, w)
    torch.cuda.synchronize()
    L.check(y, x, ids, w, "random ids")
    codes, s = hq.quantize_mxfp4(x)
    assert torch.equal(y, L.run(codes, ids, w, x_scale=s)), "quantised outside"
    bad = x.clone()
    bad[t - 1, 7] = float("nan")
    z = L.run(bad, ids, w)
    torch.cuda.synchronize()
    assert torch.equal(z[: t - 1], y[: t - 1])
    assert bool(z[t - 1].isnan().all()) == bool(((ids[t - 1] >= 0) & (ids[t - 1] < e)).any())
    one = torch.full_like(ids, e - 1)
    y = L.run(x, one, w)
    torch.cuda.synchronize()
    L.check(y, x, one, w, "one expert")
