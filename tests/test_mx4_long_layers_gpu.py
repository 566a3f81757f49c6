"""MXFP4 experts' layers as a prompt runs them, compared whole with the float64 oracle: 256 experts
with more slots than one workgroup sorts, H = 7168 past the few tokens, intermediates beyond 1024."""
import pytest
import torch

import bit_quantized_gemm_repack_amd as hq
from test_mx4_gpu import DT, Layer, _routing, _x

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t,e,topk,h,i,dt", [
    (65, 256, 8, 1024, 384, "bf16"), (200, 256, 8, 1024, 384, "f16"), (300, 256, 8, 1024, 384, "bf16"), (1500, 256, 8, 1024, 384, "bf16"),
    (4100, 256, 8, 512, 128, "f16"), (20, 256, 8, 7168, 256, "bf16"), (200, 16, 2, 7168, 256, "bf16"), (333, 12, 4, 7168, 512, "f16"),
    (70, 8, 2, 640, 1408, "bf16"), (400, 8, 2, 1152, 1536, "f16"), (1200, 6, 3, 512, 2048, "bf16"),
])
def test_layer(t, e, topk, h, i, dt):
    print(f"[gpu case] layer {t} {e} {topk} {h} {i} {dt}", flush=True)
    L = Layer(t + e, e, h, i, t, dt)
    x = _x(L.g, t, h, DT[dt])
    ids, w = _routing(L.g, t, e, topk)
    ids = ids.clone()
    ids.view(-1)[:: 97] = -1
    y = L.run(x, ids, w)
    torch.cuda.synchronize()
    L.check(y, x, ids, w, "16-bit x")
    codes, s = hq.quantize_mxfp4(x)
    assert torch.equal(y, L.run(codes, ids, w, x_scale=s)), "quantised outside"
