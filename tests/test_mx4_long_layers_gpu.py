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


def test_graphs_and_streams_of_fp16_outputs():
    """Two graphs of one layer, replayed with new inputs and eager calls between, and two streams at once."""
    e, topk, h, i, t = 12, 4, 1024, 384, 300
    L = Layer(3, e, h, i, t, "f16")
    xs = [_x(L.g, t, h, torch.float16) for _ in range(3)]
    rt = [_routing(L.g, t, e, topk) for _ in range(3)]
    want = [L.run(x, *r) for x, r in zip(xs, rt)]
    side = [torch.cuda.Stream() for _ in range(2)]
    got = [None] * 3
    for s in side:
        s.wait_stream(torch.cuda.current_stream())
    for k in range(3):
        with torch.cuda.stream(side[k % 2]):
            got[k] = L.run(xs[k], *rt[k])
    for s in side:
        torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    x, ids, w = xs[0].clone(), rt[0][0].clone(), rt[0][1].clone()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = L.run(x, ids, w)
        graphs.append((graph, out))
    for k in (1, 2, 0, 1):
        x.copy_(xs[k]), ids.copy_(rt[k][0]), w.copy_(rt[k][1])
        for graph, out in graphs:
            graph.replay()
            assert torch.equal(L.run(xs[k], *rt[k]), want[k])
        torch.cuda.synchronize()
        assert all(torch.equal(out, want[k]) for _, out in graphs), f"replay of {k}"
