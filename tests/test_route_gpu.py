"""Routing by scores on the GPU against the float64 oracle (oracle/route.py): ids equal,
weights within the roundings of their sum; scores that tie, groups of every size, experts
shut off, infinite biases, slices, streams and graphs, and refusals."""
import math

import pytest
import torch

import bit_quantized_gemm_repack_amd as hq
from oracle import route as orr

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _gen(seed):
    g = torch.Generator(DEV)
    g.manual_seed(seed)
    return g


def _check(x, topk, what="", **kw):
    ids, w = hq.route_experts(x, topk, **kw)
    torch.cuda.synchronize()
    wi, ww = orr.route(x, topk, **kw)
    assert ids.dtype == torch.int32 and w.dtype == torch.float32
    bad = (ids.cpu() != wi).any(-1)
    assert not bad.any(), f"{what}: {int(bad.sum())} rows of other experts, first {ids.cpu()[bad][0].tolist()} for {wi[bad][0].tolist()}"
    off = (w.cpu().double() - ww).abs() - orr.WEIGHT * ww.abs() - 2.0 ** -149
    assert off.max() <= 0, f"{what}: weights"
    return ids, w


CASES = [  # t, experts, topk, groups, group_topk, group_best
    (1, 256, 8, 8, 4, 2), (5, 160, 6, 8, 3, 1), (130, 64, 8, 1, 1, 2), (33, 8, 8, 4, 4, 2), (7, 1, 1, 1, 1, 1), (9, 100, 10, 5, 2, 2),
    (6, 512, 16, 16, 5, 2), (3, 1024, 64, 64, 9, 2), (4, 1024, 64, 2, 1, 1), (11, 192, 6, 3, 2, 2), (21, 65, 3, 13, 4, 2),
    (12, 64, 5, 64, 7, 2), (10, 128, 8, 8, 1, 2), (257, 384, 8, 1, 1, 1), (2, 1000, 20, 50, 3, 2), (301, 40, 2, 20, 3, 2),
]


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("biased", [False, True])
def test_route(dt, scoring, biased):
    for n, (t, experts, topk, groups, group_topk, group_best) in enumerate(CASES):
        print(f"[gpu case] route {dt} {scoring} {biased} {CASES[n]}", flush=True)
        g = _gen(100 * n + t)
        x = torch.randn(t, experts, generator=g, device=DEV) * (1 if n % 2 else 3)
        x = x.masked_fill((torch.rand(t, 1, generator=g, device=DEV) < 0.2) & (torch.rand(t, experts, generator=g, device=DEV) < 0.6), -math.inf)
        if t > 2:
            x[1] = -math.inf
            x[2, experts // 2:] = float("nan")
        bias = 0.2 * torch.randn(experts, generator=g, device=DEV) if biased else None
        _check(x.to(DT[dt]), topk, f"{dt} {scoring} {CASES[n]}", bias=bias, scoring=scoring, groups=groups, group_topk=group_topk,
               group_best=group_best, renormalize=n % 3 != 0, scale=2.5 if n % 2 else 1.0)


def test_ties():
    """Equal logits, saturated scores, biases that make keys equal: the lowest index, of experts and of groups."""
    x = torch.zeros(6, 96, device=DEV)
    x[1] = 40.0                                   # sigmoid 1 as an fp32 number
    x[2, ::2], x[2, 1::2] = 30.0, 60.0            # different logits, the same score
    x[3, 50:] = 1.0
    x[4] = -1e4                                   # score 0
    x[5, 95] = -0.0
    for kw in (dict(), dict(groups=8, group_topk=3), dict(groups=8, group_topk=3, group_best=1), dict(groups=96 // 2, group_topk=5)):
        ids, w = _check(x, 6, **kw)
        assert ids[1].tolist() == list(range(6)) and ids[2].tolist() == list(range(6))
        assert (w[4] == 0).all()
        _check(x, 6, scoring="softmax", **kw)
    bias = torch.zeros(96, device=DEV)
    bias[7] = 0.25
    y = torch.zeros(1, 96, device=DEV)
    y[0, 3] = math.log(3.0)                       # score 0.75 = 0.5 + 0.25
    ids, _ = _check(y, 2, bias=bias)
    assert ids.tolist() == [[3, 7]]


def test_neighbouring_scores():
    """Logits a last bit apart: a sigmoid formed in 32 bits chooses otherwise in three rows of four."""
    g = _gen(3)
    x = (torch.randn(400, 1, generator=g, device=DEV) + 2e-7 * torch.randn(400, 200, generator=g, device=DEV))
    _check(x, 8)
    _check(x, 8, scoring="softmax", renormalize=False)
    _check(x, 8, groups=10, group_topk=4, bias=0.1 + 0.3 * torch.rand(200, generator=g, device=DEV).round())


def test_biases_and_shut_off_groups():
    inf = math.inf
    x = torch.randn(3, 32, generator=_gen(4), device=DEV)
    bias = torch.zeros(32, device=DEV)
    bias[9], bias[20], bias[0], bias[31] = inf, inf, -inf, float("nan")
    ids, w = _check(x, 4, bias=bias)
    assert ids[:, :2].tolist() == [[9, 20]] * 3 and not torch.isin(ids, torch.tensor([0, 31], device=DEV, dtype=torch.int32)).any()
    assert torch.isfinite(w).all()
    x[0, :16] = -inf                              # two groups of four gone: the kept ones end in ids of -1
    x[1, :31] = -inf
    ids, w = _check(x, 8, groups=4, group_topk=4)
    assert ids[1].tolist() == [31] + [-1] * 7 and w[1].tolist() == [1] + [0] * 7
    _check(x, 8, groups=4, group_topk=2)
    x[2] = -60.0                                  # scores near the least fp32 numbers
    _check(x, 8, groups=4, group_topk=2)
    x[2] = -120.0                                 # below them: weights stay zero
    ids, w = _check(x, 8)
    assert (w[2] == 0).all() and ids[2].tolist() == list(range(8))


def test_many_tokens_and_slices():
    g = _gen(6)
    x = torch.randn(16384, 161, generator=g, device=DEV)
    y = x.view(-1)[1:1 + 16383 * 160].view(16383, 160)         # rows at any element
    ids, w = hq.route_experts(y, 6, groups=8, group_topk=3)
    at = torch.tensor([0, 1, 5000, 16382], device=DEV)
    wi, ww = orr.route(y[at], 6, groups=8, group_topk=3)
    assert torch.equal(ids[at].cpu(), wi) and ((w[at].cpu().double() - ww).abs() <= orr.WEIGHT * ww).all()
    one = [hq.route_experts(y[i:i + 1], 6, groups=8, group_topk=3) for i in at.tolist()]
    for i, (a, b) in zip(at.tolist(), one):                    # a row's result is its own
        assert torch.equal(ids[i], a[0]) and torch.equal(w[i], b[0])
    assert hq.route_experts(y[:0], 6)[0].shape == (0, 6)


def test_streams_and_graphs():
    g = _gen(7)
    xs = [torch.randn(50, 256, generator=g, device=DEV) for _ in range(4)]
    bias = 0.1 * torch.randn(256, generator=g, device=DEV)
    kw = dict(bias=bias, groups=8, group_topk=4, scale=2.5)
    want = [hq.route_experts(x, 8, **kw) for x in xs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [hq.route_experts(x, 8, **kw) for x in xs]
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) for a, b in zip(got, want))
    x = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = hq.route_experts(x, 8, **kw)
    for i in (1, 2, 3, 0, 2):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[i][0]) and torch.equal(out[1], want[i][1]), f"replay {i}"


def test_refusals():
    x = torch.zeros(4, 64, device=DEV)
    for kw in (dict(scoring="exp"), dict(bias=torch.zeros(32, device=DEV)), dict(bias=torch.zeros(64)), dict(bias=torch.zeros(64, device=DEV).half()),
               dict(bias=torch.zeros(128, device=DEV)[::2])):
        with pytest.raises(ValueError):
            hq.route_experts(x, 4, **kw)
    for bad in (x.double(), x.t(), x[0], x.int()):
        with pytest.raises(ValueError):
            hq.route_experts(bad, 4)
    for kw in (dict(topk=0), dict(topk=65), dict(groups=7), dict(groups=8, group_topk=9), dict(topk=9, groups=8, group_topk=1), dict(group_best=3),
               dict(scale=math.inf)):
        with pytest.raises(hq.HQError):
            hq.route_experts(x, **dict(dict(topk=4), **kw))


@pytest.mark.parametrize("t,e,topk,kw,dt", [(4096, 64, 6, dict(), "bf16"), (4100, 8, 2, dict(scoring="softmax"), "f32"),
                                           (5121, 128, 16, dict(groups=16, group_topk=5, group_best=1), "f16"), (7001, 160, 6, dict(scoring="softmax", groups=8, group_topk=3), "bf16"),
                                           (10241, 256, 8, dict(bias=True, groups=8, group_topk=4, scale=2.5), "f32"), (10250, 250, 1, dict(renormalize=False), "f32"),
                                           (4111, 100, 10, dict(groups=10, group_topk=2, bias=True), "f32"), (4097, 17, 16, dict(scoring="softmax", bias=True), "f32")])
def test_many_tokens_are_single_ones(t, e, topk, kw, dt):
    """The kernel of many tokens gives the bits of the other one, for ties, experts shut off and rows without any."""
    print(f"[gpu case] many {t} {e} {topk} {kw} {dt}", flush=True)
    g = _gen(e)
    x = torch.randn(t, e, generator=g, device=DEV)
    x[::3] = (x[::3] * 2).round() / 2                              # ties
    x[torch.rand(t, e, generator=g, device=DEV) < 0.05] = -math.inf
    x[5], x[6, 1:], x[t - 1, 0] = -math.inf, float("nan"), float("nan")
    x = x.to(DT[dt])
    if kw.get("bias"):
        kw = dict(kw, bias=torch.randn(e, generator=g, device=DEV))
    ids, w = hq.route_experts(x, topk, **kw)
    parts = [hq.route_experts(x[i:i + 1500], topk, **kw) for i in range(0, t, 1500)]
    torch.cuda.synchronize()
    assert torch.equal(ids, torch.cat([p[0] for p in parts])) and torch.equal(w, torch.cat([p[1] for p in parts]))
    rows = torch.cat([torch.arange(40, device=DEV), torch.arange(t - 40, t, device=DEV)])
    kw = {k: v.cpu() if k == "bias" else v for k, v in kw.items()}
    wi, ww = orr.route(x[rows].cpu(), topk, **kw)
    assert torch.equal(ids[rows].cpu(), wi)
    assert ((w[rows].cpu().double() - ww).abs() <= orr.WEIGHT * ww.abs() + 2.0 ** -149).all()


def test_native_calls_are_the_same(monkeypatch):
    """The binding's native call against the same call through ctypes, on another stream too."""
    x = torch.randn(9, 64, generator=_gen(41), device=DEV)
    b = torch.randn(64, generator=_gen(42), device=DEV)

    def calls():
        return [*hq.route_experts(x, 4), *hq.route_experts(x.half(), 6, b, "softmax", 8, 3, 1, False, 2.5), *hq.route_experts(x.bfloat16(), 1, b),
                *hq.route_experts(x[:0], 3), *hq.route_experts(x, 8, bias=b, groups=4, group_topk=2, scale=0.5)]
    assert hq._calls is not None and hq._calls.route_experts(x, 4, b, 0, 1, 1, 2, True, 1.0) is not None
    native = calls()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        other = calls()
    torch.cuda.synchronize()
    assert hq._calls.route_experts(x.t(), 4, None, 0, 1, 1, 2, True, 1.0) is None and hq._calls.route_experts(x, 65, None, 0, 1, 1, 2, True, 1.0) is None
    assert hq._calls.route_experts(x, 4, b[1:], 0, 1, 1, 2, True, 1.0) is None and hq._calls.route_experts(x, 4, b, 0, 7, 1, 2, True, 1.0) is None
    monkeypatch.setattr(hq, "_calls", None)
    plain = calls()
    torch.cuda.synchronize()
    for p, q, r in zip(native, other, plain):
        assert p.dtype == r.dtype and p.shape == r.shape and torch.equal(p, r) and torch.equal(q, r)
