"""MXFP4 experts' layers on the GPU against the float64 oracle (oracle/mx4.py): the two
grouped products stage by stage on every block, exact sums, whole layers, quantisation
of blocks that are not finite, rows and experts that must not touch each other, graphs
and streams, and refusals."""
import pytest
import torch

import bit_quantized_gemm_repack_amd as hq
from oracle import mx4 as om

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def _gen(seed):
    g = torch.Generator(DEV)
    g.manual_seed(seed)
    return g


def _x(g, m, k, dt, spread=0.5):
    return (torch.randn(m, k, generator=g, device=DEV) * torch.exp(spread * torch.randn(m, 1, generator=g, device=DEV))).to(dt)


def _check(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float(((got.double() - want).abs() / tol).max()):.3g} of the bound"


def _routing(g, t, e, topk):
    lg = torch.randn(t, e, generator=g, device=DEV)
    w, ids = torch.softmax(lg, -1).topk(topk)
    return ids.int().contiguous(), (w / w.sum(-1, keepdim=True)).contiguous()


def _quant(v):
    q, e = om.quantize(v.double())
    return om.pack(q), e.to(torch.uint8)


class Layer:
    def __init__(self, seed, e, h, i, t, dt="bf16", tuning=None):
        self.g = g = _gen(seed)
        self.e, self.h, self.i, self.dt = e, h, i, DT[dt]
        self.w1, self.e1 = _quant(torch.randn(e, 2 * i, h, generator=g, device=DEV) * torch.exp(0.3 * torch.randn(e, 2 * i, 1, generator=g, device=DEV)) / h ** 0.5)
        self.w2, self.e2 = _quant(torch.randn(e, h, i, generator=g, device=DEV) / i ** 0.5)
        q = hq.w4a4_mxfp4(dt)
        self.gu = hq.MoePlan(2 * i, h, q, e, t, "silu_mul_qmxfp4", tuning=tuning)
        self.dn = hq.MoePlan(h, i, q, e, t, "topk_combine", tuning=tuning)
        self.wm = (*self.gu.repack(self.w1, e8m0=self.e1), *self.dn.repack(self.w2, e8m0=self.e2))

    def run(self, x, ids, w, **kw):
        return hq.moe_layer(self.gu, self.dn, x, ids, w, *self.wm, **kw)

    def check(self, y, x, ids, w, what):
        xq = om.rows(*om.quantize(x.double())) if x.dtype != torch.float64 else x
        want, tol = om.layer(xq, ids, w, self.w1, self.e1, self.w2, self.e2)
        _check(y, want, tol + om.half_step(want.abs() + tol, self.dt) + 1e-30, what)


# ------------------------------------------------------------------ the quantiser --
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_quantize_bits(dt):
    """Every 16-bit value as its block's largest, and blocks that are not finite apart from the others."""
    v = torch.arange(0, 1 << 15, dtype=torch.int32, device=DEV).to(torch.int16).view(DT[dt])
    v = v[torch.isfinite(v)]
    f = torch.linspace(-1, 1, 32, device=DEV, dtype=torch.float64)
    x = (v.double()[:, None] * f).to(DT[dt])
    x = x[: x.shape[0] // 4 * 4].view(-1, 128)
    codes, e = hq.quantize_mxfp4(x)
    q, we = om.quantize(x.double())
    assert torch.equal(om.row_major(e).double(), we)
    assert torch.equal(codes, om.pack(q))
    x[5, 3], x[9, 64], x[11, 127] = float("nan"), float("inf"), -float("inf")
    c2, e2 = hq.quantize_mxfp4(x)
    torch.cuda.synchronize()
    r, r2 = om.row_major(e), om.row_major(e2)
    assert (r2 != r).sum() == 3 and r2[5, 0] == 255 and r2[9, 2] == 255 and r2[11, 3] == 255
    same = (r2 == r).repeat_interleave(16, 1)
    assert torch.equal(c2[same], codes[same])


# ------------------------------------------------------------- the grouped products --
@pytest.mark.parametrize("t,e,topk,h,i", [(1, 8, 2, 512, 128), (5, 8, 8, 640, 256), (40, 16, 4, 768, 384), (300, 12, 3, 512, 1024),
                                          (37, 3, 1, 1152, 640), (130, 70, 6, 256, 768), (700, 4, 2, 320, 128)])
@pytest.mark.parametrize("bm", [None, 16, 64, 128])
def test_grouped_stages(t, e, topk, h, i, bm):
    if h % 128:
        h = 384
    print(f"[gpu case] grouped {t} {e} {topk} {h} {i} {bm}", flush=True)
    L = Layer(t + e, e, h, i, t, tuning=None if bm is None else dict(tile_m=bm))
    x = _x(L.g, t, h, torch.bfloat16)
    ids, w = _routing(L.g, t, e, topk)
    ids = ids.clone()
    ids.view(-1)[:: 11] = -1                          # slots without an expert
    if t > 4:
        ids[3] = e + 5
    b = L.gu.block_m(t, topk)
    al = hq.moe_align(ids, e, b)
    xq, xs = hq.quantize_mxfp4(x)
    codes, sc = L.gu.moe_gemm(xq, t, topk, *al, *L.wm[:2], a_scale=xs)
    y = L.dn.moe_gemm(codes, t, topk, *al, *L.wm[2:], a_scale=sc, topk_w=w)
    torch.cuda.synchronize()
    used = int(al[2])
    sid, bex = al[0][:used].long(), al[1].long()
    of = bex[torch.arange(used, device=DEV) // b]
    live = (sid < t * topk) & (of >= 0)
    xv = om.rows(om.values(xq), om.row_major(xs))
    got, want = om.rows(om.values(codes), om.row_major(sc)), torch.zeros(t, h, dtype=torch.float64, device=DEV)
    tol = torch.zeros_like(want)
    for ex in range(e):
        pos = torch.nonzero(live & (of == ex)).squeeze(1)
        if not len(pos):
            continue
        tok = sid[pos] // topk
        hh, th = om.gemm(xv[tok], om.weight(L.w1[ex], L.e1[ex]))
        mid, far = om.requant_range(om.silu_mul(hh), om.act_bound(hh, th))
        _check(got[pos], mid, far, f"gate_up of expert {ex}")
        o, to = om.gemm(got[pos], om.weight(L.w2[ex], L.e2[ex]))
        p = w.view(-1)[sid[pos]].double().unsqueeze(1)
        want.index_add_(0, tok, o * p)
        tol.index_add_(0, tok, (to + om.slot_rows_bound(o) + 2.0 ** -20 * o.abs()) * p.abs())
    _check(y, want, tol + om.half_step(want.abs() + tol, torch.bfloat16) + 1e-30, "down")
    if t > 4:
        assert (y[3] == 0).all()


@pytest.mark.parametrize("bm", [16, 64, 128])
def test_down_is_exact_where_sums_are(bm):
    """Whole numbers whose sums fp32 holds: the slot rows are exact in fp16 below 2^11, so y is what integers give."""
    e, h, i, t = 3, 256, 512, 90
    L = Layer(1, e, h, i, t, "f16", tuning=dict(tile_m=bm))
    g = _gen(2)
    w2 = torch.randint(-2, 3, (e, h, i), generator=g, device=DEV).double()
    L.w2, L.e2 = om.pack(w2), torch.full((e, h, i // 32), 127, dtype=torch.uint8, device=DEV)
    L.e2[:, :, 3] = 128
    wm = L.dn.repack(L.w2, e8m0=L.e2)
    ids = torch.randint(0, e, (t, 1), generator=g, device=DEV, dtype=torch.int32)
    al = hq.moe_align(ids, e, L.dn.block_m(t, 1))
    mp = al[0].numel()
    a = torch.randint(-1, 2, (mp, i), generator=g, device=DEV).double()
    s = torch.full((mp, i // 32), 127, dtype=torch.uint8, device=DEV)
    s[::3, 1] = 129
    y = L.dn.moe_gemm(om.pack(a), t, 1, *al, *wm, a_scale=om.group_major(s), topk_w=torch.ones(t, 1, device=DEV))
    torch.cuda.synchronize()
    at = torch.empty(t, dtype=torch.long, device=DEV)
    used = int(al[2])
    live = al[0][:used] < t
    at[al[0][:used][live].long()] = torch.nonzero(live).squeeze(1)
    av = om.rows(a, s)[at]
    want = torch.stack([om.weight(L.w2[k], L.e2[k]) @ av[r] for r, k in enumerate(ids[:, 0].tolist())])
    assert want.abs().max() < 2048 and torch.equal(y.double(), want)


# ---------------------------------------------------------------------- whole layers --
@pytest.mark.parametrize("t", [1, 2, 3, 7, 8, 9, 13, 16, 17, 33, 64, 65, 200, 1500])
@pytest.mark.parametrize("e,topk,h,i,dt", [(8, 2, 512, 128, "bf16"), (60, 6, 640, 256, "f16"), (256, 8, 1024, 384, "bf16"), (16, 16, 256, 1024, "f16"),
                                           (5, 3, 2176, 128, "bf16")])
def test_layer(t, e, topk, h, i, dt):
    if t > 64 and e > 100:
        pytest.skip("covered by the smaller layers")
    print(f"[gpu case] layer {t} {e} {topk} {h} {i} {dt}", flush=True)
    topk = min(topk, e)
    L = Layer(t + e, e, h, i, t, dt)
    x = _x(L.g, t, h, DT[dt])
    ids, w = _routing(L.g, t, e, topk)
    y = L.run(x, ids, w)
    torch.cuda.synchronize()
    L.check(y, x, ids, w, "16-bit x")
    codes, s = hq.quantize_mxfp4(x)
    z = L.run(codes, ids, w, x_scale=s)
    torch.cuda.synchronize()
    assert torch.equal(y, z), "quantised outside"
    assert torch.equal(y, L.run(x, ids, w)), "twice"


@pytest.mark.parametrize("t,e,topk,h,i", [(1, 20, 16, 2048, 640), (1, 8, 1, 2048, 128), (2, 8, 8, 2176, 384), (4, 8, 8, 4096, 256), (5, 12, 8, 4096, 128),
                                          (9, 256, 8, 7168, 256), (16, 3, 2, 7168, 384), (17, 3, 1, 7168, 128), (33, 40, 2, 7168, 512), (64, 5, 1, 7168, 256),
                                          (15, 1, 4, 7168, 128), (2, 8, 1, 2048, 7168), (2, 2, 8, 2048, 7168), (4, 2, 2, 24576, 128)])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_layer_of_few_tokens(t, e, topk, h, i, dt):
    """The two kernels: slots without an expert, an expert twice in a row, NaN rows, one expert for many."""
    print(f"[gpu case] few {t} {e} {topk} {h} {i} {dt}", flush=True)
    L = Layer(t + e, e, h, i, t, dt)
    x = _x(L.g, t, h, DT[dt])
    ids = torch.randint(-1, e + 1, (t, topk), generator=L.g, device=DEV).to(torch.int32)
    w = torch.randn(t, topk, generator=L.g, device=DEV)
    y = L.run(x, ids, w)
    torch.cuda.synchronize()
    L.check(y, x, ids, w, "random ids")
    codes, s = hq.quantize_mxfp4(x)
    assert torch.equal(y, L.run(codes, ids, w, x_scale=s)), "quantised outside"
    hit = ((ids >= 0) & (ids < e)).any(-1)
    assert (y[~hit] == 0).all()
    if t > 1:
        bad = x.clone()
        bad[t - 1, 7] = float("nan")
        z = L.run(bad, ids, w)
        torch.cuda.synchronize()
        assert torch.equal(z[: t - 1], y[: t - 1]) and z[t - 1].isnan().all() == hit[t - 1]
    one = torch.full_like(ids, e - 1)
    y = L.run(x, one, w)
    torch.cuda.synchronize()
    L.check(y, x, one, w, "one expert")


@pytest.mark.parametrize("t,h", [(2, 2176), (5, 4096)])
def test_nan_weights_of_few_tokens(t, h):
    """A NaN column of one expert's gate_up, and one of its down: tokens elsewhere keep their bits."""
    e, i = 6, 128
    L = Layer(4, e, h, i, t)
    x = _x(L.g, t, h, torch.bfloat16)
    ids = torch.tensor([[4, 1], [0, 2], [3, 4], [5, 0], [1, 2]], dtype=torch.int32, device=DEV)[:t].contiguous()
    w = torch.rand(t, 2, generator=L.g, device=DEV) + 0.1
    y = L.run(x, ids, w)
    hit = (ids == 4).any(-1)
    e1, e2 = L.e1.clone(), L.e2.clone()
    e1[4, 0, 0], e2[4, 7, 1] = 255, 255
    z = hq.moe_layer(L.gu, L.dn, x, ids, w, *L.gu.repack(L.w1, e8m0=e1), *L.wm[2:])
    u = hq.moe_layer(L.gu, L.dn, x, ids, w, *L.wm[:2], *L.dn.repack(L.w2, e8m0=e2))
    torch.cuda.synchronize()
    assert z[hit].isnan().all() and torch.equal(z[~hit], y[~hit])
    assert u[hit][:, 7].isnan().all() and torch.equal(u[~hit], y[~hit])
    u[:, 7], y[:, 7] = 0, 0
    assert torch.equal(u, y)


@pytest.mark.parametrize("t,topk", [(40, 4), (3, 64), (900, 2)])
def test_layer_of_most_experts(t, topk):
    """4096 experts, the most; 64 slots a token, the most."""
    print(f"[gpu case] 4096 experts {t} {topk}", flush=True)
    L = Layer(t, 4096, 128, 128, t)
    x = _x(L.g, t, 128, torch.bfloat16)
    ids, w = _routing(L.g, t, 4096, topk)
    ids[0, 0], ids[1, :2] = 4095, 7
    y = L.run(x, ids, w)
    torch.cuda.synchronize()
    L.check(y, x, ids, w, "4096 experts")


@pytest.mark.parametrize("t", [1, 3, 70])
def test_layer_to_another_width(t):
    """down's n need not be gate_up's k."""
    e, h, i, n, topk = 6, 2048, 256, 640, 3
    L = Layer(8, e, h, i, t)
    w2, e2 = _quant(torch.randn(e, n, i, generator=L.g, device=DEV) / i ** 0.5)
    dn = hq.MoePlan(n, i, hq.w4a4_mxfp4("bf16"), e, t, "topk_combine")
    x = _x(L.g, t, h, torch.bfloat16)
    ids, w = _routing(L.g, t, e, topk)
    y0 = L.run(x, ids, w)
    y = hq.moe_layer(L.gu, dn, x, ids, w, *L.wm[:2], *dn.repack(w2, e8m0=e2))
    torch.cuda.synchronize()
    want, tol = om.layer(om.rows(*om.quantize(x.double())), ids, w, L.w1, L.e1, w2, e2)
    assert y.shape == (t, n) and y0.shape == (t, h)
    _check(y, want, tol + om.half_step(want.abs() + tol, torch.bfloat16) + 1e-30, "to 640")


def test_layer_windows():
    """Enough slots for two column windows of the down product (240 MiB of rows)."""
    t, e, topk, h, i = 9000, 8, 8, 2048, 128
    print("[gpu case] 9000 tokens", flush=True)
    L = Layer(1, e, h, i, t)
    x = _x(L.g, t, h, torch.bfloat16)
    ids, w = _routing(L.g, t, e, topk)
    y = L.run(x, ids, w)
    torch.cuda.synchronize()
    pick = torch.tensor([0, 1, 4500, t - 1], device=DEV)
    L.check(y[pick], x[pick], ids[pick], w[pick], "rows")


@pytest.mark.parametrize("t", [3, 16, 40, 300])
def test_odd_routings(t):
    """No expert at all, one expert for all, an expert twice in a row, ids out of range, weights of any sign."""
    e, h, i = 12, 384, 256
    L = Layer(t, e, h, i, t)
    x = _x(L.g, t, h, torch.bfloat16)
    for n, ids in enumerate((torch.full((t, 4), -1), torch.full((t, 4), 7), torch.tensor([[1, 1, e, -5]]).expand(t, 4), torch.arange(4 * t).view(t, 4) % e)):
        ids = ids.to(torch.int32).to(DEV).contiguous()
        w = torch.randn(t, 4, generator=L.g, device=DEV)
        y = L.run(x, ids, w)
        torch.cuda.synchronize()
        L.check(y, x, ids, w, f"routing {n}")
        if n == 0:
            assert (y == 0).all()


@pytest.mark.parametrize("t", [2, 12, 90, 600])
def test_rows_stay_apart(t):
    """A token of NaN or of infinities spoils its own row only, and every row is the same bits whatever the others hold."""
    e, h, i = 8, 512, 256
    L = Layer(9, e, h, i, t)
    x = _x(L.g, t, h, torch.bfloat16)
    ids, w = _routing(L.g, t, e, 3)
    y = L.run(x, ids, w)
    bad = x.clone()
    bad[1, 5] = float("nan")
    if t > 4:
        bad[3, 200] = float("inf")
    z = L.run(bad, ids, w)
    torch.cuda.synchronize()
    rows = [1, 3] if t > 4 else [1]
    keep = torch.ones(t, dtype=torch.bool, device=DEV)
    keep[rows] = False
    assert z[rows].isnan().all() and torch.equal(z[keep], y[keep])


def test_nan_weights_stay_in_their_expert():
    e, h, i, t = 6, 256, 128, 50
    L = Layer(3, e, h, i, t)
    x = _x(L.g, t, h, torch.bfloat16)
    ids, w = _routing(L.g, t, e, 2)
    y = L.run(x, ids, w)
    L.e1[4, 0, 0] = 255                                # a column of expert 4 is NaN
    L.wm = (*L.gu.repack(L.w1, e8m0=L.e1), *L.wm[2:])
    z = L.run(x, ids, w)
    torch.cuda.synchronize()
    hit = (ids == 4).any(-1)
    assert z[hit].isnan().all() and torch.equal(z[~hit], y[~hit])


def test_no_tokens_and_outputs():
    L = Layer(4, 8, 512, 128, 64)
    x = torch.empty(0, 512, dtype=torch.bfloat16, device=DEV)
    y = L.run(x, torch.empty(0, 2, dtype=torch.int32, device=DEV), torch.empty(0, 2, device=DEV))
    assert y.shape == (0, 512) and y.dtype == torch.bfloat16


def test_repack_gpu_is_host_repack():
    L = Layer(5, 3, 640, 128, 8)
    for plan, w, e, got in ((L.gu, L.w1, L.e1, L.wm[:2]), (L.dn, L.w2, L.e2, L.wm[2:])):
        host = plan.repack_host(w.cpu(), e8m0=e.cpu())
        assert torch.equal(got[0].cpu(), host[0])


# ------------------------------------------------------------------ streams and graphs --
@pytest.mark.parametrize("t", [1, 6, 40, 300])
def test_graph_and_streams(t):
    L = Layer(6, 16, 512, 256, 512)
    xs = [_x(L.g, t, 512, torch.bfloat16) for _ in range(4)]
    rt = [_routing(L.g, t, 16, 3) for _ in range(4)]
    want = [L.run(x, *r) for x, r in zip(xs, rt)]
    side = [torch.cuda.Stream() for _ in range(2)]
    got = [None] * 4
    for s in side:
        s.wait_stream(torch.cuda.current_stream())
    for i in range(4):                                 # two streams at once, nothing shared
        with torch.cuda.stream(side[i % 2]):
            got[i] = L.run(xs[i], *rt[i])
    for s in side:
        torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    x, ids, w = xs[0].clone(), rt[0][0].clone(), rt[0][1].clone()
    graphs = []
    for _ in range(2):                                 # two graphs of the same plans
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = L.run(x, ids, w)
        graphs.append((graph, out))
    for i in (1, 2, 3, 0, 2):
        x.copy_(xs[i]), ids.copy_(rt[i][0]), w.copy_(rt[i][1])
        for graph, out in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out, want[i]) for _, out in graphs), f"replay {i}"


# ------------------------------------------------------------------------- refusals --
def test_refusals():
    L = Layer(13, 8, 512, 128, 64)
    x = _x(L.g, 40, 512, torch.bfloat16)
    ids, w = _routing(L.g, 40, 8, 2)
    q, s = hq.quantize_mxfp4(x)
    al = hq.moe_align(ids, 8, L.gu.block_m(40, 2))
    codes, sc = L.gu.moe_gemm(q, 40, 2, *al, *L.wm[:2], a_scale=s)

    def down(a=codes, a_scale=sc, topk_w=w, wm=L.wm[2:], **kw):
        return L.dn.moe_gemm(a, 40, 2, *al, *wm, a_scale=a_scale, topk_w=topk_w, **kw)
    down()
    for kw in (dict(topk_w=w.cpu()), dict(topk_w=w.double()), dict(topk_w=w[:20].contiguous()), dict(topk_w=None), dict(a_scale=sc.cpu()),
               dict(a_scale=None), dict(a_scale=sc.float()), dict(a_scale=sc[:, :-1].contiguous()), dict(a=codes[:-1].contiguous()), dict(a=codes.half()),
               dict(out=torch.empty(39, 512, dtype=torch.bfloat16, device=DEV)), dict(out=torch.empty(40, 512, device=DEV)),
               dict(wm=(L.wm[2][:-16].contiguous(), L.wm[3])), dict(ws=torch.empty(1 << 20, dtype=torch.uint8)),
               dict(ws=torch.empty(1 << 21, dtype=torch.uint8, device=DEV)[::2])):
        with pytest.raises(ValueError):
            down(**kw)
    with pytest.raises(hq.HQError):
        down(ws=torch.empty(64, dtype=torch.uint8, device=DEV))
    for kw in (dict(out=codes[:-1].contiguous()), dict(out_scale=sc[:, 1:].contiguous())):
        with pytest.raises(ValueError):
            L.gu.moe_gemm(q, 40, 2, *al, *L.wm[:2], a_scale=s, **kw)
    for bad in (dict(x=x[:20]), dict(x=x.float()), dict(x=x[:, :256].contiguous()), dict(ids=ids.long()), dict(w=w[:20].contiguous()), dict(w=w.half()),
                dict(x=x.cpu())):
        with pytest.raises((ValueError, hq.HQError)):
            L.run(**dict(dict(x=x, ids=ids, w=w), **bad))
    with pytest.raises(hq.HQError):                    # more tokens than the plan allows
        L.run(_x(L.g, 65, 512, torch.bfloat16), *_routing(L.g, 65, 8, 2))
    with pytest.raises(hq.HQError):
        L.gu.moe_gemm_by_slot(q, 40, 2, ids, *L.wm[:2], a_scale=s)


# --------------------------------------------------------------- the layer as it is used --
@pytest.mark.parametrize("t", [1, 11, 130])
def test_norm_route_experts(t):
    """The second half of a decoder layer: the residual's sum and its norm in MXFP4, the router's scores with bias and groups, the experts."""
    from oracle import norm as on
    from oracle import route as orr
    L = Layer(20, 32, 512, 256, t)
    g = _gen(21)
    x, r = _x(g, t, 512, torch.bfloat16), _x(g, t, 512, torch.bfloat16)
    nw = (1 + 0.1 * torch.randn(512, generator=g, device=DEV)).bfloat16()
    router, bias = torch.randn(32, 512, generator=g, device=DEV).bfloat16() / 23, 0.1 * torch.randn(32, generator=g, device=DEV)
    codes, s, h = hq.rms_norm(x, nw, residual=r, out="mxfp4")
    logits = hq.rms_norm(h, nw) @ router.t()
    ids, w = hq.route_experts(logits, 4, bias=bias, groups=4, group_topk=2, scale=2.5)
    y = L.run(codes, ids, w, x_scale=s)
    torch.cuda.synchronize()
    wh, wy = on.norm(x, nw, 1e-6, r)
    assert torch.equal(h, wh)
    wi, ww = orr.route(logits, 4, bias=bias, groups=4, group_topk=2, scale=2.5)
    assert torch.equal(ids.cpu(), wi)
    L.check(y, om.rows(om.values(codes), om.row_major(s)), ids, w, "layer")
    off = (om.rows(om.values(codes), om.row_major(s)) - wy).norm() / wy.norm()
    assert off < 0.25                                  # E2M1 keeps a step of a quarter at most
