"""fp8 with 128-block scales on the GPU against the float64 oracle
(oracle/block8.py): the block quantiser bit for bit, the dense GEMM on every
kernel it may run, routing, the grouped layer stage by stage, the two-kernel
layer, and all of them as a program uses them together (captured, on other
streams, with rows and experts that must not touch each other)."""
import pytest
import torch

import bit_quantized_gemm_repack_amd as hq
from oracle import block8 as o8

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E4 = torch.float8_e4m3fn
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def _log(msg):
    print(f"[gpu case] {msg}", flush=True)


def _gen(seed):
    g = torch.Generator(DEV)
    g.manual_seed(seed)
    return g


def _x(g, m, k, dt, spread=0.5):
    x = torch.randn(m, k, generator=g, device=DEV) * torch.exp(spread * torch.randn(m, 1, generator=g, device=DEV))
    return x.to(dt)


def _w(g, n, k, experts=None):
    lead = () if experts is None else (experts,)
    codes = (torch.randn(*lead, n, k, generator=g, device=DEV) * 96).clamp_(-448, 448).to(E4)
    s = (0.5 + torch.rand(*lead, -(-n // 128), k // 128, generator=g, device=DEV)) / (96 * k ** 0.5)
    return codes, s


def _codes(t):
    return t.view(torch.uint8)


def _vals(codes, scales):
    """uint8 codes [m, k], scales [k/128, m] -> float64 values."""
    return o8.rows(codes.view(E4), scales.t())


def _check(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float(((got.double() - want).abs() / tol).max()):.3g} of the bound"


# ------------------------------------------------------------------ quantiser --
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("m,k", [(1, 128), (3, 384), (17, 7168), (300, 1152), (2049, 256)])
def test_quantize_bits(m, k, dt):
    _log(f"quantize {m} {k} {dt}")
    g = _gen(m + k)
    x = _x(g, m, k, DT[dt])
    x[0, :128] = 0                                   # a block of zeros
    x[m // 2, -1] = torch.finfo(DT[dt]).max          # a block of one huge value
    x[m - 1, :128] = 2.0 ** -20                      # equal small values
    codes, s = hq.quantize_blocks(x)
    torch.cuda.synchronize()
    want, ws = o8.quantize(x.double())
    assert torch.equal(s.t().double(), ws)
    assert torch.equal(codes.view(E4).double(), want)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_quantize_all_magnitudes(dt):
    """Every positive finite 16-bit value as its block's largest, with its
    neighbours: the scales' whole exponent range, subnormals among them."""
    top = torch.finfo(DT[dt]).max
    v = torch.arange(1, 1 << 15, dtype=torch.int32, device=DEV).to(torch.int16).view(DT[dt])
    v = v[torch.isfinite(v) & (v <= top)]
    f = torch.linspace(-1, 1, 128, device=DEV).double()
    f[0], f[-1] = -0.96875, 1.0
    x = (v.double()[:, None] * f).to(DT[dt])
    codes, s = hq.quantize_blocks(x)
    torch.cuda.synchronize()
    want, ws = o8.quantize(x.double())
    assert torch.equal(s.t().double(), ws)
    keep = (ws > 2.0 ** -120).squeeze(1)             # below, float32 quotients of subnormal scales saturate or vanish
    assert torch.equal(codes.view(E4).double()[keep], want[keep])
    assert torch.isfinite(codes.view(E4).float()).all()


@pytest.mark.parametrize("m,k,dt", [(1, 128, "bf16"), (33, 2048, "f16"), (129, 640, "bf16")])
def test_quantize_silu(m, k, dt):
    _log(f"quantize silu {m} {k} {dt}")
    h = _x(_gen(k), m, 2 * k, DT[dt])
    codes, s = hq.quantize_blocks(h, silu_mul=True)
    torch.cuda.synchronize()
    act = o8.silu_mul(h.double())
    mid, far = o8.requant_range(act, o8.act_bound(h.double(), torch.zeros_like(h.double())))
    _check(_vals(codes, s), mid, far + 2.0 ** -24 * mid.abs() + 1e-300, "silu rows")


def test_quantize_nonfinite_blocks_stay_apart():
    x = _x(_gen(1), 4, 512, torch.bfloat16)
    clean = hq.quantize_blocks(x)
    x[1, 130], x[2, 300], x[3, 0] = float("inf"), float("nan"), -float("inf")
    codes, s = hq.quantize_blocks(x)
    torch.cuda.synchronize()
    bad = torch.zeros(4, 4, dtype=torch.bool, device=DEV)
    bad[1, 1], bad[2, 2], bad[3, 0] = True, True, True
    assert torch.equal(torch.isnan(s).t(), bad)
    same = ~bad.repeat_interleave(128, 1)
    assert torch.equal(codes[same], clean[0][same])


def test_quantize_given_outputs_and_refusals():
    x = _x(_gen(2), 5, 256, torch.bfloat16)
    codes, s = torch.empty(5, 256, dtype=E4, device=DEV), torch.empty(2, 5, device=DEV)
    r = hq.quantize_blocks(x, codes=codes, scales=s)
    assert r[0] is codes and r[1] is s
    assert torch.equal(codes.double(), o8.quantize(x.double())[0])
    for bad in (x.t(), x[:, ::2], x.float(), x[0]):
        with pytest.raises(ValueError):
            hq.quantize_blocks(bad)
    with pytest.raises(hq.HQError):
        hq.quantize_blocks(x[:, :192].contiguous())
    with pytest.raises(ValueError):
        hq.quantize_blocks(x, scales=torch.empty(5, 2, device=DEV))
    assert hq.quantize_blocks(x[:0])[0].shape == (0, 256)


# ----------------------------------------------------------------- dense GEMM --
def _gemm_case(m, n, k, dt, tuning=None, seed=0):
    g = _gen(seed + m + n + k)
    codes, s = hq.quantize_blocks(_x(g, m, k, DT[dt]))
    w, sw = _w(g, n, k)
    plan = hq.Plan(n, k, hq.w8a8_block(dt), max_m=max(m, 1), tuning=tuning)
    wm = plan.repack(_codes(w), sw)
    y = plan.gemm(codes, *wm, a_scale=s)
    torch.cuda.synchronize()
    want, tol = o8.gemm(_vals(codes, s), o8.weight(w, sw))
    _check(y, want, tol + o8.half_step(want.abs() + tol, DT[dt]), plan.describe(m))
    return plan, codes, s, wm, y


@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 33, 64, 65, 129, 300])
@pytest.mark.parametrize("n,k", [(16, 128), (144, 640), (576, 1920), (1040, 4096)])
def test_gemm(m, n, k):
    dt = "bf16" if (m + n) % 3 else "f16"
    _log(f"gemm {m} {n} {k} {dt}")
    _gemm_case(m, n, k, dt)


@pytest.mark.parametrize("tuning", [dict(kernel=1, tile_n=tn, waves=w, split_k=s) for tn, w, s in
                                    ((16, 1, 1), (16, 4, 1), (16, 8, 3), (32, 4, 1), (32, 3, 2), (32, 8, 64))] +
                         [dict(kernel=2, tile_m=bm, tile_n=bn, split_k=s, tile_group=g) for bm, bn, s, g in
                          ((16, 128, 1, 8), (32, 128, 3, 1), (64, 128, 2, 8), (128, 128, 1, 3), (128, 128, 7, 8), (128, 256, 1, 8),
                           (128, 256, 2, 64))], ids=lambda t: "-".join(str(v) for v in t.values()))
def test_gemm_every_kernel(tuning):
    for m, n, k in ((1, 272, 1152), (70, 400, 896), (261, 656, 1024)):
        _log(f"gemm {m} {n} {k} {tuning}")
        _gemm_case(m, n, k, "bf16", tuning)


@pytest.mark.parametrize("tuning", [None, dict(kernel=1, tile_n=16, waves=8, split_k=2), dict(kernel=1, tile_n=32, waves=4, split_k=1),
                                    dict(kernel=2, tile_m=16, tile_n=128, split_k=1), dict(kernel=2, tile_m=32, tile_n=128, split_k=2),
                                    dict(kernel=2, tile_m=64, tile_n=128, split_k=1), dict(kernel=2, tile_m=128, tile_n=128, split_k=3),
                                    dict(kernel=2, tile_m=128, tile_n=256, split_k=1)], ids=str)
@pytest.mark.parametrize("m,n,k", [(1, 16, 128), (7, 144, 1152), (33, 576, 640), (129, 272, 1024), (300, 1040, 2048)])
def test_gemm_exact(m, n, k, tuning):
    """Small integers and scales that are powers of two: no product or sum is
    rounded, so every bit of the result is given."""
    g = _gen(m * n)
    a = torch.randint(-4, 5, (m, k), generator=g, device=DEV).float().to(E4)
    w = torch.randint(-3, 4, (n, k), generator=g, device=DEV).float().to(E4)
    sa = torch.exp2(torch.randint(-3, 3, (k // 128, m), generator=g, device=DEV).float())
    sw = torch.exp2(torch.randint(-3, 3, (-(-n // 128), k // 128), generator=g, device=DEV).float())
    plan = hq.Plan(n, k, hq.w8a8_block(), max_m=m, tuning=tuning)
    y = plan.gemm(_codes(a), *plan.repack(_codes(w), sw), a_scale=sa)
    torch.cuda.synchronize()
    assert torch.equal(y, (_vals(_codes(a), sa) @ o8.weight(w, sw).t()).to(torch.bfloat16))


def test_gemm_large_tiles():
    _log("gemm 1031 1664 2048")
    _gemm_case(1031, 1664, 2048, "bf16")
    _log("gemm 2500 4112 512")
    _gemm_case(2500, 4112, 512, "f16")


def test_gemm_weight_near_2gib():
    """Offsets up to 2^31: the last columns and the last groups of K."""
    n, k = 65488, 32768                              # 2 GiB less 1.5 MiB
    for m in (1, 20):
        _log(f"gemm {m} {n} {k}")
        g = _gen(m)
        w = torch.randint(0, 120, (n, k), generator=g, device=DEV, dtype=torch.uint8)
        sw = (0.5 + torch.rand(-(-n // 128), k // 128, generator=g, device=DEV)) * 1e-6
        codes, s = hq.quantize_blocks(_x(g, m, k, torch.bfloat16))
        plan = hq.Plan(n, k, hq.w8a8_block(), max_m=m)
        wm = plan.repack(w, sw)
        y = plan.gemm(codes, *wm, a_scale=s)
        torch.cuda.synchronize()
        for c0 in (0, 32752, n - 16):
            want, tol = o8.gemm(_vals(codes, s), o8.rows(w[c0:c0 + 16].view(E4), sw[torch.arange(c0, c0 + 16, device=DEV) // 128]))
            _check(y[:, c0:c0 + 16], want, tol + o8.half_step(want.abs() + tol, torch.bfloat16), f"columns from {c0}")
        del w, wm, y


@pytest.mark.parametrize("m", [5, 40, 200])
def test_gemm_rows_stay_apart(m):
    """A row whose scale is NaN, and rows of NaN codes, leave the others as they are."""
    plan, codes, s, wm, y = _gemm_case(m, 272, 640, "bf16")
    c2, s2 = codes.clone(), s.clone()
    s2[1, 0] = float("nan")
    c2[m - 1] = 0x7F
    z = plan.gemm(c2, *wm, a_scale=s2)
    torch.cuda.synchronize()
    assert torch.isnan(z[0]).all() and torch.isnan(z[m - 1]).all()
    assert torch.equal(z[1:m - 1], y[1:m - 1])


def test_gemm_guard_rows_and_outputs():
    """Only the call's rows are written; the given workspace and output are used."""
    plan, codes, s, wm, y = _gemm_case(64, 576, 7168, "bf16", tuning=dict(kernel=2, tile_m=32, split_k=4))
    buf = torch.full((66, 576), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = torch.full((plan.workspace_bytes(64) + 256,), 171, dtype=torch.uint8, device=DEV)
    r = plan.gemm(codes, *wm, a_scale=s, out=buf[1:65], ws=ws[:-256])
    torch.cuda.synchronize()
    assert r.data_ptr() == buf[1:65].data_ptr() and torch.equal(buf[1:65], y)
    assert (buf[0] == 7).all() and (buf[65] == 7).all() and (ws[-256:] == 171).all()
    with pytest.raises(hq.HQError):
        plan.gemm(codes, *wm, a_scale=s, ws=ws[:256])
    for kw in (dict(a_scale=s.t().contiguous().double()), dict(a_scale=s[:1].contiguous()), dict(a_scale=None),
               dict(a_scale=s, out=buf[:64].float())):
        with pytest.raises((ValueError, AttributeError)):
            plan.gemm(codes, *wm, **kw)
    with pytest.raises(ValueError):
        plan.gemm(codes, wm[0][:1024], wm[1], a_scale=s)


def test_gemm_deterministic_and_noalloc():
    for m, n, k in ((33, 4096, 7168), (1, 576, 7168)):
        plan, codes, s, wm, y = _gemm_case(m, n, k, "bf16")
        out = torch.empty_like(y)
        hq._check(hq.lib().hq_gemm_noalloc(plan._h, m, codes.data_ptr(), s.data_ptr(), wm[0].data_ptr(), wm[1].data_ptr(),
                                           out.data_ptr(), hq._stream_ptr(torch.device(DEV))))
        torch.cuda.synchronize()
        assert torch.equal(out, y)
        for _ in range(3):
            assert torch.equal(plan.gemm(codes, *wm, a_scale=s), y)


def test_gemm_autotune():
    plan, codes, s, wm, y = _gemm_case(48, 576, 2048, "bf16")
    r = plan.autotune(codes, *wm, a_scale=s, reps=2, flush_bytes=0)
    assert r["candidates"] > 5 and r["best_us"] <= r["current_us"] * 1.0001
    z = plan.gemm(codes, *wm, a_scale=s)
    torch.cuda.synchronize()
    want, tol = o8.gemm(_vals(codes, s), _deq_from(plan, wm))
    _check(z, want, tol + o8.half_step(want.abs() + tol, torch.bfloat16), plan.describe(48))


def _deq_from(plan, wm):
    """float64 weights from the device layout (fragments of 16 x 128)."""
    n, k = plan.n, plan.k
    c = wm[0].view(n // 16, k // 128, 2, 4, 16, 16).permute(0, 4, 1, 2, 3, 5).reshape(n, k)
    return o8.weight(c.view(E4), wm[1].view(torch.float32)[:-(-n // 128) * (k // 128)].view(-1, k // 128))


def test_repack_gpu_is_host_repack():
    for shape in ((144, 384), (3, 512, 256)):
        n, k = shape[-2:]
        e = shape[0] if len(shape) == 3 else 1
        codes = torch.randint(0, 256, shape, dtype=torch.uint8)
        s = torch.rand(*shape[:-2], -(-n // 128), k // 128)
        kind = dict(kind="grouped", epi="silu_mul_qfp8", num_experts=e) if e > 1 else {}
        plan = hq.Plan(n, k, hq.w8a8_block(), max_m=4, **kind)
        hw, hm = plan.repack_host(codes, s)
        w, m = plan.repack(codes.to(DEV), s.to(DEV))
        torch.cuda.synchronize()
        assert torch.equal(w.cpu(), hw) and torch.equal(m.cpu()[:s.numel() * 4], hm[:s.numel() * 4])


@pytest.mark.parametrize("m", [1, 3, 40, 200])
def test_mlp_as_used(m):
    """x -> quantise -> gate_up -> SiLU * up, quantise -> down, each against the oracle on its own input."""
    h, i = 512, 384
    g = _gen(m)
    x = _x(g, m, h, torch.bfloat16)
    w1, s1 = _w(g, 2 * i, h)
    w2, s2 = _w(g, h, i)
    up, down = (hq.Plan(a, b, hq.w8a8_block(), max_m=256) for a, b in ((2 * i, h), (h, i)))
    u, d = up.repack(_codes(w1), s1), down.repack(_codes(w2), s2)
    t = up.linear(x, *u)
    q = hq.quantize_blocks(t, silu_mul=True)
    y = down.gemm(q[0], *d, a_scale=q[1])
    torch.cuda.synchronize()
    want, tol = o8.gemm(o8.rows(*o8.quantize(x.double())), o8.weight(w1, s1))
    _check(t, want, tol + o8.half_step(want.abs() + tol, torch.bfloat16), "gate_up")
    mid, far = o8.requant_range(o8.silu_mul(t.double()), o8.act_bound(t.double(), torch.zeros_like(t.double())))
    _check(_vals(*q), mid, far + 2.0 ** -24 * mid.abs() + 1e-300, "rows")
    want, tol = o8.gemm(_vals(*q), o8.weight(w2, s2))
    _check(y, want, tol + o8.half_step(want.abs() + tol, torch.bfloat16), "down")


# -------------------------------------------------------------------- routing --
def _logits(g, t, e, dt, masked=True):
    x = torch.randn(t, e, generator=g, device=DEV)
    if masked:
        x[torch.rand(t, e, generator=g, device=DEV) < 0.1] = -float("inf")
    return x.to(dt)


@pytest.mark.parametrize("e,topk", [(1, 1), (4, 4), (60, 6), (64, 8), (65, 8), (128, 1), (160, 6), (256, 8), (257, 3), (512, 64), (513, 8),
                                    (1024, 8)])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16])
def test_route(e, topk, dt):
    for t, renorm in ((1, True), (7, False), (130, True)):
        _log(f"route {t} {e} {topk} {dt} {renorm}")
        x = _logits(_gen(e + t), t, e, dt)
        if t == 7:
            x[0] = -float("inf")                     # no expert
            x[1] = -float("inf")
            x[1, e - 1] = -3.0                       # one expert
            x[2] = 0.25                              # all equal
            x[3, : e // 2] = float("nan")
            x[4] = -x[4].abs()
            x[4, 0] = -0.0
            x[4, e - 1] = 0.0
        ids, w = hq.route_topk(x, topk, renormalize=renorm)
        torch.cuda.synchronize()
        wi, ww = o8.route(x.cpu(), topk, renorm)
        assert torch.equal(ids.cpu().long(), wi)
        # exp of a difference rounded by |x - max| 2^-24 and exp's own 2 ulp, at most 1024 terms summed in a tree of 16 + 6
        # steps, one quotient
        span = torch.where(torch.isfinite(x.double()), x.double(), torch.zeros_like(x.double())).abs().amax().item() * 2
        _check(w.cpu(), ww, ww * (span + 40) * 2.0 ** -23 + 1e-38, "weights")


def test_route_refusals():
    x = _logits(_gen(0), 4, 16, torch.float32)
    for bad in (x.double(), x[:, ::2], x[0]):
        with pytest.raises(ValueError):
            hq.route_topk(bad, 2)
    for k in (0, 17):
        with pytest.raises(hq.HQError):
            hq.route_topk(x, k)
    assert hq.route_topk(x[:0], 2)[0].shape == (0, 2)


# ------------------------------------------------------------- experts' layers --
class Layer:
    def __init__(self, seed, e, h, i, max_t, dt="bf16", tuning=None):
        g = self.g = _gen(seed)
        self.e, self.h, self.i, self.dt = e, h, i, DT[dt]
        self.w1, self.s1 = _w(g, 2 * i, h, e)
        self.w2, self.s2 = _w(g, h, i, e)
        q = hq.w8a8_block(dt)
        self.gu = hq.MoePlan(2 * i, h, q, e, max_t, "silu_mul_qfp8", tuning=tuning)
        self.dn = hq.MoePlan(h, i, q, e, max_t, "topk_combine", tuning=tuning)
        self.wm = (*self.gu.repack(_codes(self.w1), self.s1), *self.dn.repack(_codes(self.w2), self.s2))

    def run(self, x, ids, w, **kw):
        return hq.moe_layer(self.gu, self.dn, x, ids, w, *self.wm, **kw)

    def routed(self, x, logits, topk, **kw):
        return hq.moe_layer_routed(self.gu, self.dn, x, logits, topk, *self.wm, **kw)

    def check(self, y, x, ids, w, what, row_err=0.0):
        want, tol = o8.layer(x.double(), ids.long(), w, self.w1, self.s1, self.w2, self.s2, row_err)
        _check(y, want, tol + o8.half_step(want.abs() + tol, self.dt) + 1e-30, what)


ROW_ERR = 2.0 ** -14  # a stored row's integers: one unit of at most 2^-14 of the 64 columns' largest


def _routing(g, t, e, topk, logits=None):
    x = torch.randn(t, e, generator=g, device=DEV) if logits is None else logits
    ids, w = hq.route_topk(x, topk)
    return ids, w


@pytest.mark.parametrize("t,e,topk,h,i", [(1, 8, 2, 512, 128), (5, 8, 8, 640, 256), (40, 16, 4, 768, 384), (300, 12, 3, 512, 1024),
                                          (700, 8, 6, 512, 256), (65, 3, 1, 256, 2048)])
@pytest.mark.parametrize("bm", [None, 16, 64, 128])
def test_grouped_stages(t, e, topk, h, i, bm):
    _log(f"grouped {t} {e} {topk} {h} {i} {bm}")
    L = Layer(t + e, e, h, i, t, tuning=None if bm is None else dict(tile_m=bm))
    x = _x(L.g, t, h, torch.bfloat16)
    ids, w = _routing(L.g, t, e, topk)
    ids = ids.clone()
    ids.view(-1)[:: 11] = -1                          # slots without an expert
    if t > 4:
        ids[3] = e + 5
    b = L.gu.block_m(t, topk)
    al = hq.moe_align(ids, e, b)
    xq, xs = hq.quantize_blocks(x)
    codes, sc = L.gu.moe_gemm(xq, t, topk, *al, *L.wm[:2], a_scale=xs)
    y = L.dn.moe_gemm(codes, t, topk, *al, *L.wm[2:], a_scale=sc, topk_w=w)
    torch.cuda.synchronize()
    used = int(al[2])
    sid, bex = al[0][:used].long(), al[1].long()
    live = (sid < t * topk) & (bex[torch.arange(used, device=DEV) // b] >= 0)
    got, want = _vals(codes, sc), torch.zeros(t, h, dtype=torch.float64, device=DEV)
    tolr = torch.zeros_like(want)
    for ex in range(e):
        pos = torch.nonzero(live & (bex[torch.arange(used, device=DEV) // b] == ex)).squeeze(1)
        if not len(pos):
            continue
        tok = sid[pos] // topk
        hh, th = o8.gemm(_vals(xq, xs)[tok], o8.weight(L.w1[ex], L.s1[ex]))
        mid, far = o8.requant_range(o8.silu_mul(hh), o8.act_bound(hh, th))
        _check(got[pos], mid, far + 2.0 ** -24 * mid.abs() + 1e-300, f"gate_up of expert {ex}")
        o, to = o8.gemm(got[pos], o8.weight(L.w2[ex], L.s2[ex]))
        p = w.view(-1)[sid[pos]].double().unsqueeze(1)
        strip = o.unflatten(1, (-1, 64)).abs().amax(2).repeat_interleave(64, 1)
        want.index_add_(0, tok, o * p)
        tolr.index_add_(0, tok, (to + ROW_ERR * strip + 2.0 ** -20 * o.abs()) * p.abs())
    _check(y, want, tolr + o8.half_step(want.abs() + tolr, torch.bfloat16) + 1e-30, "down")
    if t > 4:
        assert (y[3] == 0).all()


@pytest.mark.parametrize("bm", [16, 64, 128])
@pytest.mark.parametrize("t", [1, 90, 700])
def test_grouped_fp16(t, bm):
    """fp16 layers on every block, alone and shared by an expert's rows."""
    L = Layer(40 + t, 5, 640, 384, t, "f16", tuning=dict(tile_m=bm))
    x = _x(L.g, t, 640, torch.float16)
    ids, w = _routing(L.g, t, 5, 2)
    q, s = hq.quantize_blocks(x)
    y = L.run(q, ids, w, x_scale=s)
    torch.cuda.synchronize()
    L.check(y, x, ids, w, f"block {bm}", ROW_ERR)


def test_grouped_windows(monkeypatch):
    """Enough slots for two column windows of the down GEMM (240 MiB of rows)."""
    t, e, topk, h, i = 9000, 8, 8, 2048, 128
    L = Layer(1, e, h, i, t)
    x = _x(L.g, t, h, torch.bfloat16)
    ids, w = _routing(L.g, t, e, topk)
    _log("grouped 9000 tokens")
    y = L.run(x, ids, w)
    torch.cuda.synchronize()
    pick = torch.tensor([0, 1, 4500, t - 1], device=DEV)
    L.check(y[pick], x[pick], ids[pick], w[pick], "rows", ROW_ERR)


@pytest.mark.parametrize("t", [1, 2, 3, 8, 9, 16])
@pytest.mark.parametrize("e,topk,h,i,dt", [(8, 2, 512, 128, "bf16"), (60, 6, 640, 256, "f16"), (256, 8, 1024, 384, "bf16"),
                                           (300, 3, 896, 512, "bf16"), (16, 16, 256, 1024, "f16")])
def test_few(t, e, topk, h, i, dt):
    L = Layer(t + e, e, h, i, 64, dt)
    x = _x(L.g, t, h, DT[dt])
    for lt, renorm in ((torch.float32, True), (torch.bfloat16, False)):
        _log(f"few {t} {e} {topk} {h} {i} {dt} {lt}")
        logits = _logits(L.g, t, e, lt)
        y, ids, w = L.routed(x, logits, topk, renormalize=renorm)
        ri, rw = hq.route_topk(logits, topk, renormalize=renorm)
        z = L.run(x, ids, w)
        torch.cuda.synchronize()
        assert torch.equal(ids, ri)
        _check(w, rw.double(), rw.double().abs() * 2.0 ** -18 + 1e-38, "weights")
        L.check(y, x, ids, w, "layer")
        assert torch.equal(y, z)                      # the same from given ids


@pytest.mark.parametrize("t", [17, 33, 64])
def test_few_more_tokens(monkeypatch, t):
    monkeypatch.setattr(hq, "MOE_FEW_MAX_TOKENS", 64)
    L = Layer(t, 24, 512, 256, 64)
    x = _x(L.g, t, 512, torch.bfloat16)
    _log(f"few {t}")
    y, ids, w = L.routed(x, _logits(L.g, t, 24, torch.float32), 4)
    torch.cuda.synchronize()
    L.check(y, x, ids, w, "layer")


@pytest.mark.parametrize("t", [2, 9, 16])
def test_few_crowded_and_odd_ids(t):
    """Every token at one expert (rows beyond what a workgroup keeps), an expert
    twice in a token's row, ids outside the experts, an idle token."""
    L = Layer(t, 12, 512, 256, 64)
    x = _x(L.g, t, 512, torch.bfloat16)
    ids = torch.randint(0, 12, (t, 4), generator=L.g, device=DEV, dtype=torch.int32)
    ids[:, 0] = 7
    ids[0] = torch.tensor([7, 7, 7, 7])
    ids[1] = torch.tensor([-1, 12, 1 << 30, -(1 << 31)])
    w = torch.rand(t, 4, generator=L.g, device=DEV)
    w[0, 1] = -0.5
    _log(f"few crowded {t}")
    y = L.run(x, ids, w)
    torch.cuda.synchronize()
    L.check(y, x, ids, w, "layer")
    assert (y[1] == 0).all()


def test_few_long_rows():
    """H beyond the blocks a workgroup loads ahead, and an intermediate that is
    taken in several pieces."""
    L = Layer(3, 6, 16384, 512, 64)
    for t, topk in ((1, 2), (5, 4), (16, 6)):
        _log(f"few long {t} {topk}")
        x = _x(L.g, t, 16384, torch.bfloat16)
        y, ids, w = L.routed(x, _logits(L.g, t, 6, torch.float32, masked=False), topk)
        torch.cuda.synchronize()
        L.check(y, x, ids, w, "layer")


@pytest.mark.parametrize("t", [2, 12])
def test_few_rows_stay_apart(t):
    L = Layer(4, 8, 512, 128, 64)
    x = _x(L.g, t, 512, torch.bfloat16)
    logits = _logits(L.g, t, 8, torch.float32, masked=False)
    y, ids, w = L.routed(x, logits, 4)
    bad = x.clone()
    bad[1, 5] = float("nan")
    z, _, _ = L.routed(bad, logits, 4)
    torch.cuda.synchronize()
    assert torch.isnan(z[1]).all()
    keep = [i for i in range(t) if i != 1]
    assert torch.equal(z[keep], y[keep])
    logits[0] = -float("inf")                         # a token without experts
    y, ids, w = L.routed(x, logits, 4)
    torch.cuda.synchronize()
    assert (y[0] == 0).all() and (ids[0] == -1).all() and (w[0] == 0).all()


def test_layers_beyond_4gib():
    """Experts whose weights lie past 2^32 bytes."""
    e, h, i = 136, 8192, 2048
    g = _gen(9)
    q = hq.w8a8_block()
    gu, dn = hq.MoePlan(2 * i, h, q, e, 64, "silu_mul_qfp8"), hq.MoePlan(h, i, q, e, 64, "topk_combine")
    w1 = torch.randint(0, 110, (e, 2 * i, h), generator=g, device=DEV, dtype=torch.uint8)
    w2 = torch.randint(0, 110, (e, h, i), generator=g, device=DEV, dtype=torch.uint8)
    w1[:, ::2] += 128                                 # half the rows negative
    s1 = torch.full((e, 2 * i // 128, h // 128), 1e-6, device=DEV)
    s2 = torch.full((e, h // 128, i // 128), 1e-4, device=DEV)
    wm = (*gu.repack(w1, s1), *dn.repack(w2, s2))
    for t in (1, 20):
        _log(f"beyond 4 GiB: {t}")
        x = _x(g, t, h, torch.bfloat16)
        ids = torch.tensor([[e - 1, 0]], dtype=torch.int32, device=DEV).repeat(t, 1)
        w = torch.full((t, 2), 0.5, device=DEV)
        y = hq.moe_layer(gu, dn, x, ids, w, *wm)
        torch.cuda.synchronize()
        want, tol = o8.layer(x.double(), ids.long(), w, w1.view(E4), s1, w2.view(E4), s2, ROW_ERR)
        _check(y, want, tol + o8.half_step(want.abs() + tol, torch.bfloat16), "layer")


def test_layer_dispatch_and_refusals():
    L = Layer(5, 8, 512, 256, 64)
    x = _x(L.g, 20, 512, torch.bfloat16)
    ids, w = _routing(L.g, 20, 8, 2)
    y = L.run(x, ids, w)                              # aligned path, x quantised inside
    xq, xs = hq.quantize_blocks(x)
    assert torch.equal(y, L.run(xq, ids, w, x_scale=xs))
    torch.cuda.synchronize()
    L.check(y, x, ids, w, "aligned", ROW_ERR)
    z, ri, rw = L.routed(x, torch.randn(20, 8, device=DEV), 2)
    torch.cuda.synchronize()
    L.check(z, x, ri, rw, "routed, aligned", ROW_ERR)
    for t, b in ((16, 4), (2, 1)):
        s = L.run(x[:t], ids[:t], w[:t])
        torch.cuda.synchronize()
        L.check(s, x[:t], ids[:t], w[:t], "few")
    with pytest.raises(ValueError):
        L.run(x, ids, w, by_slot=True)
    with pytest.raises(ValueError):
        L.run(x[:2].float(), ids[:2], w[:2])
    with pytest.raises(ValueError):
        L.run(x[:2], ids[:2].long(), w[:2])
    with pytest.raises(ValueError):
        L.routed(x[:2], torch.randn(3, 8, device=DEV), 2)
    with pytest.raises(hq.HQError):
        L.routed(x[:2], torch.randn(2, 8, device=DEV), 9)


@pytest.mark.parametrize("t", [1, 5, 13, 40, 500, 1500])
def test_layer_keeps_fp16(t):
    """The intermediate is quantised to 4-bit significands, so that sums a little
    off turn into other codes.  Where no code differs, fp16 outputs are off by
    their own rounding, eps / 2 of each value at most: the root mean square over
    all of them stays below that."""
    L = Layer(20 + t, 16, 2048, 512, t, "f16")
    x = _x(L.g, t, 2048, torch.float16)
    ids, w = _routing(L.g, t, 16, 2)
    y = L.run(x, ids, w).double()
    torch.cuda.synchronize()
    want = o8.layer(x.double(), ids.long(), w, L.w1, L.s1, L.w2, L.s2)[0]
    assert ((y - want).pow(2).mean() / want.pow(2).mean()).sqrt() < torch.finfo(torch.float16).eps / 2


def test_layer_odd_calls():
    """No tokens, slices of a batch that start anywhere, one token with an expert
    several times and ids outside the experts, codes where few tokens would run."""
    L = Layer(12, 9, 512, 128, 64)
    x = _x(L.g, 24, 512, torch.bfloat16)
    logits = _logits(L.g, 24, 9, torch.bfloat16, masked=False)
    ids, w = hq.route_topk(logits, 3)
    y, ri, rw = L.routed(x[:0], logits[:0], 3)
    assert y.shape == (0, 512) and ri.shape == rw.shape == (0, 3)
    assert L.run(x[:0], ids[:0], w[:0]).shape == (0, 512)
    for a, b in ((1, 2), (3, 8), (5, 24)):            # 18-byte rows of logits, 12-byte rows of ids
        y, ri, rw = L.routed(x[a:b], logits[a:b], 3)
        z = L.run(x[a:b], ids[a:b], w[a:b])
        torch.cuda.synchronize()
        assert torch.equal(ri, ids[a:b]) and torch.equal(hq.route_topk(logits[a:b], 3)[0], ids[a:b])
        L.check(y, x[a:b], ri, rw, "routed slice", ROW_ERR)
        L.check(z, x[a:b], ids[a:b], w[a:b], "slice", ROW_ERR)
    one = torch.tensor([[4, 4, -1, 9, 4, 0]], dtype=torch.int32, device=DEV)
    ow = torch.rand(1, 6, generator=L.g, device=DEV)
    y = L.run(x[:1], one, ow)
    torch.cuda.synchronize()
    L.check(y, x[:1], one, ow, "one token")
    none = torch.full((1, 6), -1, dtype=torch.int32, device=DEV)
    assert (L.run(x[:1], none, ow) == 0).all()
    q, s = hq.quantize_blocks(x[:4].contiguous())
    y = L.run(q, ids[:4], w[:4], x_scale=s)
    torch.cuda.synchronize()
    L.check(y, x[:4], ids[:4], w[:4], "codes of few tokens", ROW_ERR)


def test_grouped_refuses_wrong_tensors():
    L = Layer(13, 8, 512, 128, 64)
    x = _x(L.g, 40, 512, torch.bfloat16)
    ids, w = _routing(L.g, 40, 8, 2)
    q, s = hq.quantize_blocks(x)
    al = hq.moe_align(ids, 8, L.gu.block_m(40, 2))
    codes, sc = L.gu.moe_gemm(q, 40, 2, *al, *L.wm[:2], a_scale=s)
    down = lambda a_scale=sc, topk_w=w, **kw: L.dn.moe_gemm(codes, 40, 2, *al, *L.wm[2:], a_scale=a_scale, topk_w=topk_w, **kw)
    down()
    for kw in (dict(topk_w=w.cpu()), dict(topk_w=w.double()), dict(topk_w=w[:20].contiguous()), dict(topk_w=None),
               dict(a_scale=sc.cpu()), dict(out=torch.empty(39, 512, dtype=torch.bfloat16, device=DEV)),
               dict(out=torch.empty(40, 512, device=DEV))):
        with pytest.raises(ValueError):
            down(**kw)
    with pytest.raises(ValueError):
        L.gu.moe_gemm(q, 40, 2, *al, *L.wm[:2], a_scale=s, out=codes[:-1].contiguous())
    with pytest.raises(ValueError):
        L.gu.moe_gemm(q, 40, 2, *al, *L.wm[:2], a_scale=s, out_scale=sc[:0].contiguous())


def test_quantize_beyond_32_bits():
    """More than 2^31 values: the last rows are right."""
    m, k = 300001, 7168
    _log(f"quantize {m} {k}")
    x = torch.zeros(m, k, dtype=torch.bfloat16, device=DEV)
    for r in (0, m // 2, m - 1):
        x[r] = _x(_gen(r), 1, k, torch.bfloat16)[0]
    codes, s = hq.quantize_blocks(x)
    torch.cuda.synchronize()
    for r in (0, m // 2, m - 1):
        want, ws = o8.quantize(x[r:r + 1].double())
        assert torch.equal(codes[r:r + 1].view(E4).double(), want) and torch.equal(s[:, r:r + 1].t().double(), ws)
    assert (s[:, 1:m // 2] == 1).all()


def test_native_calls_are_the_same(monkeypatch):
    """The binding's native short calls against the same calls through ctypes, on
    another stream too; what they do not take goes through ctypes."""
    x = _x(_gen(30), 9, 1024, torch.bfloat16)
    h = _x(_gen(31), 9, 2048, torch.float16)
    lg = _logits(_gen(32), 9, 40, torch.float32)
    w, sw = _w(_gen(33), 272, 1024)
    plan = hq.Plan(272, 1024, hq.w8a8_block(), max_m=16, tuning=dict(kernel=1, split_k=2))
    wm = plan.repack(_codes(w), sw)
    a, s = hq.quantize_blocks(x)

    def calls():
        return [*hq.quantize_blocks(x), *hq.quantize_blocks(h, silu_mul=True), *hq.route_topk(lg, 4), *hq.route_topk(lg, 2, False),
                plan.gemm(a, *wm, a_scale=s), *hq.quantize_blocks(x[:0]), *hq.route_topk(lg[:0], 3)]
    assert hq._calls is not None
    native = calls()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        other = calls()
    torch.cuda.synchronize()
    assert hq._calls.quantize_blocks(x.t(), False) is None and hq._calls.route_topk(lg, 41, True) is None
    assert hq._calls.gemm_block(plan._h.value, 272, 1024, True, a, s.double(), *wm) is None
    assert hq._calls.gemm_block(plan._h.value, 272, 1024, True, a, None, *wm) is None
    monkeypatch.setattr(hq, "_calls", None)
    plain = calls()
    torch.cuda.synchronize()
    for p, q, r in zip(native, other, plain):
        assert p.dtype == r.dtype and p.shape == r.shape and torch.equal(p, r) and torch.equal(q, r)


# ------------------------------------------------------------ streams, graphs --
def test_graph_of_everything():
    """Quantise, split-K GEMM, routing and both layers in one graph: every replay
    on new inputs equals the eager calls, with eager work between."""
    L = Layer(6, 16, 512, 256, 64)
    g = _gen(8)
    w, sw = _w(g, 576, 7168)
    plan = hq.Plan(576, 7168, hq.w8a8_block(), max_m=64, tuning=dict(kernel=2, tile_m=64, split_k=4))
    wm = plan.repack(_codes(w), sw)
    big, x, many = _x(g, 40, 7168, torch.bfloat16), _x(g, 4, 512, torch.bfloat16), _x(g, 48, 512, torch.bfloat16)
    lg, lm = torch.randn(4, 16, device=DEV), torch.randn(48, 16, device=DEV)

    def program():
        return [plan.linear(big, *wm), *L.routed(x, lg, 3), *L.routed(many, lm, 2)]
    program()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = program()
    for r in range(4):
        for v in (big, x, many, lg, lm):
            v.copy_(torch.randn_like(v))
        torch.randn(1 << 20, device=DEV).mul_(2)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        want = program()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), f"replay {r}, output {i}"


def test_two_graphs_and_two_streams_at_once():
    """Calls of one plan that overlap in time share nothing."""
    L = Layer(7, 32, 1024, 256, 64)
    plan = hq.Plan(1024, 4096, hq.w8a8_block(), max_m=64, tuning=dict(kernel=1, split_k=4))
    w, sw = _w(_gen(3), 1024, 4096)
    wm = plan.repack(_codes(w), sw)
    ins, graphs, outs, want = [], [], [], []
    for s in range(2):
        g = _gen(20 + s)
        ins.append((_x(g, 12, 1024, torch.bfloat16), torch.randn(12, 32, generator=g, device=DEV), _x(g, 30, 4096, torch.bfloat16)))
        x, lg, b = ins[s]
        f = lambda: [L.routed(x, lg, 4)[0], plan.linear(b, *wm)]
        want.append([v.clone() for v in f()])
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[s]):
            outs.append(f())
    st = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for s in range(2):
            with torch.cuda.stream(st[s]):
                graphs[s].replay()
    torch.cuda.synchronize()
    for s in range(2):
        for a, b in zip(outs[s], want[s]):
            assert torch.equal(a, b)
    eager = [[], []]
    for _ in range(20):
        for s in range(2):
            with torch.cuda.stream(st[s]):
                x, lg, b = ins[s]
                eager[s].append((L.routed(x, lg, 4)[0], plan.linear(b, *wm)))
    torch.cuda.synchronize()
    for s in range(2):
        for y, z in eager[s]:
            assert torch.equal(y, want[s][0]) and torch.equal(z, want[s][1])


def test_timing_events():
    """hq_time_next_launch covers the calls from their first kernel to their last."""
    L = Layer(10, 8, 512, 256, 64)
    x = _x(L.g, 2, 512, torch.bfloat16)
    ids, w = _routing(L.g, 2, 8, 2)
    L.run(x, ids, w)
    xq, xs = hq.quantize_blocks(x)
    for call in (lambda: hq.quantize_blocks(x), lambda: hq.route_topk(torch.randn(2, 8, device=DEV), 2), lambda: L.run(x, ids, w)):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record(), b.record()
        torch.cuda.synchronize()
        hq._check(hq.lib().hq_time_next_launch(a.cuda_event, b.cuda_event))
        call()
        torch.cuda.synchronize()
        assert 0 < a.elapsed_time(b) < 10
