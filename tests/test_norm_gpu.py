"""Root-mean-square norm on the GPU against the float64 oracle (oracle/norm.py): every
output kind, both types, weights of both types, with and without the residual, over
row lengths that choose every kernel shape; slices, sums in place, rows that are not
finite, streams and graphs, and refusals."""
import pytest
import torch

import bit_quantized_gemm_repack_amd as hq
from oracle import norm as on

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
E4 = torch.float8_e4m3fn
KINDS = [None, "fp8", "int8", "fp8_block", "mxfp4"]


def _gen(seed):
    g = torch.Generator(DEV)
    g.manual_seed(seed)
    return g


def _x(g, m, k, dt):
    x = torch.randn(m, k, generator=g, device=DEV) * torch.exp(torch.randn(m, 1, generator=g, device=DEV))
    return (x * (1 + 20 * (torch.rand(1, k, generator=g, device=DEV) < 0.01))).to(dt)


def _check(got, x, w, eps, kind, residual=None, what=""):
    torch.cuda.synchronize()
    got = list(got) if isinstance(got, tuple) else [got]
    h, y = on.norm(x, w, eps, residual)
    if residual is not None:
        assert torch.equal(got.pop(), h), f"{what}: h"
    if kind is None:
        half = torch.finfo(x.dtype).eps / 2
        tol = y.abs() * (on.FACTOR + half * (1 + on.FACTOR)) + (2.0 ** -25 if x.dtype == torch.float16 else 0.0)
        off = ((got[0].double() - y).abs() / tol.clamp_min(1e-300)).masked_fill(y == got[0].double(), 0)
        assert got[0].dtype == x.dtype and off.max() <= 1, f"{what}: y off by {float(off.max()):.3g} of the bound"
        return
    codes, s = got
    if kind == "mxfp4":
        e = on.rows_of(s).double()
        lo, hi = on.e8m0_may_be(y)
        assert ((e >= lo) & (e <= hi)).all(), f"{what}: powers of two"
        off = on.off_scaled(on.values4(codes), torch.exp2(e - 127), y, 32, on.TOP4, on.half_step4)
    elif kind == "int8":
        assert codes.dtype == torch.int8 and (codes != -128).all()
        assert (on.off_scale(s[:, None], y, y.shape[1], 127.0) <= 1).all(), f"{what}: scales"
        off = on.off_scaled(codes, s[:, None], y, y.shape[1], 127.0, lambda v: torch.full_like(v, 0.5))
    else:
        block = 128 if kind == "fp8_block" else y.shape[1]
        sc = s.t() if kind == "fp8_block" else s[:, None]
        assert (on.off_scale(sc, y, block, on.TOP8) <= 1).all(), f"{what}: scales"
        off = on.off_scaled(codes.view(E4), sc, y, block, on.TOP8, on.half_step8)
    assert off.max() <= 1, f"{what}: codes off by {float(off.max()):.3g} of the bound"


SIZES = [(1, 128), (1, 7168), (3, 384), (17, 7168), (70, 256), (33, 512), (300, 1152), (1025, 128), (700, 4096), (5, 16384), (2, 65536),
         (3, 20480), (600, 640), (515, 2048)]
ODD = [(1, 8), (9, 24), (130, 72), (2, 1000), (40, 2056), (257, 4104), (3, 40008)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_norm(kind, dt):
    for n, (m, k) in enumerate(SIZES + ([] if kind in ("fp8_block", "mxfp4") else ODD)):
        print(f"[gpu case] norm {kind} {dt} {m} {k}", flush=True)
        g = _gen(m + k + n)
        x = _x(g, m, k, DT[dt])
        w = (1 + 0.3 * torch.randn(k, generator=g, device=DEV)).to(torch.float32 if n % 3 == 0 else DT[dt])
        r = _x(g, m, k, DT[dt]) if n % 2 == 0 else None
        if m > 2:
            x[1] = 0  # a row of zeros (but for the residual)
        _check(hq.rms_norm(x, w, 1e-5, r, kind), x, w, 1e-5, kind, r, f"{m} x {k}")


@pytest.mark.parametrize("kind", KINDS)
def test_slices_and_sums_in_place(kind):
    g = _gen(5)
    wide = _x(g, 65, 1088, torch.bfloat16)
    x, r = wide[:, :512], wide[:, 576:]
    w = 1 + 0.1 * torch.randn(512, generator=g, device=DEV)
    _check(hq.rms_norm(x, w, out=kind), x, w, 1e-6, kind)
    before, x0, r0 = wide.clone(), x.clone(), r.clone()
    got = hq.rms_norm(x, w, residual=r, out=kind, residual_out=r)   # the residual stream in place
    assert got[-1] is r
    _check(got, x0, w, 1e-6, kind, r0)
    assert torch.equal(wide[:, :576], before[:, :576])
    wide.copy_(before)
    got = hq.rms_norm(x, w, residual=r, out=kind, residual_out=x)
    _check(got, x0, w, 1e-6, kind, r0)
    assert torch.equal(wide[:, 512:], before[:, 512:])
    one = before[3:4, :512]
    rows = one.expand(65, 512)                                      # one row for all
    _check(hq.rms_norm(rows, w, residual=r0, out=kind), rows, w, 1e-6, kind, r0)
    skip = before[::2, :512]                                        # every second row
    _check(hq.rms_norm(skip, w, out=kind), skip, w, 1e-6, kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("k", [128, 640, 7168, 16384])
def test_rows_that_are_not_finite(kind, k):
    """They stay in their rows; a scale says NaN where a value of its row or block is not finite."""
    g = _gen(k)
    x = _x(g, 21, k, torch.bfloat16)
    w = torch.ones(k, device=DEV)
    want = hq.rms_norm(x, w, out=kind)
    bad = x.clone()
    bad[4, 5], bad[9, k - 1], bad[20, 64] = float("nan"), float("inf"), -float("inf")
    got = hq.rms_norm(bad, w, out=kind)
    torch.cuda.synchronize()
    rows = [4, 9, 20]
    others = [i for i in range(21) if i not in rows]
    if kind is None:
        assert torch.equal(got[others], want[others]) and got[4].isnan().all()
        assert got[9, k - 1].isnan() and (got[9, :k - 1] == 0).all() and got[20, 64].isnan() and got[20, 0] == 0
        return
    assert torch.equal(got[0][others], want[0][others])
    if kind == "mxfp4":
        s, ws = on.rows_of(got[1]), on.rows_of(want[1])
        assert torch.equal(s[others], ws[others]) and (s[4] == 255).all()
        assert s[9, -1] == 255 and (s[9, :-1] == 127).all() and s[20, 2] == 255 and s[20, 0] == 127
    else:
        s, ws = (t.t() if kind == "fp8_block" else t[:, None] for t in (got[1], want[1]))
        assert torch.equal(s[others], ws[others]) and s[4].isnan().all() and s[9, -1].isnan() and s[20, 0].isnan()


def test_zeros_and_eps():
    x = torch.zeros(3, 256, dtype=torch.float16, device=DEV)
    w = torch.ones(256, dtype=torch.float16, device=DEV)
    for kind in KINDS:
        got = hq.rms_norm(x, w, out=kind)
        y = got if kind is None else got[0]
        assert (y == 0).all()
        if kind is not None:
            assert (got[1].float() == (127 if kind == "mxfp4" else 1)).all()
    x += 6e-8                                          # the least subnormal: eps decides
    assert torch.allclose(hq.rms_norm(x, w, eps=1e-12).float(), x.float() / 1e-6, rtol=1e-2)
    assert torch.allclose(hq.rms_norm(x, w, eps=0.0).float(), torch.ones_like(x).float(), rtol=1e-3)


def test_no_rows():
    x = torch.empty(0, 256, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(256, dtype=torch.bfloat16, device=DEV)
    codes, s, h = hq.rms_norm(x, w, residual=x, out="fp8_block")
    assert codes.shape == (0, 256) and s.shape == (2, 0) and h.shape == (0, 256)


def test_streams_and_graphs():
    g = _gen(8)
    w = (1 + 0.1 * torch.randn(1024, generator=g, device=DEV)).bfloat16()
    xs = [_x(g, 37, 1024, torch.bfloat16) for _ in range(4)]
    want = [hq.rms_norm(x, w, residual=xs[0], out="mxfp4") for x in xs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [hq.rms_norm(x, w, residual=xs[0], out="mxfp4") for x in xs]
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, want):
        assert all(torch.equal(u, v) for u, v in zip(a, b))
    x = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = hq.rms_norm(x, w, residual=xs[0], out="mxfp4")
    for i in (1, 2, 3, 0, 2):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(out, want[i])), f"replay {i}"


def test_refusals():
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(256, dtype=torch.bfloat16, device=DEV)
    for bad in (dict(weight=w[:128]), dict(weight=w.half()), dict(weight=w.cpu()), dict(weight=torch.ones(512, device=DEV)[::2]),
                dict(out="fp4"), dict(residual=x[:2]), dict(residual=x.half()), dict(residual=x.cpu()), dict(residual_out=x),
                dict(residual=x, residual_out=x[:2]), dict(x=x[0]), dict(x=x.float()), dict(x=x.t())):
        kw = dict(dict(x=x, weight=w), **bad)
        with pytest.raises(ValueError):
            hq.rms_norm(kw.pop("x"), kw.pop("weight"), **kw)
    wide = torch.zeros(4, 516, dtype=torch.bfloat16, device=DEV)
    for kw in (dict(x=wide[:, :256]), dict(x=wide.view(-1)[4:4 + 1024].view(4, 256)), dict(x=x, residual=x, residual_out=x[:1].expand(4, 256)),
               dict(x=x, eps=-1.0), dict(x=x[:, :136], weight=w[:136], out="mxfp4"), dict(x=x[:, :4], weight=w[:4])):
        kw = dict(dict(weight=w), **kw)
        with pytest.raises(hq.HQError):
            hq.rms_norm(kw.pop("x"), kw.pop("weight"), **kw)


def test_native_calls_are_the_same(monkeypatch):
    """The binding's native call against the same call through ctypes, on another stream
    too: each output, strided rows, h written in place, no rows."""
    g = _gen(40)
    x, wide, odd = _x(g, 9, 512, torch.bfloat16), _x(g, 9, 1104, torch.bfloat16), _x(g, 9, 1100, torch.bfloat16)
    w, w32 = torch.randn(512, device=DEV).bfloat16(), torch.randn(512, device=DEV)

    def calls():
        r = []
        for out in KINDS:
            for a in (x, wide[:, 8:520], x[3:4], x[:0]):
                y = hq.rms_norm(a, w, out=out)
                r += y if isinstance(y, tuple) else (y,)
                r += hq.rms_norm(a, w32, 1e-5, residual=wide[: len(a), 520:1032], out=out)
            h = x.clone()
            y = hq.rms_norm(x, w, residual=h, out=out, residual_out=h)
            assert y[-1] is h or y[-1].data_ptr() == h.data_ptr()
            r += y
        return r
    assert hq._calls is not None and hq._calls.rms_norm(x, w, 1e-6, None, 4, None) is not None
    native = calls()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        other = calls()
    torch.cuda.synchronize()
    assert hq._calls.rms_norm(odd[:, :512], w, 1e-6, None, 0, None) is None                 # rows of 1100
    assert hq._calls.rms_norm(x.t(), w, 1e-6, None, 0, None) is None and hq._calls.rms_norm(x, w[1:], 1e-6, None, 0, None) is None
    assert hq._calls.rms_norm(x, w, 1e-6, None, 0, x) is None and hq._calls.rms_norm(x, w, -1.0, None, 0, None) is None
    assert hq._calls.rms_norm(x, w, 1e-6, x[1:], 0, None) is None and hq._calls.rms_norm(wide, wide[0], 1e-6, None, 3, None) is None
    monkeypatch.setattr(hq, "_calls", None)
    plain = calls()
    torch.cuda.synchronize()
    assert len(native) == len(plain)
    for p, q, r in zip(native, other, plain):
        assert p.dtype == r.dtype and p.shape == r.shape and torch.equal(p, r) and torch.equal(q, r)
