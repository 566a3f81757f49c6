"""Calls of the fp8 block path with tensors that do not fit: refused before
anything is launched, natively and through ctypes."""
import pytest
import torch

import bit_quantized_gemm_repack_amd as hq
from oracle import block8 as o8

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E4 = torch.float8_e4m3fn


def _gen(seed):
    g = torch.Generator(DEV)
    g.manual_seed(seed)
    return g


def _weight(g, n, k, experts=None):
    lead = () if experts is None else (experts,)
    codes = (torch.randn(*lead, n, k, generator=g, device=DEV) * 96).clamp_(-448, 448).to(E4)
    return codes, (0.5 + torch.rand(*lead, -(-n // 128), k // 128, generator=g, device=DEV)) / (96 * k ** 0.5)


def _dense(m=24, n=272, k=1024, **kw):
    g = _gen(m + n)
    w, s = _weight(g, n, k)
    plan = hq.Plan(n, k, hq.w8a8_block(), max_m=64, **kw)
    a, sa = hq.quantize_blocks(torch.randn(m, k, generator=g, device=DEV, dtype=torch.bfloat16))
    return plan, w, s, plan.repack(w.view(torch.uint8), s), a, sa


@pytest.fixture(params=[True, False], ids=["native", "ctypes"])
def way(request, monkeypatch):
    hq.lib()
    if not request.param:
        monkeypatch.setattr(hq, "_calls", None)


def test_layer_of_another_output_size():
    """x of 512, y of 768 columns: the same answer on both sides of the few-token switch."""
    g = _gen(1)
    w1, s1 = _weight(g, 512, 512, 6)
    w2, s2 = _weight(g, 768, 256, 6)
    gu, dn = (hq.MoePlan(n, k, hq.w8a8_block(), 6, 64, e) for n, k, e in ((512, 512, "silu_mul_qfp8"), (768, 256, "topk_combine")))
    wm = (*gu.repack(w1.view(torch.uint8), s1), *dn.repack(w2.view(torch.uint8), s2))
    for t in (1, 4, 20):
        x = torch.randn(t, 512, generator=g, device=DEV, dtype=torch.bfloat16)
        y, ids, w = hq.moe_layer_routed(gu, dn, x, torch.randn(t, 6, generator=g, device=DEV), 2, *wm)
        z = hq.moe_layer(gu, dn, x, ids, w, *wm)
        torch.cuda.synchronize()
        want, tol = o8.layer(x.double(), ids.long(), w, w1, s1, w2, s2, 2.0 ** -11)
        for v in (y, z):
            assert v.shape == (t, 768)
            assert ((v.double() - want).abs() <= tol + o8.half_step(want.abs() + tol, torch.bfloat16)).all()


def test_workspace_elsewhere_is_refused():
    """Split-K partials and slot rows are written to the workspace given: one in host memory is no place for them."""
    plan, w, s, wm, a, sa = _dense(tuning=dict(kernel=1, split_k=4))
    need = plan.workspace_bytes(24)
    assert need
    for ws in (torch.empty(need, dtype=torch.uint8), torch.empty(2 * need, dtype=torch.uint8, device=DEV)[::2], need):
        with pytest.raises(ValueError, match="ws"):
            plan.gemm(a, *wm, a_scale=sa, ws=ws)
    y = plan.gemm(a, *wm, a_scale=sa, ws=torch.empty(need // 4, device=DEV))
    assert torch.equal(y, plan.gemm(a, *wm, a_scale=sa))
    g = _gen(3)
    dn = hq.MoePlan(512, 256, hq.w8a8_block(), 4, 64, "topk_combine")
    w2, s2 = _weight(g, 512, 256, 4)
    wd = dn.repack(w2.view(torch.uint8), s2)
    ids, p = hq.route_topk(torch.randn(24, 4, generator=g, device=DEV), 2)
    al = hq.moe_align(ids, 4, dn.block_m(24, 2))
    c, sc = hq.quantize_blocks(torch.randn(al[0].numel(), 256, generator=g, device=DEV, dtype=torch.bfloat16))
    call = lambda ws: dn.moe_gemm(c, 24, 2, *al, *wd, a_scale=sc, topk_w=p, ws=ws)
    with pytest.raises(ValueError, match="ws"):
        call(torch.empty(1 << 20, dtype=torch.uint8))
    assert torch.equal(call(torch.empty(1 << 18, device=DEV)), call(None))


def test_autotune_checks_its_tensors():
    plan, w, s, wm, a, sa = _dense()
    for args in ((a[:, :512].contiguous(), *wm, sa), (a, *wm, sa[:4].contiguous()), (a, *wm, sa.double()), (a, *wm, sa.cpu()),
                 (a, wm[0][:4096], wm[1], sa), (a, wm[0], wm[1][:16], sa)):
        with pytest.raises(ValueError):
            plan.autotune(*args, reps=1, flush_bytes=0)
    assert plan.autotune(a, *wm, sa, reps=1, flush_bytes=0)["candidates"] > 0


@pytest.mark.parametrize("m", [8, 24, 64])
def test_scales_of_another_order_are_refused(way, m):
    """Row-major scales [m, k/128], which other libraries keep, hold as many values as [k/128, m]."""
    plan, w, s, wm, a, sa = _dense(m)
    want = plan.gemm(a, *wm, a_scale=sa)
    if m != 8:
        for bad in (sa.t().contiguous(), sa.flatten(), sa.unsqueeze(0)):
            with pytest.raises(ValueError, match="a_scale"):
                plan.gemm(a, *wm, a_scale=bad)
            with pytest.raises(ValueError, match="a_scale"):
                plan.autotune(a, *wm, a_scale=bad, reps=1, flush_bytes=0)
    with pytest.raises(ValueError, match="scales"):
        plan.repack(w.view(torch.uint8), s.t().contiguous())
    with pytest.raises(ValueError, match="codes"):
        plan.repack(w.view(torch.uint8).t().contiguous(), s)
    assert torch.equal(plan.gemm(a, *wm, a_scale=sa), want)


def test_grouped_scales_of_another_order_are_refused():
    g = _gen(4)
    gu = hq.MoePlan(512, 512, hq.w8a8_block(), 4, 64, "silu_mul_qfp8")
    w1, s1 = _weight(g, 512, 512, 4)
    with pytest.raises(ValueError, match="scales"):
        gu.repack(w1.view(torch.uint8), s1.flatten(0, 1).t().contiguous())
    wm = gu.repack(w1.view(torch.uint8), s1)
    x = torch.randn(24, 512, generator=g, device=DEV, dtype=torch.bfloat16)
    ids, p = hq.route_topk(torch.randn(24, 4, generator=g, device=DEV), 2)
    al = hq.moe_align(ids, 4, gu.block_m(24, 2))
    q, s = hq.quantize_blocks(x)
    gu.moe_gemm(q, 24, 2, *al, *wm, a_scale=s)
    for kw in (dict(a=q, a_scale=s.t().contiguous()), dict(a=q.view(48, 256), a_scale=s)):
        with pytest.raises(ValueError):
            gu.moe_gemm(t=24, topk=2, sorted_ids=al[0], block_expert=al[1], num_padded=al[2], w=wm[0], meta=wm[1], **kw)


@pytest.mark.parametrize("dt", [torch.float8_e5m2, torch.float8_e4m3fnuz, torch.float8_e5m2fnuz, torch.bool])
def test_codes_of_another_type_are_refused(way, dt):
    """One byte a value, but other values."""
    plan, w, s, wm, a, sa = _dense()
    with pytest.raises(ValueError, match="e4m3"):
        plan.gemm(a.view(dt), *wm, a_scale=sa)
    with pytest.raises(ValueError, match="e4m3"):
        plan.repack(w.view(dt), s)
    with pytest.raises(ValueError, match="e4m3"):
        hq.quantize_blocks(torch.zeros(2, 256, dtype=torch.bfloat16, device=DEV), codes=torch.empty(2, 256, device=DEV).to(dt))
    want = plan.gemm(a, *wm, a_scale=sa)
    for ok in (E4, torch.int8):
        assert torch.equal(plan.gemm(a.view(ok), *wm, a_scale=sa), want)
        assert torch.equal(plan.repack(w.view(ok), s)[0], wm[0])
