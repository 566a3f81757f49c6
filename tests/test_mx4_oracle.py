"""MXFP4 experts' layers without a GPU: the oracle's pins, plans and tunings that are
refused, layers of plans that do not belong together, and the host repack."""
import pytest
import torch

import bit_quantized_gemm_repack_amd as hq
from oracle import mx4 as om


def test_values_and_packing():
    b = torch.arange(256, dtype=torch.uint8)[None]
    v = om.values(b)
    assert v[0, :6].tolist() == [0, 0, 0.5, 0, 1, 0] and v[0, 2 * 0xF7:2 * 0xF7 + 2].tolist() == [6, -6]
    keep = ((b & 15) != 8) & ((b >> 4) != 8)          # -0 packs as 0
    assert torch.equal(om.pack(v).masked_select(keep), b.masked_select(keep))


def test_rounding_is_nearest_even():
    x = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.2500001, 6.9, -0.25, -2.5])
    assert om.e2m1(x.double()).tolist() == [0, 1, 1, 2, 2, 4, 4, 0.5, 6, 0, -2]


def test_quantize_powers():
    x = torch.zeros(4, 32, dtype=torch.float64)
    x[0, 3], x[1, 3], x[2, 3] = 1.0, 7.99, 2.0 ** -130
    q, e = om.quantize(x)
    assert e[:, 0].tolist() == [125, 127, 0, 127] and q[0, 3] == 4 and q[1, 3] == 6
    v = torch.arange(32.0).view(2, 16)                # rows of 16 blocks
    assert om.group_major(v).shape == (4, 2, 4) and om.group_major(v)[1, 1].tolist() == [20, 21, 22, 23]
    assert torch.equal(om.row_major(om.group_major(v)), v)


def test_bounds_see_mistakes():
    """A code a step off, a power of two off by one, and a swapped block fall outside the range."""
    g = torch.Generator().manual_seed(1)
    act = torch.randn(16, 64, generator=g, dtype=torch.float64)
    mid, far = om.requant_range(act, 1e-6 * act.abs())
    assert (far > 0).float().mean() < 0.01
    q, e = om.quantize(act)
    assert torch.equal(om.rows(q, e), mid)
    wrong = om.rows(q, e + 1)
    assert ((wrong - mid).abs() > far)[mid != 0].all()
    table = torch.tensor(om.E2M1, dtype=torch.float64)
    step = table[(torch.searchsorted(table, q.abs()) + 1) % 8] * torch.where(q < 0, -1.0, 1.0)   # the next code
    assert ((om.rows(step, e) - mid).abs() > far).float().mean() > 0.99


def test_layer_of_one_expert():
    """Weights of ones and powers of two give sums that the hand computes."""
    h, i = 128, 128
    ones = torch.full((1, 2 * i, h // 2), 0x22, dtype=torch.uint8)          # 1.0
    e1 = torch.full((1, 2 * i, h // 32), 120, dtype=torch.uint8)            # 2^-7: h = mean of x
    w2 = torch.full((1, h, i // 2), 0x44, dtype=torch.uint8)                # 2.0
    e2 = torch.full((1, h, i // 32), 127, dtype=torch.uint8)
    x = torch.full((1, h), 2.0, dtype=torch.float64)
    y, tol = om.layer(om.rows(*om.quantize(x)), torch.tensor([[0, -1]]), torch.tensor([[0.5, 9.0]]), ones, e1, w2, e2)
    s = 2 / (1 + torch.exp(torch.tensor(-2.0, dtype=torch.float64))) * 2     # 3.52 = 7.05 / 2, beyond 6 / 2
    assert om.rows(*om.quantize(s.repeat(1, 32)))[0, 0] == 3
    assert torch.equal(y, torch.full_like(y, 0.5 * 128 * 3 * 2)) and (tol < 2.0).all()


Q = hq.w4a4_mxfp4()


@pytest.mark.parametrize("n,k,epi,ok", [
    (512, 256, "silu_mul_qmxfp4", True), (256, 256, "topk_combine", True), (64, 128, "topk_combine", True),
    (384, 256, "silu_mul_qmxfp4", False),     # 192 outputs are no whole 128
    (96, 256, "topk_combine", False), (512, 256, "silu_mul", False), (512, 256, "silu_mul_qfp8", False), (512, 256, "none", False),
    (512, 200, "silu_mul_qmxfp4", False),
])
def test_plans(n, k, epi, ok):
    if ok:
        p = hq.MoePlan(n, k, Q, 4, 64, epi)
        assert "w4a4-mxfp4" in p.describe(8, 2)
        assert p.repacked_bytes() == (4 * (n * k // 2 + n * k // 32), 0)
        return
    with pytest.raises(hq.HQError) as e:
        hq.MoePlan(n, k, Q, 4, 64, epi)
    assert e.value.status == hq.HQ_ERR_UNSUPPORTED


def test_epilogue_goes_with_its_format():
    for q in (hq.w8a8_block(), hq.w4a16("bf16"), hq.w4a8_fp8()):
        with pytest.raises(hq.HQError):
            hq.MoePlan(512, 256, q, 4, 64, "silu_mul_qmxfp4")
    with pytest.raises(hq.HQError):
        hq.Plan(512, 256, Q, 64, epi="silu_mul_qmxfp4", fallback=False)


@pytest.mark.parametrize("tuning,ok", [(dict(tile_m=16), True), (dict(tile_m=64), True), (dict(tile_m=128, tile_n=256), True), (dict(tile_m=32), False),
                                       (dict(tile_n=128), False), (dict(kernel=1), False)])
def test_tunings(tuning, ok):
    if ok:
        p = hq.MoePlan(512, 256, Q, 4, 4096, "silu_mul_qmxfp4", tuning=tuning)
        assert all(p.block_m(t, 2) == tuning["tile_m"] for t in (1, 40, 4000))
    else:
        with pytest.raises(hq.HQError):
            hq.MoePlan(512, 256, Q, 4, 4096, "silu_mul_qmxfp4", tuning=tuning)


def test_both_plans_choose_one_block():
    for e, h, i in ((256, 7168, 256), (64, 2048, 768), (8, 4096, 1024), (1, 512, 128)):
        gu = hq.MoePlan(2 * i, h, Q, e, 1 << 14, "silu_mul_qmxfp4")
        dn = hq.MoePlan(h, i, Q, e, 1 << 14, "topk_combine")
        for t in (1, 2, 7, 16, 40, 100, 300, 509, 1000, 1500, 4096, 9000):
            assert gu.block_m(t, 2) == dn.block_m(t, 2), (e, h, i, t)


def test_layer_plans_belong_together():
    gu, dn = hq.MoePlan(512, 256, Q, 4, 64, "silu_mul_qmxfp4"), hq.MoePlan(256, 256, Q, 4, 64, "topk_combine")
    ids, w = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2)
    x = torch.zeros(2, 256, dtype=torch.bfloat16)
    few = hq.MoePlan(256, 256, Q, 3, 64, "topk_combine")
    more = hq.MoePlan(256, 256, Q, 5, 64, "topk_combine")
    short = hq.MoePlan(256, 128, Q, 4, 64, "topk_combine")
    fp8 = hq.MoePlan(256, 256, hq.w8a8_block(), 4, 64, "topk_combine")
    for d in (few, more, short, fp8, gu):
        with pytest.raises(ValueError):
            hq.moe_layer(gu, d, x, ids, w, x, x, x, x)
    with pytest.raises(ValueError, match="by-slot"):
        hq.moe_layer(gu, dn, x, ids, w, x, x, x, x, by_slot=True)


LAYER = dict(t=2, topk=2, type=hq.BF16, x=4096, xs=None, ids=8192, w=12288, w1=16384, w2=20480, out=24576, ws=28672, ws_bytes=1 << 20)


def _layer(gu, dn, **kw):
    a = dict(LAYER, **kw)
    return hq.lib().hq_moe_layer_mxfp4(gu._h if gu else None, dn._h if dn else None, a["t"], a["topk"], a["type"], a["x"], a["xs"], a["ids"], a["w"],
                                       a["w1"], a["w2"], a["out"], a["ws"], a["ws_bytes"], None)


def test_layer_refusals():
    """Every refusal of hq_moe_layer_mxfp4 comes before a launch."""
    import ctypes
    gu, dn = hq.MoePlan(512, 2048, Q, 4, 64, "silu_mul_qmxfp4"), hq.MoePlan(2048, 256, Q, 4, 64, "topk_combine")
    n = ctypes.c_size_t()
    need = {}
    for t, topk in ((0, 2), (1, 2), (2, 2), (40, 2), (64, 64)):
        assert hq.lib().hq_moe_mxfp4_workspace_bytes(gu._h, dn._h, t, topk, ctypes.byref(n)) == hq.HQ_OK
        need[t] = n.value
    assert need[0] == 0 < need[1] <= need[2] < need[40] < need[64]
    assert _layer(gu, dn, t=0, x=None, ws=None, ws_bytes=0) == hq.HQ_OK
    arg, un, ws = hq.HQ_ERR_INVALID_ARG, hq.HQ_ERR_UNSUPPORTED, hq.HQ_ERR_WORKSPACE
    for kw, want in ((dict(t=65), arg), (dict(t=-1), arg), (dict(topk=0), arg), (dict(topk=65), arg), (dict(type=hq.F32), un), (dict(type=hq.FP8_E4M3), un),
                     (dict(type=hq.FP4_E2M1), arg), (dict(xs=4096), arg), (dict(x=None), arg), (dict(ids=None), arg), (dict(w=None), arg),
                     (dict(w1=None), arg), (dict(w2=None), arg), (dict(out=None), arg), (dict(x=4104), arg), (dict(type=hq.FP4_E2M1, xs=4100), arg),
                     (dict(w1=16392), arg), (dict(w2=20488), arg), (dict(out=24584), arg), (dict(ids=8193), arg), (dict(w=12290), arg),
                     (dict(ws=None), ws), (dict(ws_bytes=need[2] - 1), ws), (dict(t=40, ws_bytes=need[40] - 1), ws), (dict(ws=28680), arg)):
        assert _layer(gu, dn, **kw) == want, kw
        assert hq.lib().hq_last_error()
    assert _layer(None, dn) == arg and _layer(gu, None) == arg and _layer(dn, gu) == arg and _layer(gu, gu) == arg
    assert hq.lib().hq_moe_mxfp4_workspace_bytes(gu._h, dn._h, 1, 2, None) == arg
    assert _layer(gu, hq.MoePlan(2048, 256, Q, 5, 64, "topk_combine")) == arg
    assert _layer(gu, hq.MoePlan(2048, 128, Q, 4, 64, "topk_combine")) == arg
    assert _layer(gu, hq.MoePlan(2048, 256, Q, 4, 64, "topk_combine", tuning=dict(tile_m=128))) == arg      # another block height
    assert _layer(gu, hq.MoePlan(2048, 256, Q, 4, 1, "topk_combine")) == arg
    assert _layer(gu, hq.MoePlan(2048, 256, hq.w8a8_block(), 4, 64, "topk_combine")) == un
    big = [hq.MoePlan(n, k, Q, 4, 1 << 20, epi) for n, k, epi in ((512, 2048, "silu_mul_qmxfp4"), (2048, 256, "topk_combine"))]
    assert _layer(*big, t=1 << 20) == un
    for h, i, t in ((65536, 32768, 2), (65536, 128, 70000), (128, 65536, 40000)):      # an expert, x, the intermediate of 2 GiB
        big = [hq.MoePlan(n, k, Q, 1, 1 << 17, epi) for n, k, epi in ((2 * i, h, "silu_mul_qmxfp4"), (h, i, "topk_combine"))]
        assert hq.lib().hq_moe_mxfp4_workspace_bytes(*(p._h for p in big), t, 2, ctypes.byref(n)) == un
        assert _layer(*big, t=t, ws_bytes=1 << 50) == un
    many = [hq.MoePlan(n, k, Q, 4097, 64, epi) for n, k, epi in ((512, 128, "silu_mul_qmxfp4"), (128, 256, "topk_combine"))]
    assert _layer(*many) == un


def test_host_repack_checks_shapes():
    gu = hq.MoePlan(512, 256, Q, 2, 64, "silu_mul_qmxfp4")
    codes, e = torch.zeros(2, 512, 128, dtype=torch.uint8), torch.full((2, 512, 8), 127, dtype=torch.uint8)
    w, _ = gu.repack_host(codes, e8m0=e)
    assert w.numel() == 2 * 512 * (128 + 8) and (w == 127).sum() == 2 * 512 * 8
    for c, s in ((codes[:1], e), (codes.transpose(1, 2), e), (codes, e[:1]), (codes, e.transpose(1, 2)), (codes, None), (codes.float(), e)):
        with pytest.raises(ValueError):
            gu.repack_host(c, e8m0=s)
