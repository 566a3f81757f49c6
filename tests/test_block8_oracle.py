"""The fp8 block oracle (oracle/block8.py) against torch's e4m3 casts, a scalar
brute force and hand-worked values, and the host side of the fp8 block path:
the weight repack's operand order, every refusal, and the arithmetic of the
kernels' quotient, checked for all 16-bit inputs."""
import ctypes
import math

import numpy as np
import pytest
import torch

import bit_quantized_gemm_repack_amd as hq
from oracle import block8 as o8

FAKE = 1 << 20  # an aligned address that no rejected call reads


def test_e4m3_rounds_as_torch_casts():
    v = torch.linspace(-460, 460, 200001, dtype=torch.float64).float()
    v = torch.cat([v, v * 2.0 ** -9, torch.tensor([0.0, 2.0 ** -10, 3 * 2.0 ** -10, 17.0, 18.0, 19.0])])
    want = v.clamp(-448, 448).to(torch.float8_e4m3fn).double()
    assert torch.equal(o8.e4m3(v.double()), want)


def test_quantize_by_hand():
    x = torch.zeros(2, 256, dtype=torch.float64)
    x[0, 0], x[0, 1], x[0, 2] = 448.0, 17.0, -18.0    # scale 1: 17 is the midpoint of 16 and 18 -> 16
    x[1, 130] = -7.0                                  # scale 1/64
    codes, s = o8.quantize(x)
    assert s.tolist() == [[1.0, 1.0], [1.0, 7.0 / 448]]
    assert codes[0, :3].tolist() == [448.0, 16.0, -18.0] and codes[1, 130] == -448.0


def test_gemm_and_weight_against_loops():
    g = torch.Generator().manual_seed(3)
    n, k, m = 144, 256, 3
    w = torch.randn(n, k, generator=g).clamp(-448, 448).to(torch.float8_e4m3fn)
    sw = torch.rand(2, 2, generator=g)
    a = torch.randn(m, k, generator=g).to(torch.float8_e4m3fn)
    sa = torch.rand(m, 2, generator=g)
    c, tol = o8.gemm(o8.rows(a, sa), o8.weight(w, sw))
    for i in range(m):
        for j in (0, 127, 128, 143):
            want = sum(float(a[i, q]) * float(sa[i, q // 128]) * float(w[j, q]) * float(sw[j // 128, q // 128]) for q in range(k))
            assert abs(float(c[i, j]) - want) < 1e-9
    assert (tol > 0).all()


def test_route_by_hand():
    x = torch.tensor([[1.0, 3.0, 3.0, float("nan")], [float("-inf"), 0.0, float("-inf"), float("-inf")],
                      [float("-inf")] * 4])
    ids, w = o8.route(x, 3, False)
    assert ids.tolist() == [[1, 2, 0], [1, -1, -1], [-1, -1, -1]]
    z = 2 * math.exp(3) + math.exp(1)
    assert w[0].tolist() == pytest.approx([math.exp(3) / z, math.exp(3) / z, math.exp(1) / z])
    assert w[1].tolist() == [1.0, 0.0, 0.0] and w[2].tolist() == [0.0, 0.0, 0.0]
    _, w = o8.route(x, 2, True)
    assert w[0].tolist() == pytest.approx([0.5, 0.5])


def test_act_bound_holds_under_perturbation():
    g = torch.Generator().manual_seed(5)
    h = 4 * torch.randn(64, 512, generator=g, dtype=torch.float64)
    tau = 1e-3 * torch.rand(64, 512, generator=g, dtype=torch.float64)
    b = o8.act_bound(h, tau)
    for sg in (-1, 1):
        for su in (-1, 1):
            d = torch.cat([sg * tau[:, :256], su * tau[:, 256:]], 1)
            assert ((o8.silu_mul(h + d) - o8.silu_mul(h)).abs() <= b).all()


def test_requant_range_covers_perturbed_values():
    g = torch.Generator().manual_seed(6)
    act = torch.randn(32, 256, generator=g, dtype=torch.float64)
    tau = 1e-4 * torch.ones_like(act)
    mid, far = o8.requant_range(act, tau)
    for _ in range(20):
        d = (2 * torch.rand(act.shape, generator=g, dtype=torch.float64) - 1) * tau
        assert ((o8.rows(*o8.quantize(act + d)) - mid).abs() <= far * (1 + 1e-12)).all()


def test_planted_mistakes_exceed_the_bounds():
    """A scale block taken one off, and a slot's weight left out, are seen."""
    g = torch.Generator().manual_seed(7)
    a, w = torch.randn(4, 512, generator=g), torch.randn(256, 512, generator=g)
    ac, asc = o8.quantize(a.double())
    wc = w.clamp(-448, 448).to(torch.float8_e4m3fn).double()
    sw = 0.5 + torch.rand(2, 4, generator=g)
    c, tol = o8.gemm(o8.rows(ac, asc), o8.weight(wc, sw))
    bad, _ = o8.gemm(o8.rows(ac, asc), o8.weight(wc, sw.roll(1, 1)))
    assert ((bad - c).abs() > tol + o8.half_step(c, torch.bfloat16)).float().mean() > 0.9


@pytest.mark.parametrize("bits", [8, 11])
def test_corrected_product_is_the_rounded_quotient(bits):
    """v r + r (v - s (v r)) with r = fl(1/s), s = fl(top / 448), is the
    correctly rounded v / s for every pair of significands of bf16 (8 bits) and
    fp16 (11 bits); powers of two change no step."""
    f = np.float32
    n = 1 << (bits - 1)
    mant = np.arange(n, 2 * n) / n
    for eb in (0, 1):
        s = ((mant * 2.0 ** eb).astype(f) / f(448)).astype(f)
        r = (f(1) / s).astype(f)
        for lo in range(0, n, 64):
            v = mant[lo:lo + 64].astype(f)[:, None]
            q = (v * r).astype(f)
            rem = (v.astype(np.float64) - q.astype(np.float64) * s.astype(np.float64)).astype(f)
            got = (q.astype(np.float64) + rem.astype(np.float64) * r.astype(np.float64)).astype(f)
            assert (got == (v / s).astype(f)).all()


# ------------------------------------------------------------ the host side --
@pytest.mark.parametrize("n,k,experts", [(16, 128, 1), (144, 384, 1), (256, 256, 3)])
def test_repack_host_operand_order(n, k, experts):
    """Lane l, half h of fragment (nb, g): column 16 nb + l % 16, k = 128 g + 64 h + 16 (l // 16) + [0, 16)."""
    g = torch.Generator().manual_seed(n + k)
    codes = torch.randint(0, 256, (experts, n, k), generator=g, dtype=torch.uint8)
    scales = torch.rand(experts, -(-n // 128), k // 128, generator=g)
    kind = dict(kind="grouped", epi="silu_mul_qfp8", num_experts=experts) if experts > 1 else {}
    plan = hq.Plan(n, k, hq.w8a8_block(), max_m=8, **kind)
    w, meta = plan.repack_host(codes, scales)
    w = w.view(experts, n // 16, k // 128, 2, 4, 16, 16)  # e, nb, g, h, kq, c, byte
    want = codes.view(experts, n // 16, 16, k // 128, 2, 4, 16).permute(0, 1, 3, 4, 5, 2, 6)
    assert torch.equal(w, want)
    assert torch.equal(meta[:scales.numel() * 4].view(torch.float32), scales.flatten())


def _plan(n=256, k=512, max_m=64, quant=None, **kw):
    return hq.Plan(n, k, quant or hq.w8a8_block(), max_m=max_m, fallback=False, **kw)


def test_descriptions_refused():
    def q(**kw):
        d = hq.w8a8_block()
        for f, v in kw.items():
            setattr(d, f, v)
        return d
    for kw in (dict(w_bits=4), dict(group_size=64), dict(scale=hq.BF16), dict(zp=hq.ZP_FIXED), dict(act=hq.BF16, act_scale=hq.ASCALE_NONE),
               dict(act_scale=hq.ASCALE_PER_TOKEN_F32), dict(act=hq.INT8), dict(out=hq.F32)):
        with pytest.raises(hq.HQError) as e:
            _plan(quant=q(**kw))
        assert e.value.status == hq.HQ_ERR_UNSUPPORTED, kw
    for n, k in ((24, 512), (256, 192)):
        with pytest.raises(hq.HQError) as e:
            _plan(n, k)
        assert e.value.status == hq.HQ_ERR_UNSUPPORTED
    with pytest.raises(hq.HQError):
        _plan(mfma_in="bf16")
    assert "w8a8-block" in _plan(mfma_in="fp8").describe(1)


def test_tunings():
    for t in (dict(kernel=2, tile_m=256), dict(kernel=2, tile_m=64, tile_n=256), dict(kernel=2, tile_m=16, stages=2),
              dict(kernel=1, tile_m=32), dict(kernel=1, tile_n=64), dict(kernel=1, waves=9), dict(kernel=2, tile_group=65)):
        with pytest.raises(hq.HQError):
            _plan(tuning=t)
    p = _plan(max_m=4096, n=4096, k=7168)
    for m, kernel in ((1, "skinny"), (16, "skinny"), (64, "tiled"), (4096, "tiled")):
        assert f"kernel={kernel}" in p.describe(m)
        t, tuned = p.get_tuning(m)
        p.set_tuning(m, t)                       # what the plan says of itself is a tuning it takes
        assert p.get_tuning(m) == (t, True) and not tuned
    need = p.workspace_bytes(64)
    assert need > 0 and need % 256 == 0
    for f in (p.set_jit, lambda: p.jit_cache_key(1), lambda: p.jit_prepare(1)):
        with pytest.raises(hq.HQError) as e:
            f()
        assert e.value.status == hq.HQ_ERR_UNSUPPORTED


def test_grouped_plans_refused():
    q = hq.w8a8_block()
    for n, k, epi in ((512, 256, "silu_mul"), (512, 256, "none"), (384, 256, "silu_mul_qfp8"), (96, 256, "topk_combine")):
        with pytest.raises(hq.HQError) as e:
            hq.MoePlan(n, k, q, 4, 8, epi)
        assert e.value.status == hq.HQ_ERR_UNSUPPORTED
    for t in (dict(kernel=1), dict(tile_m=32), dict(tile_n=128), dict(tile_m=48)):
        with pytest.raises(hq.HQError):
            hq.MoePlan(512, 256, q, 4, 8, "silu_mul_qfp8", tuning=t)
    g = hq.MoePlan(512, 256, q, 256, 4096, "silu_mul_qfp8")  # blocks by rows per expert, where there are plenty
    assert g.block_m(64, 8) == 16 and g.block_m(1024, 8) == 64 and g.block_m(4096, 8) == 128
    g = hq.MoePlan(512, 256, q, 4, 64, "silu_mul_qfp8")
    assert g.block_m(1, 2) == 16 and g.block_m(64, 64) == 16  # few workgroups: low blocks
    L = hq.lib()
    assert L.hq_moe_gemm_by_slot(g._h, 1, 1, *[FAKE] * 9, 1 << 30, None) == hq.HQ_ERR_UNSUPPORTED


def test_gemm_call_refused():
    L = hq.lib()
    p = _plan(n=4096, k=7168)
    args = dict(a=FAKE, s=FAKE, w=FAKE, meta=FAKE, out=FAKE, ws=FAKE, n=1 << 30)

    def call(m=1, **kw):
        v = {**args, **kw}
        return L.hq_gemm(p._h, m, v["a"], v["s"], v["w"], v["meta"], v["out"], v["ws"], v["n"], None)
    assert call(m=0) == hq.HQ_OK
    assert call(m=65) == hq.HQ_ERR_INVALID_ARG and call(m=-1) == hq.HQ_ERR_INVALID_ARG
    for k in ("a", "s", "w", "meta", "out"):
        assert call(**{k: None}) == hq.HQ_ERR_INVALID_ARG
    for k in ("a", "w", "meta", "out"):
        assert call(**{k: FAKE + 4}) == hq.HQ_ERR_INVALID_ARG
    assert call(m=64, ws=None, n=0) == hq.HQ_ERR_WORKSPACE and call(m=64, n=16) == hq.HQ_ERR_WORKSPACE
    big = _plan(n=1 << 16, k=1 << 15)            # 2 GiB of codes
    assert L.hq_gemm(big._h, 1, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 30, None) == hq.HQ_ERR_UNSUPPORTED


def test_quantize_blocks_call_refused():
    q = hq.lib().hq_quantize_blocks
    assert q(4, 128, hq.F32, 0, FAKE, FAKE, FAKE, None) == hq.HQ_ERR_UNSUPPORTED
    assert q(4, 128, hq.BF16, 2, FAKE, FAKE, FAKE, None) == hq.HQ_ERR_INVALID_ARG
    assert q(-1, 128, hq.BF16, 0, FAKE, FAKE, FAKE, None) == hq.HQ_ERR_INVALID_ARG
    for k in (0, 64, 192, (1 << 24) + 128):
        assert q(4, k, hq.BF16, 0, FAKE, FAKE, FAKE, None) == hq.HQ_ERR_INVALID_ARG
    assert q(1 << 24, 1 << 17, hq.BF16, 0, FAKE, FAKE, FAKE, None) == hq.HQ_ERR_UNSUPPORTED
    for bad in ((None, FAKE, FAKE), (FAKE, None, FAKE), (FAKE, FAKE, None), (FAKE + 8, FAKE, FAKE), (FAKE, FAKE + 8, FAKE),
                (FAKE, FAKE, FAKE + 4)):
        assert q(4, 128, hq.BF16, 0, *bad, None) == hq.HQ_ERR_INVALID_ARG
    assert q(0, 128, hq.BF16, 0, None, None, None, None) == hq.HQ_OK


def test_route_call_refused():
    r = hq.lib().hq_route_topk
    assert r(4, 8, 2, hq.INT8, FAKE, 0, FAKE, FAKE, None) == hq.HQ_ERR_UNSUPPORTED
    assert r(4, 1025, 2, hq.F32, FAKE, 0, FAKE, FAKE, None) == hq.HQ_ERR_UNSUPPORTED
    for e, k in ((0, 1), (8, 0), (8, 9), (128, 65)):
        assert r(4, e, k, hq.F32, FAKE, 0, FAKE, FAKE, None) == hq.HQ_ERR_INVALID_ARG
    assert r(-1, 8, 2, hq.F32, FAKE, 0, FAKE, FAKE, None) == hq.HQ_ERR_INVALID_ARG
    assert r(4, 8, 2, hq.F32, FAKE, 2, FAKE, FAKE, None) == hq.HQ_ERR_INVALID_ARG
    for bad in ((None, FAKE, FAKE), (FAKE, None, FAKE), (FAKE, FAKE, None), (FAKE + 2, FAKE, FAKE), (FAKE, FAKE + 2, FAKE)):
        assert r(4, 8, 2, hq.F32, bad[0], 0, bad[1], bad[2], None) == hq.HQ_ERR_INVALID_ARG
    assert r(0, 8, 2, hq.F32, None, 0, None, None, None) == hq.HQ_OK


def test_few_call_refused():
    L = hq.lib()
    q = hq.w8a8_block()
    g = hq.MoePlan(512, 1024, q, 8, 64, "silu_mul_qfp8")
    d = hq.MoePlan(1024, 256, q, 8, 64, "topk_combine")

    def call(gu=g, dn=d, t=4, topk=2, xt=hq.BF16, lt=hq.F32, logits=FAKE, renorm=1, ws=FAKE, n=1 << 30, x=FAKE, out=FAKE):
        return L.hq_moe_layer_few(gu._h, dn._h, t, topk, xt, x, lt, logits, renorm, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, out,
                                  ws, n, None)
    assert call(t=0) == hq.HQ_OK
    for kw in (dict(t=-1), dict(t=65), dict(topk=0), dict(topk=9), dict(renorm=2), dict(x=None), dict(out=None), dict(x=FAKE + 8),
               dict(gu=d, dn=g), dict(dn=hq.MoePlan(1024, 512, q, 8, 64, "topk_combine")),
               dict(dn=hq.MoePlan(1024, 256, q, 9, 64, "topk_combine"))):
        assert call(**kw) == hq.HQ_ERR_INVALID_ARG, kw
    for kw in (dict(topk=17), dict(xt=hq.F32), dict(lt=hq.INT8), dict(dn=hq.MoePlan(1024, 256, hq.w4a16("bf16"), 8, 64, "topk_combine"))):
        assert call(**kw) == hq.HQ_ERR_UNSUPPORTED, kw
    assert call(ws=None) == hq.HQ_ERR_WORKSPACE and call(n=16) == hq.HQ_ERR_WORKSPACE
    many = [hq.MoePlan(512, 1024, q, 8, 128, "silu_mul_qfp8"), hq.MoePlan(1024, 256, q, 8, 128, "topk_combine")]
    assert call(gu=many[0], dn=many[1], t=65) == hq.HQ_ERR_UNSUPPORTED
    wide = [hq.MoePlan(512, 1024, q, 1100, 64, "silu_mul_qfp8"), hq.MoePlan(1024, 256, q, 1100, 64, "topk_combine")]
    assert call(gu=wide[0], dn=wide[1]) == hq.HQ_ERR_UNSUPPORTED                      # routing: up to 1024 experts
    b = ctypes.c_size_t()
    assert L.hq_moe_few_workspace_bytes(g._h, d._h, 4, 2, ctypes.byref(b)) == hq.HQ_OK and b.value >= 4 * 2 * 256 * 4
    assert L.hq_moe_few_workspace_bytes(g._h, d._h, 65, 2, ctypes.byref(b)) == hq.HQ_ERR_INVALID_ARG


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(2, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        hq.quantize_blocks(x)
    with pytest.raises(ValueError):
        hq.route_topk(torch.zeros(2, 8), 2)
    p = _plan()
    with pytest.raises(ValueError):
        p.gemm(x, x, x, a_scale=x)
    with pytest.raises(ValueError):
        p.repack_host(torch.zeros(256, 512, dtype=torch.uint8), torch.zeros(2, 3))   # scales of another shape
    with pytest.raises(ValueError):
        p.repack_host(torch.zeros(256, 256, dtype=torch.uint8), torch.zeros(2, 4))


def test_layer_plans_share_blocks():
    """gate_up and down come to one alignment block for every call of a layer."""
    q = hq.w8a8_block()
    seen = set()
    for e, h, i in ((8, 512, 128), (16, 4096, 512), (32, 2048, 768), (256, 7168, 256), (2, 256, 1024)):
        g, d = hq.MoePlan(2 * i, h, q, e, 8192, "silu_mul_qfp8"), hq.MoePlan(h, i, q, e, 8192, "topk_combine")
        for t in (1, 2, 17, 24, 100, 300, 700, 1500, 4096, 8192):
            for k in (1, 2, 8):
                assert g.block_m(t, k) == d.block_m(t, k)
                seen.add(g.block_m(t, k))
    assert seen == {16, 64, 128}


def test_native_calls_take_nothing_else():
    """What is no GPU tensor of the right kind is left to the Python checks."""
    hq.lib()
    if hq._calls is None:
        pytest.skip("the native calls are not built")
    x = torch.zeros(2, 256, dtype=torch.bfloat16)
    for args in ((), (x,), (None, False), (x, False), (x.float(), True), ("x", 1)):
        assert hq._calls.quantize_blocks(*args) is None
    for args in ((x, 2, True), (x, "2", True), (x, 1 << 70, True), (3, 2, True), (x, 2)):
        assert hq._calls.route_topk(*args) is None
    assert hq._calls.gemm_block(0, 16, 128, True, x, x, x, x) is None and hq._calls.gemm_block() is None
    with pytest.raises(TypeError):
        hq._calls.bind(1, 2)
    with pytest.raises(ValueError):
        hq.quantize_blocks(x)


def test_repack_refuses_transposed_tensors():
    """Scales [k/128, n/128] and codes [k, n] hold as many values as the right ones."""
    p = _plan(n=256, k=512)
    codes, s = torch.zeros(256, 512, dtype=torch.uint8), torch.ones(2, 4)
    p.repack_host(codes, s)
    for c, v in ((codes, s.t()), (codes, s.flatten()), (codes.t(), s), (codes.flatten(), s), (codes.view(torch.int32), s)):
        with pytest.raises(ValueError):
            p.repack_host(c, v)


def test_repack_refuses_other_types():
    p = _plan(n=256, k=512)
    codes, s = torch.zeros(256, 512, dtype=torch.uint8), torch.ones(2, 4)
    for dt in (torch.float8_e4m3fn, torch.int8):
        p.repack_host(codes.view(dt), s)
    for dt in (torch.float8_e5m2, torch.float8_e4m3fnuz, torch.bool):
        with pytest.raises(ValueError, match="e4m3"):
            p.repack_host(codes.view(dt), s)
