"""Grouped MXFP4 plans keep no metadata: 0 bytes of it are a null pointer for a C caller."""
import pytest
import torch

import bit_quantized_gemm_repack_amd as hq

Q = hq.w4a4_mxfp4()


def _plan(epi):
    return hq.MoePlan(256, 256, Q, 3, 64, epi)


@pytest.mark.parametrize("epi", ["silu_mul_qmxfp4", "topk_combine"])
def test_repack_host(epi):
    p = _plan(epi)
    wb, mb = p.repacked_bytes()
    assert mb == 0
    codes, e = torch.randint(0, 256, (3, 256, 128), dtype=torch.uint8), torch.randint(0, 255, (3, 256, 8), dtype=torch.uint8)
    w = torch.empty(wb, dtype=torch.uint8)
    assert hq.lib().hq_repack_host(p._h, codes.data_ptr(), None, e.data_ptr(), w.data_ptr(), None) == hq.HQ_OK
    assert torch.equal(w, p.repack_host(codes, e8m0=e)[0])
    dense = hq.Plan(256, 256, Q, 64)                   # whose metadata is not empty
    assert hq.lib().hq_repack_host(dense._h, codes.data_ptr(), None, e.data_ptr(), w.data_ptr(), None) == hq.HQ_ERR_INVALID_ARG
    assert hq.lib().hq_repack(dense._h, 4096, None, 4096, 4096, None, None) == hq.HQ_ERR_INVALID_ARG


def test_checks_go_on():
    """Without metadata the calls come to their next refusal."""
    A = 1 << 16
    p = _plan("topk_combine")
    assert hq.lib().hq_repack(p._h, A, None, A, A + 8, None, None) == hq.HQ_ERR_INVALID_ARG
    assert b"aligned" in hq.lib().hq_last_error()

    def gemm(plan, meta, ws_bytes=0):
        return hq.lib().hq_moe_gemm(plan._h, 4, 2, A, A, A, A, A, A, A, meta, A, None, A, ws_bytes, None)
    assert gemm(p, None) == hq.HQ_ERR_WORKSPACE
    fp8 = hq.MoePlan(256, 256, hq.w8a8_block(), 3, 64, "topk_combine")
    assert gemm(fp8, None) == hq.HQ_ERR_INVALID_ARG and gemm(fp8, A) == hq.HQ_ERR_WORKSPACE


@pytest.mark.gpu
def test_on_the_device():
    dev = torch.device("cuda:0")
    t, topk = 40, 2
    g = torch.Generator(dev)
    g.manual_seed(1)
    gu, dn = hq.MoePlan(256, 256, Q, 3, 64, "silu_mul_qmxfp4"), hq.MoePlan(256, 128, Q, 3, 64, "topk_combine")
    st = torch.cuda.current_stream().cuda_stream
    ws = []
    for p in (gu, dn):
        codes = torch.randint(0, 256, (3, p.n, p.k // 2), generator=g, dtype=torch.uint8, device=dev)
        e = torch.randint(118, 124, (3, p.n, p.k // 32), generator=g, dtype=torch.uint8, device=dev)
        w = torch.empty(p.repacked_bytes()[0], dtype=torch.uint8, device=dev)
        assert hq.lib().hq_repack(p._h, codes.data_ptr(), None, e.data_ptr(), w.data_ptr(), None, st) == hq.HQ_OK
        given, meta = p.repack(codes, e8m0=e)
        assert torch.equal(w, given)
        ws.append((given, meta))
    x, s = hq.quantize_mxfp4(torch.randn(t, 256, generator=g, device=dev).bfloat16())
    ids = torch.randint(0, 3, (t, topk), generator=g, device=dev, dtype=torch.int32)
    al = hq.moe_align(ids, 3, gu.block_m(t, topk))
    c, sc = gu.moe_gemm(x, t, topk, *al, *ws[0], a_scale=s)
    c2, sc2 = torch.zeros_like(c), torch.zeros_like(sc)
    assert hq.lib().hq_moe_gemm(gu._h, t, topk, x.data_ptr(), s.data_ptr(), *(v.data_ptr() for v in al), None, ws[0][0].data_ptr(), None,
                                c2.data_ptr(), sc2.data_ptr(), None, 0, st) == hq.HQ_OK
    torch.cuda.synchronize()
    used = int(al[2])
    live = torch.nonzero(al[0][:used] < t * topk).squeeze(1)
    assert torch.equal(c[live], c2[live]) and torch.equal(sc[:, live], sc2[:, live])
