"""The two plans of an experts' layer: what does not belong together is refused
before any tensor is read (a down plan of fewer experts, or of other rows,
would be read past its weights)."""
import pytest
import torch

import bit_quantized_gemm_repack_amd as hq

IDS, W = torch.zeros(20, 2, dtype=torch.int32), torch.ones(20, 2)
NONE = torch.zeros(0)


def _call(gu, dn, routed, t=20):
    x = torch.zeros(t, gu.k, dtype=torch.bfloat16)
    if routed:
        return hq.moe_layer_routed(gu, dn, x, torch.zeros(t, gu.num_experts), 2, NONE, NONE, NONE, NONE)
    return hq.moe_layer(gu, dn, x, IDS[:t], W[:t], NONE, NONE, NONE, NONE)


def _block8(n, k, e, epi):
    return hq.MoePlan(n, k, hq.w8a8_block(), e, 64, epi)


@pytest.mark.parametrize("routed", [False, True])
@pytest.mark.parametrize("t", [4, 20])
def test_block8_plans_that_do_not_belong_together(t, routed):
    gu = _block8(512, 1024, 8, "silu_mul_qfp8")
    for dn, what in ((_block8(1024, 256, 7, "topk_combine"), "experts"), (_block8(1024, 256, 9, "topk_combine"), "experts"),
                     (_block8(1024, 512, 8, "topk_combine"), "rows"), (_block8(1024, 128, 8, "topk_combine"), "rows"),
                     (hq.MoePlan(1024, 256, hq.w4a8_fp8(), 8, 64, "topk_combine"), "w8a8_block")):
        with pytest.raises(ValueError, match=what):
            _call(gu, dn, routed, t)
    q4 = hq.MoePlan(512, 1024, hq.w4a8_fp8(), 8, 64, "silu_mul_qfp8")
    with pytest.raises(ValueError, match="w8a8_block"):
        _call(q4, _block8(1024, 256, 8, "topk_combine"), routed, t)


@pytest.mark.parametrize("t", [4, 20])
def test_int4_plans_that_do_not_belong_together(t):
    gu = hq.MoePlan(512, 1024, hq.w4a16("bf16"), 8, 64, "silu_mul")
    for n, k, e, what in ((1024, 256, 7, "experts"), (1024, 512, 8, "rows")):
        with pytest.raises(ValueError, match=what):
            _call(gu, hq.MoePlan(n, k, hq.w4a16("bf16"), e, 64, "topk_combine"), False, t)

def test_few_tokens_need_equal_hidden_sizes():
    """The two-kernel layer writes rows of x's size; other outputs take the aligned path."""
    gu, dn = _block8(512, 1024, 8, "silu_mul_qfp8"), _block8(512, 256, 8, "topk_combine")
    assert not hq._uses_few(gu, dn, 4, 2)
    assert hq._uses_few(gu, _block8(1024, 256, 8, "topk_combine"), 4, 2)
