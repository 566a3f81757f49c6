"""Which MXFP4 layers run in the two kernels for a few tokens: not those whose experts get so many
rows that their weights are read over and over.  (A plan with a block height of its own always takes
the aligned path, whose workspace the other form does not need.)"""
import ctypes

import pytest

import bit_quantized_gemm_repack_amd as hq

Q = hq.w4a4_mxfp4("bf16")


def _few(e, h, i, topk, t):
    n = ctypes.c_size_t()
    need = []
    for tuning in (None, dict(tile_m=16)):
        gu = hq.MoePlan(2 * i, h, Q, e, 64, "silu_mul_qmxfp4", tuning=tuning)
        dn = hq.MoePlan(h, i, Q, e, 64, "topk_combine", tuning=tuning)
        assert tuning or gu.block_m(t, topk) in (16, 64)
        assert hq.lib().hq_moe_mxfp4_workspace_bytes(gu._h, dn._h, t, topk, ctypes.byref(n)) == hq.HQ_OK
        need.append(n.value)
    return need[0] < need[1] // 2


@pytest.mark.parametrize("e,h,i,topk,t", [(256, 7168, 256, 8, 1), (256, 7168, 256, 8, 9), (64, 2048, 768, 8, 2), (64, 7168, 256, 2, 32), (256, 7168, 256, 1, 32),
                                          (8, 4096, 512, 2, 10), (8, 7168, 256, 1, 17), (8, 7168, 256, 8, 4), (16, 7168, 256, 4, 10), (8, 4096, 2048, 1, 8)])
def test_few(e, h, i, topk, t):
    assert _few(e, h, i, topk, t)


@pytest.mark.parametrize("e,h,i,topk,t", [(256, 7168, 256, 8, 13), (64, 2048, 768, 8, 3), (8, 4096, 512, 2, 16), (8, 4096, 512, 2, 21), (8, 7168, 256, 1, 24),
                                          (8, 7168, 256, 4, 18), (8, 7168, 256, 2, 37), (16, 7168, 256, 1, 40), (256, 7168, 256, 1, 64), (8, 4096, 2048, 8, 5),
                                          (8, 4096, 2048, 2, 12)])
def test_aligned(e, h, i, topk, t):
    assert not _few(e, h, i, topk, t)
