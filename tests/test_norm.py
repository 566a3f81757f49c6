"""Root-mean-square norm without a GPU: every refusal of the C entry, and the oracle's
own pins (values that the mathematics fixes, codes planted a step off)."""
import ctypes

import pytest
import torch

import bit_quantized_gemm_repack_amd as hq
from oracle import norm as on

GOOD = dict(m=4, k=256, x_type=hq.BF16, x=4096, x_stride=256, r=8192, r_stride=256, w_type=hq.BF16, w=4096, eps=1e-6,
            kind=hq.NORM_FP8_BLOCK, h=8192, h_stride=256, out=16384, scale=32768)


def _call(**kw):
    a = dict(GOOD, **kw)
    return hq.lib().hq_rms_norm(a["m"], a["k"], a["x_type"], a["x"], a["x_stride"], a["r"], a["r_stride"], a["w_type"], a["w"],
                                ctypes.c_float(a["eps"]), a["kind"], a["h"], a["h_stride"], a["out"], a["scale"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(x_type=hq.F32), hq.HQ_ERR_UNSUPPORTED),
    (dict(w_type=hq.F16), hq.HQ_ERR_UNSUPPORTED),
    (dict(kind=5), hq.HQ_ERR_INVALID_ARG),
    (dict(kind=-1), hq.HQ_ERR_INVALID_ARG),
    (dict(m=-1), hq.HQ_ERR_INVALID_ARG),
    (dict(m=(1 << 24) + 1), hq.HQ_ERR_INVALID_ARG),
    (dict(k=0), hq.HQ_ERR_INVALID_ARG),
    (dict(k=252, kind=hq.NORM_FP8), hq.HQ_ERR_INVALID_ARG),
    (dict(k=136), hq.HQ_ERR_INVALID_ARG),                       # blocks of 128
    (dict(k=136, kind=hq.NORM_MXFP4), hq.HQ_ERR_INVALID_ARG),
    (dict(k=65664, x_stride=65664, r_stride=65664, h_stride=65664), hq.HQ_ERR_UNSUPPORTED),
    (dict(eps=-1e-6), hq.HQ_ERR_INVALID_ARG),
    (dict(eps=float("nan")), hq.HQ_ERR_INVALID_ARG),
    (dict(eps=float("inf")), hq.HQ_ERR_INVALID_ARG),
    (dict(x=None), hq.HQ_ERR_INVALID_ARG),
    (dict(w=None), hq.HQ_ERR_INVALID_ARG),
    (dict(out=None), hq.HQ_ERR_INVALID_ARG),
    (dict(r=None), hq.HQ_ERR_INVALID_ARG),                      # h without a residual
    (dict(h=None), hq.HQ_ERR_INVALID_ARG),
    (dict(scale=None), hq.HQ_ERR_INVALID_ARG),
    (dict(kind=hq.NORM_SAME), hq.HQ_ERR_INVALID_ARG),           # a scale without codes
    (dict(x_stride=260), hq.HQ_ERR_INVALID_ARG),
    (dict(x_stride=-256), hq.HQ_ERR_INVALID_ARG),
    (dict(r_stride=260), hq.HQ_ERR_INVALID_ARG),
    (dict(h_stride=248), hq.HQ_ERR_INVALID_ARG),                # rows of h overlap
    (dict(x=4104), hq.HQ_ERR_INVALID_ARG),
    (dict(w=4100), hq.HQ_ERR_INVALID_ARG),
    (dict(out=16392), hq.HQ_ERR_INVALID_ARG),
    (dict(scale=32772), hq.HQ_ERR_INVALID_ARG),
    (dict(h=8200), hq.HQ_ERR_INVALID_ARG),
])
def test_refusals(kw, status):
    assert _call(**kw) == status
    assert hq.lib().hq_last_error()


def test_no_rows():
    assert _call(m=0, x=None, r=None, w=None, out=None, h=None, scale=None) == hq.HQ_OK


def test_python_refuses_cpu_tensors():
    with pytest.raises(ValueError, match="GPU"):
        hq.rms_norm(torch.zeros(2, 128, dtype=torch.bfloat16), torch.ones(128, dtype=torch.bfloat16))


def test_oracle_values():
    x = torch.tensor([[3.0, -4.0] * 64, [0.0] * 128], dtype=torch.bfloat16)
    w = torch.full((128,), 2.0)
    _, y = on.norm(x, w, 0.5)
    assert torch.allclose(y[0, :2], torch.tensor([6.0, -8.0], dtype=torch.float64) / 13 ** 0.5, rtol=1e-15)
    assert (y[1] == 0).all()
    r = torch.full((2, 128), 2.0 ** -9, dtype=torch.bfloat16)
    h, _ = on.norm(x, w, 0.5, r)                     # 3 + 2^-9 rounds to 3, 0 + 2^-9 stays
    assert h[0, 0] == 3 and h[1, 0] == 2.0 ** -9


def test_oracle_sees_a_step():
    g = torch.Generator().manual_seed(1)
    y = torch.randn(4, 256, generator=g, dtype=torch.float64)
    s = on.block_top(y, 128) / 448
    v = (y / s.repeat_interleave(128, -1)).float().to(torch.float8_e4m3fn)
    assert (on.off_scaled(v.double(), s, y, 128, 448.0, on.half_step8) <= 1).all()
    worse = (v.view(torch.uint8) + 1).view(torch.float8_e4m3fn).double()
    assert (on.off_scaled(worse, s, y, 128, 448.0, on.half_step8) > 1).float().mean() > 0.9
    assert (on.off_scale(s * (1 + 1e-5), y, 128, 448.0) > 1).all()
    lo, hi = on.e8m0_may_be(torch.tensor([[1.0] + [0.0] * 31, [1.5] + [0.0] * 31, [0.0] * 32], dtype=torch.float64))
    assert lo.flatten().tolist() == [124, 125, 127] and hi.flatten().tolist() == [125, 125, 127]


def test_oracle_values4():
    assert on.values4(torch.tensor([[0x21, 0xF8]], dtype=torch.uint8)).tolist() == [[0.5, 1.0, -0.0, -6.0]]


def test_native_call_takes_nothing_else():
    """What is no GPU tensor of the right kind is left to the Python checks."""
    hq.lib()
    if hq._calls is None:
        pytest.skip("the native calls are not built")
    x, w = torch.zeros(2, 256, dtype=torch.bfloat16), torch.zeros(256)
    for args in ((), (x,), (None, w, 1e-6, None, 0, None), (x, w, 1e-6, None, 0, None), (x, w, 1, None, 0, None), (x, w, 1e-6, None, None, None),
                 (x, w, 1e-6, None, 1 << 70, None), ("x", "w", 1e-6, 3, 0, 4)):
        assert hq._calls.rms_norm(*args) is None
