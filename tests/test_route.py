"""Routing by scores without a GPU: every refusal of the C entry, and the oracle's pins."""
import ctypes
import math

import pytest
import torch

import bit_quantized_gemm_repack_amd as hq
from oracle import route as orr

GOOD = dict(t=4, experts=64, topk=4, type=hq.F32, logits=4096, scoring=hq.SCORE_SIGMOID, bias=8192, groups=8, group_topk=2,
            group_best=2, renorm=1, scale=1.0, ids=16384, w=32768)


def _call(**kw):
    a = dict(GOOD, **kw)
    return hq.lib().hq_route_experts(a["t"], a["experts"], a["topk"], a["type"], a["logits"], a["scoring"], a["bias"], a["groups"],
                                     a["group_topk"], a["group_best"], a["renorm"], ctypes.c_float(a["scale"]), a["ids"], a["w"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(type=hq.INT8), hq.HQ_ERR_UNSUPPORTED),
    (dict(scoring=2), hq.HQ_ERR_INVALID_ARG),
    (dict(t=-1), hq.HQ_ERR_INVALID_ARG),
    (dict(t=(1 << 24) + 1), hq.HQ_ERR_INVALID_ARG),
    (dict(experts=0), hq.HQ_ERR_INVALID_ARG),
    (dict(experts=1032), hq.HQ_ERR_UNSUPPORTED),
    (dict(groups=0), hq.HQ_ERR_INVALID_ARG),
    (dict(groups=7), hq.HQ_ERR_INVALID_ARG),
    (dict(experts=1024, groups=128, group_topk=64), hq.HQ_ERR_UNSUPPORTED),
    (dict(group_topk=0), hq.HQ_ERR_INVALID_ARG),
    (dict(group_topk=9), hq.HQ_ERR_INVALID_ARG),
    (dict(group_best=0), hq.HQ_ERR_INVALID_ARG),
    (dict(group_best=3), hq.HQ_ERR_INVALID_ARG),
    (dict(topk=0), hq.HQ_ERR_INVALID_ARG),
    (dict(topk=17), hq.HQ_ERR_INVALID_ARG),                       # two groups of 8
    (dict(topk=65, experts=1024), hq.HQ_ERR_INVALID_ARG),
    (dict(renorm=2), hq.HQ_ERR_INVALID_ARG),
    (dict(scale=float("inf")), hq.HQ_ERR_INVALID_ARG),
    (dict(scale=float("nan")), hq.HQ_ERR_INVALID_ARG),
    (dict(logits=None), hq.HQ_ERR_INVALID_ARG),
    (dict(ids=None), hq.HQ_ERR_INVALID_ARG),
    (dict(w=None), hq.HQ_ERR_INVALID_ARG),
    (dict(logits=4098), hq.HQ_ERR_INVALID_ARG),
    (dict(bias=8194), hq.HQ_ERR_INVALID_ARG),
    (dict(ids=16386), hq.HQ_ERR_INVALID_ARG),
    (dict(w=32769), hq.HQ_ERR_INVALID_ARG),
])
def test_refusals(kw, status):
    assert _call(**kw) == status
    assert hq.lib().hq_last_error()


def test_no_tokens():
    assert _call(t=0, logits=None, ids=None, w=None) == hq.HQ_OK


def test_python_refuses_cpu_tensors():
    with pytest.raises(ValueError, match="GPU"):
        hq.route_experts(torch.zeros(2, 8), 2)


def test_oracle_values():
    inf = math.inf
    x = torch.tensor([[0.0, 1.0, 0.0, -inf], [-inf, -inf, -inf, -inf], [5.0, 5.0, 5.0, float("nan")]])
    ids, w = orr.route(x, 2)
    assert ids.tolist() == [[1, 0], [-1, -1], [0, 1]]
    a, b = 1 / (1 + math.exp(-1)), 0.5
    assert torch.allclose(w[0], torch.tensor([a / (a + b), b / (a + b)], dtype=torch.float64), rtol=1e-7)
    assert w[1].tolist() == [0, 0] and w[2].tolist() == [0.5, 0.5]
    ids, w = orr.route(x[:1], 2, bias=torch.tensor([0.0, -1.0, 0.1, 9.0]), renormalize=False, scale=2.0)
    assert ids.tolist() == [[2, 0]] and w.tolist() == [[1.0, 1.0]]     # the bias chooses, the score weighs
    ids, _ = orr.route(torch.tensor([[3.0, -9.0, 2.0, 2.0]]), 2, groups=2, group_topk=1)
    assert ids.tolist() == [[2, 3]]                                   # two good ones beat one
    ids, _ = orr.route(torch.tensor([[3.0, -9.0, 2.0, 2.0]]), 2, groups=2, group_topk=1, group_best=1, scoring="softmax")
    assert ids.tolist() == [[0, 1]]


def test_native_call_takes_nothing_else():
    """What is no GPU tensor of the right kind is left to the Python checks."""
    hq.lib()
    if hq._calls is None:
        pytest.skip("the native calls are not built")
    x = torch.zeros(2, 8)
    for args in ((), (x,), (x, 2, None, 0, 1, 1, 2, True, 1.0), (x, 2, x, None, 1, 1, 2, True, 1.0), (3, 2, None, 0, 1, 1, 2, True, 1.0),
                 (x, 1 << 70, None, 0, 1, 1, 2, True, 1.0), (x, 2, None, 0, 1, 1, 1 << 70, True, 1.0), (x, 2, None, 0, 1, 1, 2, True, 1)):
        assert hq._calls.route_experts(*args) is None
