"""Down products of more slots than 32-bit addresses reach with a tile's 256 columns a row:
2^23 and more, from alignments of the caller's own (hq_moe_align makes up to 2^20)."""
import pytest
import torch

import bit_quantized_gemm_repack_amd as hq
from oracle import block8 as ob
from oracle import mx4 as om

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _room(gib):
    torch.cuda.empty_cache()
    free = torch.cuda.mem_get_info()[0]
    if free < gib * 2 ** 30:
        pytest.skip(f"needs {gib} GiB of device memory, {free / 2 ** 30:.0f} are free")


def _alignment(plan, t, topk):
    """Every slot in order, expert 0's, and a last block of no expert's: two slots of it."""
    bm, n = plan.block_m(t, topk), t * topk
    blocks = (n + 2 * (bm - 1) + bm - 1) // bm            # what one expert's alignment may take
    ids = torch.full((blocks * bm,), n, dtype=torch.int32, device=DEV)
    live = (n - 2 + bm - 1) // bm                         # blocks of expert 0
    ids[:n - 2] = torch.arange(n - 2, dtype=torch.int32, device=DEV)
    ids[live * bm:live * bm + 2] = torch.tensor([n - 2, n - 1], dtype=torch.int32, device=DEV)
    bex = torch.zeros(blocks, dtype=torch.int32, device=DEV)
    bex[live:] = -1
    return ids, bex, torch.tensor([(live + 1) * bm], dtype=torch.int32, device=DEV)


def _rows(g, rows, width):
    """Random bytes [rows, width], made in pieces."""
    a = torch.empty(rows, width, dtype=torch.uint8, device=DEV)
    for i in range(0, rows, 1 << 21):
        a[i:i + (1 << 21)] = torch.randint(0, 256, (min(1 << 21, rows - i), width), generator=g, dtype=torch.uint8, device=DEV)
    return a


def _picks(t):
    return sorted({0, 1, t - 1, t - 2} | {min(2 ** i // 64 + d, t - 1) for i in (20, 22, 23, 24) for d in (-1, 0, 1)})


def _check(y, o, to, w, last, dtype, what):
    """y = sum_j w_j o_j, the last two slots of the last token without an expert.  Beyond the
    products' bound: a slot's row in fp16, 64 additions (each 2^-24 of a partial sum, twice
    that for both forms), and the output's rounding."""
    p = w.double().unsqueeze(1).clone()
    if last:
        p[-2:] = 0
    want = (p * o).sum(0)
    tol = (p * (to + om.slot_rows_bound(o) + 2.0 ** -17 * o.abs())).sum(0)
    tol = tol + om.half_step(want.abs() + tol, dtype) + 1e-30
    off = (y.double() - want).abs()
    assert (off <= tol).all(), f"{what}: worst {float((off / tol).max()):.3g} of the bound"


@pytest.mark.parametrize("t,n", [((1 << 17) + 3, 320), ((1 << 17) - 1, 256)])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_fp8_block(t, n, dt):
    topk, k = 64, 128
    print(f"[gpu case] fp8 block down {t} x {topk} n {n} {dt}", flush=True)
    _room(24)
    g = torch.Generator(DEV)
    g.manual_seed(t)
    T = torch.bfloat16 if dt == "bf16" else torch.float16
    plan = hq.MoePlan(n, k, hq.w8a8_block(dt), 1, t, "topk_combine")
    codes = torch.randint(0, 120, (1, n, k), generator=g, dtype=torch.uint8, device=DEV) | (torch.randint(0, 2, (1, n, k), generator=g, dtype=torch.uint8, device=DEV) << 7)
    ws = torch.rand(1, (n + 127) // 128, 1, generator=g, device=DEV) * 1e-3 + 1e-4
    w = plan.repack(codes, ws)
    ids, bex, used = _alignment(plan, t, topk)
    a = _rows(g, ids.numel(), k) & 0xB7                   # magnitudes up to 0x37, finite
    sa = torch.rand(1, ids.numel(), generator=g, device=DEV) + 0.5
    tw = torch.rand(t, topk, generator=g, device=DEV)
    y = plan.moe_gemm(a, t, topk, ids, bex, used, *w, a_scale=sa, topk_w=tw)
    torch.cuda.synchronize()
    wf = ob.weight(codes[0].view(torch.float8_e4m3fn), ws[0])
    for i in _picks(t):
        slots = torch.arange(i * topk, (i + 1) * topk, device=DEV)
        o, to = ob.gemm(ob.rows(a[slots].view(torch.float8_e4m3fn), sa[:, slots].t()), wf)
        _check(y[i], o, to, tw[i], i == t - 1, T, f"token {i}")


@pytest.mark.parametrize("t,n", [((1 << 17) + 3, 320), ((1 << 18) + 1, 192)])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_mxfp4(t, n, dt):
    topk, k = 64, 128
    print(f"[gpu case] MXFP4 down {t} x {topk} n {n} {dt}", flush=True)
    _room(24)
    g = torch.Generator(DEV)
    g.manual_seed(t)
    T = torch.bfloat16 if dt == "bf16" else torch.float16
    plan = hq.MoePlan(n, k, hq.w4a4_mxfp4(dt), 1, t, "topk_combine")
    codes = torch.randint(0, 256, (1, n, k // 2), generator=g, dtype=torch.uint8, device=DEV)
    e = torch.randint(118, 124, (1, n, k // 32), generator=g, dtype=torch.uint8, device=DEV)
    w = plan.repack(codes, e8m0=e)
    ids, bex, used = _alignment(plan, t, topk)
    a = _rows(g, ids.numel(), k // 2)
    s = torch.randint(125, 129, (1, ids.numel(), 4), generator=g, dtype=torch.uint8, device=DEV)
    tw = torch.rand(t, topk, generator=g, device=DEV)
    y = plan.moe_gemm(a, t, topk, ids, bex, used, *w, a_scale=s, topk_w=tw)
    torch.cuda.synchronize()
    for i in _picks(t):
        slots = torch.arange(i * topk, (i + 1) * topk, device=DEV)
        o, to = om.gemm(om.rows(om.values(a[slots]), om.row_major(s[:, slots])), om.weight(codes[0], e[0]))
        _check(y[i], o, to, tw[i], i == t - 1, T, f"token {i}")
