"""Row-wise operators on inputs whose launch has more work-items than one of its dimensions
holds (2^32): rows from the whole input against the same rows by themselves."""
import pytest
import torch

import bit_quantized_gemm_repack_amd as hq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _room(gib):
    torch.cuda.empty_cache()
    free = torch.cuda.mem_get_info()[0]
    if free < gib * 2 ** 30:
        pytest.skip(f"needs {gib} GiB of device memory, {free / 2 ** 30:.0f} are free")


def _parts(m, n):
    """Where to look: the start, the end, and either side of every power of two of rows, n rows each."""
    at = {0, m - n} | {min(max(0, 2 ** i - n // 2), m - n) for i in range(10, m.bit_length())}
    return sorted(at)


def _long_rows(m, k, dt, seed):
    """[m, k] contiguous, rows unlike each other, made in pieces."""
    g = torch.Generator(DEV)
    g.manual_seed(seed)
    base = torch.randn(1 << 20, generator=g, device=DEV).to(dt)
    x = torch.empty(m * k, dtype=dt, device=DEV)
    for i in range(0, m * k, 1 << 20):
        n = min(1 << 20, m * k - i)
        torch.mul(base[:n], 2.0 ** (i // (1 << 20) % 13 - 6), out=x[i:i + n])
    return x.view(m, k)


@pytest.mark.parametrize("m,k", [((1 << 24) - 3, 2176), ((1 << 17) + 5, 1 << 18)])
def test_quantize_mxfp4(m, k):
    """2^35 values and more; 2^36 are allowed."""
    print(f"[gpu case] quantize_mxfp4 {m} x {k}", flush=True)
    _room(100)
    x = _long_rows(m, k, torch.bfloat16, 1)
    codes, e = hq.quantize_mxfp4(x)
    torch.cuda.synchronize()
    for r in _parts(m, 8):
        c1, e1 = hq.quantize_mxfp4(x[r:r + 8].clone())
        assert torch.equal(codes[r:r + 8], c1) and torch.equal(e[:, r:r + 8], e1), f"rows from {r}"
    del x, codes, e
    torch.cuda.empty_cache()


@pytest.mark.parametrize("m,k,kind", [(1 << 24, 1152, "mxfp4"), ((1 << 23) + 1, 4224, "mxfp4"), ((1 << 22) + 3, 8320, "fp8_block"), ((1 << 22) + 1, 8200, "int8"),
                                      ((1 << 22) + 1, 16392, "fp8"), ((1 << 23) + 7, 4104, None)])
def test_rms_norm(m, k, kind):
    """Workgroups of 256, 512 and 1024 threads a row; the rows overlap in memory, eight elements apart.  In 16
    bits with a residual of one row for all."""
    print(f"[gpu case] rms_norm {m} x {k} {kind}", flush=True)
    _room(150)
    g = torch.Generator(DEV)
    g.manual_seed(2)
    base = torch.randn(8 * m + k, generator=g, device=DEV).bfloat16()
    x = base.as_strided((m, k), (8, 1))
    w = (1 + 0.1 * torch.randn(k, generator=g, device=DEV)).bfloat16()
    residual = None if kind else x.new_ones(k).expand(m, k)
    out = hq.rms_norm(x, w, out=kind, residual=residual)
    torch.cuda.synchronize()
    n = 300  # (few rows may be summed by other threads than many)
    for r in _parts(m, n):
        part = hq.rms_norm(x[r:r + n], w, out=kind, residual=None if kind else residual[r:r + n])
        for whole, one in zip(out, part):
            rows = whole[:, r:r + n] if kind in ("mxfp4", "fp8_block") and whole is out[1] else whole[r:r + n]
            assert torch.equal(rows, one), f"rows from {r}"
    del x, base, out, part, whole, one, rows
    torch.cuda.empty_cache()


@pytest.mark.parametrize("way,m,k", [("int8", 1 << 24, 1544), ("blocks", (1 << 24) - 3, 2176), ("blocks", (1 << 17) + 5, 1 << 18)])
def test_other_quantisers(way, m, k):
    print(f"[gpu case] quantize {way} {m} x {k}", flush=True)
    _room(130)
    f = (lambda v: hq.quantize_per_token(v, out="int8")) if way == "int8" else hq.quantize_blocks
    x = _long_rows(m, k, torch.float16, 3)
    codes, scale = f(x)
    torch.cuda.synchronize()
    for r in _parts(m, 260):
        c1, s1 = f(x[r:r + 260].clone())
        s = scale[r:r + 260] if scale.dim() == 1 else scale[:, r:r + 260]
        assert torch.equal(codes[r:r + 260], c1) and torch.equal(s, s1), f"rows from {r}"
    del x, codes, scale
    torch.cuda.empty_cache()
