"""Tunings of fp8 block plans: a zero field is the library's choice, so a tuning
that some kernel has runs at every number of rows, with the fields that were
given, and one that none has is refused when the plan is made."""
import itertools

import pytest

import bit_quantized_gemm_repack_amd as hq

SHAPES = [(4096, 7168), (576, 7168), (14336, 4096), (1024, 1024), (24576, 1536), (48, 128)]
ROWS = [1, 2, 15, 16, 17, 32, 33, 40, 64, 65, 100, 128, 129, 200, 256, 300, 512, 1000, 2048, 4096]
VALUES = dict(kernel=(1, 2), tile_m=(16, 32, 64, 128, 256), tile_n=(16, 32, 64, 128, 256), waves=(1, 4, 8, 9), split_k=(1, 3, 64),
              stages=(2, 3, 4), tile_group=(1, 64, 65))


def _exists(t):
    """Whether a kernel has the shape that the given fields name."""
    skinny = t.get("kernel") != 2 and t.get("tile_m", 16) == 16 and t.get("tile_n", 16) in (16, 32) and t.get("waves", 4) <= 8
    shapes = [(16, 128, 4), (32, 128, 4), (64, 128, 3), (128, 128, 2), (128, 256, 2)]
    tiled = t.get("kernel") != 1 and t.get("tile_group", 8) <= 64 and any(
        t.get("tile_m", bm) == bm and t.get("tile_n", bn) == bn and t.get("stages", st) == st for bm, bn, st in shapes)
    return skinny, tiled


def _tunings():
    names = list(VALUES)
    for n in (1, 2, 3):
        for fields in itertools.combinations(names, n):
            for values in itertools.product(*(VALUES[f] for f in fields)):
                yield dict(zip(fields, values))


@pytest.mark.parametrize("n,k", SHAPES)
def test_every_partial_tuning_runs_or_is_refused(n, k):
    for t in _tunings():
        skinny, tiled = _exists(t)
        if not skinny and not tiled or t.get("waves", 1) > 8 or t.get("tile_group", 1) > 64:
            for max_m in (1, 64, 4096):
                with pytest.raises(hq.HQError):
                    hq.Plan(n, k, hq.w8a8_block(), max_m=max_m, tuning=t, fallback=False)
            continue
        plan = hq.Plan(n, k, hq.w8a8_block(), max_m=4096, tuning=t, fallback=False)
        fields = [f for f in ("kernel", "tile_m", "tile_n") if f in t]
        for m in ROWS:
            got, _ = plan.get_tuning(m)
            assert [got[f] for f in fields] == [t[f] for f in fields], (t, m, got)
            if got["kernel"] == 1:
                assert skinny and got["tile_m"] == 16 and got["tile_n"] in (16, 32) and 1 <= got["waves"] <= 8, (t, m, got)
                assert "waves" not in t or got["waves"] == t["waves"]
            else:
                assert tiled and (got["tile_m"], got["tile_n"], got["stages"]) in \
                    [(16, 128, 4), (32, 128, 4), (64, 128, 3), (128, 128, 2), (128, 256, 2)], (t, m, got)
                assert "stages" not in t or got["stages"] == t["stages"]
            plan.set_tuning(m, got)                  # a complete shape that the library accepts


def test_no_tuning_is_as_before():
    """The library's own choices at sizes that its comments give times for."""
    pick = lambda n, k, m: hq.Plan(n, k, hq.w8a8_block(), max_m=4096).get_tuning(m)[0]
    shape = lambda n, k, m: tuple(pick(n, k, m)[f] for f in ("kernel", "tile_m", "tile_n", "split_k"))
    assert shape(4096, 7168, 1) == (1, 16, 16, 1) and shape(576, 7168, 33) == (1, 16, 16, 1)
    assert shape(14336, 4096, 200) == (2, 64, 128, 1) and shape(4096, 7168, 4096) == (2, 128, 256, 1)
    assert shape(4096, 7168, 128) == (2, 64, 128, 4) and shape(576, 7168, 200) == (2, 32, 128, 4)
