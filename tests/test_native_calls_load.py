"""The native short calls are optional: a file that does not load, or was built
for another torch, costs a warning and leaves every call to ctypes."""
import os
import shutil
import subprocess
import sys

import pytest

import bit_quantized_gemm_repack_amd as hq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
USE = """
import warnings
import bit_quantized_gemm_repack_amd as hq
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    p = hq.Plan(256, 512, hq.w4a16("bf16"), max_m=4)
    q = hq.Plan(256, 512, hq.w8a8_block(), max_m=4)
print(p.describe(1), q.describe(1))
print("native", hq._calls is not None, "warned", [str(w.message) for w in seen if w.category is RuntimeWarning])
"""


def _package(tmp_path, calls):
    """The package in a folder of its own, with `calls` for its native part."""
    pkg = tmp_path / "bit_quantized_gemm_repack_amd"
    pkg.mkdir()
    (tmp_path / "include").symlink_to(os.path.join(ROOT, "include"))
    shutil.copy(os.path.join(ROOT, "bit_quantized_gemm_repack_amd", "__init__.py"), pkg)
    (pkg / "libhq.so").symlink_to(hq.LIB_PATH)
    if calls is not None:
        (pkg / "_calls.so").write_bytes(calls)
    return subprocess.run([sys.executable, "-c", USE], cwd=tmp_path, capture_output=True, text=True, timeout=300)


@pytest.mark.parametrize("kind", ["damaged", "cut short", "missing"])
def test_first_call_without_the_native_part(tmp_path, kind):
    hq.lib()
    if kind == "cut short" and not os.path.exists(hq.CALLS_PATH):
        pytest.skip("the native calls are not built")
    calls = {"damaged": b"\x7fELF damaged", "missing": None}.get(kind)
    if kind == "cut short":
        with open(hq.CALLS_PATH, "rb") as f:
            calls = f.read(4096)
    r = _package(tmp_path, calls)
    assert r.returncode == 0, r.stderr
    assert "kernel=" in r.stdout and "native False" in r.stdout
    assert ("is not used" in r.stdout) == (kind != "missing")


def test_native_part_of_another_torch_is_not_used(monkeypatch):
    L = hq.lib()
    if hq._calls is None:
        pytest.skip("the native calls are not built")
    native = hq._calls
    assert native.built_for == hq.torch.__version__
    monkeypatch.setattr(hq, "_calls", None)
    monkeypatch.setattr(hq.torch, "__version__", "0.0")
    with pytest.warns(RuntimeWarning, match="built for torch"):
        hq._bind_calls(L)
    assert hq._calls is None


def test_build_goes_on_without_the_native_part(tmp_path, monkeypatch):
    """No compiler for it, or headers that do not fit: a warning, and no file of an earlier build stays."""
    from bit_quantized_gemm_repack_amd import build as b
    monkeypatch.setattr(b, "CALLS", str(tmp_path / "_calls.so"))
    no_headers = subprocess.CompletedProcess([], 1, "", "fatal error: ATen/core/Tensor.h: No such file or directory")

    def no_compiler(*a, **kw):
        raise FileNotFoundError("g++")
    for run, what in ((no_compiler, r"g\+\+"), (lambda *a, **kw: no_headers, "Tensor.h")):
        (tmp_path / "_calls.so").write_bytes(b"old")
        monkeypatch.setattr(b.subprocess, "run", run)
        with pytest.warns(RuntimeWarning, match=what):
            assert b._build_calls_if_possible() is None
        assert not (tmp_path / "_calls.so").exists()
