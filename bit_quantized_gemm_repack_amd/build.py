"""Build the HIP library (libhq.so) in-tree for gfx950 with hipcc, and the
binding's native calls (_calls.so) with g++; where those do not compile the
build goes on without them, and the binding calls through ctypes.

Every source is compiled to an object in parallel, then linked into
``bit_quantized_gemm_repack_amd/libhq.so``.  HIP device code is built with
packed-FP32 instruction selection disabled (``-packed-fp32-ops``).
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libhq.so")
CALLS = os.path.join(PKG, "_calls.so")
ARCH = os.environ.get("HQ_OFFLOAD_ARCH", "gfx950")

HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
COMMON = ["-O3", "-std=c++20", "-fPIC", "-I", os.path.join(ROOT, "include"), "-Wno-unused-command-line-argument"]
DEVICE = [f"--offload-arch={ARCH}", "-mcode-object-version=5", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]
# Matrix-instruction results in ordinary VGPRs, so that the per-group
# epilogues read them without a v_accvgpr_read copy each; sources named
# *_f16.hip (an fp16 k loop without per-group epilogue) keep the default.
VGPR_FORM = ["-mllvm", "-amdgpu-mfma-vgpr-form=1"]
# hipRTC for the run-time specialised kernels (hq_plan_set_jit)
LINK = ["-lhiprtc", "-Wl,-z,defs"]  # every symbol resolved at link time


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".hip", ".cpp")))


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [HIPCC, *COMMON, "-c", src, "-o", obj]
    if src.endswith(".hip"):
        cmd[1:1] = DEVICE + ([] if src.endswith("_f16.hip") else VGPR_FORM)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def build_calls() -> str:
    """The binding's native short calls (csrc/binding/calls.cpp), host code
    against the installed torch."""
    import sysconfig

    import torch

    t = os.path.dirname(torch.__file__)
    tmp = CALLS + ".tmp"
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           "-D__HIP_PLATFORM_AMD__", "-DUSE_ROCM", f'-DHQ_TORCH_VERSION="{torch.__version__}"', f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", os.path.join(ROOT, "include"), "-isystem", os.path.join(t, "include"),
           "-isystem", os.path.join(t, "include", "torch", "csrc", "api", "include"), "-isystem", "/opt/rocm/include",
           "-isystem", sysconfig.get_paths()["include"], os.path.join(CSRC, "binding", "calls.cpp"), "-o", tmp,
           "-L", os.path.join(t, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_hip"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for calls.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALLS)
    return CALLS


def _build_calls_if_possible():
    """CALLS, or None with a warning.  One of an earlier build is taken away first:
    it may call the library otherwise than the headers now say."""
    if os.path.exists(CALLS):
        os.remove(CALLS)
    try:
        return build_calls()
    except Exception as e:
        warnings.warn(f"the native short calls are not built, calls go through ctypes: {e}", RuntimeWarning)
        return None


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources()
    with ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        calls = ex.submit(_build_calls_if_possible)
        objs = list(ex.map(_compile, srcs))
        calls = calls.result()
    tmp = LIB + ".tmp"
    cmd = [HIPCC, *DEVICE, "-shared", "-fPIC", "-o", tmp, *objs, *LINK]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}" + (f" and {calls}" if calls else ""), file=sys.stderr)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
