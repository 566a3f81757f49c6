"""Python binding of the MI355X quantized GEMM library (libhq.so).

Argument marshalling only: every step of the computation runs in the HIP
kernels behind the C ABI declared in ``include/hq.h``.  PyTorch supplies the
device memory (tensors) and the stream (the current HIP stream); there is no
CPU fallback, and every entry point raises if the library is not built or a
tensor is not on the GPU.  The short calls of the fp8 block layers go through
native code where it is built (csrc/binding/calls.cpp).

Quick use::

    import bit_quantized_gemm_repack_amd as hq
    plan = hq.Plan(n=4096, k=4096, quant=hq.w4a16(act="bf16", zp="u4"), max_m=64)
    w, meta = plan.repack(codes, scales, zeros)        # canonical -> device layout
    out = plan.gemm(a, w, meta)                         # [m, n] bf16
"""
from __future__ import annotations

import ctypes
import importlib
import json
import os
import re
import warnings
from dataclasses import dataclass
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libhq.so")
CALLS_PATH = os.path.join(_HERE, "_calls.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "hq.h")

# ------------------------------------------------------------------ enums --
HQ_OK, HQ_ERR_INVALID_ARG, HQ_ERR_UNSUPPORTED, HQ_ERR_WORKSPACE, HQ_ERR_HIP, HQ_ERR_INTERNAL = range(6)
F16, BF16, F32, FP8_E4M3, INT8, U4, FP4_E2M1, E8M0, I32, U8, U2, U3, I4 = range(13)
ZP_NONE, ZP_FIXED, ZP_PER_GROUP_U4 = range(3)
ASCALE_NONE, ASCALE_PER_TOKEN_F32, ASCALE_MX_E8M0, ASCALE_BLOCK_F32 = range(4)
GEMM_DENSE, GEMM_GROUPED = range(2)
EPI_NONE, EPI_SILU_MUL, EPI_SILU_MUL_QFP8, EPI_TOPK_COMBINE, EPI_I32_ACC = range(5)
PEAK_F16, PEAK_BF16, PEAK_FP8, PEAK_FP8_FP4, PEAK_FP4, PEAK_INT8 = range(6)
MFMA_AUTO, MFMA_F16, MFMA_BF16, MFMA_FP8, MFMA_INT8, MFMA_FP8_FP4, MFMA_FP4 = range(7)
_MFMA = {None: MFMA_AUTO, "auto": MFMA_AUTO, "f16": MFMA_F16, "bf16": MFMA_BF16, "fp8": MFMA_FP8,
         "int8": MFMA_INT8, "fp8xfp4": MFMA_FP8_FP4, "fp4": MFMA_FP4}

_DT = {"f16": F16, "bf16": BF16, "fp8": FP8_E4M3, "int8": INT8}
_EPI = {"none": EPI_NONE, "silu_mul": EPI_SILU_MUL, "silu_mul_qfp8": EPI_SILU_MUL_QFP8,
        "topk_combine": EPI_TOPK_COMBINE, "i32_acc": EPI_I32_ACC}


class HQError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{_status_name(status)}: {msg}")
        self.status = status


def _status_name(s: int) -> str:
    names = ["HQ_OK", "HQ_ERR_INVALID_ARG", "HQ_ERR_UNSUPPORTED", "HQ_ERR_WORKSPACE", "HQ_ERR_HIP",
             "HQ_ERR_INTERNAL"]
    return names[s] if 0 <= s < len(names) else f"HQ_ERR_{s}"


# ------------------------------------------------------------- structures --
class QuantDesc(ctypes.Structure):
    _fields_ = [("w_elem", ctypes.c_int), ("w_bits", ctypes.c_int), ("group_size", ctypes.c_int),
                ("scale", ctypes.c_int), ("zp", ctypes.c_int), ("zp_value", ctypes.c_int),
                ("act", ctypes.c_int), ("act_scale", ctypes.c_int), ("out", ctypes.c_int)]


class LayerDesc(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("k", ctypes.c_int64), ("num_experts", ctypes.c_int),
                ("q", QuantDesc)]


class Compute(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("epi", ctypes.c_int), ("mfma_in", ctypes.c_int)]


class Tuning(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int), ("tile_m", ctypes.c_int), ("tile_n", ctypes.c_int),
                ("waves", ctypes.c_int), ("split_k", ctypes.c_int), ("stages", ctypes.c_int),
                ("mfma", ctypes.c_int), ("tile_group", ctypes.c_int)]


class JitStats(ctypes.Structure):
    _fields_ = [("compiles", ctypes.c_int64), ("disk_hits", ctypes.c_int64), ("memory_hits", ctypes.c_int64),
                ("launches", ctypes.c_int64), ("compile_seconds", ctypes.c_double), ("load_seconds", ctypes.c_double)]


class AutotuneResult(ctypes.Structure):
    _fields_ = [("best", Tuning), ("best_us", ctypes.c_float), ("current_us", ctypes.c_float),
                ("candidates", ctypes.c_int)]


_TUNING_FIELDS = ("kernel", "tile_m", "tile_n", "waves", "split_k", "stages", "tile_group")


def _tuning_dict(t: Tuning) -> dict:
    return {f: int(getattr(t, f)) for f in _TUNING_FIELDS}


def w4a16(act: str = "f16", scale: Optional[str] = None, zp="fixed", zp_value: int = 8,
          out: Optional[str] = None) -> QuantDesc:
    """INT4 (group 128) weights x fp16/bf16 activations.  zp: 'fixed' or 'u4'."""
    return QuantDesc(U4, 4, 128, _DT[scale or act], ZP_FIXED if zp == "fixed" else ZP_PER_GROUP_U4,
                     zp_value, _DT[act], ASCALE_NONE, _DT[out or act])


def w8a16(act: str = "f16", scale: Optional[str] = None, zp_value: int = 128, out: Optional[str] = None) -> QuantDesc:
    """INT8 (group 128, fixed zero point) weights x fp16/bf16 activations; codes
    are uint8 [N, K], one byte per weight."""
    return QuantDesc(U8, 8, 128, _DT[scale or act], ZP_FIXED, zp_value, _DT[act], ASCALE_NONE, _DT[out or act])


def w2a16(act: str = "f16", scale: Optional[str] = None, zp_value: int = 2, out: Optional[str] = None) -> QuantDesc:
    """INT2 (group 128, fixed zero point) weights x fp16/bf16 activations; codes
    are int32 [N, K/16], sixteen 2-bit codes per word, lowest bits first."""
    return QuantDesc(U2, 2, 128, _DT[scale or act], ZP_FIXED, zp_value, _DT[act], ASCALE_NONE, _DT[out or act])


def w3a16(act: str = "f16", scale: Optional[str] = None, zp_value: int = 4, out: Optional[str] = None) -> QuantDesc:
    """INT3 (group 128, fixed zero point) weights x fp16/bf16 activations; codes
    are int32 [N, 3K/32], the dense 3-bit packing of GPTQ INT3 along K (each
    row one little-endian bit stream, code k in bits [3k, 3k+3))."""
    return QuantDesc(U3, 3, 128, _DT[scale or act], ZP_FIXED, zp_value, _DT[act], ASCALE_NONE, _DT[out or act])


def w4a16_mxint4(act: str = "bf16", out: Optional[str] = None) -> QuantDesc:
    """MXINT4 weights (two's-complement 4-bit codes times 2^-2, one E8M0 scale
    per 32 k; codes packed as INT4, scales uint8 [N, K/32]) x fp16/bf16
    activations."""
    return QuantDesc(I4, 4, 32, E8M0, ZP_NONE, 0, _DT[act], ASCALE_NONE, _DT[out or act])


def w4a16_nvfp4(act: str = "bf16", out: Optional[str] = None) -> QuantDesc:
    """NVFP4 weights (E2M1 codes packed as INT4, one E4M3 scale per 16 k as
    uint8 [N, K/16], one fp32 tensor scale) x fp16/bf16 activations.  Repack
    with scales = the tensor scale (float32 [1], or [E] for stacked weights)
    and e8m0 = the E4M3 block scales."""
    return QuantDesc(FP4_E2M1, 4, 16, FP8_E4M3, ZP_NONE, 0, _DT[act], ASCALE_NONE, _DT[out or act])


def w4a8_int(scale: str = "f16", out: str = "bf16") -> QuantDesc:
    """INT4 (group 128, zero 8) weights x int8 per-token activations."""
    return QuantDesc(U4, 4, 128, _DT[scale], ZP_FIXED, 8, INT8, ASCALE_PER_TOKEN_F32, _DT[out])


def w4a8_fp8(scale: str = "f16", zp="fixed", zp_value: int = 8, out: str = "bf16") -> QuantDesc:
    """INT4 (group 128) weights x fp8 e4m3 per-token activations."""
    return QuantDesc(U4, 4, 128, _DT[scale], ZP_FIXED if zp == "fixed" else ZP_PER_GROUP_U4, zp_value,
                     FP8_E4M3, ASCALE_PER_TOKEN_F32, _DT[out])


def w4a8_mxfp4(out: str = "bf16") -> QuantDesc:
    """MXFP4 (E2M1 + E8M0 per 32) weights x fp8 e4m3 per-token activations."""
    return QuantDesc(FP4_E2M1, 4, 32, E8M0, ZP_NONE, 0, FP8_E4M3, ASCALE_PER_TOKEN_F32, _DT[out])


def w4a4_mxfp4(out: str = "bf16") -> QuantDesc:
    """MXFP4 weights x MXFP4 activations (E2M1 codes packed two per byte along
    K; E8M0 block scales passed as a_scale in the group-major layout
    [K/128, m, 4], see mx_scales_group_major)."""
    return QuantDesc(FP4_E2M1, 4, 32, E8M0, ZP_NONE, 0, FP4_E2M1, ASCALE_MX_E8M0, _DT[out])


def w8a8_block(out: str = "bf16") -> QuantDesc:
    """fp8 e4m3 weights with one fp32 scale per 128 x 128 x fp8 e4m3 activations
    with one fp32 scale per row and 128 k.  Repack takes codes uint8 (or
    float8_e4m3fn) [N, K] and scales float32 [ceil(N/128), K/128] (stacked
    [E, ...] for a grouped plan); a_scale is float32 [K/128, m], as
    quantize_blocks writes it."""
    return QuantDesc(FP8_E4M3, 8, 128, F32, ZP_NONE, 0, FP8_E4M3, ASCALE_BLOCK_F32, _DT[out])


# ---------------------------------------------------------------- library --
_lib = None

_SIGS = {
    "hq_abi_version": (ctypes.c_int, []),
    "hq_status_str": (ctypes.c_char_p, [ctypes.c_int]),
    "hq_last_error": (ctypes.c_char_p, []),
    "hq_plan_create": (ctypes.c_int, [ctypes.POINTER(LayerDesc), ctypes.POINTER(Compute), ctypes.c_int64,
                                      ctypes.POINTER(Tuning), ctypes.POINTER(ctypes.c_void_p)]),
    "hq_plan_destroy": (ctypes.c_int, [ctypes.c_void_p]),
    "hq_plan_describe": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_char_p, ctypes.c_size_t]),
    "hq_plan_workspace_bytes": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64,
                                               ctypes.POINTER(ctypes.c_size_t)]),
    "hq_repacked_bytes": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(ctypes.c_size_t),
                                         ctypes.POINTER(ctypes.c_size_t)]),
    "hq_repack": (ctypes.c_int, [ctypes.c_void_p] + [ctypes.c_void_p] * 5 + [ctypes.c_void_p]),
    "hq_repack_host": (ctypes.c_int, [ctypes.c_void_p] + [ctypes.c_void_p] * 5),
    "hq_time_next_launch": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]),
    "hq_moe_block_m": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.POINTER(ctypes.c_int)]),
    "hq_moe_max_padded": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                         ctypes.POINTER(ctypes.c_int64)]),
    "hq_moe_align": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int] +
                     [ctypes.c_void_p] * 5),
    "hq_moe_workspace_bytes": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int,
                                              ctypes.POINTER(ctypes.c_size_t)]),
    "hq_moe_gemm": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int] + [ctypes.c_void_p] * 11 +
                    [ctypes.c_size_t, ctypes.c_void_p]),
    "hq_moe_gemm_by_slot": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int] + [ctypes.c_void_p] * 9 +
                            [ctypes.c_size_t, ctypes.c_void_p]),
    "hq_stream_read": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_int,
                                      ctypes.c_void_p]),
    "hq_mfma_peak": (ctypes.c_int, [ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_void_p,
                                    ctypes.POINTER(ctypes.c_double), ctypes.c_void_p]),
    "hq_quantize_per_token": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_int] +
                              [ctypes.c_void_p] * 4),
    "hq_quantize_mxfp4": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int] + [ctypes.c_void_p] * 4),
    "hq_route_topk": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_void_p,
                                     ctypes.c_int] + [ctypes.c_void_p] * 3),
    "hq_moe_few_workspace_bytes": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int,
                                                  ctypes.POINTER(ctypes.c_size_t)]),
    "hq_moe_layer_few": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                                        ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_int] +
                         [ctypes.c_void_p] * 8 + [ctypes.c_size_t, ctypes.c_void_p]),
    "hq_quantize_blocks": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_int] +
                           [ctypes.c_void_p] * 4),
    "hq_plan_autotune": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64] + [ctypes.c_void_p] * 6 +
                         [ctypes.c_size_t, ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p,
                          ctypes.POINTER(AutotuneResult)]),
    "hq_plan_set_tuning": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(Tuning)]),
    "hq_plan_get_tuning": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(Tuning),
                                          ctypes.POINTER(ctypes.c_int)]),
    "hq_gemm": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
                               ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                               ctypes.c_size_t, ctypes.c_void_p]),
    "hq_gemm_noalloc": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64] + [ctypes.c_void_p] * 5 +
                        [ctypes.c_void_p]),
    "hq_plan_set_jit": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_char_p]),
    "hq_jit_cache_key": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_char_p, ctypes.c_char_p,
                                        ctypes.c_size_t]),
    "hq_jit_get_stats": (ctypes.c_int, [ctypes.POINTER(JitStats)]),
    "hq_jit_prepare": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_char_p]),
}


def jit_stats() -> dict:
    """Counters of the run-time specialisation since the library was loaded
    (hq_jit_get_stats)."""
    st = JitStats()
    _check(lib().hq_jit_get_stats(ctypes.byref(st)))
    return {f: getattr(st, f) for f, _ in JitStats._fields_}


def lib():
    """Load libhq.so (built in-tree by ``__graft_entry__.build()``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run __graft_entry__.build() first")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
        _bind_calls(L)
    return _lib


# The native form of the short calls (csrc/binding/calls.cpp), once the library
# is loaded and if it is built and loads with this torch; it answers None to
# anything but the ordinary call, which the Python below then checks.
_calls = None


def _whole(path: str) -> bool:
    """Whether an ELF file is as long as its header says: mapping one that was cut
    short ends the process instead of raising."""
    with open(path, "rb") as f:
        h = f.read(64)
    if len(h) < 64 or h[:4] != b"\x7fELF":
        return False
    at = int.from_bytes(h[40:48], "little")           # the section table, which comes last
    size, count = (int.from_bytes(h[i:i + 2], "little") for i in (58, 60))
    return os.path.getsize(path) >= at + size * count


def _bind_calls(L):
    global _calls
    if not os.path.exists(CALLS_PATH):
        return
    try:
        if not _whole(CALLS_PATH):
            raise ImportError("the file is cut short")
        native = importlib.import_module("._calls", __package__)
        if native.built_for != torch.__version__:
            raise ImportError(f"built for torch {native.built_for}, this is {torch.__version__}")
        native.bind(*(ctypes.cast(f, ctypes.c_void_p).value
                      for f in (L.hq_quantize_blocks, L.hq_route_topk, L.hq_gemm, L.hq_plan_workspace_bytes)))
    except Exception as e:  # a damaged file, another torch's: every call works without it
        warnings.warn(f"{CALLS_PATH} is not used ({e}): short calls go through ctypes; build again to have it", RuntimeWarning)
        return
    _calls = native


def header_functions(path: str = HEADER_PATH):
    """Names of the functions declared in include/hq.h."""
    text = open(path).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[A-Za-z_][A-Za-z0-9_]*\s*\**\s*(hq_[a-z0-9_]+)\s*\(",
                                 text, flags=re.M)))


def _check(status: int):
    if status != HQ_OK:
        raise HQError(status, lib().hq_last_error().decode())


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _dev(t: torch.Tensor, name: str):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _stream_ptr(device) -> int:
    """The current stream of `device` (the raw handle: a Stream object costs
    more than the rest of a small call)."""
    return torch._C._cuda_getCurrentRawStream(device.index if device.index is not None else torch.cuda.current_device())


class _on:
    """Makes `device` current where it is not (a launch goes to the current
    device, its stream to the tensors')."""
    __slots__ = ("index", "was")

    def __init__(self, device):
        self.index = device.index

    def __enter__(self):
        self.was = torch.cuda.current_device()
        if self.was != self.index:
            torch.cuda.set_device(self.index)

    def __exit__(self, *exc):
        if self.was != self.index:
            torch.cuda.set_device(self.was)


def _run(dev, fn, *args):
    """fn(*args, dev's current stream) with dev current."""
    i = dev.index
    if torch._C._cuda_getDevice() == i:
        status = fn(*args, torch._C._cuda_getCurrentRawStream(i))
    else:
        with _on(dev):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(i))
    if status != HQ_OK:
        _check(status)


def _same_device(dev, *tensors) -> bool:
    """All contiguous tensors on dev, a GPU (the quick form of _dev's checks)."""
    for t in tensors:
        if not isinstance(t, torch.Tensor) or t.device != dev or not t.is_contiguous():
            return False
    return dev.type == "cuda"


def _block_ws(ws, dev):
    """A given workspace of a block-scaled call: the kernels write it."""
    if ws is not None and not _same_device(dev, ws):
        raise ValueError("ws must be contiguous and on the inputs' device")


_TORCH_OUT = {F16: torch.float16, BF16: torch.bfloat16}
# What may hold e4m3 codes: the type itself, or raw bytes (not another fp8 type's)
_E4M3 = (torch.uint8, torch.int8, torch.float8_e4m3fn)
_LOGITS = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
_DT_NAME = {F16: "f16", BF16: "bf16", FP8_E4M3: "fp8", INT8: "int8", FP4_E2M1: "mxfp4"}


# ------------------------------------------------------------------ plan --
def _as16(q: QuantDesc) -> QuantDesc:
    """The same weights with 16-bit activations (the output dtype's type)."""
    act = q.out if q.out in (F16, BF16) else BF16
    return QuantDesc(q.w_elem, q.w_bits, q.group_size, q.scale, q.zp, q.zp_value, act, ASCALE_NONE, q.out)


class Plan:
    """A layer description + execution choice (owns an hq_plan).

    mfma_in names the matrix-instruction operand type ('f16', 'bf16', 'fp8',
    'int8', 'fp8xfp4', 'fp4'; None: the description's).  When the library
    cannot run the description (HQ_ERR_UNSUPPORTED) and its activations are 8-
    or 4-bit, the plan is built again for the same weights with 16-bit
    activations -- the pages' fallback to a higher-precision compute type
    (Humming page on news.ditty.ir, summary) -- unless fallback=False.  Then
    `fallback` holds the reason, `quant` the description that runs and
    `requested_quant` the one asked for; `linear` takes 16-bit activations
    either way."""

    def __init__(self, n: int, k: int, quant: QuantDesc, max_m: int, epi: str = "none",
                 kind: str = "dense", num_experts: int = 1, tuning: Optional[dict] = None,
                 mfma_in: Optional[str] = None, fallback: bool = True):
        L = lib()
        self.n, self.k, self.max_m, self.num_experts = int(n), int(k), int(max_m), int(num_experts)
        self.requested_quant = quant
        self.quant = quant
        self.fallback = None
        self.epi = _EPI[epi]
        if mfma_in not in _MFMA:
            raise ValueError(f"mfma_in must be one of {sorted(k for k in _MFMA if k)}")
        tun = None
        if tuning:
            tun = Tuning(**{key: int(v) for key, v in tuning.items()})

        def create(q, mi):
            layer = LayerDesc(self.n, self.k, self.num_experts, q)
            comp = Compute(GEMM_DENSE if kind == "dense" else GEMM_GROUPED, self.epi, mi)
            h = ctypes.c_void_p()
            _check(L.hq_plan_create(ctypes.byref(layer), ctypes.byref(comp), self.max_m,
                                    ctypes.byref(tun) if tun is not None else None, ctypes.byref(h)))
            return h

        try:
            handle = create(quant, _MFMA[mfma_in])
        except HQError as e:
            if not fallback or e.status != HQ_ERR_UNSUPPORTED or quant.act in (F16, BF16) or \
                    self.epi == EPI_I32_ACC:
                raise
            q16 = _as16(quant)
            try:
                handle = create(q16, MFMA_AUTO)
            except HQError:
                raise e from None
            self.quant = q16
            self.fallback = (f"{_DT_NAME.get(quant.act, quant.act)} activations requested: {e}; running "
                             f"{_DT_NAME[q16.act]} activations")
        self._h = handle
        self._block8 = self.quant.act_scale == ASCALE_BLOCK_F32
        self._ws_need = {}  # rows -> workspace bytes of a block-scaled GEMM
        self._few_need = {}  # (tokens, topk, down's k) -> workspace bytes of a layer of a few tokens
        self._ws = {}
        self._act_buf = {}

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value and _lib is not None:
            _lib.hq_plan_destroy(h)
            self._h = None

    # -- sizes ----------------------------------------------------------
    def repacked_bytes(self):
        w, m = ctypes.c_size_t(), ctypes.c_size_t()
        _check(lib().hq_repacked_bytes(self._h, ctypes.byref(w), ctypes.byref(m)))
        return w.value, m.value

    def workspace_bytes(self, m: int) -> int:
        b = ctypes.c_size_t()
        _check(lib().hq_plan_workspace_bytes(self._h, int(m), ctypes.byref(b)))
        return b.value

    def describe(self, m: int) -> str:
        buf = ctypes.create_string_buffer(512)
        _check(lib().hq_plan_describe(self._h, int(m), buf, 512))
        d = buf.value.decode()
        return d if self.fallback is None else f"{d} fallback=16-bit-activations ({self.fallback})"

    def workspace(self, m: int, device) -> Optional[torch.Tensor]:
        """A zero-initialised workspace kept per device (reused across calls;
        the kernels leave it ready for the next call on the same stream)."""
        need = self.workspace_bytes(m)
        if need == 0:
            return None
        dev = torch.device(device)
        ws = self._ws.get(dev)
        if ws is None or ws.numel() < need:
            ws = torch.zeros(max(need, 256), dtype=torch.uint8, device=dev)
            self._ws[dev] = ws
        return ws

    # -- repack ---------------------------------------------------------
    def _check_block_weight(self, codes, scales):
        if not self._block8:
            return
        # by shape: [k, n] codes, or scales of [k/128, n/128], hold as many values
        if codes.dtype not in _E4M3 or codes.shape[-2:] != (self.n, self.k) or \
                codes.numel() != self.num_experts * self.n * self.k:
            raise ValueError(f"codes must hold {self.num_experts} x [{self.n}, {self.k}] e4m3 codes (or their bytes)")
        blocks = (-(-self.n // 128), self.k // 128)
        if scales is None or scales.dtype != torch.float32 or scales.shape[-2:] != blocks or \
                scales.numel() != self.num_experts * blocks[0] * blocks[1]:
            raise ValueError(f"scales must be float32, {self.num_experts} x [{blocks[0]}, {blocks[1]}]")

    def _repack_outputs(self, device):
        wb, mb = self.repacked_bytes()
        w = torch.empty(wb, dtype=torch.uint8, device=device)
        meta = torch.empty(max(mb, 16), dtype=torch.uint8, device=device)
        return w, meta

    def repack(self, codes: torch.Tensor, scales: Optional[torch.Tensor] = None,
               zeros: Optional[torch.Tensor] = None, e8m0: Optional[torch.Tensor] = None):
        """Canonical device tensors -> (w, meta) device-layout tensors (GPU kernel)."""
        _dev(codes, "codes")
        for t, nm in ((scales, "scales"), (zeros, "zeros"), (e8m0, "e8m0")):
            if t is not None:
                _dev(t, nm)
        self._check_block_weight(codes, scales)
        w, meta = self._repack_outputs(codes.device)
        zx = e8m0 if e8m0 is not None else zeros
        _run(codes.device, lib().hq_repack, self._h, _ptr(codes), _ptr(scales), _ptr(zx), _ptr(w), _ptr(meta))
        return w, meta

    def repack_host(self, codes: torch.Tensor, scales: Optional[torch.Tensor] = None,
                    zeros: Optional[torch.Tensor] = None, e8m0: Optional[torch.Tensor] = None):
        """The same permutation on CPU tensors (offline preparation)."""
        ts = [t.contiguous() if t is not None else None for t in (codes, scales, zeros, e8m0)]
        for t in ts:
            if t is not None and t.is_cuda:
                raise ValueError("repack_host takes CPU tensors")
        codes, scales, zeros, e8m0 = ts
        self._check_block_weight(codes, scales)
        w, meta = self._repack_outputs("cpu")
        zx = e8m0 if e8m0 is not None else zeros
        _check(lib().hq_repack_host(self._h, _ptr(codes), _ptr(scales), _ptr(zx), _ptr(w), _ptr(meta)))
        return w, meta

    # -- GEMM -----------------------------------------------------------
    def gemm(self, a: torch.Tensor, w: torch.Tensor, meta: torch.Tensor, a_scale: Optional[torch.Tensor] = None,
             out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None) -> torch.Tensor:
        """out[m, n] = A . W_deq^T (see include/hq.h, hq_gemm)."""
        if self._block8:
            if _calls is not None and out is None and ws is None:
                r = _calls.gemm_block(self._h.value, self.n, self.k, self.quant.out == BF16, a, a_scale, w, meta)
                if r is not None:
                    return r
            return self._gemm_block(a, w, meta, a_scale, out, ws)
        _dev(a, "a"), _dev(w, "w"), _dev(meta, "meta")
        act4 = self.quant.act == FP4_E2M1
        if a_scale is not None:
            _dev(a_scale, "a_scale")
            if a_scale.dtype != (torch.uint8 if act4 else torch.float32):
                raise ValueError("a_scale must be uint8 E8M0 [m, k/32] (MXFP4 activations) or float32 [m]")
        m = a.shape[0]
        if act4:  # MXFP4 codes two per byte: [m, k/2] bytes (or [m, k/8] int32 words)
            if a.dim() != 2 or a.shape[1] * a.element_size() != self.k // 2:
                raise ValueError(f"a must hold [m, {self.k // 2}] bytes of packed MXFP4 codes")
        elif a.dim() != 2 or a.shape[1] != self.k:
            raise ValueError(f"a must be [m, {self.k}]")
        if out is None:
            if self.epi == EPI_I32_ACC:
                out = torch.empty((m, self.n, self.k // 128), dtype=torch.int32, device=a.device)
            else:
                out = torch.empty((m, self.n), dtype=_TORCH_OUT[self.quant.out], device=a.device)
        _dev(out, "out")
        if ws is None:
            ws = self.workspace(m, a.device)
        ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
        _check(lib().hq_gemm(self._h, m, _ptr(a), _ptr(a_scale), _ptr(w), _ptr(meta), _ptr(out), _ptr(ws),
                             ws_bytes, _stream_ptr(a.device)))
        return out


    def _gemm_block(self, a, w, meta, a_scale, out, ws):
        """gemm of a w8a8_block plan.  Split-K partials live in a workspace of
        the call's own unless one is given, so that calls on several streams, or
        captured into several graphs, do not share one."""
        self._check_block_inputs(a, w, meta, a_scale)
        dev, m = a.device, a.shape[0]
        _block_ws(ws, dev)
        if out is None:
            out = a.new_empty((m, self.n), dtype=_TORCH_OUT[self.quant.out])
        elif _dev(out, "out").shape != (m, self.n) or out.dtype != _TORCH_OUT[self.quant.out] or out.device != dev:
            raise ValueError(f"out must be {_TORCH_OUT[self.quant.out]} [m, {self.n}] on a's device")
        need = self._ws_need.get(m)
        if need is None:
            need = self._ws_need[m] = self.workspace_bytes(m)
        if ws is None and need:
            ws = a.new_empty(need, dtype=torch.uint8)
        _run(dev, lib().hq_gemm, self._h, m, a.data_ptr(), a_scale.data_ptr(), w.data_ptr(), meta.data_ptr(), out.data_ptr(),
             None if ws is None else ws.data_ptr(), 0 if ws is None else ws.nbytes)
        return out

    def _check_block_inputs(self, a, w, meta, a_scale):
        dev = a.device
        if not _same_device(dev, a, w, meta, a_scale):
            for t, name in ((a, "a"), (w, "w"), (meta, "meta"), (a_scale, "a_scale")):
                if _dev(t, name).device != dev:
                    raise ValueError(f"{name} must be on a's device")
        if a.dim() != 2 or a.shape[1] != self.k or a.dtype not in _E4M3:
            raise ValueError(f"a must hold e4m3 codes (or their bytes) [m, {self.k}]")
        # by shape: row-major [m, k/128] scales hold as many values
        if a_scale.dtype != torch.float32 or a_scale.shape != (self.k // 128, a.shape[0]):
            raise ValueError(f"a_scale must be float32 [{self.k // 128}, m]")
        self._check_block_layout(w, meta)

    def _check_block_layout(self, w, meta):
        if w.nbytes < self.num_experts * self.n * self.k or \
                meta.nbytes < self.num_experts * (-(-self.n // 128)) * (self.k // 128) * 4:
            raise ValueError("w and meta must be what repack returned for this plan")

    def linear(self, x: torch.Tensor, w: torch.Tensor, meta: torch.Tensor, out: Optional[torch.Tensor] = None,
               ws: Optional[torch.Tensor] = None) -> torch.Tensor:
        """out = x . W_deq^T for 16-bit activations x [m, k]: a plan that runs
        8-bit activations quantises x per token first (hq_quantize_per_token:
        fp8 e4m3 or int8), one that runs MXFP4 activations block-quantises it
        (hq_quantize_mxfp4), one that runs fp8 with block scales quantises it
        by row and 128 k (hq_quantize_blocks), a 16-bit plan -- including one that fell back --
        multiplies x as it is.  Every step is a library kernel on x's stream;
        the activation codes live in a buffer kept per device and m."""
        _dev(x, "x")
        if x.dtype not in (torch.float16, torch.bfloat16) or x.dim() != 2 or x.shape[1] != self.k:
            raise ValueError(f"x must be fp16 / bf16 [m, {self.k}]")
        q = self.quant
        if q.act in (F16, BF16):
            if x.dtype != _TORCH_OUT[q.act]:
                raise ValueError(f"this plan multiplies {_DT_NAME[q.act]} activations")
            return self.gemm(x, w, meta, out=out, ws=ws)
        m = x.shape[0]
        if self._block8:
            codes, sc = quantize_blocks(x)
            return self.gemm(codes, w, meta, a_scale=sc, out=out, ws=ws)
        key = (x.device, m)
        buf = self._act_buf.get(key)
        if q.act == FP4_E2M1:
            if buf is None:
                buf = (torch.empty((m, self.k // 2), dtype=torch.uint8, device=x.device),
                       torch.empty((self.k // 128, m, 4), dtype=torch.uint8, device=x.device))
                self._act_buf[key] = buf
            codes, sc = quantize_mxfp4(x, codes=buf[0], e8m0=buf[1])
        else:
            kind = "fp8" if q.act == FP8_E4M3 else "int8"
            if buf is None:
                buf = (torch.empty((m, self.k), dtype=torch.uint8 if kind == "fp8" else torch.int8, device=x.device),
                       torch.empty(m, dtype=torch.float32, device=x.device))
                self._act_buf[key] = buf
            codes, sc = quantize_per_token(x, kind, codes=buf[0], scales=buf[1])
        return self.gemm(codes, w, meta, a_scale=sc, out=out, ws=ws)

    # -- measured execution choices --------------------------------------
    def autotune(self, a: torch.Tensor, w: torch.Tensor, meta: torch.Tensor, a_scale: Optional[torch.Tensor] = None,
                 reps: int = 10, flush_bytes: int = 512 << 20, max_ws_bytes: int = 512 << 20) -> dict:
        """Time the candidate execution choices for m = a.shape[0] rows on these
        buffers and install the fastest for that m (see hq_plan_autotune).
        Returns {"tuning", "best_us", "current_us", "candidates"}."""
        if self._block8:
            self._check_block_inputs(a, w, meta, a_scale)
        _dev(a, "a"), _dev(w, "w"), _dev(meta, "meta")
        if a_scale is not None:
            _dev(a_scale, "a_scale")
        m = a.shape[0]
        self._ws_need.pop(m, None)
        out = torch.empty((m, self.n), dtype=_TORCH_OUT.get(self.quant.out, torch.float16), device=a.device)
        if self.epi == EPI_I32_ACC:
            out = torch.empty((m, self.n, self.k // 128), dtype=torch.int32, device=a.device)
        ws_bytes = min(int(max_ws_bytes), 8 * m * self.n * 4)
        ws = torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device=a.device)
        res = AutotuneResult()
        _check(lib().hq_plan_autotune(self._h, m, _ptr(a), _ptr(a_scale), _ptr(w), _ptr(meta), _ptr(out), _ptr(ws),
                                      ws_bytes, int(reps), int(flush_bytes), _stream_ptr(a.device),
                                      ctypes.byref(res)))
        return {"tuning": _tuning_dict(res.best), "best_us": float(res.best_us),
                "current_us": float(res.current_us), "candidates": int(res.candidates)}

    def set_jit(self, enable: bool = True, cache_dir: Optional[str] = None):
        """Run-time specialised kernels for this dense plan (hq_plan_set_jit):
        each call's shape compiled once by hipRTC, code objects cached on disk
        under cache_dir (None: the library's default directory)."""
        _check(lib().hq_plan_set_jit(self._h, 1 if enable else 0,
                                     None if cache_dir is None else os.fsencode(cache_dir)))

    def jit_cache_key(self, m: int, arch: str = "gfx950") -> str:
        """The code-object cache key of the kernel a call with m rows runs under
        run-time specialisation (hq_jit_cache_key; host only)."""
        buf = ctypes.create_string_buffer(128)
        _check(lib().hq_jit_cache_key(self._h, int(m), arch.encode(), buf, len(buf)))
        return buf.value.decode()

    def jit_prepare(self, m: int, arch: str = "gfx950"):
        """Compile the m-row kernel of run-time specialisation into the plan's
        code-object cache without a device (hq_jit_prepare)."""
        _check(lib().hq_jit_prepare(self._h, int(m), arch.encode()))

    def set_tuning(self, m: int, tuning: Optional[dict]):
        """Install a tuning for exactly m rows (None removes m's entry)."""
        self._ws_need.pop(int(m), None)
        t = None if tuning is None else Tuning(**{f: int(tuning.get(f, 0)) for f in _TUNING_FIELDS})
        _check(lib().hq_plan_set_tuning(self._h, int(m), None if t is None else ctypes.byref(t)))

    def get_tuning(self, m: int):
        """(resolved tuning dict for m rows, whether it comes from the table)."""
        t, flag = Tuning(), ctypes.c_int(0)
        _check(lib().hq_plan_get_tuning(self._h, int(m), ctypes.byref(t), ctypes.byref(flag)))
        return _tuning_dict(t), bool(flag.value)

    def tuning_key(self, m: int, device) -> str:
        """Cache key of m rows of this plan on `device`: format, shape, GPU, rows."""
        q = self.quant
        fmt = "-".join(str(int(getattr(q, f))) for f, _ in QuantDesc._fields_)
        name = torch.cuda.get_device_name(torch.device(device)).replace("|", "/")
        return f"{fmt}|epi{self.epi}|n{self.n}|k{self.k}|{name}|abi{lib().hq_abi_version()}|m{int(m)}"


class TuningCache:
    """Measured execution choices kept across processes: a JSON file that maps
    Plan.tuning_key(m, device) to a resolved tuning."""

    def __init__(self, path: str):
        self.path = path
        self.entries = {}
        if os.path.exists(path):
            with open(path) as f:
                self.entries = json.load(f)

    def save(self):
        tmp = self.path + ".tmp"
        with open(tmp, "w") as f:
            json.dump(self.entries, f, indent=1, sort_keys=True)
        os.replace(tmp, self.path)

    def apply(self, plan: Plan, device) -> int:
        """Install every cached tuning of this plan on `device`; returns how many."""
        prefix = plan.tuning_key(0, device)[:-1]  # everything but the row count
        n = 0
        for key, t in self.entries.items():
            if key.startswith(prefix) and key[len(prefix):].isdigit() and 1 <= int(key[len(prefix):]) <= plan.max_m:
                plan.set_tuning(int(key[len(prefix):]), t)
                n += 1
        return n

    def tune(self, plan: Plan, a: torch.Tensor, w: torch.Tensor, meta: torch.Tensor,
             a_scale: Optional[torch.Tensor] = None, **kw) -> dict:
        """The cached tuning for a's rows if there is one (installed), else an
        autotune run whose result is installed and saved."""
        key = plan.tuning_key(a.shape[0], a.device)
        if key in self.entries:
            plan.set_tuning(a.shape[0], self.entries[key])
            return {"tuning": dict(self.entries[key]), "cached": True}
        r = plan.autotune(a, w, meta, a_scale, **kw)
        self.entries[key] = r["tuning"]
        self.save()
        return dict(r, cached=False)


def stream_read(buf: torch.Tensor, sink: torch.Tensor, workgroups: int, nbytes: Optional[int] = None):
    """Bandwidth probe: read `nbytes` (default all) of `buf` once (see hq_stream_read)."""
    _dev(buf, "buf"), _dev(sink, "sink")
    n = buf.numel() * buf.element_size() if nbytes is None else int(nbytes)
    _check(lib().hq_stream_read(_ptr(buf), n, _ptr(sink), int(workgroups), _stream_ptr(buf.device)))


def mfma_peak(kind: int, sink: torch.Tensor, workgroups: int = 1024, iters: int = 2000) -> float:
    """Matrix-core throughput probe (see hq_mfma_peak): one launch of `kind`
    (PEAK_F16 .. PEAK_INT8) on the stream of `sink`; returns its operations."""
    _dev(sink, "sink")
    fl = ctypes.c_double()
    _check(lib().hq_mfma_peak(int(kind), int(workgroups), int(iters), _ptr(sink), ctypes.byref(fl),
                              _stream_ptr(sink.device)))
    return fl.value


def quantize_per_token(x: torch.Tensor, out: str = "fp8", codes: Optional[torch.Tensor] = None,
                       scales: Optional[torch.Tensor] = None):
    """Per-row 8-bit quantisation of fp16 / bf16 activations [m, k] (see
    hq_quantize_per_token): scales = max|row| / Q, codes = RNE(x / scale).
    out "fp8" gives uint8 e4m3 codes (Q = 448), "int8" int8 codes (Q = 127).
    Returns (codes [m, k], scales fp32 [m]), the (a, a_scale) of a W4A8 GEMM."""
    _dev(x, "x")
    if x.dim() != 2 or x.dtype not in (torch.float16, torch.bfloat16):
        raise ValueError("x must be fp16 / bf16 [m, k]")
    if out not in ("fp8", "int8"):
        raise ValueError("out must be 'fp8' or 'int8'")
    m, k = x.shape
    cdt = torch.uint8 if out == "fp8" else torch.int8
    if codes is None:
        codes = torch.empty((m, k), dtype=cdt, device=x.device)
    if scales is None:
        scales = torch.empty(m, dtype=torch.float32, device=x.device)
    _dev(codes, "codes"), _dev(scales, "scales")
    if codes.shape != (m, k) or codes.element_size() != 1 or scales.numel() != m or scales.dtype != torch.float32:
        raise ValueError("codes must be 1-byte [m, k] and scales fp32 [m]")
    _check(lib().hq_quantize_per_token(m, k, BF16 if x.dtype == torch.bfloat16 else F16,
                                       FP8_E4M3 if out == "fp8" else INT8, _ptr(x), _ptr(codes), _ptr(scales),
                                       _stream_ptr(x.device)))
    return codes, scales


def quantize_blocks(x: torch.Tensor, silu_mul: bool = False, codes: Optional[torch.Tensor] = None,
                    scales: Optional[torch.Tensor] = None):
    """fp8 e4m3 quantisation of fp16 / bf16 activations by row and 128 columns
    (see hq_quantize_blocks): x [m, k], or with silu_mul the [m, 2k] output of
    a gate_up GEMM, of which SiLU(x[:, :k]) * x[:, k:] is quantised.  Returns
    (codes uint8 [m, k], scales float32 [k/128, m]), the (a, a_scale) of a
    w8a8_block GEMM."""
    if _calls is not None and codes is None and scales is None:
        r = _calls.quantize_blocks(x, silu_mul)
        if r is not None:
            return r
    _dev(x, "x")
    if x.dim() != 2 or x.dtype not in (torch.float16, torch.bfloat16):
        raise ValueError("x must be fp16 / bf16 [m, k]")
    m, k = x.shape
    if silu_mul:
        if k % 2:
            raise ValueError("x must be [m, 2k] with silu_mul")
        k //= 2
    dev = x.device
    if codes is None:
        codes = x.new_empty((m, k), dtype=torch.uint8) if silu_mul else torch.empty_like(x, dtype=torch.uint8)
    elif _dev(codes, "codes").shape != (m, k) or codes.dtype not in _E4M3 or codes.device != dev:
        raise ValueError("codes must be e4m3 (or bytes) [m, k] on x's device")
    if scales is None:
        scales = x.new_empty((k // 128, m), dtype=torch.float32)
    elif _dev(scales, "scales").shape != (k // 128, m) or scales.dtype != torch.float32 or scales.device != dev:
        raise ValueError("scales must be float32 [k/128, m] on x's device")
    _run(dev, lib().hq_quantize_blocks, m, k, BF16 if x.dtype == torch.bfloat16 else F16, 1 if silu_mul else 0,
         x.data_ptr(), codes.data_ptr(), scales.data_ptr())
    return codes, scales


def mx_scales_group_major(e8m0_rows: torch.Tensor) -> torch.Tensor:
    """Row-major E8M0 block scales [m, K/32] -> the group-major words
    [K/128, m, 4] that a W4A4 GEMM reads (a copy; runs where the tensor is)."""
    m, kb = e8m0_rows.shape
    return e8m0_rows.reshape(m, kb // 4, 4).transpose(0, 1).contiguous()


def quantize_mxfp4(x: torch.Tensor, codes: Optional[torch.Tensor] = None, e8m0: Optional[torch.Tensor] = None):
    """MXFP4 block quantisation of fp16 / bf16 activations [m, k] (see
    hq_quantize_mxfp4).  Returns (codes uint8 [m, k/2], e8m0 uint8
    [k/128, m, 4] group-major), the (a, a_scale) of a W4A4 GEMM."""
    _dev(x, "x")
    if x.dim() != 2 or x.dtype not in (torch.float16, torch.bfloat16):
        raise ValueError("x must be fp16 / bf16 [m, k]")
    m, k = x.shape
    if codes is None:
        codes = torch.empty((m, k // 2), dtype=torch.uint8, device=x.device)
    if e8m0 is None:
        e8m0 = torch.empty((k // 128, m, 4), dtype=torch.uint8, device=x.device)
    _dev(codes, "codes"), _dev(e8m0, "e8m0")
    if codes.numel() * codes.element_size() != m * (k // 2) or e8m0.numel() != m * (k // 32) or \
            e8m0.dtype != torch.uint8:
        raise ValueError("codes must hold [m, k/2] bytes and e8m0 be uint8 [k/128, m, 4]")
    _check(lib().hq_quantize_mxfp4(m, k, BF16 if x.dtype == torch.bfloat16 else F16, _ptr(x), _ptr(codes),
                                   _ptr(e8m0), _stream_ptr(x.device)))
    return codes, e8m0


# ------------------------------------------------------------------- MoE --
def moe_max_padded(t: int, topk: int, num_experts: int, block_m: int) -> int:
    v = ctypes.c_int64()
    _check(lib().hq_moe_max_padded(int(t), int(topk), int(num_experts), int(block_m), ctypes.byref(v)))
    return v.value


def moe_align(topk_ids: torch.Tensor, num_experts: int, block_m: int):
    """Token sort / align by expert (see hq_moe_align).  topk_ids: int32 [t, topk] on the GPU.
    Returns (sorted_ids, block_expert, num_padded) device int32 tensors."""
    _dev(topk_ids, "topk_ids")
    if topk_ids.dtype != torch.int32 or topk_ids.dim() != 2:
        raise ValueError("topk_ids must be int32 [t, topk]")
    t, topk = topk_ids.shape
    mp = moe_max_padded(t, topk, num_experts, block_m)
    dev = topk_ids.device
    sorted_ids = torch.empty(mp, dtype=torch.int32, device=dev)
    block_expert = torch.empty(max(mp // block_m, 1), dtype=torch.int32, device=dev)
    num_padded = torch.empty(1, dtype=torch.int32, device=dev)
    _run(dev, lib().hq_moe_align, t, topk, int(num_experts), int(block_m), _ptr(topk_ids), _ptr(sorted_ids),
         _ptr(block_expert), _ptr(num_padded))
    return sorted_ids, block_expert, num_padded


class MoePlan(Plan):
    """A grouped plan: num_experts weights of [n, k]; epi one of 'silu_mul',
    'silu_mul_qfp8' (gate_up), 'topk_combine' (down) or 'none'."""

    def __init__(self, n: int, k: int, quant: QuantDesc, num_experts: int, max_t: int, epi: str,
                 tuning: Optional[dict] = None, mfma_in: Optional[str] = None, fallback: bool = False):
        super().__init__(n, k, quant, max_m=max_t, epi=epi, kind="grouped", num_experts=num_experts, tuning=tuning,
                         mfma_in=mfma_in, fallback=fallback)

    def describe(self, t: int, topk: int = 1) -> str:
        """The kernel a grouped call with t tokens of topk slots launches."""
        return super().describe(int(t) * int(topk))

    def block_m(self, t: int, topk: int) -> int:
        v = ctypes.c_int()
        _check(lib().hq_moe_block_m(self._h, int(t), int(topk), ctypes.byref(v)))
        return v.value

    def moe_workspace(self, t: int, topk: int, device) -> Optional[torch.Tensor]:
        b = ctypes.c_size_t()
        _check(lib().hq_moe_workspace_bytes(self._h, int(t), int(topk), ctypes.byref(b)))
        if b.value == 0:
            return None
        dev = torch.device(device)
        ws = self._ws.get(dev)
        if ws is None or ws.numel() < b.value:
            ws = torch.zeros(b.value, dtype=torch.uint8, device=dev)
            self._ws[dev] = ws
        return ws

    def moe_gemm(self, a: torch.Tensor, t: int, topk: int, sorted_ids: torch.Tensor, block_expert: torch.Tensor,
                 num_padded: torch.Tensor, w: torch.Tensor, meta: torch.Tensor, a_scale=None, topk_w=None,
                 out=None, out_scale=None, ws=None):
        for x, nm in ((a, "a"), (sorted_ids, "sorted_ids"), (block_expert, "block_expert"),
                      (num_padded, "num_padded"), (w, "w"), (meta, "meta")):
            _dev(x, nm)
        dev = a.device
        bm = self.block_m(t, topk)
        need = moe_max_padded(t, topk, self.num_experts, bm)
        if sorted_ids.numel() < need or block_expert.numel() < max(need // bm, 1):
            raise ValueError(f"sorted_ids / block_expert are smaller than an alignment with block_m={bm} "
                             f"for t={t}, topk={topk} needs ({need}, {need // bm}); align with block_m(t, topk)")
        mp = sorted_ids.numel()
        if out is None:
            if self.epi == EPI_TOPK_COMBINE:
                out = torch.empty((t, self.n), dtype=_TORCH_OUT[self.quant.out], device=dev)
            elif self.epi == EPI_SILU_MUL_QFP8:
                out = torch.empty((mp, self.n // 2), dtype=torch.uint8, device=dev)
            elif self.epi == EPI_SILU_MUL:
                out = torch.empty((mp, self.n // 2), dtype=_TORCH_OUT[self.quant.out], device=dev)
            else:
                out = torch.empty((mp, self.n), dtype=_TORCH_OUT[self.quant.out], device=dev)
        if self.epi == EPI_SILU_MUL_QFP8 and out_scale is None:
            shape = (self.n // 256, mp) if self._block8 else (mp,)
            out_scale = torch.empty(shape, dtype=torch.float32, device=dev)
        if self._block8:
            rows = mp if self.epi == EPI_TOPK_COMBINE else t
            if mp != need:
                raise ValueError(f"sorted_ids must hold {need} ids: the block scales are laid out for that many rows")
            if a_scale is None or a_scale.dtype != torch.float32 or a_scale.shape != (self.k // 128, rows) or \
                    a.dtype not in _E4M3 or a.shape != (rows, self.k):
                raise ValueError(f"a must hold [{rows}, {self.k}] e4m3 codes (or their bytes) and a_scale float32 [{self.k // 128}, {rows}]")
            self._check_block_layout(w, meta)
            _block_ws(ws, dev)
            down = self.epi == EPI_TOPK_COMBINE
            if not _same_device(dev, a_scale, sorted_ids, block_expert, num_padded, w, meta, out) or \
                    not _same_device(dev, topk_w if down else out_scale):
                raise ValueError("the tensors of a w8a8_block GEMM must be contiguous and on a's device")
            if any(v.dtype != torch.int32 for v in (sorted_ids, block_expert, num_padded)):
                raise ValueError("sorted_ids, block_expert and num_padded must be int32")
            if down and (topk_w.dtype != torch.float32 or topk_w.numel() != t * topk):
                raise ValueError(f"topk_w must be float32 [{t}, {topk}]")
            if out.dtype != (_TORCH_OUT[self.quant.out] if down else torch.uint8) or \
                    out.numel() != (t * self.n if down else mp * (self.n // 2)):
                raise ValueError("out must be [t, n] of the output type, or uint8 codes [rows, n/2]")
            if not down and (out_scale.dtype != torch.float32 or out_scale.numel() != mp * (self.n // 256)):
                raise ValueError(f"out_scale must be float32 [{self.n // 256}, {mp}]")
            if ws is None and self.epi == EPI_TOPK_COMBINE:  # of the call's own, as in gemm
                b = ctypes.c_size_t()
                _check(lib().hq_moe_workspace_bytes(self._h, int(t), int(topk), ctypes.byref(b)))
                ws = torch.empty(b.value, dtype=torch.uint8, device=dev)
        if ws is None and not self._block8:
            ws = self.moe_workspace(t, topk, dev)
        ws_bytes = 0 if ws is None else ws.nbytes
        _run(dev, lib().hq_moe_gemm, self._h, int(t), int(topk), _ptr(a), _ptr(a_scale), _ptr(sorted_ids),
             _ptr(block_expert), _ptr(num_padded), _ptr(topk_w), _ptr(w), _ptr(meta), _ptr(out), _ptr(out_scale),
             _ptr(ws), ws_bytes)
        return (out, out_scale) if self.epi == EPI_SILU_MUL_QFP8 else out

    def moe_gemm_by_slot(self, a: torch.Tensor, t: int, topk: int, topk_ids: torch.Tensor, w: torch.Tensor,
                         meta: torch.Tensor, a_scale=None, topk_w=None, out=None, out_scale=None, ws=None):
        """hq_moe_gemm_by_slot: the grouped GEMM with rows indexed by routed
        slot (no alignment).  gate_up returns [t*topk, n/2] (fp8: codes and
        per-slot scales); down takes those slot rows and returns y [t, n]."""
        for x, nm in ((a, "a"), (topk_ids, "topk_ids"), (w, "w"), (meta, "meta")):
            _dev(x, nm)
        dev = a.device
        slots = int(t) * int(topk)
        if topk_ids.numel() < slots:
            raise ValueError(f"topk_ids holds {topk_ids.numel()} ids, t * topk = {slots}")
        if out is None:
            if self.epi == EPI_TOPK_COMBINE:
                out = torch.empty((t, self.n), dtype=_TORCH_OUT[self.quant.out], device=dev)
            elif self.epi == EPI_SILU_MUL_QFP8:
                out = torch.empty((slots, self.n // 2), dtype=torch.uint8, device=dev)
            elif self.epi == EPI_SILU_MUL:
                out = torch.empty((slots, self.n // 2), dtype=_TORCH_OUT[self.quant.out], device=dev)
            else:
                out = torch.empty((slots, self.n), dtype=_TORCH_OUT[self.quant.out], device=dev)
        if self.epi == EPI_SILU_MUL_QFP8 and out_scale is None:
            out_scale = torch.empty(slots, dtype=torch.float32, device=dev)
        if ws is None and self.epi == EPI_SILU_MUL_QFP8:
            ws = self.moe_workspace(t, topk, dev)
        ws_bytes = 0 if ws is None else ws.numel()
        _check(lib().hq_moe_gemm_by_slot(self._h, int(t), int(topk), _ptr(a), _ptr(a_scale), _ptr(topk_ids),
                                         _ptr(topk_w), _ptr(w), _ptr(meta), _ptr(out), _ptr(out_scale), _ptr(ws),
                                         ws_bytes, _stream_ptr(dev)))
        return (out, out_scale) if self.epi == EPI_SILU_MUL_QFP8 else out


# Routed slots (t * topk) up to which moe_layer takes the unaligned by-slot
# path: measured on MI355X (256 experts, top 8, H = 7168, I = 256) it is the
# faster one up to 32 slots and level with the aligned path at 64, where an
# expert picked by several slots starts to be read once per slot.
# routed slots up to which moe_layer takes the by-slot path: the measured
# crossover on MI355X (256 experts, top 8, H = 7168, I = 256, graph-timed
# layers): bf16 by slot against aligned 60.7 / 71.0 us at T = 12 and 82.9 /
# 85.4 us at T = 16; fp8 64.0 / 66.3 us at T = 12 and 78.0 / 76.3 us at T = 16
MOE_BY_SLOT_MAX_SLOTS = 128
MOE_BY_SLOT_MAX_SLOTS_FP8 = 96


def moe_uses_by_slot(t: int, topk: int, fp8: bool = False) -> bool:
    """Whether moe_layer runs a call of t tokens routed to topk experts each
    (fp8: W4A8-FP8 activations) through hq_moe_gemm_by_slot (else the aligned
    hq_moe_align + hq_moe_gemm)."""
    limit = MOE_BY_SLOT_MAX_SLOTS_FP8 if fp8 else MOE_BY_SLOT_MAX_SLOTS
    return 0 < int(t) * int(topk) <= limit


def route_topk(logits: torch.Tensor, topk: int, renormalize: bool = True):
    """The topk experts of each row of logits [t, experts] (fp32, fp16 or bf16)
    and their softmax weights (see hq_route_topk): (ids int32 [t, topk],
    weights float32 [t, topk]), the (topk_ids, topk_w) of moe_layer."""
    if _calls is not None:
        r = _calls.route_topk(logits, topk, renormalize)
        if r is not None:
            return r
    _dev(logits, "logits")
    if logits.dim() != 2 or logits.dtype not in _LOGITS:
        raise ValueError("logits must be fp32 / fp16 / bf16 [t, experts]")
    t, experts = logits.shape
    topk = int(topk)
    ids = logits.new_empty((t, topk), dtype=torch.int32)
    w = logits.new_empty((t, topk), dtype=torch.float32)
    _run(logits.device, lib().hq_route_topk, t, experts, topk, _LOGITS[logits.dtype], logits.data_ptr(),
         1 if renormalize else 0, ids.data_ptr(), w.data_ptr())
    return ids, w


# Tokens up to which a w8a8_block layer runs in two kernels (hq_moe_layer_few): the
# crossover with 256 experts, top 8, H = 7168, I = 256 (16 tokens 97 us against 106
# aligned, 24 tokens 150 against 117).  With fewer experts it lies lower (64 experts,
# top 8, H = 2048, I = 768: 4 tokens 43 against 42, 16 tokens 89 against 71).
MOE_FEW_MAX_TOKENS = 16


def _uses_few(gate_up: "MoePlan", down: "MoePlan", t: int, topk: int) -> bool:
    return gate_up._block8 and 0 < t <= MOE_FEW_MAX_TOKENS and topk <= 16 and gate_up.k == down.n <= 98304


def _check_layer_plans(gate_up: "MoePlan", down: "MoePlan"):
    """Both plans of a layer index one set of experts, and down takes gate_up's
    rows: a plan of another shape would read past its weights."""
    if down.epi != EPI_TOPK_COMBINE or gate_up.epi not in (EPI_SILU_MUL, EPI_SILU_MUL_QFP8):
        raise ValueError("moe_layer takes a gate_up plan (silu_mul / silu_mul_qfp8) and a topk_combine plan")
    if gate_up._block8 != down._block8:
        raise ValueError("gate_up and down must both be w8a8_block plans, or neither")
    if down.num_experts < gate_up.num_experts or (gate_up._block8 and down.num_experts != gate_up.num_experts):
        raise ValueError(f"gate_up has {gate_up.num_experts} experts, down {down.num_experts}")
    if gate_up.n != 2 * down.k:
        raise ValueError(f"gate_up gives rows of {gate_up.n // 2}, down takes {down.k}")


def _moe_few(gate_up, down, x, topk, ids, w, logits, renormalize, w1, m1, w2, m2):
    dev = x.device
    if not _same_device(dev, x, ids, w, w1, m1, w2, m2):
        for v, nm in ((x, "x"), (ids, "topk_ids"), (w, "topk_w"), (w1, "w1"), (m1, "m1"), (w2, "w2"), (m2, "m2")):
            if _dev(v, nm).device != dev:
                raise ValueError(f"{nm} must be on x's device")
    t = x.shape[0]
    if x.dim() != 2 or x.shape[1] != gate_up.k or x.dtype not in (torch.float16, torch.bfloat16):
        raise ValueError(f"x must be fp16 / bf16 [t, {gate_up.k}]")
    if ids.shape != (t, topk) or ids.dtype != torch.int32 or w.shape != (t, topk) or w.dtype != torch.float32:
        raise ValueError(f"topk_ids / topk_w must be int32 / float32 [{t}, {topk}]")
    need = gate_up._few_need.get((t, topk, down.k))
    if need is None:
        n = ctypes.c_size_t()
        _check(lib().hq_moe_few_workspace_bytes(gate_up._h, down._h, t, topk, ctypes.byref(n)))
        need = gate_up._few_need[t, topk, down.k] = n.value
    ws = x.new_empty(need, dtype=torch.uint8)
    out = x.new_empty((t, down.n), dtype=_TORCH_OUT[down.quant.out])
    gate_up._check_block_layout(w1, m1), down._check_block_layout(w2, m2)
    _run(dev, lib().hq_moe_layer_few, gate_up._h, down._h, t, topk, BF16 if x.dtype == torch.bfloat16 else F16, x.data_ptr(),
         F32 if logits is None else _LOGITS[logits.dtype], _ptr(logits), 1 if renormalize else 0, ids.data_ptr(), w.data_ptr(),
         w1.data_ptr(), m1.data_ptr(), w2.data_ptr(), m2.data_ptr(), out.data_ptr(), ws.data_ptr(), need)
    return out


def moe_layer_routed(gate_up: "MoePlan", down: "MoePlan", x: torch.Tensor, logits: torch.Tensor, topk: int,
                     w1: torch.Tensor, m1: torch.Tensor, w2: torch.Tensor, m2: torch.Tensor, renormalize: bool = True):
    """An MoE layer from the router's logits [t, experts] on: (y [t, n_down],
    topk_ids, topk_w).  w8a8_block plans run a few tokens in two kernels
    (hq_moe_layer_few); otherwise route_topk, then moe_layer."""
    _check_layer_plans(gate_up, down)
    _dev(logits, "logits")
    topk = int(topk)
    if logits.dim() != 2 or logits.shape != (x.shape[0], gate_up.num_experts) or logits.dtype not in _LOGITS or \
            logits.device != x.device:
        raise ValueError(f"logits must be fp32 / fp16 / bf16 [{x.shape[0]}, {gate_up.num_experts}] on x's device")
    if _uses_few(gate_up, down, x.shape[0], topk) and gate_up.num_experts <= 1024:
        ids = x.new_empty((x.shape[0], topk), dtype=torch.int32)
        w = x.new_empty((x.shape[0], topk), dtype=torch.float32)
        return _moe_few(gate_up, down, x, topk, ids, w, logits, renormalize, w1, m1, w2, m2), ids, w
    ids, w = route_topk(logits, topk, renormalize)
    return moe_layer(gate_up, down, x, ids, w, w1, m1, w2, m2), ids, w


def moe_layer(gate_up: "MoePlan", down: "MoePlan", x: torch.Tensor, topk_ids: torch.Tensor, topk_w: torch.Tensor,
              w1: torch.Tensor, m1: torch.Tensor, w2: torch.Tensor, m2: torch.Tensor, x_scale=None,
              by_slot: Optional[bool] = None) -> torch.Tensor:
    """One MoE layer, y [t, n_down]: gate_up (SiLU * up, or with the fp8
    requant) then down with the top-k combine, on the by-slot path for
    decode-sized calls (moe_uses_by_slot) and the aligned path otherwise;
    `by_slot` forces one.  w8a8_block plans take 16-bit x (quantised here, or
    inside the two kernels that few tokens run in) or the codes and scales of
    quantize_blocks, and always the aligned path beyond.  x: [t, k] activations (fp8 codes with x_scale for
    W4A8); topk_ids int32 / topk_w fp32 [t, topk] on the GPU."""
    t, topk = topk_ids.shape
    _check_layer_plans(gate_up, down)
    fp8 = gate_up.epi == EPI_SILU_MUL_QFP8
    if gate_up._block8:
        if by_slot:
            raise ValueError("w8a8_block layers have no by-slot path")
        if t == 0:
            return x.new_empty((0, down.n), dtype=_TORCH_OUT[down.quant.out])
        if x_scale is None and _uses_few(gate_up, down, t, topk):
            return _moe_few(gate_up, down, x, topk, topk_ids, topk_w, None, False, w1, m1, w2, m2)
        by_slot = False
        if x_scale is None:
            x, x_scale = quantize_blocks(x)
    if by_slot is None:
        by_slot = moe_uses_by_slot(t, topk, fp8)
    if by_slot:
        r = gate_up.moe_gemm_by_slot(x, t, topk, topk_ids, w1, m1, a_scale=x_scale)
        act, scl = r if fp8 else (r, None)
        return down.moe_gemm_by_slot(act, t, topk, topk_ids, w2, m2, a_scale=scl, topk_w=topk_w)
    bm = gate_up.block_m(t, topk)
    if down.block_m(t, topk) != bm:
        raise ValueError("the gate_up and down plans must share one alignment block size (equal tuning)")
    sid, bex, npad = moe_align(topk_ids, gate_up.num_experts, bm)
    r = gate_up.moe_gemm(x, t, topk, sid, bex, npad, w1, m1, a_scale=x_scale)
    act, scl = r if fp8 else (r, None)
    return down.moe_gemm(act, t, topk, sid, bex, npad, w2, m2, a_scale=scl, topk_w=topk_w)
