"""The native short calls beside other Python threads: while one of them waits
in the library, for memory or a place in the launch queue, the others run."""
import ctypes
import threading
import time

import pytest
import torch

import bit_quantized_gemm_repack_amd as hq

pytestmark = pytest.mark.gpu


def test_other_threads_run_while_a_call_waits():
    """libc's usleep stands in for the library's quantiser: its first argument, here
    the number of rows, is the time it waits, and 0 is success.  No kernel runs."""
    L = hq.lib()
    assert hq._calls is not None
    real = [ctypes.cast(f, ctypes.c_void_p).value for f in (L.hq_quantize_blocks, L.hq_route_topk, L.hq_gemm, L.hq_plan_workspace_bytes)]
    usleep = ctypes.cast(ctypes.CDLL(None).usleep, ctypes.c_void_p).value
    x = torch.zeros(500_000, 128, dtype=torch.bfloat16, device="cuda:0")
    hq.quantize_blocks(x)
    torch.cuda.synchronize()
    ticks, stop = [], threading.Event()

    def beside():
        while not stop.is_set():
            ticks.append(time.perf_counter())
            time.sleep(0.005)
    other = threading.Thread(target=beside)
    hq._calls.bind(usleep, *real[1:])
    try:
        other.start()
        t0 = time.perf_counter()
        r = hq._calls.quantize_blocks(x, False)
        t1 = time.perf_counter()
    finally:
        hq._calls.bind(*real)
        stop.set()
        other.join()
    assert r is not None and t1 - t0 > 0.45
    assert sum(t0 + 0.05 < t < t1 - 0.05 for t in ticks) > 10
