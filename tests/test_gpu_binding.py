"""What the compiled part of the binding owes its callers beside the results."""
import ctypes
import threading
import time

import pytest
import torch

import mxfp4_expert_gemm_b200 as moe

pytestmark = pytest.mark.gpu


def test_other_threads_run_while_a_call_is_in_the_library():
    """The call's address is libc's sleep, its first argument (kind: 1, "layer") the seconds."""
    x, w = torch.ones(4, 64, device="cuda"), torch.ones(64, device="cuda")
    moe.moe_norm(x, w)
    sleep = ctypes.cast(ctypes.CDLL(None).sleep, ctypes.c_void_p).value
    seen, stop = [], threading.Event()

    def tick():
        while not stop.is_set():
            seen.append(time.monotonic())
            time.sleep(0.01)

    t = threading.Thread(target=tick)
    with moe.use_library(moe.LIB_PATH):
        moe._calls().bind(*[sleep] * 8)
        t.start()
        t0 = time.monotonic()
        moe.moe_norm(x, w, kind="layer")
        t1 = time.monotonic()
        stop.set()
        t.join()
    assert t1 - t0 >= 0.9
    assert len([s for s in seen if t0 + 0.1 < s < t1 - 0.1]) >= 10
    assert bool((moe.moe_norm(x, w) - 1 / (1 + 1e-5) ** 0.5).abs().max() < 1e-6)   # the library's own call again


def test_a_flag_without_a_truth_value_is_refused():
    x, w = torch.ones(4, 64, device="cuda"), torch.ones(64, device="cuda")
    with pytest.raises(RuntimeError, match="ambiguous"):
        moe.moe_norm(x, w, want_stats=torch.ones(2))
