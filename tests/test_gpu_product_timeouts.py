"""A pipeline wait that runs out, in every form of the tiled products: the call ends, reports it, and
the next call is whole.  (No GPU fault: one arrival is withheld, and the bounded waits end.)"""
import pytest
import torch

import mxfp4_expert_gemm_b200 as moe
from _train_ref import generator, normal

pytestmark = pytest.mark.gpu


def _shared(fn, M, K, N):
    """Few tiles: clusters that share a contraction and join it over distributed shared memory."""
    g = generator(M)
    x, w = normal(g, M, K), normal(g, N, K, std=0.05)
    return lambda st: [moe.moe_linear(x, w, fn=fn, status_word=st)]


def _input_gradient():
    g = generator(2)
    dy, x, w = normal(g, 70, 2048), normal(g, 70, 4096), normal(g, 2048, 4096, std=0.05)
    return lambda st: moe.moe_linear_backward(dy, x, w, status_word=st)[:2]


def _weight_gradient():
    g = generator(3)
    dy, x, w = normal(g, 2000, 64), normal(g, 2000, 64), normal(g, 64, 64)
    return lambda st: [moe.moe_linear_backward(dy, x, w, need_dx=False, status_word=st)[1]]


def _pairs(way):
    g = generator(4)
    counts, K, N = [700, 0, 900, 600], 1024, 2048
    P, off = sum(counts), torch.tensor([0, 700, 700, 1600, 2200], dtype=torch.int32, device="cuda")
    x, w, dy, z = normal(g, P, K), normal(g, 4, N, K, std=0.05), normal(g, P, N // 2), normal(g, P, N)
    if way == "forward":
        return lambda st: [moe.moe_grouped_linear(x, w, off, fn="swiglu", status_word=st)]
    return lambda st: moe.moe_grouped_linear_backward(dy, x, w, off, z, fn="swiglu", status_word=st)[:2]


CASES = {
    "shared 64 wide": lambda: _shared("none", 40, 2880, 2880),
    "shared 32 wide": lambda: _shared("swiglu", 20, 2880, 5760),
    "shared by two": lambda: _shared("silu", 256, 1024, 1024),
    "input gradient": _input_gradient,
    "weight gradient": _weight_gradient,
    "pairs": lambda: _pairs("forward"),
    "pairs backward": lambda: _pairs("backward"),
}


@pytest.mark.parametrize("name", CASES)
def test_timeout_ends_and_the_next_call_is_whole(name):
    call, st = CASES[name](), torch.zeros(4, dtype=torch.int32, device="cuda")
    want = [t.clone() for t in call(st)]
    assert moe.moe_device_status(st) == moe.MOE_OK
    moe.moe_debug_inject_timeout()
    call(st)
    assert moe.moe_device_status(st) == moe.MOE_ERR_TIMEOUT
    for _ in range(3):
        for a, b in zip(call(st), want):
            assert torch.equal(a, b)
    assert moe.moe_device_status(st) == moe.MOE_OK


def test_calls_without_a_pipeline_clear_the_hook():
    g = generator(5)
    x, w, dy = normal(g, 4, 256), normal(g, 512, 256), normal(g, 4, 512)
    big, st = normal(g, 40, 256), torch.zeros(4, dtype=torch.int32, device="cuda")
    want, db = moe.moe_linear(x, w), moe.moe_linear_backward(dy, x, w, need_db=True)[2]
    for call, ref in ((lambda: moe.moe_linear(x, w, status_word=st), want),
                      (lambda: moe.moe_linear_backward(dy, x, w, need_dx=False, need_dw=False, need_db=True,
                                                       status_word=st)[2], db)):
        moe.moe_debug_inject_timeout()
        assert torch.equal(call(), ref)
        moe.moe_linear(big, w, status_word=st)
        assert moe.moe_device_status(st) == moe.MOE_OK
