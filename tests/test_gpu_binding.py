"""What the compiled part of the binding owes its callers beside the results."""
import ctypes
import threading
import time
import warnings

import pytest
import torch

import mxfp4_expert_gemm_b200 as moe
from _train_ref import generator, normal

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


def _calls():
    g = generator(1)
    x, w1, dy = normal(g, 6, 64), normal(g, 32, 64), normal(g, 6, 32)
    gamma, w3 = normal(g, 64, dtype=torch.float32), normal(g, 2, 32, 64)
    off = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    rstd = torch.ones(6, device="cuda")
    return dict(
        norm=(lambda a: moe.moe_norm(*a), (x, gamma)),
        norm_backward=(lambda a: moe.moe_norm_backward(a[0], a[0], a[1], None, rstd), (x, gamma)),
        linear=(lambda a: moe.moe_linear(*a), (x, w1)),
        linear_backward=(lambda a: moe.moe_linear_backward(dy, *a), (x, w1)),
        grouped=(lambda a: moe.moe_grouped_linear(*a, off), (x, w3)),
        grouped_backward=(lambda a: moe.moe_grouped_linear_backward(dy, *a, off), (x, w3)))


@pytest.mark.parametrize("name", ["norm", "norm_backward", "linear", "linear_backward", "grouped", "grouped_backward"])
def test_a_tensor_that_requires_grad_is_named(name, request):
    """No call records a graph: with gradients on, an argument that requires one gets a warning."""
    call, args = _calls()[name]
    torch.set_warn_always(True)   # (otherwise the first time only)
    request.addfinalizer(lambda: torch.set_warn_always(False))
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        call(args)
    for i in range(len(args)):
        a = [t.clone() for t in args]
        a[i].requires_grad_()
        with pytest.warns(UserWarning, match="no graph"):
            out = call(a)
        assert not any(t.requires_grad for t in (out if isinstance(out, tuple) else (out,)) if t is not None)
        with warnings.catch_warnings(), torch.no_grad():
            warnings.simplefilter("error")
            call(a)


def test_inside_a_function_of_autograd():
    """The calls as the two halves of a torch.autograd.Function: its graph's gradients are theirs."""

    class Linear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w):
            y, z = moe.moe_linear(x, w, fn="silu", want_z=True)
            ctx.save_for_backward(x, w, z)
            return y

        @staticmethod
        def backward(ctx, dy):
            x, w, z = ctx.saved_tensors
            return moe.moe_linear_backward(dy, x, w, z, fn="silu")[:2]

    g = generator(2)
    x, w, dy = normal(g, 20, 64).requires_grad_(), normal(g, 32, 64, std=0.1).requires_grad_(), normal(g, 20, 32)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        Linear.apply(x, w).backward(dy)
    with torch.no_grad():
        _, z = moe.moe_linear(x, w, fn="silu", want_z=True)
        dx, dw, _ = moe.moe_linear_backward(dy, x, w, z, fn="silu")
    assert torch.equal(x.grad, dx) and torch.equal(w.grad, dw)
