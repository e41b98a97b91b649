"""Calls on a stream that is not the current one own the memory that they make: nothing that the
current stream still uses is written, and nothing that the call still writes goes to the current
stream."""
import pytest
import torch

import mxfp4_expert_gemm_b200 as moe
from _train_ref import generator, normal

pytestmark = pytest.mark.gpu

BUSY = 60_000_000   # clock cycles (30 ms) that a stream is kept from what comes next


def _norm():
    g = generator(1)
    x, w = normal(g, 3000, 1024), normal(g, 1024, dtype=torch.float32)
    return lambda **kw: moe.moe_norm(x, w, kind="layer", want_stats=True, **kw), 0


def _norm_backward():
    g = generator(2)
    x, dy, w = normal(g, 3000, 1024), normal(g, 3000, 1024), normal(g, 1024, dtype=torch.float32)
    _, mean, rstd = moe.moe_norm(x, w, kind="layer", want_stats=True)
    return (lambda **kw: moe.moe_norm_backward(dy, x, w, mean, rstd, kind="layer", **kw),
            moe.moe_norm_workspace_bytes(3000, 1024))


def _linear():
    g = generator(3)
    x, w = normal(g, 300, 256), normal(g, 640, 256, std=0.1)
    return lambda **kw: moe.moe_linear(x, w, fn="swiglu", want_z=True, **kw), 0


def _linear_backward():
    g = generator(4)
    M, K, N = 300, 256, 640
    x, w, dy, z = normal(g, M, K), normal(g, N, K, std=0.1), normal(g, M, N // 2), normal(g, M, N)
    ws = moe.moe_linear_workspace_bytes(moe.make_linear_dims(K, N, 1, x.dtype, "swiglu"), M)
    return lambda **kw: moe.moe_linear_backward(dy, x, w, z, fn="swiglu", need_db=True, **kw), ws


def _grouped():
    g = generator(5)
    x, w, off = normal(g, 300, 256), normal(g, 3, 640, 256, std=0.1), torch.tensor([0, 100, 130, 300]).int().cuda()
    return lambda **kw: moe.moe_grouped_linear(x, w, off, fn="silu", want_z=True, **kw), 0


def _grouped_backward():
    g = generator(6)
    P, K, N = 300, 256, 640
    x, w, off = normal(g, P, K), normal(g, 3, N, K, std=0.1), torch.tensor([0, 100, 130, 300]).int().cuda()
    dy, z = normal(g, P, N), normal(g, P, N)
    ws = moe.moe_linear_workspace_bytes(moe.make_linear_dims(K, N, 3, x.dtype, "silu"), P)
    return lambda **kw: moe.moe_grouped_linear_backward(dy, x, w, off, z, fn="silu", need_db=True, **kw), ws


CALLS = dict(norm=_norm, norm_backward=_norm_backward, linear=_linear, linear_backward=_linear_backward,
             grouped=_grouped, grouped_backward=_grouped_backward)


def _blanks(want, ws, value):
    out = [torch.full_like(t, value) for t in want]
    return out + [torch.full((ws // 4,), value, device="cuda")] if ws else out


@pytest.mark.parametrize("name", CALLS)
def test_memory_still_in_use_on_the_current_stream_is_left_alone(name):
    """The current stream is busy and still has to read tensors that were dropped: of the sizes of the
    call's outputs and scratch, so that their blocks would be the first choice."""
    call, ws = CALLS[name]()
    want = [t.clone() for t in call()]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        torch.cuda.empty_cache()
        dropped = _blanks(want, ws, 3.0)
        copies = [torch.empty_like(t) for t in dropped]
        torch.cuda.synchronize()
        torch.cuda._sleep(BUSY)
        for c, t in zip(copies, dropped):
            c.copy_(t)
        del dropped, t
        got = call(stream=s)
        s.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        torch.cuda.synchronize()
        for c in copies:
            assert bool((c == 3).all())


@pytest.mark.parametrize("name", CALLS)
def test_memory_still_written_on_the_calls_stream_is_not_handed_out(name):
    """Outputs dropped while their stream is busy do not turn up in the current stream's tensors."""
    call, ws = CALLS[name]()
    want = [t.clone() for t in call()]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        torch.cuda.empty_cache()
        with torch.cuda.stream(s):
            torch.cuda._sleep(BUSY)
        call(stream=s)
        kept = _blanks(want, ws, 5.0)
        torch.cuda.synchronize()
        for t in kept:
            assert bool((t == 5).all())


@pytest.mark.parametrize("name", CALLS)
def test_outputs_are_of_the_calls_stream(name):
    """The segments that the outputs lie in are the given stream's."""
    call, _ = CALLS[name]()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = call(stream=s)
    s.synchronize()
    segments = torch.cuda.memory_snapshot()
    for t in out:
        mine = [q for q in segments if q["address"] <= t.data_ptr() < q["address"] + q["total_size"]]
        assert [q["stream"] for q in mine] == [s.cuda_stream]
    before = torch.cuda.current_stream()
    call(stream=s)
    assert torch.cuda.current_stream() == before
    with pytest.raises((TypeError, ValueError, moe.MoeError)):
        call(stream=s, ws=torch.empty(16, device="cuda")) if "backward" in name else call(stream=s, y=s)
    assert torch.cuda.current_stream() == before   # after an error too
    s.synchronize()


@pytest.mark.parametrize("name", CALLS)
def test_the_default_stream_named_from_another(name):
    call, _ = CALLS[name]()
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = call(stream=torch.cuda.default_stream())
    for a, b in zip(got, want):
        assert torch.equal(a, b)
