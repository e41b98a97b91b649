"""Argument checks of the norms and the 16-bit products: they answer before any device work, so
they run without a GPU."""
import ctypes

import pytest
import torch

import mxfp4_expert_gemm_b200 as moe
from mxfp4_expert_gemm_b200 import build

BAD, SHAPE, WS = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED_SHAPE, moe.MOE_ERR_WORKSPACE


@pytest.fixture(scope="module")
def L():
    build.build()
    return moe.lib()


def dims(K=64, N=64, E=1, dtype=0, fn=0, limit=7.0):
    return moe.moe_linear_dims(K, N, E, dtype, fn, limit)


def _linear(L, dm, M=4, x=256, ldx=64, w=4096, bias=None, res=None, ldr=0, y=8192, ldy=64, z=None, status=None):
    return L.moe_linear(ctypes.byref(dm) if dm else None, M, x, ldx, w, bias, res, ldr, y, ldy, z, status, None)


def _grouped(L, dm, P=4, x=256, ldx=64, w=4096, off=512, bias=None, y=8192, ldy=64, z=None, status=None):
    return L.moe_grouped_linear(ctypes.byref(dm), P, x, ldx, w, off, bias, y, ldy, z, status, None)


def _backward(L, dm, M=4, dy=256, lddy=64, x=1024, ldx=64, w=4096, z=2048, dx=8192, lddx=64, dw=16384, db=32768,
              ws=65536, n=1 << 40):
    return L.moe_linear_backward(ctypes.byref(dm), M, dy, lddy, x, ldx, w, z, dx, lddx, dw, db, ws, n, None, None)


def test_linear_refusals(L):
    assert _linear(L, None) == BAD
    assert _linear(L, dims(), M=-1) == BAD
    assert _linear(L, dims(), M=0, x=None, y=None, w=None) == moe.MOE_OK       # nothing to do
    assert _linear(L, dims(dtype=2)) == BAD                                     # fp32 products are not offered
    assert _linear(L, dims(fn=6)) == BAD and _linear(L, dims(fn=-1)) == BAD
    for limit in (0.0, -1.0, float("nan"), float("inf")):
        assert _linear(L, dims(fn=5, limit=limit), ldy=32) == BAD
    for kw in (dict(K=0), dict(K=12), dict(N=4), dict(N=100), dict(K=(1 << 16) + 8), dict(N=(1 << 17) + 8), dict(E=2),
               dict(N=72, fn=5), dict(E=0)):
        assert _linear(L, dims(**kw)) == SHAPE, kw
    assert _linear(L, dims(), M=(1 << 24) + 1) == SHAPE
    for kw in (dict(x=None), dict(x=264), dict(w=None), dict(w=4100), dict(y=None), dict(y=8200), dict(ldx=56),
               dict(ldx=68), dict(ldy=60), dict(ldy=68), dict(bias=4098), dict(res=264, ldr=64), dict(res=256, ldr=60),
               dict(z=8), dict(status=2), dict(y=256), dict(z=8192), dict(res=8192, ldr=72), dict(ldx=1 << 40)):
        assert _linear(L, dims(), **kw) == BAD, kw


def test_grouped_refusals(L):
    assert _grouped(L, dims(E=3), off=None) == BAD
    assert _grouped(L, dims(E=3), off=514) == BAD
    assert _grouped(L, dims(E=257)) == SHAPE
    assert _grouped(L, dims(E=3), P=0, off=None, x=None, y=None) == moe.MOE_OK


def test_backward_refusals(L):
    for kw in (dict(dy=None), dict(dy=264), dict(lddy=60), dict(x=None), dict(ldx=60), dict(w=None), dict(dx=8200),
               dict(lddx=60), dict(dw=16388), dict(db=32770), dict(ws=None), dict(ws=65544), dict(dx=256),
               dict(dw=4096), dict(dw=1024)):
        assert _backward(L, dims(), **kw) == BAD, kw
    assert _backward(L, dims(fn=4), z=None) == BAD
    need = moe.moe_linear_workspace_bytes(dims(fn=4), 4)
    assert need > 0 and _backward(L, dims(fn=4), n=need - 1) == WS
    assert _backward(L, dims(), M=0, dx=None, dw=None, db=None) == moe.MOE_OK
    assert _backward(L, dims(), dx=None, dw=None, db=None) == moe.MOE_OK       # nothing asked for
    assert moe.moe_linear_workspace_bytes(dims(K=12), 4) == 0
    assert moe.moe_linear_workspace_bytes(dims(E=32, N=5760, K=2880, fn=5), 16384) >= 2 * 16384 * 5760


def _norm(L, kind=1, dtype=0, T=4, d=64, x=256, ldx=64, w=512, b=None, eps=1e-5, y=8192, ldy=64, mean=None, rstd=None):
    return L.moe_norm(kind, dtype, T, d, x, ldx, w, b, eps, y, ldy, mean, rstd, None)


def _norm_backward(L, kind=1, dtype=0, T=4, d=64, dy=256, lddy=64, x=1024, ldx=64, w=512, mean=128, rstd=64, dres=None,
                   lddres=0, dx=8192, lddx=64, dw=16384, db=32768, ws=65536, n=1 << 40):
    return L.moe_norm_backward(kind, dtype, T, d, dy, lddy, x, ldx, w, mean, rstd, dres, lddres, dx, lddx, dw, db, ws,
                               n, None)


def test_norm_refusals(L):
    for kw in (dict(kind=2), dict(dtype=3), dict(T=-1), dict(d=0), dict(eps=-1.0), dict(eps=float("nan")),
               dict(kind=0, b=512), dict(x=None), dict(x=257), dict(dtype=2, x=258), dict(w=None), dict(w=514),
               dict(y=None), dict(ldx=63), dict(ldy=63), dict(mean=2), dict(rstd=2), dict(y=256, ldy=72)):
        assert _norm(L, **kw) == BAD, kw
    assert _norm(L, d=(1 << 16) + 1) == SHAPE and _norm(L, T=(1 << 24) + 1) == SHAPE
    assert _norm(L, T=0, x=None, y=None, w=None) == moe.MOE_OK
    for kw in (dict(dy=None), dict(x=None), dict(w=None), dict(rstd=None), dict(mean=None), dict(dx=None),
               dict(dy=257), dict(dres=256, lddres=60), dict(lddx=60), dict(ws=None), dict(ws=65544), dict(dw=2),
               dict(dx=256, lddx=72), dict(dres=8192, lddres=72), dict(kind=0)):
        assert _norm_backward(L, **kw) == BAD, kw
    need = moe.moe_norm_workspace_bytes(4, 64)
    assert need > 0 and _norm_backward(L, n=need - 1) == WS
    assert _norm_backward(L, d=(1 << 16) + 1) == SHAPE
    assert moe.moe_norm_workspace_bytes(-1, 64) == 0 and moe.moe_norm_workspace_bytes(4, 1 << 17) == 0


def test_valid_arguments_reach_the_device(L):
    """With valid arguments and no usable GPU the calls fail; there is no CPU path."""
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for st in (_linear(L, dims()), _grouped(L, dims(E=3)), _backward(L, dims()), _norm(L), _norm_backward(L)):
        assert st in (moe.MOE_ERR_CUDA, moe.MOE_ERR_DEVICE)


def test_binding_refuses_host_tensors_and_bad_names():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(64, 64, dtype=torch.bfloat16)
    for call in (lambda: moe.moe_linear(x, w), lambda: moe.moe_grouped_linear(x, w[None], torch.zeros(2)),
                 lambda: moe.moe_linear_backward(x, x, w), lambda: moe.moe_norm(x, torch.ones(64)),
                 lambda: moe.moe_grouped_linear(x, w[None], None),
                 lambda: moe.moe_norm_backward(x, x, torch.ones(64), None, torch.ones(4))):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError):
        moe.make_linear_dims(64, 64, fn="tanh")
    with pytest.raises(TypeError):
        moe.make_linear_dims(64, 64, dtype=torch.float32)
