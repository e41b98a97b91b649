"""The norms and grouped products run together as a layer, forward and back:
norm -> moe_route -> grouped gate_up with SwiGLU -> grouped down -> weighted combine.

Forward, on MXFP4 weights decoded to bf16 (E2M1 times a power of two: exact), it has to give the
expert mix of the library's own MXFP4 layer; backward, the gradients of the layer in 64 bits.
"""
import pytest
import torch

import mxfp4_expert_gemm_b200 as moe
from __graft_entry__ import _decode_stored
from _gpu_case import case
from _train_ref import f_ref, generator, half_step, normal
from test_gpu_parity import SMALL

pytestmark = pytest.mark.gpu

STEP = half_step(torch.bfloat16)   # 2^-8: a rounding's largest relative error


def _decoded(codes, scales, N, K, gate_up):
    W = [torch.from_numpy(_decode_stored(c.cpu().numpy(), s.cpu().numpy(), N, K, gate_up)) for c, s in zip(codes, scales)]
    W = torch.stack(W)
    assert torch.equal(W, W.to(torch.bfloat16).double())
    return W.to(torch.bfloat16).cuda()


def _route(c, dims):
    cfg = c["cfg"]
    ws = moe.new_workspace(dims, cfg.T)
    r = moe.moe_route(dims, c["x_dev"], c["gamma_dev"], c["rw_dev"], c["rb_dev"], ws)
    assert moe.moe_device_status(ws) == moe.MOE_OK
    perm = r["perm"].long()
    return r["offsets"], perm, perm // cfg.k, r["topk_w"].reshape(-1)[perm]   # offsets, pair, token, weight per row


def _rel(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


@pytest.mark.parametrize("name", ["tiny", "odd", "single", "wide_E", "clamp", "mid_ragged"])
def test_forward_matches_the_mxfp4_layer(name):
    c = case(SMALL[name])
    cfg = c["cfg"]
    dims = moe.make_dims(cfg.d, cfg.I, cfg.E, cfg.k, cfg.rms_eps, cfg.swiglu_limit)
    c1, s1, c2, s2 = c["W"]["gpu"]
    W1, W2 = _decoded(c1, s1, 2 * cfg.I, cfg.d, True), _decoded(c2, s2, cfg.d, cfg.I, False)
    off, perm, tok, w = _route(c, dims)
    st = torch.zeros(4, dtype=torch.int32, device="cuda")
    xn = moe.moe_norm(c["x_dev"], c["gamma_dev"], kind="rms", eps=cfg.rms_eps)
    h = moe.moe_grouped_linear(xn[tok], W1, off, fn="swiglu", limit=cfg.swiglu_limit, status_word=st)
    o = moe.moe_grouped_linear(h, W2, off, status_word=st)
    assert moe.moe_device_status(st) == moe.MOE_OK
    mix = torch.zeros(cfg.T, cfg.d, device="cuda").index_add_(0, tok, w[:, None] * o.float())
    ws = moe.new_workspace(dims, cfg.T)
    want = moe.moe_forward_partial(dims, c["x_dev"], c["gamma_dev"], c["rw_dev"], c["rb_dev"], *c["W"]["gpu"], ws)
    assert moe.moe_device_status(ws) == moe.MOE_OK
    # the library's layer keeps o in fp32: here it is rounded, by 2^-8 of itself at most; xn and h are
    # rounded alike on both sides but for values next to a rounding border
    assert _rel(mix, want) <= STEP


@pytest.mark.parametrize("T,d,I,E,k,seed", [(48, 192, 320, 6, 2, 1), (700, 512, 640, 16, 4, 2), (5, 64, 64, 8, 1, 3)])
def test_gradients_of_the_layer(T, d, I, E, k, seed):
    g = generator(seed)
    x, dy = normal(g, T, d), normal(g, T, d)
    gamma = normal(g, d, dtype=torch.float32, std=0.1, mean=1.0)
    rw, rb = normal(g, E, d, dtype=torch.float32, std=0.02), normal(g, E, dtype=torch.float32, std=0.01)
    W1, W2 = normal(g, E, 2 * I, d, std=d ** -0.5), normal(g, E, d, I, std=I ** -0.5)
    dims = moe.make_dims(d, I, E, k)
    ws = moe.new_workspace(dims, T)
    r = moe.moe_route(dims, x, gamma, rw, rb, ws)
    assert moe.moe_device_status(ws) == moe.MOE_OK
    off, perm = r["offsets"], r["perm"].long()
    tok, w = perm // k, r["topk_w"].reshape(-1)[perm]

    xn, _, rstd = moe.moe_norm(x, gamma, want_stats=True)
    xp = xn[tok]
    h, z = moe.moe_grouped_linear(xp, W1, off, fn="swiglu", want_z=True)
    o = moe.moe_grouped_linear(h, W2, off)
    y = x.float() + torch.zeros(T, d, device="cuda").index_add_(0, tok, w[:, None] * o.float())

    do = (w[:, None] * dy[tok].float()).to(torch.bfloat16)
    dh, dW2, _ = moe.moe_grouped_linear_backward(do, h, W2, off)
    dxp, dW1, _ = moe.moe_grouped_linear_backward(dh, xp, W1, off, z, fn="swiglu")
    dxn = torch.zeros(T, d, device="cuda").index_add_(0, tok, dxp.float()).to(torch.bfloat16)
    dx, dgamma, _ = moe.moe_norm_backward(dxn, x, gamma, None, rstd, dres=dy)

    # the layer in 64 bits, with the experts and weights that the router chose
    xd, gd = x.double().requires_grad_(), gamma.double().requires_grad_()
    w1, w2 = W1.double().requires_grad_(), W2.double().requires_grad_()
    xnd = xd * torch.rsqrt(xd.square().mean(1, keepdim=True) + 1e-5) * gd
    ends, parts = off.tolist(), []
    for e in range(E):
        s = slice(ends[e], ends[e + 1])
        parts.append(f_ref("swiglu", xnd[tok[s]] @ w1[e].t()) @ w2[e].t())
    yd = xd + torch.zeros(T, d, dtype=torch.float64, device="cuda").index_add(0, tok, w.double()[:, None] * torch.cat(parts))
    yd.backward(dy.double())

    # A rounding to bf16 moves a tensor by at most 2^-8 of its norm; on the way to y there are 3 (xn,
    # h, o), to dW2 4 (xn, h, do, dW2), to dW1 6 (xn, z, do, dh, dz, dW1), to dx and dgamma 8 (those
    # but dW1, then dxp, dxn and dx), each carried on by maps that do not enlarge a random
    # perturbation relative to their result by more than 2 (the activation's slopes).
    for got, want, steps, what in ((y, yd, 3, "y"), (dW2, w2.grad, 4, "dW2"), (dW1, w1.grad, 6, "dW1"),
                                   (dx, xd.grad, 8, "dx"), (dgamma, gd.grad, 8, "dgamma")):
        assert got.shape == want.shape and _rel(got, want.detach()) <= 2 * steps * STEP, what
