"""Operands that lie at the very end, or the very start, of an allocation of their own: nothing is read
or written beside them."""
import pytest
import torch

import mxfp4_expert_gemm_b200 as moe
from _train_ref import generator, normal

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
OWN = 34 << 20   # bytes: an allocation of its own in torch's allocator, ending where its mapping ends


class Place:
    """Copies of tensors in allocations of their own, against the end or the start."""

    def __init__(self, end):
        self.end, self.kept = end, []

    def __call__(self, t):
        if t is None:
            return None
        n = t.numel() * t.element_size()
        buf = torch.full((OWN,), 0xA5, dtype=torch.uint8, device="cuda")
        at = (OWN - n) // 16 * 16 if self.end else 0
        view = buf[at:at + n].view(t.dtype).view(t.shape)
        view.copy_(t)
        self.kept.append((buf, at, n))
        return view

    def intact(self):
        return all(bool((b[:a] == 0xA5).all()) and bool((b[a + n:] == 0xA5).all()) for b, a, n in self.kept)


def _same(got, want):
    for a, b in zip(got, want):
        assert (a is None and b is None) or torch.equal(a, b)


@pytest.mark.parametrize("end", [True, False])
@pytest.mark.parametrize("M,K,N,fn,dt", [
    (17, 2024, 16, "gelu", HF), (1, 2880, 320, "swiglu", BF), (2, 1432, 1040, "none", BF), (9, 848, 64, "relu", HF),
    (63, 1000, 136, "silu", BF), (65, 2024, 264, "gelu_tanh", BF), (100, 72, 2880, "none", HF), (700, 1024, 2048, "swiglu", BF)])
def test_dense(M, K, N, fn, dt, end):
    g = generator(M + K)
    No = N // 2 if fn == "swiglu" else N
    x, w, b = normal(g, M, K, dtype=dt), normal(g, N, K, dtype=dt, std=K ** -0.5), normal(g, N, dtype=torch.float32)
    r, dy, z = normal(g, M, No, dtype=dt), normal(g, M, No, dtype=dt), normal(g, M, N, dtype=dt)
    zz = z if fn != "none" else None
    forward = moe.moe_linear(x, w, b, fn=fn, residual=r, want_z=True)
    back = moe.moe_linear_backward(dy, x, w, zz, fn=fn, need_db=True)
    p = Place(end)
    px, pw, pdy, pz = p(x), p(w), p(dy), p(zz)
    _same(moe.moe_linear(px, pw, p(b), fn=fn, residual=p(r), y=p(torch.zeros_like(r)), z=p(torch.zeros_like(z)), want_z=True),
          forward)
    _same(moe.moe_linear_backward(pdy, px, pw, pz, fn=fn, need_db=True, dx=p(torch.zeros_like(x)), dw=p(torch.zeros_like(w))),
          back)
    assert p.intact()


@pytest.mark.parametrize("end", [True, False])
@pytest.mark.parametrize("counts,pad,first,K,N,fn,dt", [
    ([17], 0, 0, 2024, 16, "gelu", HF),
    ([5, 0, 12, 3], 0, 0, 2024, 64, "silu", BF),
    ([1, 2, 3, 4, 5, 6, 7, 8, 9, 10], 0, 0, 512, 320, "none", BF),
    ([62], 1, 0, 1000, 528, "swiglu", BF),
    ([30, 40, 63, 1], 2, 3, 2024, 2576, "swiglu", BF),
    ([3, 0, 20, 1, 500, 63], 0, 7, 1032, 2576, "gelu", HF),
    ([0, 0, 11, 0], 0, 0, 2880, 5760, "none", BF)])
def test_grouped(counts, pad, first, K, N, fn, dt, end):
    g = generator(sum(counts) + K)
    E, offs = len(counts), [first]
    for c in counts:
        offs.append(offs[-1] + c)
    P, No = offs[-1] + pad, N // 2 if fn == "swiglu" else N
    off = torch.tensor(offs, dtype=torch.int32, device="cuda")
    x, w = normal(g, P, K, dtype=dt), normal(g, E, N, K, dtype=dt, std=K ** -0.5)
    dy, z = normal(g, P, No, dtype=dt), normal(g, P, N, dtype=dt)
    zz, s = z if fn != "none" else None, slice(first, offs[-1])
    y = moe.moe_grouped_linear(x, w, off, fn=fn)
    dx, dw, db = moe.moe_grouped_linear_backward(dy, x, w, off, zz, fn=fn, need_db=True)
    for e in range(E):   # the weight gradient in 64 bits, from dz as the products take it (its rounding, then their sum's)
        r = slice(offs[e], offs[e + 1])
        if fn == "none":
            ref = dy[r].double().t() @ x[r].double()
            mag = dy[r].double().abs().t() @ x[r].double().abs()
            assert bool(((dw[e].double() - ref).abs() <= torch.finfo(dt).eps / 2 * ref.abs() + 32 * 2.0 ** -23 * mag).all())
        if offs[e] == offs[e + 1]:
            assert not bool(dw[e].any())
    p = Place(end)
    keep = [t for t in (w, dw) if t.numel() * t.element_size() > OWN]
    pw, pdw = (w, torch.zeros_like(w)) if keep else (p(w), p(torch.zeros_like(w)))
    px, pdy, pz = p(x), p(dy), p(zz)
    py = moe.moe_grouped_linear(px, pw, off, fn=fn, y=p(torch.zeros_like(y)))
    assert torch.equal(py[s], y[s])
    pdx, pdw, pdb = moe.moe_grouped_linear_backward(pdy, px, pw, off, pz, fn=fn, need_db=True, dx=p(torch.zeros_like(x)), dw=pdw)
    assert torch.equal(pdx[s], dx[s]) and torch.equal(pdw, dw) and torch.equal(pdb, db)
    assert p.intact()


@pytest.mark.parametrize("end", [True, False])
@pytest.mark.parametrize("T,d,dt", [(5, 2880, BF), (300, 1001, HF), (300, 1002, BF), (2400, 2880, torch.float32), (3, 20001, BF)])
def test_norms(T, d, dt, end):
    g = generator(T + d)
    x, dy, r = (normal(g, T, d, dtype=dt) for _ in range(3))
    w, b = normal(g, d, dtype=torch.float32), normal(g, d, dtype=torch.float32)
    y, mean, rstd = moe.moe_norm(x, w, b, kind="layer", want_stats=True)
    back = moe.moe_norm_backward(dy, x, w, mean, rstd, kind="layer", dres=r)
    p = Place(end)
    px, pw = p(x), p(w)
    assert torch.equal(moe.moe_norm(px, pw, p(b), kind="layer", y=p(torch.zeros_like(x))), y)
    _same(moe.moe_norm_backward(p(dy), px, pw, p(mean), p(rstd), kind="layer", dres=p(r), dx=p(torch.zeros_like(x))), back)
    assert p.intact()


LOW, HIGH = -2 ** 31, 2 ** 31 - 1


@pytest.mark.parametrize("fn", ["none", "swiglu"])
@pytest.mark.parametrize("offs", [
    [0, HIGH, LOW, 20], [LOW, LOW, LOW, LOW], [HIGH] * 4, [60, 40, 20, 0], [0, 63, 62, 63], [5, 5, 64, 63], [0, 0, 0, 64]])
def test_offsets_out_of_range_or_order(offs, fn):
    """Reported, and nothing beside the outputs is touched."""
    g = generator(4)
    P, K, N, E = 63, 72, 144, 3
    No = N // 2 if fn == "swiglu" else N
    off, p = torch.tensor(offs, dtype=torch.int32, device="cuda"), Place(True)
    x, w, dy, z = p(normal(g, P, K)), p(normal(g, E, N, K)), p(normal(g, P, No)), p(normal(g, P, N))
    y, dx, dw = p(torch.zeros_like(dy)), p(torch.zeros_like(x)), p(torch.zeros_like(w))
    st = torch.zeros(4, dtype=torch.int32, device="cuda")
    moe.moe_grouped_linear(x, w, off, fn=fn, y=y, status_word=st)
    assert moe.moe_device_status(st) == moe.MOE_ERR_INVALID_ARG
    moe.moe_grouped_linear_backward(dy, x, w, off, z if fn != "none" else None, fn=fn, dx=dx, dw=dw, need_db=True, status_word=st)
    assert moe.moe_device_status(st) == moe.MOE_ERR_INVALID_ARG
    assert p.intact()


@pytest.mark.parametrize("end", [True, False])
@pytest.mark.parametrize("act", ["bf16", "mxfp8", "mxfp4"])
@pytest.mark.parametrize("path", ["gemm", "gemv"])
@pytest.mark.parametrize("T,d,I,E,k", [(37, 192, 320, 5, 3), (200, 576, 448, 8, 4), (300, 256, 128, 64, 4), (1, 2880, 704, 4, 2)])
def test_layer(T, d, I, E, k, path, act, end):
    """The MXFP4 layer with its weights, workspace and tokens so placed."""
    g = generator(T + d)
    F = torch.float32
    x, gamma = normal(g, T, d), normal(g, d, dtype=F, mean=1.0, std=0.1)
    rw, rb = normal(g, E, d, dtype=F, std=0.1), normal(g, E, dtype=F, std=0.1)
    w1, w2 = normal(g, E, 2 * I, d, dtype=F, std=d ** -0.5), normal(g, E, d, I, dtype=F, std=I ** -0.5)
    dims = moe.make_dims(d, I, E, k, path=path, act=act)
    W = [*moe.moe_mxfp4_quantize(w1, role="gate_up"), *moe.moe_mxfp4_quantize(w2, role="down")]
    ws = moe.new_workspace(dims, T)
    want = moe.moe_forward(dims, x, gamma, rw, rb, *W, ws)
    assert moe.moe_device_status(ws) == moe.MOE_OK
    p = Place(end)
    n = ws.numel()
    pws = p(torch.zeros((n + 255) // 256 * 256, dtype=torch.uint8, device="cuda"))
    pW = [p(t) for t in W]
    got = moe.moe_forward(dims, p(x), p(gamma), p(rw), p(rb), *pW, pws, y=p(torch.zeros_like(x)))
    assert moe.moe_device_status(pws) == moe.MOE_OK
    assert torch.equal(got, want) and p.intact()
    q = [p(torch.zeros_like(t)) for t in W[:2]]
    moe.moe_mxfp4_quantize(p(w1) if w1.numel() * 4 < OWN else w1, *q, role="gate_up")
    assert torch.equal(q[0], W[0]) and torch.equal(q[1], W[1]) and p.intact()
