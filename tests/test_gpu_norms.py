"""moe_norm and moe_norm_backward against 64-bit references."""
import pytest
import torch

import mxfp4_expert_gemm_b200 as moe
from _train_ref import assert_close, generator, normal

pytestmark = pytest.mark.gpu

BF, HF, SF = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-5


def forward_ref(x, w, b, kind):
    x = x.double()
    m = x.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(x[:, :1])
    r = 1 / torch.sqrt((x - m).square().mean(1, keepdim=True) + EPS)
    y = (x - m) * r * w.double()
    if b is not None:
        y = y + b.double()
    return y, m, r


def errors(x, w, b, m, r, kind):
    """Bound of y's fp32 error: the mean is off by (d + 8) 2^-24 of mean |x| (sums of any order), r
    by as much relative to itself, and a handful of roundings."""
    n = (x.shape[1] + 8) * 2.0 ** -24 if x.shape[1] < 64 else (x.shape[1] / 32 + 40) * 2.0 ** -24
    x = x.double()
    em = n * x.abs().mean(1, keepdim=True) if kind == "layer" else 0.0
    xc = (x - m).abs()
    er = n + 4 * 2.0 ** -24 + r * em
    return (em * r + xc * r * (er + 6 * 2.0 ** -24)) * w.double().abs() + (
        0 if b is None else 2.0 ** -23 * b.double().abs())


SHAPES = [(1, 1), (1, 2880), (3, 7), (5, 33), (16, 2880), (33, 64), (100, 257), (129, 1000), (7, 8192), (300, 512),
          (2, 65536), (4, 20001), (1021, 96), (2000, 2880)]


@pytest.mark.parametrize("dt", [BF, HF, SF])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("T,d", SHAPES)
def test_norm(T, d, kind, dt):
    g = generator(T + d)
    x = normal(g, T, d, dtype=dt, std=2.0, mean=0.5)
    w = normal(g, d, dtype=SF, std=0.3, mean=1.0)
    b = normal(g, d, dtype=SF) if kind == "layer" else None
    y, mean, rstd = moe.moe_norm(x, w, b, kind=kind, eps=EPS, want_stats=True)
    yr, m, r = forward_ref(x, w, b, kind)
    assert_close(y, yr, errors(x, w, b, m, r, kind) + 1e-30)
    assert (mean is None) == (kind == "rms")
    dy, dres = normal(g, T, d, dtype=dt), normal(g, T, d, dtype=dt)
    dx, dw, db = moe.moe_norm_backward(dy, x, w, mean, rstd, kind=kind, dres=dres)
    assert (db is None) == (kind == "rms")
    # the formulas in 64 bits from the same fp32 statistics
    m = mean.double().unsqueeze(1) if mean is not None else 0.0
    r = rstd.double().unsqueeze(1)
    xh, dyd = (x.double() - m) * r, dy.double()
    gg = dyd * w.double()
    c1, c2 = (gg * xh).mean(1, keepdim=True), gg.mean(1, keepdim=True)
    want = r * (gg - xh * c1 - (c2 if kind == "layer" else 0.0)) + dres.double()
    n = (d / 32 + 48) * 2.0 ** -24
    mag = gg.abs() + xh.abs() * (gg * xh).abs().mean(1, keepdim=True) + gg.abs().mean(1, keepdim=True)
    assert_close(dx, want, r * n * mag + 4 * 2.0 ** -24 * (want.abs() + dres.double().abs()), "dx")
    nt = (T + 16) * 2.0 ** -24
    xr = (x.double().abs() + (m.abs() if kind == "layer" else 0)) * r
    assert_close(dw, (dyd * xh).sum(0), nt * (dyd.abs() * xr).sum(0) + 1e-30, "dw")
    if db is not None:
        assert_close(db, dyd.sum(0), nt * dyd.abs().sum(0) + 1e-30, "db")
    again = moe.moe_norm_backward(dy, x, w, mean, rstd, kind=kind, dres=dres)
    for p, q in zip((dx, dw, db), again):
        assert (p is None and q is None) or torch.equal(p, q)


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_gradients_against_differences(kind):
    g = generator(3)
    T, d, h = 12, 56, 1e-5
    x, w = normal(g, T, d, dtype=SF), normal(g, d, dtype=SF, std=0.3, mean=1.0)
    b = normal(g, d, dtype=SF) if kind == "layer" else None
    dy = normal(g, T, d, dtype=SF)
    _, mean, rstd = moe.moe_norm(x, w, b, kind=kind, eps=EPS, want_stats=True)
    dx, dw, db = moe.moe_norm_backward(dy, x, w, mean, rstd, kind=kind)

    def loss(xx, ww, bb):
        return float((forward_ref(xx, ww, bb, kind)[0] * dy.double()).sum())

    xd, wd, bd = x.double(), w.double(), None if b is None else b.double()
    vx, vw = torch.randn_like(xd), torch.randn_like(wd)
    pairs = [(dx, vx, loss(xd + h * vx, wd, bd) - loss(xd - h * vx, wd, bd)),
             (dw, vw, loss(xd, wd + h * vw, bd) - loss(xd, wd - h * vw, bd))]
    if b is not None:
        vb = torch.randn_like(bd)
        pairs.append((db, vb, loss(xd, wd, bd + h * vb) - loss(xd, wd, bd - h * vb)))
    for grad, v, diff in pairs:
        got, want = float((grad.double() * v).sum()), diff / (2 * h)
        # fp32 gradients (d 2^-24 of their magnitudes at most) and differences with h^2 error
        assert abs(got - want) <= 1e-4 * float((grad.double() * v).abs().sum()) + 1e-6


@pytest.mark.parametrize("dt", [BF, SF])
def test_strides_alignment_and_in_place(dt):
    """Rows of a wider buffer at an odd offset (the scalar path), y over x, dx over dres and dy."""
    g = generator(9)
    T, d = 37, 480
    w, b = normal(g, d, dtype=SF, mean=1.0, std=0.2), normal(g, d, dtype=SF)
    for off in (0, 3, 8):
        buf = normal(g, T, d + 24, dtype=dt)
        x = buf[:, off:off + d]
        y, mean, rstd = moe.moe_norm(x, w, b, kind="layer", want_stats=True)
        yr, m, r = forward_ref(x, w, b, "layer")
        assert_close(y, yr, errors(x, w, b, m, r, "layer"))
        dy, dres = normal(g, T, d + 24, dtype=dt)[:, off:off + d], normal(g, T, d + 8, dtype=dt)[:, :d]
        want, dw, db = moe.moe_norm_backward(dy, x, w, mean, rstd, kind="layer", dres=dres)
        keep = dres.clone()
        moe.moe_norm_backward(dy, x, w, mean, rstd, kind="layer", dres=dres, dx=dres)
        assert torch.equal(dres, want)
        dyc = dy.clone()
        dw2 = moe.moe_norm_backward(dyc, x, w, mean, rstd, kind="layer", dres=keep, dx=dyc)[1]
        assert torch.equal(dyc, want) and torch.equal(dw2, dw)
        before = buf.clone()
        moe.moe_norm(x, w, b, kind="layer", y=x)
        assert torch.equal(x, y)
        assert torch.equal(buf[:, :off], before[:, :off]) and torch.equal(buf[:, off + d:], before[:, off + d:])


def test_long_rows_in_place():
    """Rows too long for registers: dx over dy and over x leaves the column sums right."""
    g = generator(10)
    T, d = 5, 40000
    x, dy, w = normal(g, T, d, dtype=SF), normal(g, T, d, dtype=SF), normal(g, d, dtype=SF, mean=1.0)
    _, mean, rstd = moe.moe_norm(x, w, kind="layer", want_stats=True)
    dx, dw, db = moe.moe_norm_backward(dy, x, w, mean, rstd, kind="layer")
    for over in (dy.clone(), x.clone()):
        a = over if torch.equal(over, dy) else dy
        c = over if torch.equal(over, x) else x
        got = moe.moe_norm_backward(a, c, w, mean, rstd, kind="layer", dx=over)
        assert torch.equal(got[0], dx) and torch.equal(got[1], dw) and torch.equal(got[2], db)


def test_rms_matches_the_layers_own_norm():
    """moe_norm(kind="rms") and moe_residual_norm compute the same norm."""
    g = generator(12)
    x, w = normal(g, 50, 2880), normal(g, 2880, dtype=SF, std=0.1, mean=1.0)
    y, yn = moe.moe_residual_norm(x, torch.zeros(50, 2880, device="cuda"), w)
    assert torch.equal(y, x)
    got, err = moe.moe_norm(x, w), forward_ref(x, w, None, "rms")[0]
    for t in (got, yn):
        assert_close(t, err, (2880 / 32 + 60) * 2.0 ** -24 * err.abs())


def test_non_finite_rows_and_constant_rows():
    x = torch.zeros(6, 64, dtype=BF, device="cuda")
    x[1] = 3.0                      # no variance: y = b, gradients finite
    x[2, 5] = float("nan")
    x[3, 5] = float("inf")
    x[4] = 3.0e38
    x[5, 1] = -2.0
    w, b = torch.ones(64, device="cuda"), torch.full((64,), 0.5, device="cuda")
    y, mean, rstd = moe.moe_norm(x, w, b, kind="layer", want_stats=True)
    assert bool((y[:2] == 0.5).all()) and bool(torch.isnan(y[2]).all()) and bool(torch.isnan(y[3]).all())
    assert bool(torch.isfinite(y[5]).all())
    dx = moe.moe_norm_backward(torch.ones_like(x), x, w, mean, rstd, kind="layer")[0]
    assert bool(torch.isfinite(dx[:2]).all()) and bool(torch.isfinite(dx[5]).all())


def test_empty_and_graph():
    w = torch.ones(64, device="cuda")
    x = torch.empty(0, 64, dtype=BF, device="cuda")
    y, mean, rstd = moe.moe_norm(x, w, kind="layer", want_stats=True)
    assert y.shape == (0, 64)
    _, dw, db = moe.moe_norm_backward(x, x, w, mean, rstd, kind="layer")
    assert not bool(dw.any()) and not bool(db.any())
    g = generator(13)
    x, dy = normal(g, 70, 64), normal(g, 70, 64)

    def step():
        y, mean, rstd = moe.moe_norm(x, w, kind="layer", want_stats=True)
        return (y, *moe.moe_norm_backward(dy, x, w, mean, rstd, kind="layer"))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    x.copy_(normal(g, 70, 64))
    graph.replay()
    for a, e in zip(out, step()):
        assert torch.equal(a, e)
