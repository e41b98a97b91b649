"""moe_linear, moe_grouped_linear and their backward passes against 64-bit references."""
import pytest
import torch

import mxfp4_expert_gemm_b200 as moe
from _train_ref import (LIMIT, assert_close, backward_ref, f_ref, forward_ref, generator, half_step, normal, offsets_of)

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def _status():
    return torch.zeros(4, dtype=torch.int32, device="cuda")


def _ok(status):
    assert moe.moe_device_status(status) == moe.MOE_OK


# M, K, N, fn, dtype, bias, residual, want_z
FORWARD = [
    (1, 8, 16, "none", BF, False, False, False),
    (1, 2880, 2880, "none", BF, True, True, False),
    (2, 64, 8, "relu", HF, True, False, True),
    (5, 72, 136, "silu", BF, True, True, True),
    (16, 2880, 5760, "swiglu", BF, True, False, False),
    (17, 200, 336, "swiglu", HF, True, True, True),
    (32, 1024, 4096, "gelu_tanh", BF, True, False, True),
    (33, 320, 64, "gelu", BF, False, True, False),
    (1, 136, 16392, "none", BF, True, False, False),
    (8, 40, 16384, "silu", HF, True, True, True),
    (16, 104, 8192, "swiglu", BF, True, True, True),
    (9, 104, 8208, "swiglu", BF, False, False, True),
    (9, 4104, 1552, "swiglu", HF, False, True, True),
    (24, 2880, 200, "relu", BF, True, False, False),
    (8, 65536, 16, "gelu", BF, True, False, True),
    (100, 1000, 24, "gelu", HF, True, True, True),
    (129, 136, 1288, "none", BF, True, False, True),
    (257, 2880, 320, "swiglu", BF, False, False, True),
    (700, 4096, 128, "silu", BF, True, False, False),
    (1031, 512, 2880, "gelu_tanh", HF, True, True, False),
    (2500, 192, 640, "swiglu", BF, True, True, True),
    (2111, 2880, 1304, "none", BF, True, True, True),
    (4096, 72, 5760, "swiglu", HF, True, False, True),
    (3000, 1024, 4096, "gelu", BF, False, False, False),
]


@pytest.mark.parametrize("M,K,N,fn,dt,bias,residual,want_z", FORWARD)
def test_linear_forward(M, K, N, fn, dt, bias, residual, want_z):
    g = generator(M + K + N)
    No = N // 2 if fn == "swiglu" else N
    x, w = normal(g, M, K, dtype=dt), normal(g, N, K, dtype=dt, std=2.0 / K ** 0.5)
    b = normal(g, N, dtype=torch.float32) if bias else None
    r = normal(g, M, No, dtype=dt) if residual else None
    st = _status()
    out = moe.moe_linear(x, w, b, fn=fn, residual=r, want_z=want_z, status_word=st)
    y, z = out if want_z else (out, None)
    yr, zr, ey, ez = forward_ref(x, w, b, fn, r)
    assert y.shape == (M, No) and y.dtype == dt
    assert_close(y, yr, ey, "y")
    if want_z:
        assert_close(z, zr, ez, "z")
    _ok(st)
    again = moe.moe_linear(x, w, b, fn=fn, residual=r, want_z=want_z)
    assert torch.equal(again[0] if want_z else again, y)


@pytest.mark.parametrize("M", [3, 20, 77])
def test_linear_strided_rows_and_residual_in_place(M):
    """Rows of wider buffers, and y written over the residual it adds."""
    g = generator(5)
    K, N = 264, 144
    xb, yb = normal(g, M, K + 56), normal(g, M, N + 24)
    x, y = xb[:, 16:16 + K], yb[:, 8:8 + N]
    w = normal(g, N, K, std=0.1)
    before = yb.clone()
    yr, _, ey, _ = forward_ref(x, w, None, "none", y.clone())
    got = moe.moe_linear(x, w, residual=y, y=y)
    assert got.data_ptr() == y.data_ptr()
    assert_close(y, yr, ey)
    assert torch.equal(yb[:, :8], before[:, :8]) and torch.equal(yb[:, 8 + N:], before[:, 8 + N:])


def test_swiglu_rows_come_in_pairs_of_eight():
    """N = 1544 is a multiple of 8 but not of 16: half of it is no whole 16-byte row."""
    x, w = torch.ones(9, 4104, dtype=HF, device="cuda"), torch.ones(1544, 4104, dtype=HF, device="cuda")
    with pytest.raises(moe.MoeError) as e:
        moe.moe_linear(x, w, fn="swiglu")
    assert e.value.status == moe.MOE_ERR_UNSUPPORTED_SHAPE


def test_linear_clamp_and_large_values():
    """SwiGLU at and past its clamps, and saturated activations."""
    K, N = 16, 32
    x = torch.zeros(8, K, dtype=BF, device="cuda")
    x[:, 0] = torch.tensor([7.0, 7.03125, -7.0, -7.03125, 100.0, -100.0, 0.0, 3.0e38], dtype=BF)
    w = torch.zeros(N, K, dtype=BF, device="cuda")
    w[:, 0] = 1.0
    y = moe.moe_linear(x, w, fn="swiglu")
    assert_close(y, f_ref("swiglu", (x.double() @ w.double().t())), torch.full((8, 16), 1e-5, device="cuda"))
    for fn in ("relu", "silu", "gelu", "gelu_tanh"):
        y = moe.moe_linear(x, w, fn=fn).float()
        assert bool((y[4] == 100).all()) and bool((y[5].abs() < 1e-30).all()) and bool((y[6] == 0).all()), fn
        assert bool((y[7] > 2.9e38).all()), fn


def test_linear_nan_and_inf_stay_in_their_rows():
    g = generator(6)
    M, K, N = 40, 72, 64
    x, w = normal(g, M, K), normal(g, N, K, std=0.1)
    x[3, 71] = float("nan")
    x[7, 0] = float("inf")
    y = moe.moe_linear(x, w)
    fine = [r for r in range(M) if r not in (3, 7)]
    assert bool(torch.isnan(y[3]).all()) and not bool(torch.isfinite(y[7]).any())
    yr, _, ey, _ = forward_ref(x[fine], w, None, "none", None)
    assert_close(y[fine], yr, ey)


BACKWARD = [
    (1, 8, 16, "none", BF, True),
    (1, 2880, 320, "swiglu", BF, True),
    (3, 72, 136, "relu", HF, False),
    (16, 1024, 512, "gelu", BF, True),
    (33, 328, 640, "swiglu", HF, True),
    (64, 64, 64, "silu", BF, True),
    (65, 136, 264, "gelu_tanh", BF, True),
    (200, 2880, 96, "none", HF, True),
    (1000, 192, 320, "gelu_tanh", HF, False),
    (4099, 320, 192, "swiglu", BF, True),
    (2000, 2888, 1304, "silu", BF, True),
    (777, 2880, 5760, "swiglu", HF, True),
    (70, 4096, 2048, "none", BF, True),
]


def _check_backward(got, refs, errs, norms, dt, what=""):
    for k, name in enumerate(("dx", "dw", "db")):
        if got[k] is None:
            continue
        assert_close(got[k], refs[k], errs[k], f"{what}{name}")
        if k < 2 and refs[k].numel() > 4096:   # rounding errors are independent: their norm is far below the bound
            assert float((got[k].double() - refs[k]).norm()) <= float(norms[k]) + 1e-6 * float(refs[k].norm()), name


@pytest.mark.parametrize("M,K,N,fn,dt,want_db", BACKWARD)
def test_linear_backward(M, K, N, fn, dt, want_db):
    g = generator(M + 3 * K + N)
    No = N // 2 if fn == "swiglu" else N
    x, w = normal(g, M, K, dtype=dt), normal(g, N, K, dtype=dt, std=2.0 / K ** 0.5)
    dy, z = normal(g, M, No, dtype=dt), normal(g, M, N, dtype=dt, std=3.0)
    zz = z if fn != "none" else None
    st = _status()
    got = moe.moe_linear_backward(dy, x, w, zz, fn=fn, need_db=want_db, status_word=st)
    refs, errs, norms = backward_ref(dy, x, w, zz, fn)
    assert (got[2] is not None) == want_db
    _check_backward(got, refs, errs, norms, dt)
    _ok(st)
    again = moe.moe_linear_backward(dy, x, w, zz, fn=fn, need_db=want_db)
    for a, b in zip(got, again):
        assert (a is None and b is None) or torch.equal(a, b)
    only = moe.moe_linear_backward(dy, x, w, zz, fn=fn, need_dx=False, need_dw=True)
    assert only[0] is None and only[2] is None and torch.equal(only[1], got[1])


@pytest.mark.parametrize("fn", ["none", "relu", "gelu", "gelu_tanh", "silu", "swiglu"])
def test_linear_gradients_against_differences(fn):
    """The kernel's gradients against central differences of the 64-bit forward formula."""
    g = generator(11)
    M, K, N = 24, 40, 32
    x, w, b = normal(g, M, K), normal(g, N, K, std=0.3), normal(g, N, dtype=torch.float32)
    _, z = moe.moe_linear(x, w, b, fn=fn, want_z=True)
    dy = normal(g, M, N // 2 if fn == "swiglu" else N)
    dx, dw, db = moe.moe_linear_backward(dy, x, w, z, fn=fn, need_db=True)
    # the differences are taken at z as kept (rounded to 16 bits): z + h d(x w^T + b)
    h = 1e-5
    for name, grad, dirn in (("dx", dx, (torch.randn(M, K, dtype=torch.float64, device="cuda", generator=g), 0, 0)),
                             ("dw", dw, (0, torch.randn(N, K, dtype=torch.float64, device="cuda", generator=g), 0)),
                             ("db", db, (0, 0, torch.randn(N, dtype=torch.float64, device="cuda", generator=g)))):
        vx, vw, vb = dirn
        dz = (vx @ w.double().t() if name == "dx" else x.double() @ vw.t() if name == "dw" else vb.expand(M, N))
        zd = z.double()
        want = float((dy.double() * (f_ref(fn, zd + h * dz) - f_ref(fn, zd - h * dz))).sum()) / (2 * h)
        v = vx if name == "dx" else vw if name == "dw" else vb
        got = float((grad.double() * v).sum())
        # two roundings of 16 bits per gradient element, independent: their sum in the root mean square,
        # four standard deviations (a rounding's is at most its bound over sqrt 3); 1e-6: the differences
        scale = float((grad.double() * v).square().sum().sqrt())
        rows = float((dz * df(fn, zd, dy)).square().sum().sqrt())
        tol = 4 / 3 ** 0.5 * half_step(x.dtype) * (scale + rows) + 1e-6 * (abs(want) + rows)
        assert abs(got - want) <= tol, (name, got, want, tol)


def df(fn, z, dy):
    from _train_ref import df_ref
    return df_ref(fn, z, dy.double())


# counts per expert, rows behind the last, first offset, K, N, fn, dtype
GROUPED = [
    ([4], 0, 0, 64, 64, "none", BF),
    ([0, 0, 3, 0], 5, 0, 72, 144, "swiglu", BF),
    ([1] * 40, 0, 0, 200, 96, "silu", HF),
    ([2, 0, 7, 1, 30, 16, 0, 8], 3, 2, 2880, 320, "swiglu", BF),
    ([0, 500, 1, 33, 0, 129], 40, 0, 192, 320, "gelu", HF),
    ([64, 128, 32, 63, 65, 127], 0, 7, 328, 136, "relu", BF),
    ([300, 0, 0, 0, 2, 900, 31], 9, 0, 136, 272, "gelu_tanh", BF),
    ([0] * 255 + [17], 1, 0, 64, 128, "none", HF),
    ([0, 0, 0], 6, 0, 64, 64, "none", BF),
    ([3, 1, 4, 1, 5, 9, 2, 6] * 32, 0, 0, 128, 640, "swiglu", BF),
    ([0, 500, 1, 33, 0, 129, 700, 256], 5, 3, 1032, 2576, "swiglu", BF),
    ([130, 0, 600, 257, 31, 0, 64, 1000], 0, 0, 2880, 1096, "none", HF),
    ([97] * 20 + [0] * 3 + [300], 2, 0, 520, 1544, "gelu", BF),
]


def _grouped_case(counts, pad, first, K, N, fn, dt, seed=1):
    g = generator(sum(counts) + K + N + seed)
    E, off = len(counts), offsets_of(counts, first)
    P = int(off[-1]) + pad
    No = N // 2 if fn == "swiglu" else N
    x, w = normal(g, P, K, dtype=dt), normal(g, E, N, K, dtype=dt, std=2.0 / K ** 0.5)
    b = normal(g, E, N, dtype=torch.float32)
    return g, E, off, P, No, x, w, b


@pytest.mark.parametrize("counts,pad,first,K,N,fn,dt", GROUPED)
def test_grouped_forward(counts, pad, first, K, N, fn, dt):
    g, E, off, P, No, x, w, b = _grouped_case(counts, pad, first, K, N, fn, dt)
    x[:first] = float("nan")              # rows no expert covers hold anything
    if pad:
        x[-pad:] = float("inf")
    y, z = normal(g, P, No, dtype=dt), normal(g, P, N, dtype=dt)
    y0, z0 = y.clone(), z.clone()
    st = _status()
    moe.moe_grouped_linear(x, w, off.cuda(), b, fn=fn, y=y, z=z, want_z=True, status_word=st)
    o = off.tolist()
    for e in range(E):
        s = slice(o[e], o[e + 1])
        if o[e] == o[e + 1]:
            continue
        yr, zr, ey, ez = forward_ref(x[s], w[e], b[e], fn, None)
        assert_close(y[s], yr, ey, f"y of expert {e}")
        assert_close(z[s], zr, ez, f"z of expert {e}")
    for buf, was in ((y, y0), (z, z0)):   # untouched outside the experts' rows
        assert torch.equal(buf[:first], was[:first]) and torch.equal(buf[o[-1]:], was[o[-1]:])
    _ok(st)


@pytest.mark.parametrize("counts,pad,first,K,N,fn,dt", GROUPED)
def test_grouped_backward(counts, pad, first, K, N, fn, dt):
    g, E, off, P, No, x, w, b = _grouped_case(counts, pad, first, K, N, fn, dt, seed=2)
    dy, z = normal(g, P, No, dtype=dt), normal(g, P, N, dtype=dt, std=3.0)
    for t in (x, dy, z):                  # rows no expert covers hold anything
        t[:first] = float("nan")
        if pad:
            t[-pad:] = float("inf")
    dx = normal(g, P, K, dtype=dt)
    dx0 = dx.clone()
    zz = z if fn != "none" else None
    st = _status()
    _, dw, db = moe.moe_grouped_linear_backward(dy, x, w, off.cuda(), zz, fn=fn, dx=dx, need_db=True, status_word=st)
    o = off.tolist()
    for e in range(E):
        s = slice(o[e], o[e + 1])
        if o[e] == o[e + 1]:
            assert not bool(dw[e].any()) and not bool(db[e].any())
            continue
        refs, errs, norms = backward_ref(dy[s], x[s], w[e], None if zz is None else z[s], fn)
        _check_backward((dx[s], dw[e], db[e]), refs, errs, norms, dt, f"expert {e} ")
    assert torch.equal(dx[:first], dx0[:first]) and torch.equal(dx[o[-1]:], dx0[o[-1]:])
    _ok(st)


def test_grouped_nan_rows_and_weights_of_one_expert_stay_there():
    """A neighbour's NaN or infinite rows and weights do not reach an expert's results: tiles
    and contraction blocks straddle both."""
    counts, K, N = [37, 30, 90], 72, 72
    g, E, off, P, No, x, w, b = _grouped_case(counts, 0, 0, K, N, "none", BF)
    dy = normal(g, P, N)
    o = off.tolist()
    x[o[1]:o[2]] = float("inf")
    dy[o[1]:o[2]] = float("nan")
    w[1] = float("nan")
    y = moe.moe_grouped_linear(x, w, off.cuda(), b)
    dx, dw, db = moe.moe_grouped_linear_backward(dy, x, w, off.cuda(), need_db=True)
    for e in (0, 2):
        s = slice(o[e], o[e + 1])
        yr, _, ey, _ = forward_ref(x[s], w[e], b[e], "none", None)
        assert_close(y[s], yr, ey)
        refs, errs, norms = backward_ref(dy[s], x[s], w[e], None, "none")
        _check_backward((dx[s], dw[e], db[e]), refs, errs, norms, BF)


def test_grouped_bad_offsets_are_reported():
    """Decreasing or out-of-range offsets: recorded in the status word, nothing outside the buffers
    is touched (the kernels force the ranges into the buffer)."""
    K, N, P = 64, 64, 50
    x = torch.ones(P, K, dtype=BF, device="cuda")
    w = torch.ones(3, N, K, dtype=BF, device="cuda")
    for off in ([0, 20, 10, 50], [0, 20, 40, 70], [-5, 20, 40, 50]):
        o = torch.tensor(off, dtype=torch.int32, device="cuda")
        st = _status()
        moe.moe_grouped_linear(x, w, o, status_word=st)
        assert moe.moe_device_status(st) == moe.MOE_ERR_INVALID_ARG
        moe.moe_grouped_linear_backward(torch.ones(P, N, dtype=BF, device="cuda"), x, w, o, need_db=True, status_word=st)
        assert moe.moe_device_status(st) == moe.MOE_ERR_INVALID_ARG


def test_empty_batches():
    x, w = torch.empty(0, 64, dtype=BF, device="cuda"), torch.ones(32, 64, dtype=BF, device="cuda")
    assert moe.moe_linear(x, w).shape == (0, 32)
    dw, db = moe.moe_linear_backward(torch.empty(0, 32, dtype=BF, device="cuda"), x, w, need_db=True)[1:]
    assert not bool(dw.any()) and not bool(db.any())
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    w2 = torch.ones(2, 32, 64, dtype=BF, device="cuda")
    assert moe.moe_grouped_linear(x, w2, off).shape == (0, 32)
    dw, db = moe.moe_grouped_linear_backward(torch.empty(0, 32, dtype=BF, device="cuda"), x, w2, off, need_db=True)[1:]
    assert not bool(dw.any()) and not bool(db.any())


def test_graph_replay_and_streams():
    """A captured forward + backward replays on new contents; two streams run side by side."""
    g = generator(21)
    counts, K, N = [5, 0, 40, 90], 192, 320
    _, E, off, P, No, x, w, b = _grouped_case(counts, 0, 0, K, N, "swiglu", BF)
    dy, offd = normal(g, P, No), off.cuda()

    def step():
        y, z = moe.moe_grouped_linear(x, w, offd, b, fn="swiglu", want_z=True)
        return (y, z, *moe.moe_grouped_linear_backward(dy, x, w, offd, z, fn="swiglu", need_db=True))

    first = [t.clone() for t in step()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    x2 = normal(g, P, K)
    keep = x.clone()
    x.copy_(x2)
    graph.replay()
    new = [t.clone() for t in out]
    for a, e in zip(new, step()):
        assert torch.equal(a, e)
    x.copy_(keep)
    offd.copy_(offsets_of([60, 30, 45, 0]).cuda())   # other row counts in the same graph
    graph.replay()
    for a, e in zip(out, step()):
        assert torch.equal(a, e)
    offd.copy_(off.cuda())
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    with torch.cuda.stream(other):
        two = step()
    one = step()
    torch.cuda.synchronize()
    for a, c, e in zip(one, two, first):
        assert torch.equal(a, e) and torch.equal(c, e)


def test_injected_timeout_is_reported_and_cleared():
    x, w = torch.ones(40, 256, dtype=BF, device="cuda"), torch.ones(64, 256, dtype=BF, device="cuda")
    st = _status()
    moe.moe_debug_inject_timeout()
    moe.moe_linear(x, w, status_word=st)
    assert moe.moe_device_status(st) == moe.MOE_ERR_TIMEOUT
    y = moe.moe_linear(x, w, status_word=st)
    assert moe.moe_device_status(st) == moe.MOE_OK and bool((y == 256).all())


def test_on_a_stream_that_is_not_current():
    """`stream=`: the call's own scratch stays with that stream until it has passed."""
    g = generator(31)
    M, K, N = 300, 256, 640
    x, w, dy, z = normal(g, M, K), normal(g, N, K, std=0.1), normal(g, M, N // 2), normal(g, M, N)
    want = moe.moe_linear_backward(dy, x, w, z, fn="swiglu", need_db=True)
    s = torch.cuda.Stream()
    for _ in range(20):
        s.wait_stream(torch.cuda.current_stream())
        got = moe.moe_linear_backward(dy, x, w, z, fn="swiglu", need_db=True, stream=s)
        torch.empty(1 << 20, dtype=torch.uint8, device="cuda").fill_(255)   # would take the scratch's place
        s.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    big = [torch.empty(50 * 1024 * 1024, dtype=torch.uint8, device="cuda")]   # a workspace of the caller's
    got = moe.moe_linear_backward(dy, x, w, z, fn="swiglu", need_db=True, ws=big[0])
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    with pytest.raises(moe.MoeError):
        moe.moe_linear_backward(dy, x, w, z, fn="swiglu", ws=big[0][:4096])


BAND = 4096   # bytes of canary on each side (keeps 16-byte alignment)


def _banded(t):
    """The tensor's values inside a larger buffer of canary bytes: (buffer, view)."""
    n = t.numel() * t.element_size()
    buf = torch.full((n + 2 * BAND,), 0xA5, dtype=torch.uint8, device="cuda")
    view = buf[BAND:BAND + n].view(t.dtype).view(t.shape)
    view.copy_(t)
    return buf, view


def _intact(buf):
    return bool((buf[:BAND] == 0xA5).all()) and bool((buf[-BAND:] == 0xA5).all())


@pytest.mark.parametrize("counts,pad,first,K,N,fn,dt", [c for c in GROUPED if sum(c[0]) < 2000])
def test_no_store_outside_the_outputs(counts, pad, first, K, N, fn, dt):
    """Guard bands around every output and the workspace, and the bounds-checking build, whose
    stores at computed addresses report one outside its buffer."""
    from mxfp4_expert_gemm_b200 import build as libbuild
    g, E, off, P, No, x, w, b = _grouped_case(counts, pad, first, K, N, fn, dt, seed=5)
    dy, z, offd = normal(g, P, No, dtype=dt), normal(g, P, N, dtype=dt), off.cuda()
    zz = z if fn != "none" else None
    blank = lambda *s: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    bufs = [_banded(t) for t in (blank(P, No), blank(P, N), blank(P, K), blank(E, N, K))]
    (yb, y), (zb, zo), (dxb, dx), (dwb, dw) = bufs
    dims = moe.make_linear_dims(K, N, E, dt, fn)
    wsb, ws = _banded(torch.zeros(moe.moe_linear_workspace_bytes(dims, P), dtype=torch.uint8, device="cuda"))

    def run():
        st = _status()
        moe.moe_grouped_linear(x, w, offd, b, fn=fn, y=y, z=zo, want_z=True, status_word=st)
        moe.moe_grouped_linear_backward(dy, x, w, offd, zz, fn=fn, dx=dx, dw=dw, need_db=True, ws=ws, status_word=st)
        _ok(st)
        return [t.clone() for t in (y, zo, dx, dw)]

    first_run = run()
    assert all(_intact(t) for t in (yb, zb, dxb, dwb, wsb))
    for t in (y, zo, dx, dw):
        t.zero_()
    with moe.use_library(libbuild.build(bounds=True)):
        second = run()
    for a, c in zip(first_run, second):
        assert torch.equal(a, c)
