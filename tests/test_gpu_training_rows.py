"""The kernels that a training batch's row counts choose: the norm's backward pass over a ring of
asynchronous copies, the forward norm of a warp a row at every pack width, and the large products'
SwiGLU with a residual.  The checks are those of the smaller shapes."""
import pytest
import torch

import mxfp4_expert_gemm_b200 as moe
import test_gpu_norms as norms
import test_gpu_products as products
from _train_ref import generator, normal

pytestmark = pytest.mark.gpu

BF, HF, SF = torch.bfloat16, torch.float16, torch.float32


def ring_rows(d, dt):
    """The fewest rows for which the backward pass takes several rows at a time (16-byte packs)."""
    threads = (d * (4 if dt == SF else 2) // 16 + 1) // 2
    threads = (threads + 31) // 32 * 32
    groups = 8 if threads == 32 else 1
    blocks = torch.cuda.get_device_properties(0).multi_processor_count * max(1, 576 // (threads * groups))
    return 16 * blocks * groups


# one row past the threshold: the last step holds a single row
RING = [(2880, BF), (2880, HF), (2880, SF), (8192, BF), (4096, SF), (1024, HF), (1000, SF), (64, BF), (512, HF), (24, SF)]


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("d,dt", RING)
def test_norm_backward_of_many_rows(d, dt, kind):
    norms.test_norm(ring_rows(d, dt) + 1, d, kind, dt)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("d,dt,more", [(2880, BF, 1), (2880, SF, 2), (64, HF, 3)])
def test_norm_backward_of_many_rows_in_place(d, dt, more, kind):
    """dx over dy, x and dres, whose later rows are on their way while earlier ones are stored; and
    rows of wider buffers, whose other columns stay."""
    T = ring_rows(d, dt) + more
    g = generator(T + d)
    x, dy, dres = (normal(g, T, d + 16, dtype=dt) for _ in range(3))
    w = normal(g, d, dtype=SF, mean=1.0, std=0.2)
    view = lambda t: t[:, 8:8 + d]  # noqa: E731
    _, mean, rstd = moe.moe_norm(view(x), w, kind=kind, want_stats=True)
    want = moe.moe_norm_backward(view(dy), view(x), w, mean, rstd, kind=kind, dres=view(dres))
    plain = moe.moe_norm_backward(view(dy), view(x), w, mean, rstd, kind=kind)
    for dr, ref in ((dres, want), (None, plain)):
        for which in range(3 if dr is not None else 2):
            a = [dy.clone(), x.clone(), dr.clone() if dr is not None else None]
            before = a[which].clone()
            got = moe.moe_norm_backward(view(a[0]), view(a[1]), w, mean, rstd, kind=kind,
                                        dres=view(a[2]) if dr is not None else None, dx=view(a[which]))
            for p, q in zip(got, ref):
                assert (p is None and q is None) or torch.equal(p, q), which
            assert torch.equal(a[which][:, :8], before[:, :8]) and torch.equal(a[which][:, 8 + d:], before[:, 8 + d:])
    assert torch.equal(plain[1], want[1])   # the residual's gradient has no part in the column sums
    for need in (dict(need_dw=False, need_db=False), dict(need_dw=False)):
        got = moe.moe_norm_backward(view(dy), view(x), w, mean, rstd, kind=kind, dres=view(dres), **need)
        assert got[1] is None and torch.equal(got[0], want[0])


# each pack width (8 or 4, 2, 1 values) at each of the four row lengths that a warp's registers hold
WARP = [(512, BF), (776, HF), (1544, BF), (2880, HF), (258, BF), (1002, HF), (2002, BF), (3002, HF), (33, BF), (257, HF),
        (601, BF), (1001, HF), (200, SF), (500, SF), (1000, SF), (1500, SF), (31, SF), (255, SF), (603, SF), (1149, SF),
        (1153, BF), (3074, BF), (3080, HF)]


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("d,dt", WARP)
def test_norm_of_a_warp_a_row(d, dt, kind):
    norms.test_norm(2 * torch.cuda.get_device_properties(0).multi_processor_count + 5, d, kind, dt)


@pytest.mark.parametrize("off", [1, 2])
def test_norm_of_a_warp_a_row_in_views(off):
    """Rows that start on no 16-byte boundary: single values and pairs, in place."""
    g = generator(off)
    T, d = 301, 776
    buf = normal(g, T, d + 8)
    w, b = normal(g, d, dtype=SF, mean=1.0, std=0.2), normal(g, d, dtype=SF)
    x, before = buf[:, off:off + d], buf.clone()
    yr, m, r = norms.forward_ref(x, w, b, "layer")
    err = norms.errors(x, w, b, m, r, "layer")
    moe.moe_norm(x, w, b, kind="layer", eps=norms.EPS, y=x)
    norms.assert_close(x, yr, err)
    assert torch.equal(buf[:, :off], before[:, :off]) and torch.equal(buf[:, off + d:], before[:, off + d:])


@pytest.mark.parametrize("M,K,N,fn,dt,bias,residual,want_z", [
    (2111, 512, 2896, "swiglu", BF, True, True, True),
    (2111, 512, 2896, "swiglu", HF, False, True, False),
    (4099, 72, 2064, "swiglu", BF, True, True, False),
    (2500, 1024, 1040, "gelu_tanh", BF, True, True, True),
    (5001, 64, 1288, "silu", HF, False, True, False),
])
def test_large_products_with_a_residual(M, K, N, fn, dt, bias, residual, want_z):
    products.test_linear_forward(M, K, N, fn, dt, bias, residual, want_z)


@pytest.mark.parametrize("fn", ["none", "swiglu"])
def test_large_products_over_their_residual(fn):
    """y written over the residual it adds, in rows of a wider buffer."""
    g = generator(8)
    M, K, N = 2111, 520, 2896
    No = N // 2 if fn == "swiglu" else N
    x, w = normal(g, M, K), normal(g, N, K, std=2.0 / K ** 0.5)
    buf = normal(g, M, No + 24)
    y, before = buf[:, 8:8 + No], buf.clone()
    want = moe.moe_linear(x, w, fn=fn, residual=y)
    moe.moe_linear(x, w, fn=fn, residual=y, y=y)
    assert torch.equal(y, want)
    assert torch.equal(buf[:, :8], before[:, :8]) and torch.equal(buf[:, 8 + No:], before[:, 8 + No:])


@pytest.mark.parametrize("d,dt", [(768, BF), (1024, HF), (384, SF)])
def test_norm_backward_at_the_most_blocks(d, dt):
    """Rows of two warps: more blocks fit than write partial sums (592), and the rows at which each has
    eight steps of two rows follow from those."""
    for T in (16 * 592 - 1, 16 * 592 + 1):
        norms.test_norm(T, d, "layer", dt)
