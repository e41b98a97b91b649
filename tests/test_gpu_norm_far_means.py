"""The layer norm's backward pass on rows whose mean is far larger than their spread, and on rows of two
and three values, whose gradients nearly cancel: from the same statistics the gradients keep the
accuracy of the formula, which subtracts the mean first."""
import pytest
import torch

import mxfp4_expert_gemm_b200 as moe
from _train_ref import assert_close, generator, normal
from test_gpu_training_rows import ring_rows

pytestmark = pytest.mark.gpu

BF, HF, SF = torch.bfloat16, torch.float16, torch.float32


@pytest.mark.parametrize("T,d,dt,mean,std", [
    (386, 2, SF, 0.5, 2.0), (5869, 2, SF, 0.5, 2.0), (2499, 3, SF, 0.5, 2.0), (2988, 2, HF, 0.5, 2.0), (100, 2, HF, 0.5, 2.0),
    (700, 33, SF, 1000.0, 1.0), (300, 1000, SF, 1000.0, 0.25), (300, 2880, BF, 256.0, 6.0), (300, 1002, HF, 512.0, 1.0),
    (-1, 2880, SF, -3000.0, 2.0), (-1, 2880, BF, 256.0, 6.0), (-1, 64, HF, -512.0, 1.5), (3, 20000, SF, 1000.0, 1.0)])
def test_gradients(T, d, dt, mean, std):
    T = ring_rows(d, dt) + 1 if T < 0 else T
    g = generator(T + d)
    x = normal(g, T, d, dtype=dt, std=std, mean=mean)
    w, b = normal(g, d, dtype=SF, std=0.3, mean=1.0), normal(g, d, dtype=SF)
    dy = normal(g, T, d, dtype=dt)
    _, m, rstd = moe.moe_norm(x, w, b, kind="layer", eps=1e-5, want_stats=True)
    dx, dw, db = moe.moe_norm_backward(dy, x, w, m, rstd, kind="layer")
    m, r = m.double()[:, None], rstd.double()[:, None]
    xh, dyd = (x.double() - m) * r, dy.double()
    gg = dyd * w.double()
    want = r * (gg - xh * (gg * xh).mean(1, keepdim=True) - gg.mean(1, keepdim=True))
    # every term carries a few roundings of 2^-24, a sum of d terms d / 32 + 40 at most (32 lanes or more)
    n = (d / 32 + 48) * 2.0 ** -24
    mag = gg.abs() + xh.abs() * (gg * xh).abs().mean(1, keepdim=True) + gg.abs().mean(1, keepdim=True)
    assert_close(dx, want, r * n * mag, "dx")
    nt = (T + 16) * 2.0 ** -24
    assert_close(dw, (dyd * xh).sum(0), nt * (dyd * xh).abs().sum(0) + 1e-30, "dw")
    assert_close(db, dyd.sum(0), nt * dyd.abs().sum(0) + 1e-30, "db")
