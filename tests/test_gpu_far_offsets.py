"""Tensors of more than 2^31 values: rows on both sides of the border, and the sums over all of them."""
import pytest
import torch

import mxfp4_expert_gemm_b200 as moe
import test_gpu_norms as norms
from _train_ref import FN_REL, assert_close, backward_ref, df_ref, forward_ref, generator, half_step, normal

pytestmark = pytest.mark.gpu

ROWS, D = 1_060_000, 2056   # 2.18e9 values
CHUNK = 53_000


def _sampled(lo=0, hi=ROWS):
    border = 2 ** 31 // D
    r = torch.cat([torch.arange(lo, lo + 200), torch.arange(border - 100, border + 100), torch.arange(hi - 200, hi)])
    return r.cuda()


def _big(g, n, std=1.0):
    t = torch.empty(ROWS, n, dtype=torch.bfloat16, device="cuda")
    for s in range(0, ROWS, CHUNK):
        t[s:s + CHUNK] = normal(g, min(CHUNK, ROWS - s), n, std=std)
    return t


def test_grouped_product():
    g = generator(1)
    K, N, fn = 64, D, "silu"
    ends = [7, 400_001, 400_001, ROWS - 5]
    off = torch.tensor(ends, dtype=torch.int32, device="cuda")
    x, dy = _big(g, K), _big(g, N)
    w, b = normal(g, 3, N, K, std=0.2), normal(g, 3, N, dtype=torch.float32)
    st = torch.zeros(4, dtype=torch.int32, device="cuda")
    y, z = moe.moe_grouped_linear(x, w, off, b, fn=fn, want_z=True, status_word=st)
    dx, dw, db = moe.moe_grouped_linear_backward(dy, x, w, off, z, fn=fn, need_db=True, status_word=st)
    assert moe.moe_device_status(st) == moe.MOE_OK
    rows = _sampled(7, ROWS - 5)
    for e in (0, 2):
        r = rows[(rows >= ends[e]) & (rows < ends[e + 1])]
        assert r.numel() >= 200
        yr, zr, ey, ez = forward_ref(x[r], w[e], b[e], fn, None)
        assert_close(y[r], yr, ey, "y")
        assert_close(z[r], zr, ez, "z")
        refs, errs, _ = backward_ref(dy[r], x[r], w[e], z[r], fn)
        assert_close(dx[r], refs[0], errs[0], "dx")
        # dw and db over the expert's n rows.  The terms have random signs: a running sum stays within
        # three times the root of their squares' sum q.  dw: dz is rounded to bf16 (half a step of each
        # term, independently), and the accumulator takes 16 rows a step, each off by 2^-23 of it at
        # most.  db: 8 rows a warp, 8 warps, every eighth of n / 64 chunks, 8 sums: n / 512 + 24 additions
        # in a chain.
        sw, sb, qw, qb = 0.0, 0.0, 0.0, 0.0
        for s in range(ends[e], ends[e + 1], CHUNK):
            c = slice(s, min(s + CHUNK, ends[e + 1]))
            dz, xd = df_ref(fn, z[c].double(), dy[c].double()), x[c].double()
            sw, sb = sw + dz.t() @ xd, sb + dz.sum(0)
            qw, qb = qw + dz.square().t() @ xd.square(), qb + dz.square().sum(0)
        n = ends[e + 1] - ends[e]
        ew, eb = (dw[e].double() - sw).norm(), (db[e].double() - sb).norm()
        tw = half_step(x.dtype) + 8 * FN_REL + 3 * (n / 16 + 16) * 2.0 ** -23
        tb = 8 * FN_REL + 3 * (n / 512 + 32) * 2.0 ** -24
        assert float(ew) <= float(tw * qw.sqrt().norm() + half_step(x.dtype) * sw.norm())
        assert float(eb) <= float(tb * qb.sqrt().norm())
    assert not bool(dw[1].any()) and not bool(db[1].any())


def test_norm():
    g = generator(2)
    x, dy, dres = _big(g, D, std=2.0), _big(g, D), _big(g, D)
    w, b = normal(g, D, dtype=torch.float32, mean=1.0, std=0.2), normal(g, D, dtype=torch.float32)
    y, mean, rstd = moe.moe_norm(x, w, b, kind="layer", eps=norms.EPS, want_stats=True)
    r = _sampled()
    yr, m, rs = norms.forward_ref(x[r], w, b, "layer")
    assert_close(y[r], yr, norms.errors(x[r], w, b, m, rs, "layer"))
    dx, dw, db = moe.moe_norm_backward(dy, x, w, mean, rstd, kind="layer", dres=dres)
    few = moe.moe_norm_backward(dy[r], x[r], w, mean[r], rstd[r], kind="layer", dres=dres[r])[0]
    assert_close(dx[r], few.double(), 2.0 ** -20 * (few.double().abs() + dres[r].double().abs() + 1), "dx")   # (two kernels)
    sw, sb, qw, qb = 0.0, 0.0, 0.0, 0.0
    for s in range(0, ROWS, CHUNK):
        c = slice(s, s + CHUNK)
        d = dy[c].double()
        t = d * ((x[c].double() - mean[c].double()[:, None]) * rstd[c].double()[:, None])
        sw, sb, qw, qb = sw + t.sum(0), sb + d.sum(0), qw + t.square().sum(0), qb + d.square().sum(0)
    # a block's rows (one of 444) in a chain, then the blocks': 2^-24 of a running sum each, which stays
    # within three times the root of the terms' squares; 8 roundings of each term on the way to it
    steps = 3 * (ROWS / 444 + 64) + 8
    for got, want, q in ((dw, sw, qw), (db, sb, qb)):
        assert float((got.double() - want).norm()) <= float(steps * 2.0 ** -24 * q.sqrt().norm())
