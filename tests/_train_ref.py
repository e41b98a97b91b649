"""64-bit references of the norms and 16-bit products, and the error bounds their tests use.

A rounding to a type of machine epsilon eps is off by at most eps / 2 relative to the value.
The tensor cores add products of 16-bit values in fp32, 16 at a time: for a contraction of
length C at most C / 16 + 16 steps, each off by at most 2^-23 of the sum of magnitudes
(truncation included), which `acc_bound` counts.
"""
import math

import torch

LIMIT = 7.0


def f_ref(fn, z, limit=LIMIT):
    if fn == "swiglu":
        g, u = z.chunk(2, -1)
        g, u = g.clamp(max=limit), u.clamp(-limit, limit)
        return g * torch.sigmoid(g) * u
    if fn == "relu":
        return z.clamp(min=0)
    if fn == "silu":
        return z * torch.sigmoid(z)
    if fn == "gelu":
        return 0.5 * z * torch.erfc(-z * math.sqrt(0.5))
    if fn == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return z


def df_ref(fn, z, dy, limit=LIMIT):
    """dz = dy f'(z), written out (a clamp passes the gradient up to and at its bound)."""
    if fn == "swiglu":
        g0, u0 = z.chunk(2, -1)
        g, u = g0.clamp(max=limit), u0.clamp(-limit, limit)
        s = torch.sigmoid(g)
        return torch.cat([dy * u * s * (1 + g * (1 - s)) * (g0 <= limit), dy * g * s * (u0.abs() <= limit)], -1)
    if fn == "relu":
        return dy * (z > 0)
    if fn == "silu":
        s = torch.sigmoid(z)
        return dy * s * (1 + z * (1 - s))
    if fn == "gelu":
        return dy * (0.5 * torch.erfc(-z * math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi))
    if fn == "gelu_tanh":
        a = math.sqrt(2 / math.pi)
        s = torch.sigmoid(2 * a * (z + 0.044715 * z ** 3))
        return dy * (s + 2 * z * s * (1 - s) * a * (1 + 3 * 0.044715 * z * z))
    return dy


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def floor_of(dtype):
    """Half the spacing of the type's smallest values (fp16 outputs may be subnormal)."""
    fi = torch.finfo(dtype)
    return fi.tiny * fi.eps / 2


def acc_bound(a, b, C):
    """Bound of a @ b's accumulation error, from the magnitudes."""
    return (C / 16 + 16) * 2.0 ** -23 * (a.abs() @ b.abs())


# Relative error of an activation and of its derivative as computed in fp32: the hardware
# exponential and divide (2 ulp of the result each, the exponent's own rounding times |z| <= 30)
# and a handful of fp32 roundings.
FN_REL = 64 * 2.0 ** -24
# |f'| <= 1.13 for every activation here.
SLOPE = 1.13


def forward_ref(x, w, bias, fn, residual, limit=LIMIT):
    """(y, z, bound of y, bound of z) in 64 bits; the bounds without the outputs' rounding."""
    x, w = x.double(), w.double()
    z = x @ w.t()
    ez = acc_bound(x, w.t(), x.shape[1])
    if bias is not None:
        z = z + bias.double()
        ez = ez + 2.0 ** -24 * z.abs()
    y = f_ref(fn, z, limit)
    if fn == "swiglu":
        g, u = z.chunk(2, -1)
        eg, eu = ez.chunk(2, -1)
        gc, uc = g.clamp(max=limit), u.clamp(-limit, limit)
        ey = SLOPE * eg * (uc.abs() + eu) + (gc * torch.sigmoid(gc)).abs() * eu
    else:
        ey = SLOPE * ez if fn != "none" else ez
    if fn != "none":
        ey = ey + FN_REL * y.abs()
    if residual is not None:
        y = y + residual.double()
        ey = ey + 2.0 ** -24 * (y.abs() + ey)
    return y, z, ey, ez


def assert_close(got, ref, err, what=""):
    """got (rounded to its type) against ref, whose computation is off by at most err."""
    dt = got.dtype
    g = got.double()
    tol = half_step(dt) * (ref.abs() + err) + err + floor_of(dt)
    bad = ~((g - ref).abs() <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), got.numel(), float((g - ref).abs()[bad].max()),
                                 float(ref.abs().max()), torch.nonzero(bad)[:4].tolist())


def backward_ref(dy, x, w, z, fn, limit=LIMIT):
    """dx, dw, db and bounds of their errors.  dz enters the products rounded to the inputs' type:
    off by at most half a step (and FN_REL) of |dz| per element."""
    dt = x.dtype
    dy, x, w = dy.double(), x.double(), w.double()
    dz = df_ref(fn, None if z is None else z.double(), dy, limit)
    rel = 0.0 if fn == "none" else half_step(dt) + SLOPE * 4 * FN_REL
    # where f' nearly cancels, its fp32 evaluation is off by FN_REL of its terms (at most 2 |dy|
    # times the other factor), not of their sum
    mag = dz.abs()
    if fn != "none":
        other = 1.0
        if fn == "swiglu":
            g, u = z.double().chunk(2, -1)
            other = torch.cat([u.clamp(-limit, limit).abs(), g.clamp(max=limit).abs()], -1)
            dcat = torch.cat([dy, dy], -1)
        else:
            dcat = dy * (1 + z.double().abs())
        mag_fn = 4 * FN_REL * dcat.abs() * other
    else:
        mag_fn = 0.0 * mag
    edz = rel * mag + mag_fn + (floor_of(dt) if fn != "none" else 0.0)
    dx, dw, db = dz @ w, dz.t() @ x, dz.sum(0)
    edx = acc_bound(dz, w, dz.shape[1]) + edz @ w.abs()
    edw = acc_bound(dz.t(), x, dz.shape[0]) + edz.t() @ x.abs()
    edb = (dz.shape[0] + 8) * 2.0 ** -24 * dz.abs().sum(0) + (mag_fn + 4 * FN_REL * mag * (fn != "none")).sum(0)
    # the same with independent roundings: root of the summed squares, for a check of the norms
    rss = lambda a, b: torch.sqrt(a.square() @ b.square())  # noqa: E731
    sdx = rel * rss(dz, w).norm() + half_step(dt) * dx.norm()
    sdw = rel * rss(dz.t(), x).norm() + half_step(dt) * dw.norm()
    return (dx, dw, db), (edx, edw, edb), (sdx, sdw)


def normal(g, *shape, dtype=torch.bfloat16, std=1.0, mean=0.0, device="cuda"):
    t = torch.empty(shape, dtype=torch.float32, device=device).normal_(mean, std, generator=g)
    return t.to(dtype)


def generator(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def offsets_of(counts, first=0):
    out = [first]
    for c in counts:
        out.append(out[-1] + c)
    return torch.tensor(out, dtype=torch.int32)
