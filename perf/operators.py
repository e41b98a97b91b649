"""Cases for measuring the training and dense-block operators of this library.

Three operators: the norm of a row (layer norm, or the RMSNorm of the MoE layer) with its
backward pass, the matrix product with bias, activation and residual in its epilogue with its
backward pass, and the same product grouped by expert over ragged row ranges, as moe_route's
offsets give them.  Each has its plain form here in elementary torch operations in 32 bits;
with ``own`` true, ``run`` makes the library's calls instead.

Formulas (per row; w, b and the statistics are fp32 in the norm, bias is fp32 in the products):
  norm     y = (x - m) * r * w + b,  m = mean(x) (0 for "rms"),  r = 1 / sqrt(mean((x - m)^2) + eps)
  product  z = x W^T + bias,  y = f(z) [+ residual];  "swiglu": W = [gate rows | up rows],
           y = silu(min(g, L)) * clamp(u, -L, L)
  grouped  the rows offsets[e] .. offsets[e + 1] - 1 take W[e] and bias[e]
"""
import math

import torch

own = False

LIMIT = 7.0
EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # the norm before a block at a decode batch of 16 tokens: latency
        dict(name="norm_rms_decode", op="norm", way="forward", kind="rms", dtype="bf16", T=16, d=2880, dres=False),
        # a training step's norm at 16384 tokens, forward, then backward with the residual's gradient added
        dict(name="norm_layer_train", op="norm", way="both", kind="layer", dtype="bf16", T=16384, d=2880, dres=True),
        # an odd number of rows of an fp32 model whose width is no power of two
        dict(name="norm_layer_fp32", op="norm", way="both", kind="layer", dtype="fp32", T=1021, d=1000, dres=False),
        # one token's output projection with its bias and the residual stream: the weights' bytes
        dict(name="linear_token", op="linear", way="forward", fn="none", dtype="bf16", M=1, K=2880, N=2880,
             bias=True, residual=True, want_z=False),
        # a dense block's first product at width 1024, with what its backward pass needs kept
        dict(name="linear_gelu", op="linear", way="forward", fn="gelu_tanh", dtype="fp16", M=4096, K=1024, N=4096,
             bias=True, residual=False, want_z=True),
        # a shared expert's gate_up at the largest prefill batch
        dict(name="linear_swiglu", op="linear", way="forward", fn="swiglu", dtype="bf16", M=16384, K=2880, N=5760,
             bias=True, residual=False, want_z=False),
        # the gradients of the width-1024 block at an odd number of rows
        dict(name="linear_backward", op="linear", way="backward", fn="gelu", dtype="bf16", M=4099, K=1024, N=4096,
             bias=True, residual=False, want_z=False),
        # a decode batch's 16 x 4 (token, expert) pairs over 32 experts: the used experts' bytes
        dict(name="grouped_decode", op="grouped", way="forward", fn="swiglu", dtype="bf16", P=64, pad=0, E=32,
             K=2880, N=5760, bias=True, want_z=False, spread="uniform"),
        # the gate_up products of 4096 tokens, top 4 of 32 experts
        dict(name="grouped_prefill", op="grouped", way="forward", fn="swiglu", dtype="bf16", P=16384, pad=0, E=32,
             K=2880, N=5760, bias=True, want_z=True, spread="uniform"),
        # the down products of 16384 tokens, top 4 of 128 experts of Zipf popularity
        dict(name="grouped_skew", op="grouped", way="forward", fn="none", dtype="bf16", P=65536, pad=0, E=128,
             K=2880, N=2880, bias=False, want_z=False, spread="zipf"),
        # all gradients of the gate_up products of 4096 tokens
        dict(name="grouped_backward", op="grouped", way="backward", fn="swiglu", dtype="bf16", P=16384, pad=0, E=32,
             K=2880, N=5760, bias=True, want_z=False, spread="uniform"),
        # a small layer's gradients in fp16: odd counts, empty experts, a buffer longer than its rows
        dict(name="grouped_backward_ragged", op="grouped", way="backward", fn="silu", dtype="fp16", P=777, pad=23,
             E=40, K=192, N=320, bias=True, want_z=False, spread="zipf"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _log_8(rng, lo, hi, unit=8):
    return unit * _log_int(rng, lo // unit, hi // unit)


def draw(rng):
    op = rng.choice(["norm", "linear", "linear", "grouped", "grouped"])
    if op == "norm":
        return dict(op=op, way=rng.choice(["forward", "both"]), kind=rng.choice(["rms", "layer"]),
                    dtype=rng.choice(["bf16", "fp16", "fp32"]), T=_log_int(rng, 1, 16384), d=_log_int(rng, 33, 6000),
                    dres=rng.random() < 0.5)
    fn = rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu", "swiglu", "swiglu"])
    way = rng.choice(["forward", "forward", "backward"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    K = _log_8(rng, 64, 4096)
    N = _log_8(rng, 64, 5760, 16)
    bias = rng.random() < 0.7
    want_z = way == "forward" and fn != "none" and rng.random() < 0.5
    if op == "linear":
        return dict(op=op, way=way, fn=fn, dtype=dtype, M=_log_int(rng, 1, 16384), K=K, N=N, bias=bias,
                    residual=way == "forward" and rng.random() < 0.5, want_z=want_z)
    return dict(op=op, way=way, fn=fn, dtype=dtype, P=_log_int(rng, 1, 16384), pad=rng.choice([0, 0, 1, 40]),
                E=_log_int(rng, 1, 128), K=min(K, 2880), N=N, bias=bias, want_z=want_z,
                spread=rng.choice(["uniform", "zipf"]))


def _popularity(c):
    ranks = torch.arange(1, c["E"] + 1, dtype=torch.float64)
    w = ranks.pow(-1.2) if c["spread"] == "zipf" else torch.ones_like(ranks)
    return w / w.sum()


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[c["dtype"]]

    def normal(*shape, dtype=dt, std=1.0, mean=0.0):
        t = torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, 1.0, generator=g)
        return t.mul_(std).add_(mean) if std != 1.0 or mean != 0.0 else t

    s = dict(c)
    if c["op"] == "norm":
        T, d = c["T"], c["d"]
        s["x"] = normal(T, d, mean=0.25)
        s["w"] = normal(d, dtype=torch.float32, std=0.1, mean=1.0)
        s["b"] = normal(d, dtype=torch.float32, std=0.1) if c["kind"] == "layer" else None
        if c["way"] == "both":
            s["dy"] = normal(T, d)
            s["r"] = normal(T, d) if c["dres"] else None
        return s
    K, N = c["K"], c["N"]
    No = N // 2 if c["fn"] == "swiglu" else N
    if c["op"] == "linear":
        rows, lead = c["M"], ()
    else:
        rows, lead = c["P"] + c["pad"], (c["E"],)
        cpu = torch.Generator().manual_seed(seed)
        pop = _popularity(c)[torch.randperm(c["E"], generator=cpu)]
        counts = torch.bincount(torch.multinomial(pop, c["P"], replacement=True, generator=cpu), minlength=c["E"])
        ends = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)])
        s["offsets"] = ends.to(torch.int32).cuda()
        s["ends"] = ends.tolist()   # the counts as a host program knows them
    s["x"] = normal(rows, K)
    s["W"] = normal(*lead, N, K, std=0.02)
    s["bias"] = normal(*lead, N, dtype=torch.float32, std=0.1) if c["bias"] else None
    if c["way"] == "backward":
        s["dy"] = normal(rows, No)
        s["z"] = normal(rows, N, std=0.02 * math.sqrt(K)) if c["fn"] != "none" else None
        if c["op"] == "grouped":
            s["dx"] = torch.zeros(rows, K, dtype=dt, device="cuda")
    else:
        s["residual"] = normal(rows, No) if c.get("residual") else None
        if c["op"] == "grouped":   # buffers that may be longer than their rows: those stay as they were
            s["y"] = torch.zeros(rows, No, dtype=dt, device="cuda")
            s["zout"] = torch.zeros(rows, N, dtype=dt, device="cuda") if c["want_z"] else None
    return s


# ------------------------------------------------------------------------------- plain forms (32 bits)
def _act(fn, z):
    if fn == "swiglu":
        g, u = z[:, : z.shape[1] // 2].clamp(max=LIMIT), z[:, z.shape[1] // 2:].clamp(-LIMIT, LIMIT)
        return g / (1 + torch.exp(-g)) * u
    if fn == "relu":
        return z.clamp(min=0)
    if fn == "silu":
        return z / (1 + torch.exp(-z))
    if fn == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if fn == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _dact(fn, z, dy):
    """The gradient of z from that of f(z); a clamp passes it on up to and at its bound."""
    if fn == "swiglu":
        I = dy.shape[1]
        g0, u0 = z[:, :I], z[:, I:]
        g, u = g0.clamp(max=LIMIT), u0.clamp(-LIMIT, LIMIT)
        sig = 1 / (1 + torch.exp(-g))
        dg = dy * u * sig * (1 + g * (1 - sig)) * (g0 <= LIMIT)
        du = dy * g * sig * ((u0 >= -LIMIT) & (u0 <= LIMIT))
        return torch.cat([dg, du], 1)
    if fn == "relu":
        return dy * (z > 0)
    if fn == "silu":
        sig = 1 / (1 + torch.exp(-z))
        return dy * sig * (1 + z * (1 - sig))
    if fn == "gelu":
        return dy * (0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi))
    if fn == "gelu_tanh":
        a = math.sqrt(2 / math.pi)
        t = torch.tanh(a * (z + 0.044715 * z * z * z))
        return dy * (0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * 0.044715 * z * z))
    return dy


def _plain_norm(s):
    dt = s["x"].dtype
    x, w = s["x"].float(), s["w"]
    m = x.mean(1, keepdim=True) if s["kind"] == "layer" else 0.0
    xc = x - m
    r = 1 / torch.sqrt((xc * xc).mean(1, keepdim=True) + EPS)
    xh = xc * r
    y = xh * w if s["b"] is None else xh * w + s["b"]
    if s["way"] == "forward":
        return y.to(dt)
    dy = s["dy"].float()
    dxh = dy * w
    dx = dxh - xh * (dxh * xh).mean(1, keepdim=True)
    if s["kind"] == "layer":
        dx = dx - dxh.mean(1, keepdim=True)
    dx = dx * r
    if s["r"] is not None:
        dx = dx + s["r"].float()
    out = [y.to(dt), dx.to(dt), (dy * xh).sum(0)]
    return out + [dy.sum(0)] if s["kind"] == "layer" else out


def _plain_forward(s, x, W, bias):
    z = x.float() @ W.float().t()
    if bias is not None:
        z = z + bias
    return z, _act(s["fn"], z)


def _plain_backward(s, x, W, z, dy):
    dz = dy.float() if z is None else _dact(s["fn"], z.float(), dy.float())
    return dz @ W.float(), dz.t() @ x.float(), dz.sum(0)


def _plain_linear(s):
    dt = s["x"].dtype
    if s["way"] == "forward":
        z, y = _plain_forward(s, s["x"], s["W"], s["bias"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return [y.to(dt), z.to(dt)] if s["want_z"] else [y.to(dt)]
    dx, dw, db = _plain_backward(s, s["x"], s["W"], s["z"], s["dy"])
    return [dx.to(dt), dw.to(dt), db] if s["bias"] is not None else [dx.to(dt), dw.to(dt)]


def _plain_grouped(s):
    # expert by expert: the row ranges are ragged, and padding them to the longest would hold
    # up to E times the rows
    dt, ends = s["x"].dtype, s["ends"]
    if s["way"] == "forward":
        y, zo = torch.zeros_like(s["y"]), None
        if s["want_z"]:
            zo = torch.zeros_like(s["zout"])
        for e in range(s["E"]):
            a, b = ends[e], ends[e + 1]
            if a < b:
                z, h = _plain_forward(s, s["x"][a:b], s["W"][e], None if s["bias"] is None else s["bias"][e])
                y[a:b] = h.to(dt)
                if zo is not None:
                    zo[a:b] = z.to(dt)
        return [y] if zo is None else [y, zo]
    dx, dw = torch.zeros_like(s["dx"]), torch.zeros_like(s["W"])
    db = torch.zeros(s["E"], s["N"], device="cuda")
    for e in range(s["E"]):
        a, b = ends[e], ends[e + 1]
        if a < b:
            z = None if s["z"] is None else s["z"][a:b]
            dxe, dwe, db[e] = _plain_backward(s, s["x"][a:b], s["W"][e], z, s["dy"][a:b])
            dx[a:b], dw[e] = dxe.to(dt), dwe.to(dt)
    return [dx, dw, db] if s["bias"] is not None else [dx, dw]


# ------------------------------------------------------------------------------- the library's calls
def _own_norm(s):
    import mxfp4_expert_gemm_b200 as moe
    if s["way"] == "forward":
        return moe.moe_norm(s["x"], s["w"], s["b"], kind=s["kind"], eps=EPS)
    y, mean, rstd = moe.moe_norm(s["x"], s["w"], s["b"], kind=s["kind"], eps=EPS, want_stats=True)
    dx, dw, db = moe.moe_norm_backward(s["dy"], s["x"], s["w"], mean, rstd, kind=s["kind"], dres=s["r"])
    return [y, dx, dw, db] if s["kind"] == "layer" else [y, dx, dw]


def _own_linear(s):
    import mxfp4_expert_gemm_b200 as moe
    if s["way"] == "forward":
        r = moe.moe_linear(s["x"], s["W"], s["bias"], fn=s["fn"], limit=LIMIT, residual=s["residual"],
                           want_z=s["want_z"])
        return list(r) if s["want_z"] else [r]
    dx, dw, db = moe.moe_linear_backward(s["dy"], s["x"], s["W"], s["z"], fn=s["fn"], limit=LIMIT,
                                         need_db=s["bias"] is not None)
    return [dx, dw, db] if s["bias"] is not None else [dx, dw]


def _own_grouped(s):
    import mxfp4_expert_gemm_b200 as moe
    if s["way"] == "forward":
        r = moe.moe_grouped_linear(s["x"], s["W"], s["offsets"], s["bias"], fn=s["fn"], limit=LIMIT, y=s["y"],
                                   z=s["zout"], want_z=s["want_z"])
        return list(r) if s["want_z"] else [r]
    dx, dw, db = moe.moe_grouped_linear_backward(s["dy"], s["x"], s["W"], s["offsets"], s["z"], fn=s["fn"],
                                                 limit=LIMIT, dx=s["dx"], need_db=s["bias"] is not None)
    return [dx, dw, db] if s["bias"] is not None else [dx, dw]


def run(state):
    if own:
        return {"norm": _own_norm, "linear": _own_linear, "grouped": _own_grouped}[state["op"]](state)
    return {"norm": _plain_norm, "linear": _plain_linear, "grouped": _plain_grouped}[state["op"]](state)


# ------------------------------------------------------------------------------- work and 64-bit values
def work(case):
    c = case
    size = 4 if c["dtype"] == "fp32" else 2
    if c["op"] == "norm":
        n = c["T"] * c["d"]
        moved = 2 * n if c["way"] == "forward" else (4 + (1 if c["dres"] else 0)) * n   # x, y; dy, dx [, dres]
        return {"bytes": size * moved + 4 * c["d"] * (2 if c["way"] == "forward" else 4),
                "flops": n * (6 if c["way"] == "forward" else 20)}
    K, N = c["K"], c["N"]
    No = N // 2 if c["fn"] == "swiglu" else N
    if c["op"] == "linear":
        M, experts, used = c["M"], 1, 1.0
    else:
        M, experts = c["P"], c["E"]
        used = float((1 - (1 - _popularity(c)).pow(c["P"])).sum())   # experts that get a row, on average
    if c["way"] == "forward":
        elems = M * (K + No * (2 if c.get("residual") else 1) + (N if c["want_z"] else 0)) + used * N * K
        return {"bytes": size * elems + 4 * N * used * c["bias"], "flops": 2.0 * M * N * K}
    elems = M * (No + (N if c["fn"] != "none" else 0) + 2 * K) + used * N * K + experts * N * K
    return {"bytes": size * elems + 4 * N * experts * c["bias"], "flops": 4.0 * M * N * K}


def _f64(fn, z):
    f = torch.nn.functional
    if fn == "swiglu":
        g, u = z.chunk(2, 1)
        return f.silu(g.clamp(max=LIMIT)) * u.clamp(-LIMIT, LIMIT)
    return {"none": lambda v: v, "relu": f.relu, "silu": f.silu, "gelu": f.gelu,
            "gelu_tanh": lambda v: f.gelu(v, approximate="tanh")}[fn](z)


def exact(case, seed):
    """What run() returns, in 64 bits: the forward formulas, and their gradients by differentiation."""
    s = prepare(case, seed)
    if s["op"] == "norm":
        x = s["x"].double().requires_grad_()
        w = s["w"].double().requires_grad_()
        b = None if s["b"] is None else s["b"].double().requires_grad_()
        if s["kind"] == "layer":
            y = torch.nn.functional.layer_norm(x, (s["d"],), w, b, EPS)
        else:
            y = x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * w
        if s["way"] == "forward":
            return y.detach()
        y.backward(s["dy"].double())
        dx = x.grad if s["r"] is None else x.grad + s["r"].double()
        return [y.detach(), dx, w.grad] if b is None else [y.detach(), dx, w.grad, b.grad]
    grouped = s["op"] == "grouped"
    parts = [(a, b) for a, b in zip(s["ends"], s["ends"][1:])] if grouped else [(0, s["M"])]
    rows, K, N = s["x"].shape[0], s["K"], s["N"]
    No = N // 2 if s["fn"] == "swiglu" else N
    new = lambda *shape: torch.zeros(shape, dtype=torch.float64, device="cuda")  # noqa: E731
    if s["way"] == "forward":
        out = [new(rows, No)] + ([new(rows, N)] if s["want_z"] else [])
    else:
        out = [new(rows, K), new(len(parts), N, K)] + ([new(len(parts), N)] if s["bias"] is not None else [])
    for e, (a, b) in enumerate(parts):
        if a == b:
            continue
        x = s["x"][a:b].double()
        W = (s["W"][e] if grouped else s["W"]).double()
        if s["way"] == "forward":
            z = torch.einsum("mk,nk->mn", x, W)
            if s["bias"] is not None:
                z += s["bias"].double().view(-1, N)[e]
            y = _f64(s["fn"], z)
            out[0][a:b] = y if s["residual"] is None else y + s["residual"][a:b].double()
            if s["want_z"]:
                out[1][a:b] = z
            continue
        dz = s["dy"][a:b].double()
        if s["z"] is not None:
            z = s["z"][a:b].double().requires_grad_()
            dz, = torch.autograd.grad(_f64(s["fn"], z), z, dz)
        out[0][a:b] = torch.einsum("mn,nk->mk", dz, W)
        out[1][e] = torch.einsum("mn,mk->nk", dz, x)
        if s["bias"] is not None:
            out[2][e] = dz.sum(0)
    if s["way"] == "backward" and not grouped:
        out[1:] = [t[0] for t in out[1:]]
    return out
