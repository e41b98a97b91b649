"""Calls of several streams at once, some of them replayed from graphs: each gives what it gives alone.
A call's later kernels start under their predecessors, and what they hold meanwhile must not keep
another stream's kernels from going on."""
import random

import pytest
import torch

import mxfp4_expert_gemm_b200 as moe
from _gpu_case import case
from _train_ref import generator, normal
from test_gpu_parity import SMALL

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(120)]

BF, HF, SF = torch.bfloat16, torch.float16, torch.float32


def _grouped(g, E, P, K, N, fn, dt):
    ids = torch.randint(0, E, (P,), generator=torch.Generator().manual_seed(P))
    off = torch.cat([torch.zeros(1, dtype=torch.int64), torch.bincount(ids, minlength=E).cumsum(0)]).int().cuda()
    No = N // 2 if fn == "swiglu" else N
    x, w = normal(g, P, K, dtype=dt), normal(g, E, N, K, dtype=dt, std=K ** -0.5)
    dy, z = normal(g, P, No, dtype=dt), normal(g, P, N, dtype=dt)
    return lambda s=None: [moe.moe_grouped_linear(x, w, off, fn=fn, stream=s), *moe.moe_grouped_linear_backward(
        dy, x, w, off, z if fn != "none" else None, fn=fn, need_db=True, stream=s)]


def _dense(g, M, K, N, fn, dt):
    No = N // 2 if fn == "swiglu" else N
    x, w = normal(g, M, K, dtype=dt), normal(g, N, K, dtype=dt, std=K ** -0.5)
    dy, z = normal(g, M, No, dtype=dt), normal(g, M, N, dtype=dt)
    return lambda s=None: [moe.moe_linear(x, w, fn=fn, residual=dy, stream=s), *moe.moe_linear_backward(
        dy, x, w, z if fn != "none" else None, fn=fn, need_db=True, stream=s)]


def _norm(g, T, d, dt):
    x, dy, w = normal(g, T, d, dtype=dt), normal(g, T, d, dtype=dt), normal(g, d, dtype=SF)

    def call(s=None):
        y, m, r = moe.moe_norm(x, w, kind="layer", want_stats=True, stream=s)
        return [y, *moe.moe_norm_backward(dy, x, w, m, r, kind="layer", stream=s)]
    return call


def _operators(g):
    return [_grouped(g, 8, 700, 256, 640, "swiglu", BF), _grouped(g, 32, 64, 512, 512, "silu", HF),
            _grouped(g, 5, 3000, 1024, 2048, "none", BF), _dense(g, 40, 2880, 2880, "gelu", BF),
            _dense(g, 300, 256, 64, "none", HF), _dense(g, 4099, 320, 1024, "swiglu", BF), _dense(g, 4, 2880, 2880, "none", BF),
            _dense(g, 2000, 64, 64, "relu", BF), _norm(g, 16, 2880, BF), _norm(g, 8000, 2880, BF), _norm(g, 300, 1001, HF)]


def _graph(call):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    return graph, out


def _run(calls, graphed, own, rounds, seed):
    """calls in random order on four streams; graphed: calls replayed on a stream each; own: calls that
    keep to one stream (their workspaces)."""
    rng = random.Random(seed)
    want = [[None if t is None else t.clone() for t in f()] for f in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    graphs = {s: (i, *_graph(calls[i])) for s, i in graphed.items()}
    free = [i for i in range(len(calls)) if i not in own.values()]
    for _ in range(rounds):
        done = []
        for _ in range(40):
            s = rng.randrange(4)
            if s in graphs and rng.random() < 0.2:
                i, graph, out = graphs[s]
                with torch.cuda.stream(streams[s]):
                    graph.replay()
            else:
                i = own[s] if s in own and rng.random() < 0.4 else rng.choice(free)
                out = calls[i](streams[s])
            done.append((i, out))
        torch.cuda.synchronize()
        for i, out in done:
            for a, b in zip(out, want[i]):
                assert (a is None and b is None) or torch.equal(a, b), i


def test_norms_and_products():
    _run(_operators(generator(1)), {0: 0, 1: 3, 2: 5, 3: 9}, {}, 40, 1)


def test_layers_of_both_paths_beside_them():
    """The MXFP4 layer's two paths on streams of their own, and the other calls around them."""
    c = case(SMALL["mid_ragged"])
    cfg, layers = c["cfg"], []
    for path in ("gemm", "gemv", "gemm", "gemv"):
        dims = moe.make_dims(cfg.d, cfg.I, cfg.E, cfg.k, cfg.rms_eps, cfg.swiglu_limit, path=path)
        ws = moe.new_workspace(dims, cfg.T)

        def layer(s=None, dims=dims, ws=ws):
            with torch.cuda.stream(s or torch.cuda.current_stream()):
                return [moe.moe_forward(dims, c["x_dev"], c["gamma_dev"], c["rw_dev"], c["rb_dev"], *c["W"]["gpu"], ws)]
        layers.append(layer)
    calls = _operators(generator(2))
    n = len(calls)
    _run(calls + layers, {2: 3}, {0: n, 1: n + 1, 2: n + 2, 3: n + 3}, 40, 2)
