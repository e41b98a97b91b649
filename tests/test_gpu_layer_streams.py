"""The MXFP4 layer's calls on a stream that is not the current one: what they make is that stream's."""
import pytest
import torch

import mxfp4_expert_gemm_b200 as moe
from _train_ref import generator, normal

pytestmark = pytest.mark.gpu


def _calls():
    g = generator(7)
    T, d, I, E, k = 24, 128, 192, 4, 2
    x, s = normal(g, T, d), normal(g, T, d, dtype=torch.float32)
    gamma, rw, rb = normal(g, d, dtype=torch.float32, mean=1.0, std=0.1), normal(g, E, d, dtype=torch.float32), normal(g, E, dtype=torch.float32)
    w1, w2 = normal(g, E, 2 * I, d, dtype=torch.float32, std=0.1), normal(g, E, d, I, dtype=torch.float32, std=0.1)
    W = [*moe.moe_mxfp4_quantize(w1, role="gate_up"), *moe.moe_mxfp4_quantize(w2, role="down")]
    dims = moe.make_dims(d, I, E, k)
    ws = moe.new_workspace(dims, T)
    base = (dims, x, gamma, rw, rb)

    def routed(r):
        return [r[0], *r[1].values()]

    return dict(
        quantize=lambda st: list(moe.moe_mxfp4_quantize(w1, role="gate_up", stream=st)),
        route=lambda st: list(moe.moe_route(*base, ws, stream=st).values()),
        forward=lambda st: routed(moe.moe_forward(*base, *W, ws, want_routing=True, stream=st)),
        partial=lambda st: routed(moe.moe_forward_partial(*base, *W, ws, want_routing=True, stream=st)),
        norm=lambda st: list(moe.moe_forward_norm(*base, *W, ws, gamma, stream=st)),
        residual=lambda st: list(moe.moe_residual_norm(x, s, gamma, stream=st)),
        timed=lambda st: [moe.moe_forward_timed(*base, *W, ws, stream=st)],
        no_alloc=lambda st: [moe.moe_forward_no_alloc(*base, *W, stream=st)])


@pytest.mark.parametrize("name", ["quantize", "route", "forward", "partial", "norm", "residual", "timed", "no_alloc"])
def test_outputs_are_of_the_calls_stream(name):
    call = _calls()[name]
    want = call(None)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(s)
    s.synchronize()
    segments = torch.cuda.memory_snapshot()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
        mine = [q for q in segments if q["address"] <= a.data_ptr() < q["address"] + q["total_size"]]
        assert [q["stream"] for q in mine] == [s.cuda_stream]
