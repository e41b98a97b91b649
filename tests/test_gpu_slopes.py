"""Slopes of the activations at the ends of the types' ranges."""
import pytest
import torch

import mxfp4_expert_gemm_b200 as moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fn", ["relu", "gelu", "gelu_tanh", "silu"])
def test_slopes_far_from_zero(fn):
    """At the ends of bf16's range an activation's slope is 1 or 0 (db of one row is its dz)."""
    z = torch.tensor([1e4, 1e10, 1e19, 2e19, 1e20, 1e30, 3e38, 1e3], dtype=torch.bfloat16, device="cuda")
    z = torch.cat([z, -z])[None]
    w = torch.zeros(16, 8, dtype=torch.bfloat16, device="cuda")
    x, dy = torch.ones(1, 8, dtype=torch.bfloat16, device="cuda"), torch.full_like(z, 1.5)
    dx, dw, db = moe.moe_linear_backward(dy, x, w, z, fn=fn, need_db=True)
    want = torch.tensor([1.5] * 8 + [0.0] * 8, device="cuda")
    assert torch.equal(db, want), db
    assert torch.equal(dw, want[:, None].expand(16, 8).to(dw.dtype)) and not bool(dx.any())
