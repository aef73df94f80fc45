"""Calls of the adapters' entry points that the documentation refuses or leaves to the callee."""
import pytest
import torch

from test_gpu_adapters import Case, plans, tc      # noqa: F401

pytestmark = pytest.mark.gpu


def test_gradient_without_hidden(plans):      # noqa: F811
    """hidden is an input of the backward pass: without it there is nothing to make d_up of."""
    plan = plans["bf16"]
    c = Case(40, 264, 520, 16, 3, "bf16", seed=40, index="mixed")
    with pytest.raises(ValueError, match="hidden"):
        plan.linear_adapters_grad(c.dY, c.B, c.X, None, c.down, c.up, c.index, c.scale)
    z = Case(40, 264, 520, 16, 0, "bf16", seed=40, index="none", scale=False)
    g = plan.linear_adapters_grad(z.dY, z.B, z.X, None, z.down, z.up, z.index)
    want = plan.gemm(z.dY, z.B.t(), out_dtype="bf16")
    assert torch.equal(g.dX, want) and g.d_down.shape == (0, 16, 520) and g.d_up.shape == (0, 264, 16)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    g = plan.linear_adapters_grad(c.dY[:0], c.B, c.X[:0], None, c.down, c.up, none, c.scale)
    assert g.dX.shape == (0, 520) and not g.d_down.any() and not g.d_up.any()
