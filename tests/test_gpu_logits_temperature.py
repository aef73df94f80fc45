"""Distillation at temperatures whose square is no fp32 number: the loss is
t^2 sum P (log P - log Q), of the order of t where t is small.  Tolerances as
in test_gpu_logits.py, relative to the size of the terms (their logarithms are
of the order of 1 / t)."""
import numpy as np
import pytest
import torch

from test_gpu_logits import err_log_sum, make, ref_distill, teacher

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [1e-4, 1e-18, 3e-20, 1e-22, 1e-25])
def test_small(t):
    from tensor_core_dense_tma_gb300 import build as tcbuild
    tcbuild.build()
    import tensor_core_dense_tma_gb300 as tc
    T, V, K = 4, 5000, 7
    t = float(np.float32(t))
    view, z = make(T, V, "f32", seed=8)
    tt, tv, tok, val = teacher(T, V, K, 9)
    loss, _ = tc.distill_topk(view, tt, tv, temperature=t)
    loss2, _ = tc.distill_topk_grad(view, tt, tv, torch.ones(T, device="cuda"), temperature=t)
    want, size, _ = ref_distill(z, tok, val, t)
    # terms of z / t: a difference of two logits, its scaling, the product with P and the sum
    tol = 2.0 ** -20 * (size + t * np.abs(z).max()) + t * t * err_log_sum(V)
    assert want[0] > 0.1 * t
    for got in (loss, loss2):
        assert np.all(np.abs(got.double().cpu().numpy() - want) <= tol)
