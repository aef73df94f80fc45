"""The distillation example runs and learns: the operators as they are used
together (8-bit head, alternatives, loss and gradient in place, products)."""
import importlib.util
import math
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_loss_falls():
    from tensor_core_dense_tma_gb300 import build as tcbuild
    tcbuild.build()
    spec = importlib.util.spec_from_file_location("distill_head", os.path.join(ROOT, "examples", "distill_head.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    h = m.run(steps=30, tokens=256, vocab=5003, width=256, report=lambda s: None)
    # the first step's student is uniform over the vocabulary
    assert abs(h[0]["first_choice"] + math.log(5003)) < 1e-3 and abs(h[0]["entropy"] - math.log(5003)) < 1e-3
    assert all(math.isfinite(x["loss"]) for x in h)
    assert h[-1]["loss"] < 0.9 * h[0]["loss"]
    assert h[-1]["first_choice"] > h[0]["first_choice"] + 0.5
