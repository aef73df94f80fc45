"""The example that uses the adapters and the two losses together: it runs, and
its gradients are those of the whole chain in 64 bits."""
import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def adapted(x, head, lower, upper, index, scale):
    y = x @ head.t()
    for a in range(lower.shape[0]):
        mine = (index == a)[:, None]
        y = y + torch.where(mine, scale[a] * (x @ lower[a].t()) @ upper[a].t(), torch.zeros_like(y))
    return y


def check(s):
    """Gradients of both losses for factors and hidden states, by torch in 64
    bits from the same 16-bit logits: dlogits are rounded to bf16 once (half a
    unit, 2^-8 of each), which the sums that follow average but do not exceed:
    2^-8 of the sum of the magnitudes, and the outputs' own rounding of dX."""
    d = lambda t: t.detach().double()      # noqa: E731
    n = s["w_token"].numel()
    z = d(s["seen"]).requires_grad_()
    lp = torch.log_softmax(z, 1)
    at = lp.gather(1, s["answers"][:, None])[:, 0]
    diff = at[:n] - d(s["ref"])[:n]
    o = s["offsets"].tolist()
    reward = s["beta"] * torch.stack([diff[i:j].sum() for i, j in zip(o, o[1:])])
    pref = torch.nn.functional.softplus(reward[1::2] - reward[0::2])
    new, old, A = at[n:], d(s["ref"])[n:], d(s["advantage"])
    r = torch.exp(new - old)
    k = torch.exp(old - new) - (old - new) - 1
    ent = -(lp[n:].exp() * lp[n:]).sum(1)
    pol = -torch.minimum(r * A, r.clamp(0.8, 1.28) * A) + 0.05 * k - 0.001 * ent
    ((d(s["w_pair"]) * pref).sum() + (d(s["w_token"]) * pol).sum()).backward()
    assert torch.allclose(d(s["pref"].loss), pref.detach(), rtol=1e-4, atol=1e-5)
    assert torch.allclose(d(s["pol"].loss), pol.detach(), rtol=1e-4, atol=1e-5)
    # a ratio next to a border of the clipped range may fall on either side
    near = ((r - 0.8).abs() < 1e-4) | ((r - 1.28).abs() < 1e-4)
    assert not bool(near.any())
    dz = z.grad
    tol = 2.0 ** -8 * dz.abs() + 1e-4 * dz.abs().amax(1, keepdim=True)
    assert bool(((d(s["dlogits"]) - dz).abs() <= tol).all())
    # the chain from the rounded logits' gradient on is exact but for fp32 sums
    dz = d(s["dlogits"])
    leaves = [d(s[k]).requires_grad_() for k in ("hidden_states", "lower", "upper")]
    adapted(leaves[0], d(s["head"]), leaves[1], leaves[2], s["index"], d(s["scale"])).backward(dz)
    for got, leaf, half in zip(s["grads"], leaves, (2.0 ** -8, 0.0, 0.0)):
        size = leaf.grad.abs().amax()
        assert bool(((d(got) - leaf.grad).abs() <= half * leaf.grad.abs() + 1e-3 * size).all())


def test_runs_and_gradients():
    from tensor_core_dense_tma_gb300 import build as tcbuild
    tcbuild.build()
    spec = importlib.util.spec_from_file_location("preference_adapters",
                                                  os.path.join(ROOT, "examples", "preference_adapters.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    h = m.run(steps=4, tokens=128, vocab=1003, width=264, report=lambda s: None, check=check)
    # the first step's policy is the reference
    assert abs(h[0]["preference"] - math.log(2)) < 1e-5 and abs(h[0]["margin"]) < 1e-5 and abs(h[0]["kl"]) < 1e-6
    assert all(math.isfinite(v) for x in h[:-1] for v in x.values())
    served, which, state = h[-1]["served"], h[-1]["which"], h[-1]["state"]
    x, head, lower, upper, scale = (t.double() for t in state)
    want = adapted(x, head, lower, upper, which, scale)
    assert bool(((served.double() - want).abs() <= 1e-4 * want.abs().amax()).all())
