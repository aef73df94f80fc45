"""The preference loss and its slope at margins of all sizes, relative to themselves.

The rows' log-probabilities are taken as the kernel gives them; their sums are 64-bit, so the margin m is known
to 2^-50.  In units of eps = 2^-24: the exponential is off by 4 (two units in the last place), its correction by 1, 1 + x,
the quotient, 1 - smoothing, the product with it and those with beta and w by 1 each, and log1p by 2: the terms of a loss
and of a slope by at most 12 of themselves.  (A margin rounded to fp32 is off by |m| eps, and e^-m with it.)
"""
import numpy as np
import pytest
import torch

from test_gpu_logits import tc      # noqa: F401

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24


@pytest.mark.parametrize("e", [0.0, 0.1, 0.5, 1.0])
@pytest.mark.parametrize("beta", [1.0, 0.3, -0.7])
def test_margins(tc, e, beta):      # noqa: F811
    """Sequences of one row, whose token has a probability of e^-40: its gradient is the slope itself."""
    P = 4000
    rng = np.random.default_rng(1)
    z = torch.zeros((2 * P, 2), device="cuda")
    z[:, 1] = -40
    tokens = torch.ones(2 * P, dtype=torch.int64, device="cuda")
    size = np.concatenate([rng.uniform(-80, 80, P), rng.normal(size=P) * np.exp2(rng.uniform(-30, 4, P))])
    ref = (-40 - size / beta).astype(np.float32)
    w = rng.random(P).astype(np.float32) + np.float32(0.1)
    r = tc.preference_loss_grad(z, tokens, torch.arange(2 * P + 1, device="cuda"), torch.from_numpy(w).cuda(),
                                torch.from_numpy(ref).cuda(), beta=beta, smoothing=e)
    beta, e = float(np.float32(beta)), float(np.float32(e))
    reward = beta * (r.logprob.double().cpu().numpy() - ref.astype(np.float64))
    m = reward[0::2] - reward[1::2]
    assert np.abs(m).max() > 60 and np.abs(m).min() < 1e-2
    right, wrong = (1 - e) * np.logaddexp(0, -m), (e * np.logaddexp(0, m) if e else 0 * m)
    loss = right + wrong
    off = np.abs(r.loss.double().cpu().numpy() - loss)
    assert (off <= 12 * EPS * loss + 1e-37).all(), (off / (EPS * loss)).max()
    up, down = e / (1 + np.exp(-m)), (1 - e) / (1 + np.exp(m))
    g = r.dlogits[:, 1].double().cpu().numpy()
    for side, sign in ((0, 1), (1, -1)):
        off = np.abs(g[side::2] - sign * w * beta * (up - down))
        assert (off <= 12 * EPS * np.abs(w * beta) * (up + down) + 1e-37).all(), (off / (EPS * np.abs(w * beta) * (up + down))).max()


def test_far_margins(tc):      # noqa: F811
    """Beyond fp32's range, infinite and equal: no NaN comes of them."""
    z = torch.zeros((8, 2), device="cuda")
    tokens = torch.zeros(8, dtype=torch.int64, device="cuda")
    top = torch.finfo(torch.float32).max
    ref = torch.tensor([-top, top, top, -top, 1.0, 1.0, -300.0, 300.0], device="cuda")
    r = tc.preference_loss_grad(z, tokens, torch.arange(9, device="cuda"), torch.ones(4, device="cuda"), ref, beta=1.0)
    assert r.loss[0].item() == 0 and r.loss[1].item() == float("inf") and abs(r.loss[2].item() - np.log(2)) < EPS
    assert r.loss[3].item() == 0 and not r.dlogits[:2].any() and not r.dlogits[6:].any()
    # (sigma(-m) is 1: the preferred token's p is 1/2)
    assert r.dlogits[2].tolist() == [-0.5, 0.5] and r.dlogits[3].tolist() == [0.5, -0.5]
    assert r.dlogits[4].tolist() == [-0.25, 0.25]
