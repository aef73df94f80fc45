"""The policy loss where its ratio leaves fp32's range, and the KL term near 0 (bounds as in test_gpu_losses.py)."""
import numpy as np
import pytest
import torch

from test_gpu_logits import tc      # noqa: F401

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24


def test_ratio_beyond_fp32(tc):      # noqa: F811
    """r A of a ratio above 2^128: 0 for an advantage of 0, finite where the product is, infinite where it is not."""
    x = np.array([90.0, 100, 150, 170, 200, 500, 90, 100, 120, 150, 100, 100], dtype=np.float32)
    adv = np.array([0.0, -0.0, 0, 0, 0, 0, -1e-3, -1e-30, -1e-35, -1e-30, -1.0, 2.0], dtype=np.float32)
    T = len(x)
    z = torch.zeros((T, 4), device="cuda")
    tokens = torch.zeros(T, dtype=torch.int64, device="cuda")
    lp = tc.token_logprobs(z, tokens).logprob
    old = (lp - torch.from_numpy(x).cuda()).float()
    r = tc.policy_loss_grad(z, tokens, old, torch.from_numpy(adv).cuda(), torch.ones(T, device="cuda"))
    d = lp.double().cpu().numpy() - old.double().cpu().numpy()
    with np.errstate(over="ignore"):
        free, top = np.exp(d) * adv, np.float64(1) + 0.2
        want = -np.minimum(free, np.clip(np.exp(d), 0.8, top) * adv)
        want = np.where(np.abs(want) > np.finfo(np.float32).max, np.inf, want)
    got = r.loss.double().cpu().numpy()
    with np.errstate(invalid="ignore"):
        # two exponentials of half the argument, each off by 2 units and the argument's rounding
        near = np.abs(got - want) <= np.abs(want) * (12 * EPS + 2 * EPS * np.abs(d))
    assert ((got == want) | near).all(), (got, want)
    g = r.dlogits.double().cpu().numpy()
    assert not g[:6].any() and np.isfinite(g[6:10]).all() and (g[6:10, 0] > 0).all() and not g[11].any()
    assert not np.isnan(r.dlogits[:10].cpu().numpy()).any()
    # an old log-probability of -inf is a ratio of infinity: 0 times that has no value
    old[0] = -float("inf")
    assert torch.isnan(tc.policy_loss(z, tokens, old, torch.from_numpy(adv).cuda()).loss).tolist() == [True] + [False] * (T - 1)


def test_kl_is_never_negative(tc):      # noqa: F811
    """References a few units in the last place to some tenths from the log-probability."""
    T = 20000
    g = torch.Generator(device="cuda").manual_seed(3)
    z = torch.randn((T, 50), generator=g, device="cuda") * 2
    tokens = torch.randint(0, 50, (T,), generator=g, device="cuda")
    lp = tc.token_logprobs(z, tokens).logprob
    d = torch.randn(T, generator=g, device="cuda") * torch.exp2(-24 * torch.rand(T, generator=g, device="cuda"))
    ref = lp + d
    zero = torch.zeros(T, device="cuda")
    for r in (tc.policy_loss(z, tokens, lp, zero, ref, kl=1.0),
              tc.policy_loss_grad(z, tokens, lp, zero, zero + 1, ref, kl=1.0)):
        d = ref.double() - r.logprob.double()
        k = torch.expm1(d) - d
        assert bool((r.kl >= 0).all()) and torch.equal(r.loss, r.kl)
        assert bool(((r.kl.double() - k).abs() <= EPS * (4 * torch.expm1(d).abs() + 4 * d.abs()) + EPS * k).all())
