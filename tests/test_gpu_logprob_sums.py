"""Log-probabilities as callers add them up (include/logits.h): the same from every operator on equal logits,
and without an error to one side.

Tolerance of a mean over N rows.  A log-probability of 16 or less in size is rounded three times at most, each
off by half a unit, 2^-21, at most: a row is off by less than 2^-20 rms, to either side, and the mean over N rows, at six
times its deviation, by 6 * 2^-20 / sqrt(N).  (Errors to one side that are left out are larger: 2e-8 to 5e-8 for each
of the two to five exponentials on a value's way into the sum, up to 2e-7 for a logarithm of lg2.approx.  What is put
back for the exponentials is their mean over all arguments, 2^-28 more.)
"""
import math

import pytest
import torch

from test_gpu_logits import tc      # noqa: F401

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def logits(T, V, kind, seed, size):
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = (torch.randn((T, V), generator=g, device="cuda") * size).to(TYPES[kind])
    return z, torch.randint(0, V, (T,), generator=g, device="cuda"), g


def exact(z, tokens, t):
    out = []
    for part, tok in zip(z.split(1024), tokens.split(1024)):
        x = part.double() / t
        out.append(x.gather(1, tok[:, None])[:, 0] - torch.logsumexp(x, 1))
    return torch.cat(out)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("size", [0.5, 2.0])
@pytest.mark.parametrize("t", [1.0, 0.75])
def test_mean_error(tc, kind, size, t):      # noqa: F811
    T, V = 16384, 4099
    z, tokens, _ = logits(T, V, kind, 1, size)
    want = exact(z, tokens, t)
    assert want.min() > -32
    tokens[::7] = z[::7].argmax(1)
    want = exact(z, tokens, t)
    bound = 6 * 2.0 ** -20 / math.sqrt(T) + 2.0 ** -28
    old, one = torch.zeros(T, device="cuda"), torch.ones(T, device="cuda")
    at = torch.tensor([0, T, T], device="cuda")
    top = tc.token_logprobs(z, tokens, top=1, temperature=t)
    for what, lp in (("token_logprobs", tc.token_logprobs(z, tokens, temperature=t).logprob),
                     ("with alternatives", top.logprob),
                     ("token_logprobs_grad", tc.token_logprobs_grad(z, tokens, one, temperature=t).logprob),
                     ("policy_loss", tc.policy_loss(z, tokens, old, one, temperature=t).logprob),
                     ("policy_loss_grad", tc.policy_loss_grad(z, tokens, old, one, one, temperature=t).logprob),
                     ("preference_loss", tc.preference_loss(z, tokens, at, temperature=t).logprob)):
        e = lp.double() - want
        assert abs(e.mean().item()) <= bound, (what, e.mean().item(), bound)
    e = top.top_logprob[:, 0].double() - exact(z, z.float().argmax(1), t)
    assert abs(e.mean().item()) <= bound, ("alternatives", e.mean().item(), bound)
    # a reward is the sum of all of them
    r = tc.preference_loss(z, tokens, at, beta=1.0, temperature=t).reward[0].item()
    assert abs(r - want.sum().item()) <= T * bound + abs(r) * 2.0 ** -24


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("V,size,t", [(7, 1.0, 1.0), (5003, 3.0, 1.0), (70000, 2.0, 0.8)])
def test_equal_models(tc, kind, V, size, t):      # noqa: F811
    """A policy that is its reference: ratios of 1, rewards and KL terms of 0, exactly."""
    T = 3000
    z, tokens, g = logits(T, V, kind, 2, size)
    tokens[::9] = -1
    given = tokens >= 0
    ref = tc.token_logprobs(z, tokens, temperature=t).logprob
    at = torch.tensor([0, 1900, 2000, 2000, 3000], device="cuda")
    w = torch.ones(2, device="cuda")
    for r in (tc.preference_loss(z, tokens, at, ref, beta=0.5, temperature=t),
              tc.preference_loss_grad(z, tokens, at, w, ref, beta=0.5, temperature=t)):
        assert torch.equal(r.logprob, ref) and not r.reward.any()
        assert bool(((r.loss - math.log(2)).abs() <= 2.0 ** -24).all())
    adv = torch.randn(T, generator=g, device="cuda")
    r = tc.policy_loss(z, tokens, ref, adv, ref, kl=0.3, clip=(0.0, 0.0), temperature=t)
    assert torch.equal(r.logprob, ref) and not r.kl.any() and torch.equal(r.loss, torch.where(given, -adv, 0.0))


@pytest.mark.parametrize("kind", list(TYPES))
def test_extremes(tc, kind):      # noqa: F811
    """Masked tokens, rows of nothing but -inf, infinities and NaN, the type's lowest value, far temperatures."""
    inf, nan, low = math.inf, math.nan, torch.finfo(TYPES[kind]).min
    z = torch.zeros((8, 64), device="cuda", dtype=TYPES[kind])
    z[0, 3] = -inf
    z[1] = -inf
    z[2, 5] = inf
    z[3, 5] = nan
    z[4, 3] = low
    z[5] = low
    z[6, 3:] = -inf
    tokens = torch.tensor([3, 3, 3, 3, 3, 3, 2, 64], device="cuda")
    old = torch.zeros(8, device="cuda")
    at = torch.arange(9, device="cuda")
    for call in (lambda t: tc.token_logprobs(z, tokens, temperature=t), lambda t: tc.policy_loss(z, tokens, old, old, temperature=t),
                 lambda t: tc.preference_loss(z, tokens, at, temperature=t)):
        for t in (1.0, 2.0 ** -100, 2.0 ** 100):
            lp = call(t).logprob.tolist()
            assert lp[0] == -inf and lp[1] == -inf and math.isnan(lp[2]) and math.isnan(lp[3]), (t, lp)
            want = low / t - math.log(63 if low / t < -200 else 64)
            if want < torch.finfo(torch.float32).min:
                assert lp[4] == -inf or lp[4] == torch.finfo(torch.float32).min
            else:
                assert abs(lp[4] - want) <= abs(want) * 2.0 ** -22 + 2.0 ** -20
            assert abs(lp[5] + math.log(64)) <= 2.0 ** -20 and abs(lp[6] + math.log(3)) <= 2.0 ** -21 and lp[7] == 0
    r = tc.token_logprobs(z, tokens, top=4)
    assert r.top_token[0].tolist() == [0, 1, 2, 4] and r.top_token[1].tolist() == [-1] * 4 and r.top_token[6].tolist() == [0, 1, 2, -1]
    assert bool((r.top_logprob[6, :3] == r.logprob[6]).all()) and r.top_logprob[6, 3].item() == -inf


@pytest.mark.parametrize("V,T,size", [(4099, 16384, 2.0), (32768, 4096, 2.0), (32768, 4096, 0.5)])
def test_mean_of_logits(tc, V, T, size):      # noqa: F811
    """entropy - lse is minus the mean logit: both have the same logarithm of S, so what is left is the sum of u 2^u over S,
    whose two sums lack the same.  Its mean error: the roundings of two numbers of 16 or less, as above, and 2^-25 of itself."""
    z, _, _ = logits(T, V, "f32", 3, size)
    want, least = [], []
    for part in z.split(1024):
        x = part.double()
        want.append(-(torch.softmax(x, 1) * x).sum(1))
        least.append(x.amax(1))
    want = torch.cat(want)
    one = torch.ones(T, device="cuda")
    tokens = torch.zeros(T, dtype=torch.int64, device="cuda")
    for r in (tc.token_logprobs(z), tc.token_logprobs(z, top=2), tc.token_logprobs_grad(z, tokens, one, one)):
        e = r.entropy.double() - r.lse.double() - want
        assert abs(e.mean().item()) <= 6 * 2.0 ** -20 / math.sqrt(T) + (torch.cat(least) + want).mean().item() * 2.0 ** -25
