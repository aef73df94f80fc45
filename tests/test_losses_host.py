"""Argument checks of the policy and preference losses on the host (no GPU
needed): the documented status before anything is launched."""
import ctypes

import pytest

from tensor_core_dense_tma_gb300.logits import _Policy, _Preference
from test_logits_host import BAD_ROWS, INVALID, MISALIGNED, OK, P, UNSUPPORTED, lib, rows  # noqa: F401

NAN, INF = float("nan"), float("inf")
POLICY = BAD_ROWS + [
    (dict(tokens=None), INVALID), (dict(old=None), INVALID), (dict(adv=None), INVALID), (dict(loss=None), INVALID),
    (dict(policy=None), INVALID), (dict(low=-0.1), INVALID), (dict(low=1.5), INVALID), (dict(low=NAN), INVALID),
    (dict(high=-0.1), INVALID), (dict(high=INF), INVALID), (dict(high=NAN), INVALID), (dict(kl=0.1, ref=None), INVALID),
    (dict(kl=NAN), INVALID), (dict(bonus=INF), INVALID), (dict(tokens=P + 4), MISALIGNED), (dict(old=P + 2), MISALIGNED),
    (dict(adv=P + 1), MISALIGNED), (dict(ref=P + 2), MISALIGNED), (dict(loss=P + 2), MISALIGNED),
    (dict(lp=P + 2), MISALIGNED), (dict(k=P + 2), MISALIGNED), (dict(ent=P + 2), MISALIGNED), (dict(T=0), OK),
    (dict(T=0, z=None, tokens=None, old=None, adv=None, loss=None), OK),
]
GRADIENT = [(dict(w=None), INVALID), (dict(dz=None), INVALID), (dict(ldd=99), INVALID), (dict(ldd=1 << 41), UNSUPPORTED),
            (dict(dz=P + 2), MISALIGNED), (dict(w=P + 2), MISALIGNED)]


def policy_args(kw):
    a = dict(tokens=P, temperature=1.0, old=P, adv=P, ref=P, low=0.2, high=0.2, kl=0.0, bonus=0.0, loss=P, lp=P, k=P,
             ent=P, w=P, dz=P, ldd=100)
    a.update(kw)
    if a.get("V", 0) > 100:
        a["ldd"] = a["V"]
    a.setdefault("policy", ctypes.byref(_Policy(a["old"], a["adv"], a["ref"], a["low"], a["high"], a["kl"], a["bonus"])))
    return a


@pytest.mark.parametrize("kw,code", POLICY)
def test_policy(lib, kw, code):      # noqa: F811
    a = policy_args(kw)
    assert lib.logits_policy(*rows(a, "tokens", "temperature", "policy", "loss", "lp", "k", "ent"), None) == code


@pytest.mark.parametrize("kw,code", POLICY + GRADIENT)
def test_policy_grad(lib, kw, code):      # noqa: F811
    a = policy_args(kw)
    assert lib.logits_policy_grad(*rows(a, "tokens", "temperature", "policy", "w", "loss", "lp", "k", "ent", "dz", "ldd"),
                                  None) == code


PREFERENCE = [(k, c) for k, c in BAD_ROWS] + [
    (dict(tokens=None), INVALID), (dict(preference=None), INVALID), (dict(pairs=-1), INVALID),
    (dict(pairs=1 << 32), UNSUPPORTED), (dict(offsets=None), INVALID), (dict(beta=NAN), INVALID), (dict(beta=INF), INVALID),
    (dict(smoothing=-0.1), INVALID), (dict(smoothing=1.1), INVALID), (dict(smoothing=NAN), INVALID),
    (dict(loss=None), INVALID), (dict(reward=None), INVALID), (dict(lp=None), INVALID), (dict(tokens=P + 4), MISALIGNED),
    (dict(offsets=P + 4), MISALIGNED), (dict(ref=P + 2), MISALIGNED), (dict(loss=P + 2), MISALIGNED),
    (dict(reward=P + 2), MISALIGNED), (dict(lp=P + 2), MISALIGNED), (dict(T=0, pairs=0), OK),
    (dict(T=0, pairs=0, z=None, tokens=None, offsets=None, loss=None, reward=None, lp=None), OK),
]


def preference_args(kw):
    a = dict(tokens=P, temperature=1.0, offsets=P, pairs=2, ref=P, beta=0.1, smoothing=0.0, loss=P, reward=P, lp=P, w=P,
             dz=P, ldd=100, work=P)
    a.update(kw)
    if a.get("V", 0) > 100:
        a["ldd"] = a["V"]
    a.setdefault("preference",
                 ctypes.byref(_Preference(a["offsets"], a["pairs"], a["ref"], a["beta"], a["smoothing"])))
    return a


@pytest.mark.parametrize("kw,code", PREFERENCE)
def test_preference(lib, kw, code):      # noqa: F811
    a = preference_args(kw)
    assert lib.logits_preference(*rows(a, "tokens", "temperature", "preference", "loss", "reward", "lp"), None) == code


@pytest.mark.parametrize("kw,code", PREFERENCE + GRADIENT + [(dict(work=None), INVALID), (dict(work=P + 8), MISALIGNED)])
def test_preference_grad(lib, kw, code):      # noqa: F811
    a = preference_args(kw)
    assert lib.logits_preference_grad(*rows(a, "tokens", "temperature", "preference", "w", "loss", "reward", "lp", "dz",
                                            "ldd", "work"), None) == code
