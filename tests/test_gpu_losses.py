"""The policy and the preference loss (include/logits.h) against a plain numpy
implementation in 64 bits, written from the definitions.

Tolerances start from the bounds of tests/test_gpu_logits.py: b for a
log-probability and the relative error of a probability p.  With eps = 2^-24 (half
a unit of fp32):

policy      the ratio's argument is off by b and eps |lp - old|, its exponential
            by 2 units: relatively by q = b + eps |lp - old| + 4 eps, and a border
            by one rounding, so both products by q + 4 eps; the minimum by the larger.
            d = ref - lp is off by v = b + eps |d|; k's derivative is e^d - 1 and
            expm1 and the two roundings lose 4 eps (|e^d - 1| + |d|).  The slope is off
            by (q + 4 eps) |r A| and, c the coefficient, |c| (e^d v + 4 eps |e^d - 1|).
preference  a reward is beta times a 64-bit sum: off by |beta| sum b, and one rounding; m
            by both and a rounding; the loss has a slope of at most 1 in m, and sigma of
            at most 1/4; the exponential, logarithm and quotient lose 8 eps each.
gradients   the bound of the log-probabilities' gradient plus the slope's error
            times (1[j = y] + p_j) / temperature.
"""
import numpy as np
import pytest
import torch

from test_gpu_logits import (HALF_ULP, SMALLEST, TYPES, bound_log, err_log_sum, make, near, ref_logprobs, tc)  # noqa: F401

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24
CLIP = (0.2, 0.28)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def p_error(z, t):
    """of a probability, relatively (its exponent's own rounding grows with its size)"""
    top = np.nan_to_num(np.abs(np.where(np.isneginf(z), 0, z)).max(axis=1, initial=0.0))[:, None] / t
    return 2 * err_log_sum(z.shape[1]) + 2.0 ** -22 * (64 + np.minimum(top, 200))


# ---- policy --------------------------------------------------------------------
def ref_policy(z, tokens, t, old, adv, ref, ck, ce, clip=CLIP):
    """(loss, lp, k, ent, slope), their errors, and log p."""
    with np.errstate(all="ignore"):
        lp, ent, lse, logp = ref_logprobs(z, tokens, t)
        given = (tokens >= 0) & (tokens < z.shape[1])
        b = bound_log(z, t, lse, lp)
        r = np.exp(lp - old)
        u, c = r * adv, np.clip(r, 1 - clip[0], 1 + clip[1]) * adv
        q = b + EPS * np.abs(np.nan_to_num(lp - old, neginf=0)) + 8 * EPS
        loss = -np.minimum(u, c)
        slope = np.where(u <= c, -u, 0.0)
        e_loss, e_slope = q * np.maximum(np.abs(u), np.abs(c)), q * np.abs(u)
        k = e_k = np.zeros_like(lp)
        if ref is not None:
            d = ref - lp
            m = np.expm1(d)
            k = m - d
            v = b + EPS * np.abs(d)
            e_k = np.abs(m) * v + 4 * EPS * (np.abs(m) + np.abs(d)) + EPS * k
            loss, slope = loss + ck * k, slope - ck * m
            e_loss, e_slope = e_loss + abs(ck) * e_k, e_slope + abs(ck) * (np.exp(d) * v + 4 * EPS * np.abs(m))
        e_ent = (2 * err_log_sum(z.shape[1]) + 2.0 ** -22) * (1 + ent)
        loss = loss - ce * ent
        e_loss = e_loss + abs(ce) * e_ent + 4 * EPS * (np.abs(loss) + abs(ce) * ent)
        zero = lambda x: np.where(given, x, 0.0)      # noqa: E731
        return tuple(map(zero, (loss, lp, k, ent, slope))), tuple(map(zero, (e_loss, b, e_k, e_ent, e_slope))), logp


def check_policy(got, want, err):
    for name, w, e in zip(("loss", "logprob", "kl", "entropy"), want, err):
        near(getattr(got, name), w, e, name)


def check_gradient(got, z, tokens, t, logp, ent, g, e_g, h, kind):
    """dlogits = (g (1[y] - p) - h p (log p + H)) / t with an error e_g of g."""
    with np.errstate(all="ignore"):
        p = np.exp(logp)
        plogp = np.where(p > 0, p * np.where(p > 0, logp, 0), 0)
        one = np.zeros_like(p)
        given = (tokens >= 0) & (tokens < z.shape[1])
        one[np.flatnonzero(given), tokens[given]] = 1
        g, e_g, h, ent = g[:, None], e_g[:, None], h[:, None], ent[:, None]
        d = (g * (one - p) - h * (plogp + p * ent)) / t
        G = (np.abs(g) * (one + p) + np.abs(h) * (np.abs(plogp) + p * ent)) / t
        dead = ~given | np.isneginf(z).all(axis=1) | ((g == 0) & (h == 0))[:, 0]
        d[dead] = G[dead] = 0
        tol = HALF_ULP[kind] * np.abs(d) * (1 + 1e-6) + SMALLEST[kind] + G * p_error(z, t) + e_g * (one + p) / t
        tol[dead] = 0
    near(got, d, tol, "gradient")


def policy_inputs(z, tokens, t, seed, with_ref):
    """old and ref near the log-probabilities; no ratio within 0.1 % of a border."""
    T = len(z)
    rng = np.random.default_rng(seed)
    lp = np.nan_to_num(ref_logprobs(z, tokens, t)[0], neginf=-50.0)
    old = (lp + 0.3 * rng.normal(size=T)).astype(np.float32).astype(np.float64)
    for border in (np.log(1 - CLIP[0]), np.log(1 + CLIP[1])):
        old = np.where(np.abs(lp - old - border) < 1e-3, old - 0.01, old)
    old = old.astype(np.float32).astype(np.float64)
    adv = rng.normal(size=T).astype(np.float32).astype(np.float64)
    ref = (lp + 0.3 * rng.normal(size=T)).astype(np.float32).astype(np.float64) if with_ref else None
    w = rng.random(T).astype(np.float32).astype(np.float64)
    return old, adv, ref, w


def f32(a):
    return None if a is None else dev(a.astype(np.float32))


def run_policy(tc, view, z, tokens, t, kind, seed, with_ref, ck, ce, out=None):      # noqa: F811
    old, adv, ref, w = policy_inputs(z, tokens, t, seed, with_ref)
    if len(w) > 3:
        w[3] = 0.0
    args = (dev(tokens), f32(old), f32(adv))
    kw = dict(clip=CLIP, kl=ck, entropy_bonus=ce, temperature=t)
    want, err, logp = ref_policy(z, tokens, t, old, adv, ref, np.float32(ck), np.float32(ce))
    check_policy(tc.policy_loss(view, *args, f32(ref), **kw), want, err)
    r = tc.policy_loss_grad(view, *args, f32(w), f32(ref), dlogits=out, **kw)
    torch.cuda.synchronize()
    check_policy(r, want, err)
    given = (tokens >= 0) & (tokens < z.shape[1])
    w = np.where(given, w, 0)
    check_gradient(r.dlogits, z, tokens, t, logp, want[3], w * want[4], w * err[4] + 4 * EPS * np.abs(w * want[4]),
                   -np.float64(np.float32(ce)) * w, kind)
    return r


SIZES = [(5, 1), (4, 7), (5, 9), (4, 511), (5, 4103), (4, 50001), (1, 131072), (3, 262147)]


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("T,V", SIZES, ids=str)
@pytest.mark.parametrize("form", ["plain", "full", "inplace"])
def test_policy(tc, kind, T, V, form):      # noqa: F811
    view, z = make(T, V, kind, seed=V, pad=5, shift=2)
    tokens = np.random.default_rng(V).integers(0, V, T)
    if T > 2:
        tokens[2] = -1
    # apart: another row stride and another start within 16 bytes
    out = view if form == "inplace" else torch.full((T, V + 9), 7.0, dtype=TYPES[kind], device="cuda")[:, 1:V + 1]
    full = form != "plain"
    run_policy(tc, view, z, tokens, 0.8, kind, V, full, 0.05 if full else 0.0, 0.01 if full else 0.0, out)
    if form != "inplace":      # nothing beside the row is written
        whole = torch.as_strided(out, (T, V + 9), (V + 9, 1), out.storage_offset() - 1)
        assert bool((whole[:, 0] == 7).all()) and bool((whole[:, V + 1:] == 7).all())


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("mask", ["banned", "empty", "one", "lowest", "few", "equal"])
def test_policy_masks(tc, kind, mask):      # noqa: F811
    view, z = make(6, 9001, kind, mask, seed=3)
    tokens = np.random.default_rng(8).integers(0, 9001, 6)
    tokens[1], tokens[5] = 9001, -9
    run_policy(tc, view, z, tokens, 1.0, kind, 4, False, 0.0, 0.02)


def test_policy_many_rows(tc):      # noqa: F811
    """Rows two to a CTA, a third of them without a token."""
    T, V = 9000, 300
    view, z = make(T, V, "bf16", seed=9, pad=4)
    tokens = np.random.default_rng(2).integers(0, V, T)
    tokens[::3] = -1
    run_policy(tc, view, z, tokens, 1.1, "bf16", 5, True, 0.1, 0.01)


def test_rows_that_do_not_count(tc):      # noqa: F811
    """NaN in rows without a token and in rows of weight 0 reaches nothing."""
    T, V = 6, 70000
    for kind in TYPES:
        view, _ = make(T, V, kind, seed=1)
        view[1], view[4] = float("nan"), float("inf")
        tokens = torch.tensor([5, -1, 7, V, 9, 11], device="cuda")
        f = torch.zeros(T, device="cuda") - 9
        bad = f.clone()
        bad[1] = float("nan")
        w = torch.tensor([1.0, 1, 1, 1, 0, 1], device="cuda")
        r = tc.policy_loss_grad(view, tokens, bad, bad, w, bad, kl=0.1, entropy_bonus=0.1)
        assert torch.isnan(r.loss).tolist() == [False] * 4 + [True, False]
        assert not torch.isnan(r.dlogits).any()
        assert not r.dlogits[[1, 3, 4]].any() and bool(r.dlogits[[0, 2, 5]].any(1).all())
        for v in (r.loss, r.logprob, r.kl, r.entropy):
            assert v[[1, 3]].tolist() == [0.0, 0.0]
        # pairs: rows 0..1 / 2..3 and row 5 / none; row 4 is in no sequence
        o = torch.tensor([0, 2, 4, 4, 4], device="cuda")
        r = tc.preference_loss_grad(view, tokens, o, torch.ones(2, device="cuda"), bad)
        assert not torch.isnan(r.loss).any() and not torch.isnan(r.dlogits).any()
        assert bool(r.dlogits[[0, 2]].any(1).all()) and not r.dlogits[[1, 3, 4, 5]].any()
        assert r.loss[1].item() == pytest.approx(np.log(2), rel=1e-6) and r.reward[2:].tolist() == [0, 0]


def test_policy_extremes(tc):      # noqa: F811
    """Ratios that overflow, masked tokens, a NaN advantage."""
    z = torch.zeros((6, 8), device="cuda")
    z[1, 3] = -float("inf")
    tok = torch.tensor([0, 3, 0, 0, 0, 0], device="cuda")
    old = torch.tensor([-200.0, -2, -200, -2, -2, -2], device="cuda")
    adv = torch.tensor([2.0, 3, -2, float("nan"), 1, -1], device="cuda")
    w = torch.ones(6, device="cuda")
    r = tc.policy_loss_grad(z, tok, old, adv, w)
    assert r.loss[0].item() == pytest.approx(-2.4, rel=1e-6) and not r.dlogits[0].any()      # clipped
    assert r.logprob[1].item() == -np.inf and r.loss[1].item() == 0 and not r.dlogits[1].any()
    assert r.loss[2].item() == np.inf
    assert torch.isnan(r.loss).tolist() == [False, False, False, True, False, False]
    assert torch.isnan(r.dlogits[3]).all() and torch.isfinite(r.dlogits[4:]).all()
    assert not r.kl.any()


def differences(f, z, eps=1e-5):
    d = np.zeros_like(z)
    for i in range(z.shape[0]):
        for j in range(z.shape[1]):
            zp, zm = z.copy(), z.copy()
            zp[i, j] += eps
            zm[i, j] -= eps
            d[i, j] = (f(zp) - f(zm)) / (2 * eps)
    return d


def test_policy_differences(tc):      # noqa: F811
    T, V, t = 4, 20, 0.9
    view, z = make(T, V, "f32", seed=11)
    tokens = np.array([3, 19, 0, -1])
    old, adv, ref, w = policy_inputs(z, tokens, t, 2, True)

    def f(zz):
        return float((w * ref_policy(zz, tokens, t, old, adv, ref, 0.3, 0.2)[0][0]).sum())

    r = tc.policy_loss_grad(view, dev(tokens), f32(old), f32(adv), f32(w), f32(ref), clip=CLIP, kl=0.3,
                            entropy_bonus=0.2, temperature=t)
    # differences: third derivatives of some tens times eps^2 / 6 and 1e-15 / eps of rounding; fp32 itself 1e-6
    assert np.abs(r.dlogits.double().cpu().numpy() - differences(f, z)).max() < 1e-5


# ---- preference ----------------------------------------------------------------
def ref_preference(z, tokens, t, offsets, ref, beta, e):
    """(loss, reward, lp), the rewards' bound, each row's factor with weights of 1 and log p."""
    with np.errstate(all="ignore"):
        lp, _, lse, logp = ref_logprobs(z, tokens, t)
        given = (tokens >= 0) & (tokens < z.shape[1])
        b = np.where(given, bound_log(z, t, lse, lp), 0)
        diff = np.where(given, lp - (0 if ref is None else ref), 0)
        S = len(offsets) - 1
        reward = beta * np.array([diff[offsets[s]:offsets[s + 1]].sum() for s in range(S)])
        bound = abs(beta) * np.array([b[offsets[s]:offsets[s + 1]].sum() for s in range(S)])
        m = reward[0::2] - reward[1::2]
        loss = (1 - e) * np.logaddexp(0, -m) + (e * np.logaddexp(0, m) if e else 0)
        slope = beta * (e / (1 + np.exp(-m)) - (1 - e) / (1 + np.exp(m)))
        return loss, reward, lp, bound, slope, logp


def check_preference(tc, view, z, tokens, t, kind, lengths, seed, e=0.1, beta=0.1, out=None, first=0,      # noqa: F811
                     with_ref=True):
    T, P = len(z), len(lengths) // 2
    rng = np.random.default_rng(seed)
    ref = np.nan_to_num(ref_logprobs(z, tokens, t)[0], neginf=-9.0) + 0.3 * rng.normal(size=T)
    ref = ref.astype(np.float32).astype(np.float64) if with_ref else None
    w = rng.random(P).astype(np.float32).astype(np.float64)
    offsets = np.cumsum([first] + list(lengths)).astype(np.int64)
    beta, e = float(np.float32(beta)), float(np.float32(e))
    kw = dict(beta=beta, smoothing=e, temperature=t)
    loss, reward, lp, bound, slope, logp = ref_preference(z, tokens, t, offsets, ref, beta, e)
    e_m = bound[0::2] + bound[1::2]

    def results(r):
        near(r.logprob, lp, bound_log(z, t, ref_logprobs(z, tokens, t)[2], lp), "logprob")
        near(r.reward, reward, bound + EPS * np.abs(reward) + 1e-37, "reward")
        near(r.loss, loss, e_m + EPS * np.abs(reward[0::2] - reward[1::2]) + 16 * EPS * np.abs(loss) + 1e-37, "loss")

    results(tc.preference_loss(view, dev(tokens), dev(offsets), f32(ref), **kw))
    r = tc.preference_loss_grad(view, dev(tokens), dev(offsets), f32(w), f32(ref), dlogits=out, **kw)
    torch.cuda.synchronize()
    results(r)
    g, e_g = np.zeros(T), np.zeros(T)
    given = (tokens >= 0) & (tokens < z.shape[1])
    for q in range(P):
        for s, sign in ((2 * q, 1), (2 * q + 1, -1)):
            part = slice(offsets[s], offsets[s + 1])
            g[part] = sign * w[q] * slope[q] * given[part]
            e_g[part] = given[part] * w[q] * (abs(beta) * (e_m[q] + EPS * abs(reward[2 * q] - reward[2 * q + 1])) / 4
                                         + 24 * EPS * abs(beta))
    zero = np.zeros(T)
    check_gradient(r.dlogits, z, tokens, t, logp, zero, g, e_g, zero, kind)
    return r


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("V", [1, 7, 511, 4103, 50001, 131072])
@pytest.mark.parametrize("form", ["apart", "inplace", "no_ref"])
def test_preference(tc, kind, V, form):      # noqa: F811
    T = 9
    view, z = make(T, V, kind, seed=V, pad=5, shift=2)
    tokens = np.random.default_rng(V).integers(0, V, T)
    tokens[[0, 4]] = -1, V
    out = view if form == "inplace" else torch.full((T, V + 9), 7.0, dtype=TYPES[kind], device="cuda")[:, 1:V + 1]
    # rows before the first and behind the last sequence, a sequence without rows
    check_preference(tc, view, z, tokens, 0.8, kind, [3, 1, 0, 2], V, 0.0 if form == "no_ref" else 0.1, 0.3, out, 1,
                     form != "no_ref")
    if form != "inplace":
        whole = torch.as_strided(out, (T, V + 9), (V + 9, 1), out.storage_offset() - 1)
        assert bool((whole[:, 0] == 7).all()) and bool((whole[:, V + 1:] == 7).all())


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("mask", ["lowest", "few", "equal"])
def test_preference_masks(tc, kind, mask):      # noqa: F811
    view, z = make(6, 9001, kind, mask, seed=3)
    tokens = np.random.default_rng(8).integers(0, 9001, 6)
    if mask == "lowest":
        for i in range(6):      # a token that is not at the type's lowest value, which would be a reward of -1e38
            tokens[i] = z[i].argmax()
    if mask == "few":
        tokens %= 3
    check_preference(tc, view, z, tokens, 1.0, kind, [3, 3], 4)


def test_preference_masked_tokens(tc):      # noqa: F811
    """-inf: a masked token in the preferred or the other sequence, and a row of nothing but -inf."""
    z = torch.zeros((4, 16), device="cuda")
    z[0, 2] = z[3, 2] = -float("inf")
    tok = torch.tensor([2, 0, 0, 2], device="cuda")
    r = tc.preference_loss_grad(z, tok, torch.arange(5, device="cuda"), torch.ones(2, device="cuda"), beta=1.0)
    assert r.reward[0].item() == -np.inf and r.reward[3].item() == -np.inf
    assert r.loss.tolist() == [np.inf, 0.0]
    assert r.dlogits[0, 2].item() == -1 and r.dlogits[1, 0].item() == pytest.approx(1 - 1 / 16, rel=1e-6)
    assert not r.dlogits[2:].any()
    z[1] = -float("inf")
    r = tc.preference_loss_grad(z, torch.zeros_like(tok), torch.tensor([0, 1, 2], device="cuda"),
                                torch.ones(1, device="cuda"), beta=1.0)
    assert r.loss.tolist() == [0.0] and not torch.isnan(r.dlogits).any() and not r.dlogits[1:].any()


def test_preference_many_pairs(tc):      # noqa: F811
    T, V = 9000, 300
    view, z = make(T, V, "f16", seed=9, pad=4)
    rng = np.random.default_rng(2)
    tokens = rng.integers(0, V, T)
    tokens[::5] = -1
    lengths = np.diff(np.sort(np.concatenate([[0, T], rng.integers(0, T, 199)])))
    check_preference(tc, view, z, tokens, 1.1, "f16", lengths, 5)


def test_preference_one_long_pair(tc):      # noqa: F811
    T, V = 30000, 60
    view, z = make(T, V, "f32", seed=4)
    tokens = np.random.default_rng(2).integers(0, V, T)
    check_preference(tc, view, z, tokens, 1.0, "f32", [17001, 12999], 5, beta=0.001)


def test_preference_offsets_out_of_order(tc):      # noqa: F811
    """What offsets that decrease or leave 0..T give is undefined, but nothing else is touched."""
    view, z = make(6, 1000, "bf16", seed=4)
    guard = torch.full((10, 1000), 7.0, dtype=torch.bfloat16, device="cuda")
    tok = torch.zeros(6, dtype=torch.int64, device="cuda")
    for o in ([5, 2, 1], [-7, 3, 1 << 40], [9, 9, 9], [-(1 << 62), 0, (1 << 62)]):
        tc.preference_loss_grad(view, tok, torch.tensor(o, device="cuda"), torch.ones(1, device="cuda"),
                                dlogits=guard[2:8])
        torch.cuda.synchronize()
        assert bool((guard[:2] == 7).all()) and bool((guard[8:] == 7).all())


def test_preference_differences(tc):      # noqa: F811
    T, V, t = 5, 12, 0.9
    view, z = make(T, V, "f32", seed=11)
    tokens, offsets = np.array([3, 11, -1, 0, 5]), np.array([0, 2, 5])
    ref = np.random.default_rng(1).normal(size=T) - 3
    ref = ref.astype(np.float32).astype(np.float64)

    def f(zz):
        return float(2.5 * ref_preference(zz, tokens, t, offsets, ref, 0.5, 0.125)[0].sum())

    r = tc.preference_loss_grad(view, dev(tokens), dev(offsets), torch.full((1,), 2.5, device="cuda"), f32(ref),
                                beta=0.5, smoothing=0.125, temperature=t)
    assert np.abs(r.dlogits.double().cpu().numpy() - differences(f, z)).max() < 1e-5


# ---- both ----------------------------------------------------------------------
def test_streams_and_graphs(tc):      # noqa: F811
    """On a stream of its own, from two graphs replayed together, and again: the same bits."""
    T, V = 40, 30011
    view, _ = make(T, V, "bf16", seed=2, pad=5)
    tok = torch.arange(T, device="cuda") * 100
    o = torch.tensor([0, 9, 21, 30, 40], device="cuda")
    f = torch.linspace(-12, -9, T, device="cuda")
    w = torch.rand(T, device="cuda")

    def calls(dl):
        a = tc.policy_loss_grad(view, tok, f, w, w, f, kl=0.1, entropy_bonus=0.1, dlogits=dl[0])
        b = tc.preference_loss_grad(view, tok, o, w[:2], f, dlogits=dl[1])
        return [x for r in (a, b) for x in r]

    def outs():
        return [torch.empty_like(view) for _ in range(2)]

    want = [x.clone() for x in calls(outs())]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = calls(outs())
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r = calls(outs())
        graphs.append((g, r, torch.cuda.Stream()))
    for _ in range(3):
        for g, _, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for _, r, _ in graphs:
        assert all(torch.equal(a, b) for a, b in zip(r, want))


def test_given_stream(tc):      # noqa: F811
    """`stream` another than the current one, which takes what memory it can get
    meanwhile: the call's own buffer is not among it."""
    view, _ = make(200, 5000, "bf16", seed=6)
    tok = torch.arange(200, device="cuda")
    o, w = torch.tensor([0, 90, 200], device="cuda"), torch.ones(1, device="cuda")
    want = tc.preference_loss_grad(view, tok, o, w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)
        got = tc.preference_loss_grad(view, tok, o, w, stream=s.cuda_stream)
        for _ in range(8):
            torch.full((800,), float("nan"), device="cuda")
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_empty_calls(tc):      # noqa: F811
    z = torch.empty((0, 100), device="cuda")
    e, i = torch.empty(0, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    assert tc.policy_loss_grad(z, i, e, e, e).dlogits.shape == (0, 100)
    r = tc.preference_loss_grad(z, i, torch.zeros(5, dtype=torch.int64, device="cuda"), torch.ones(2, device="cuda"))
    assert r.reward.tolist() == [0.0] * 4 and r.loss.tolist() == pytest.approx([np.log(2)] * 2)
    z = torch.ones((3, 100), device="cuda")
    i = torch.zeros(3, dtype=torch.int64, device="cuda")
    r = tc.preference_loss_grad(z, i, torch.zeros(1, dtype=torch.int64, device="cuda"), e)
    assert r.loss.shape == (0,) and not r.dlogits.any() and r.logprob.tolist() == pytest.approx([-np.log(100)] * 3)
    z = torch.empty((2, 0), device="cuda")
    r = tc.policy_loss(z, i[:2], torch.zeros(2, device="cuda"), torch.ones(2, device="cuda"))
    assert r.loss.tolist() == [0, 0] and r.logprob.tolist() == [0, 0]


def test_refusals(tc):      # noqa: F811
    z = torch.zeros((4, 64), device="cuda")
    i, f = torch.zeros(4, dtype=torch.int64, device="cuda"), torch.zeros(4, device="cuda")
    ok = dict(logits=z, tokens=i, old=f, adv=f, w=f, ref=None)
    for kw in (dict(logits=z.double()), dict(logits=z.t()), dict(tokens=i.int()), dict(tokens=None), dict(old=None),
               dict(old=f[:3]), dict(adv=f.cpu()), dict(adv=f.half()), dict(ref=f.double()), dict(w=None), dict(w=f[:2])):
        a = dict(ok, **kw)
        with pytest.raises(ValueError):
            tc.policy_loss_grad(a["logits"], a["tokens"], a["old"], a["adv"], a["w"], a["ref"])
    with pytest.raises(ValueError):
        tc.policy_loss(z, i, f, f, kl=0.1)
    for kw in (dict(clip=(-0.1, 0.2)), dict(clip=(1.1, 0.2)), dict(clip=(0.1, float("inf"))), dict(clip=(0.1, -0.5)),
               dict(entropy_bonus=float("nan")), dict(temperature=0.0)):
        with pytest.raises(tc.GemmError):
            tc.policy_loss(z, i, f, f, **kw)
    o, w = torch.zeros(3, dtype=torch.int64, device="cuda"), torch.zeros(1, device="cuda")
    for kw in (dict(offsets=o.int()), dict(offsets=o[:2]), dict(offsets=None), dict(tokens=None), dict(w=None),
               dict(w=f), dict(ref=f[:1])):
        a = dict(tokens=i, offsets=o, w=w, ref=None)
        a.update(kw)
        with pytest.raises(ValueError):
            tc.preference_loss_grad(z, a["tokens"], a["offsets"], a["w"], a["ref"])
    for kw in (dict(beta=float("inf")), dict(smoothing=-0.1), dict(smoothing=1.5), dict(temperature=-1.0)):
        with pytest.raises(tc.GemmError):
            tc.preference_loss(z, i, o, **kw)
