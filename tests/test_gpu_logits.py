"""Operators on the rows of a logits matrix (include/logits.h) against a plain
numpy implementation in 64 bits, written from the definitions.

Tolerances follow from the arithmetic.  A row's sum S of 2^u is fp32: 512
threads add at most n = ceil(V / 512) + 8 terms one after another, joined by a
tree of fewer than 24 steps, each step off by at most 2^-24 relatively (two
roundings at a change of the maximum); a term is off by the exponential's 2
units (2^-22) and by its argument's two roundings, 2^-23 |u| ln 2 with
|u| 2^u < 0.54.  So ln S is off by at most

    e = 2^-24 (2 n + 48 + 8)

and lse and a log-probability x - lse by e plus 2^-24 times 4 (|x| + |m| + |lse|)
for their own roundings.  The entropy's second sum weighs the same errors with
|log p|: 2 e (1 + H) and 2^-22 (1 + H) of rounding.  A gradient element is a
sum of terms of total size G, each with the relative error of p (that of its
logarithm), and is rounded once to its type (half a unit in the last place).
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_ULP = {k: torch.finfo(v).eps / 2 for k, v in TYPES.items()}      # of the rounding to the type, relative
SMALLEST = {"f32": 1e-37, "f16": 2.0 ** -25, "bf16": 1e-37}
LOWEST = {"f32": -3.4028235e38, "f16": -65504.0, "bf16": -3.3895314e38}


@pytest.fixture(scope="module")
def tc():
    from tensor_core_dense_tma_gb300 import build as tcbuild
    tcbuild.build()
    import tensor_core_dense_tma_gb300 as tc
    return tc


# ---- the definitions in 64 bits ------------------------------------------------
def softmax_rows(x):
    """(lse, log p) of the rows of x; a row without finite entries: -inf, -inf."""
    with np.errstate(all="ignore"):
        m = x.max(axis=1, keepdims=True, initial=-np.inf)
        m0 = np.where(np.isfinite(m), m, 0.0)
        log_sum = np.log(np.exp(x - m0).sum(axis=1))
        lse = m0[:, 0] + log_sum
        # from x - m, not x - lse: next to a maximum of -3e38 the logarithm is lost in lse
        logp = np.where(np.isneginf(x), -np.inf, (x - m0) - np.where(np.isneginf(lse), 0.0, log_sum)[:, None])
    return lse, logp


def entropy_rows(logp):
    with np.errstate(all="ignore"):
        t = np.exp(logp) * logp
    return -np.where(np.isneginf(logp), 0.0, t).sum(axis=1)


def ref_logprobs(z, tokens, t):
    lse, logp = softmax_rows(z / t)
    given = (tokens >= 0) & (tokens < z.shape[1])
    at = np.array([logp[i, y] if ok else 0.0 for i, (y, ok) in enumerate(zip(tokens, given))])
    return at, entropy_rows(logp), lse, logp


def ref_top(z, logp, n):
    T, V = z.shape
    tok = np.full((T, n), -1, np.int64)
    val = np.full((T, n), -np.inf)
    for i in range(T):
        order = np.lexsort((np.arange(V), -z[i]))
        order = [j for j in order[:n] if z[i, j] > -np.inf]
        tok[i, :len(order)] = order
        val[i, :len(order)] = logp[i, order]
    return tok, val


def ref_logprobs_grad(z, tokens, g, h, t):
    _, ent, lse, logp = ref_logprobs(z, tokens, t)
    V = z.shape[1]
    given = (tokens >= 0) & (tokens < V)
    p = np.exp(logp)
    plogp = np.where(p > 0, p * np.where(p > 0, logp, 0.0), 0.0)
    d = -np.where(given, g, 0.0)[:, None] * p - h[:, None] * (plogp + p * ent[:, None])
    G = np.abs(np.where(given, g, 0.0))[:, None] * p + np.abs(h)[:, None] * (np.abs(plogp) + p * ent[:, None])
    for i in np.flatnonzero(given & ~np.isneginf(lse)):
        d[i, tokens[i]] += g[i]
        G[i, tokens[i]] += abs(g[i])
    d[np.isneginf(lse)] = 0.0
    G[np.isneginf(lse)] = 0.0
    return d / t, G / t


def teacher_softmax(tok, val, V, t):
    real = (tok >= 0) & (tok < V)
    v = np.where(real, val, -np.inf) / t
    lse, logP = softmax_rows(v)
    P = np.exp(logP)
    return P, logP


def ref_distill(z, tok, val, t):
    lse, logq = softmax_rows(z / t)
    P, logP = teacher_softmax(tok, val, z.shape[1], t)
    loss, size = np.zeros(len(z)), np.zeros(len(z))
    for i in range(len(z)):
        for k in np.flatnonzero(P[i] > 0):
            lq = logq[i, tok[i, k]] if not np.isneginf(lse[i]) else -np.inf
            loss[i] += P[i, k] * (logP[i, k] - lq)
            size[i] += P[i, k] * (abs(logP[i, k]) + abs(lq))
    return t * t * loss, t * t * size, lse


def ref_distill_grad(z, tok, val, w, t):
    lse, logq = softmax_rows(z / t)
    P, _ = teacher_softmax(tok, val, z.shape[1], t)
    d = np.exp(logq) * (w * t * P.sum(axis=1))[:, None]
    G = np.abs(d)
    for i in range(len(z)):
        if np.isneginf(lse[i]):
            d[i] = G[i] = 0.0
            continue
        for k in np.flatnonzero(P[i] > 0):
            d[i, tok[i, k]] -= w[i] * t * P[i, k]
            G[i, tok[i, k]] += abs(w[i]) * t * P[i, k]
    return d, G


def err_log_sum(V):
    return 2.0 ** -24 * (2 * (-(-V // 512) + 8) + 56)


def bound_log(z, t, lse, x):
    """of a log-probability or log-sum-exp of value x"""
    with np.errstate(all="ignore"):
        top = np.nan_to_num(np.abs(np.where(np.isneginf(z), 0, z)).max(axis=1, initial=0.0)) / t
    return err_log_sum(z.shape[1]) + 2.0 ** -22 * (np.abs(np.nan_to_num(x, neginf=0.0)) + top
                                                   + np.abs(np.nan_to_num(lse, neginf=0.0)))


def near(got, want, tol, what):
    got = got.detach().double().cpu().numpy() if isinstance(got, torch.Tensor) else got
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    with np.errstate(all="ignore"):
        ok = same | (np.abs(got - want) <= tol)
    bad = np.argwhere(~ok)
    assert bad.size == 0, (f"{what}: {len(bad)} of {ok.size} outside tolerance, first at {tuple(bad[0])}: "
                           f"got {got[tuple(bad[0])]!r}, want {want[tuple(bad[0])]!r}")


def make(T, V, kind, mask="none", seed=0, pad=0, shift=0):
    """(device view, its values in 64 bits): rows padded by `pad` elements
    (NaN there) and starting `shift` elements into the buffer."""
    g = np.random.default_rng(seed)
    z = g.normal(size=(T, V)) * 3
    low = LOWEST[kind]
    if mask == "banned":
        z[g.random((T, V)) < 0.6] = -np.inf
    elif mask == "empty":
        z[::2] = -np.inf
    elif mask == "one":
        keep = g.integers(0, V, T)
        y = z[np.arange(T), keep]
        z[:] = -np.inf
        z[np.arange(T), keep] = y
    elif mask == "lowest":
        z[g.random((T, V)) < 0.9] = low
        z[0] = low
    elif mask == "few":
        z[:, 3:] = low
    elif mask == "equal":
        z[:] = 1.25
    elif mask == "ties":
        z = np.round(z)
    elif mask == "rising":
        z = np.sort(z, axis=1)
    buf = torch.full((T * (V + pad) + shift + 8,), float("nan"), dtype=TYPES[kind], device="cuda")
    view = torch.as_strided(buf, (T, V), (V + pad, 1), shift)
    view.copy_(torch.from_numpy(z))
    return view, view.double().cpu().numpy()


def check_logprobs(tc, view, z, tokens, top, t):
    tok = torch.from_numpy(tokens).cuda()
    r = tc.token_logprobs(view, tok, top, temperature=t)
    torch.cuda.synchronize()
    lp, ent, lse, logp = ref_logprobs(z, tokens, t)
    near(r.lse, lse, bound_log(z, t, lse, lse), "lse")
    near(r.logprob, lp, bound_log(z, t, lse, lp), "logprob")
    e = err_log_sum(z.shape[1])
    near(r.entropy, ent, (2 * e + 2.0 ** -22) * (1 + ent), "entropy")
    want_tok, want_val = ref_top(z, logp, top)
    assert np.array_equal(r.top_token.cpu().numpy(), want_tok)
    near(r.top_logprob, want_val, bound_log(z, t, lse, want_val.max(axis=1, initial=0.0))[:, None]
         + 2.0 ** -22 * np.abs(np.nan_to_num(want_val, neginf=0.0)), "top_logprob")
    return r


SIZES = [(3, 1), (2, 7), (4, 8), (3, 9), (2, 50), (3, 511), (2, 4096), (3, 4103), (2, 50001), (1, 131072), (2, 262147)]


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("T,V", SIZES, ids=lambda v: str(v))
@pytest.mark.parametrize("top", [0, 1, 20, 128])
def test_logprobs_sizes(tc, kind, T, V, top):
    view, z = make(T, V, kind, seed=V + top, pad=3, shift=1)
    tokens = np.random.default_rng(V).integers(0, V, T)
    tokens[-1] = -1 if T > 2 else tokens[-1]
    check_logprobs(tc, view, z, tokens, top, 0.8)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("mask", ["banned", "empty", "one", "lowest", "few", "equal", "ties", "rising"])
@pytest.mark.parametrize("V", [200, 9001, 70000])
def test_logprobs_masks(tc, kind, mask, V):
    view, z = make(5, V, kind, mask, seed=V)
    tokens = np.random.default_rng(1).integers(0, V, 5)
    tokens[2], tokens[3] = V, -7          # outside the vocabulary: nothing is given
    check_logprobs(tc, view, z, tokens, 33, 1.0)


@pytest.mark.parametrize("kind", list(TYPES))
def test_logprobs_concentrated(tc, kind):
    """All large logits at positions a multiple of 4096 (and 8192) apart, the
    places that one thread of a block reads."""
    V = 140000
    view, z = make(2, V, kind, seed=4)
    z[:, :] = -5.0
    for off in range(8):
        z[:, off::4096] = 3.0 + 0.125 * ((np.arange(z[0, off::4096].size) * 7 + off * 3) % 61)
    view.copy_(torch.from_numpy(z))
    z = view.double().cpu().numpy()
    check_logprobs(tc, view, z, np.array([8, 4097]), 128, 1.0)


def test_logprobs_many_rows(tc):
    view, z = make(1500, 333, "bf16", "ties", seed=9, pad=1)
    check_logprobs(tc, view, z, np.random.default_rng(2).integers(0, 333, 1500), 5, 1.3)


def test_nan_and_inf_rows(tc):
    view, z = make(4, 5000, "f32", seed=5)
    z[1, 77], z[2, 4999], z[3, 0] = np.nan, np.inf, -np.inf
    view.copy_(torch.from_numpy(z))
    r = tc.token_logprobs(view, torch.zeros(4, dtype=torch.int64, device="cuda"), 3)
    bad = torch.isnan(r.lse).tolist()
    assert bad == [False, True, True, False]
    assert torch.isnan(r.entropy).tolist() == bad
    assert torch.isnan(r.logprob).tolist() == bad
    assert r.logprob[3].item() == -np.inf
    assert 77 not in r.top_token[1].tolist()
    gr = tc.token_logprobs_grad(view, torch.zeros(4, dtype=torch.int64, device="cuda"),
                                torch.ones(4, device="cuda"))
    assert torch.isnan(gr.dlogits).any(1).tolist() == bad


def check_grad(got, d, G, kind, z, t, lse):
    e = err_log_sum(z.shape[1])
    top = np.nan_to_num(np.abs(np.where(np.isneginf(z), 0, z)).max(axis=1, initial=0.0))[:, None] / t
    # the exponent of p: its own rounding grows with its size (p is at most 1
    # and |log p| p at most 1/e, so a size of 120 covers every p above 2^-150)
    tol = HALF_ULP[kind] * np.abs(d) * (1 + 1e-6) + SMALLEST[kind] + G * (2 * e + 2.0 ** -22 * (4 + 60 + np.minimum(top, 200)))
    near(got, d, tol, "gradient")


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("T,V", SIZES, ids=lambda v: str(v))
@pytest.mark.parametrize("inplace", [False, True], ids=["apart", "inplace"])
def test_logprobs_grad(tc, kind, T, V, inplace):
    view, z = make(T, V, kind, seed=V, pad=5, shift=2)
    rng = np.random.default_rng(V)
    tokens = rng.integers(0, V, T)
    tokens[-1] = -1 if T > 2 else tokens[-1]
    g, h = rng.normal(size=T).astype(np.float32), rng.normal(size=T).astype(np.float32)
    t = 1.7
    # apart: another row stride and another start within 16 bytes
    out = view if inplace else torch.full((T, V + 9), 7.0, dtype=TYPES[kind], device="cuda")[:, 1:V + 1]
    r = tc.token_logprobs_grad(view, torch.from_numpy(tokens).cuda(), torch.from_numpy(g).cuda(),
                               torch.from_numpy(h).cuda(), temperature=t, dlogits=out)
    torch.cuda.synchronize()
    lp, ent, lse, _ = ref_logprobs(z, tokens, t)
    near(r.lse, lse, bound_log(z, t, lse, lse), "lse")
    near(r.logprob, lp, bound_log(z, t, lse, lp), "logprob")
    near(r.entropy, ent, (2 * err_log_sum(V) + 2.0 ** -22) * (1 + ent), "entropy")
    d, G = ref_logprobs_grad(z, tokens, g.astype(np.float64), h.astype(np.float64), t)
    check_grad(r.dlogits, d, G, kind, z, t, lse)
    if not inplace:      # nothing beside the row is written
        whole = torch.as_strided(out, (T, V + 9), (V + 9, 1), out.storage_offset() - 1)
        assert bool((whole[:, 0] == 7).all()) and bool((whole[:, V + 1:] == 7).all())


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("mask", ["banned", "empty", "one", "lowest", "few", "equal"])
def test_logprobs_grad_masks(tc, kind, mask):
    T, V = 6, 9001
    view, z = make(T, V, kind, mask, seed=3)
    rng = np.random.default_rng(8)
    tokens = rng.integers(0, V, T)
    tokens[1] = V
    g, h = rng.normal(size=T).astype(np.float32), rng.normal(size=T).astype(np.float32)
    r = tc.token_logprobs_grad(view, torch.from_numpy(tokens).cuda(), torch.from_numpy(g).cuda(),
                               torch.from_numpy(h).cuda())
    torch.cuda.synchronize()
    d, G = ref_logprobs_grad(z, tokens, g.astype(np.float64), h.astype(np.float64), 1.0)
    lse = ref_logprobs(z, tokens, 1.0)[2]
    check_grad(r.dlogits, d, G, kind, z, 1.0, lse)


def test_logprobs_grad_differences(tc):
    """The gradient against central differences of the 64-bit definition."""
    T, V, t = 3, 40, 0.9
    view, z = make(T, V, "f32", seed=11)
    tokens = np.array([3, 39, 0])
    g, h = np.array([1.0, -0.5, 2.0]), np.array([0.3, 1.0, -0.7])
    r = tc.token_logprobs_grad(view, torch.from_numpy(tokens).cuda(), torch.from_numpy(g).float().cuda(),
                               torch.from_numpy(h).float().cuda(), temperature=t)
    got = r.dlogits.double().cpu().numpy()
    eps = 1e-5

    def f(zz):
        lp, ent, _, _ = ref_logprobs(zz, tokens, t)
        return g * lp + h * ent

    for j in range(V):
        zp, zm = z.copy(), z.copy()
        zp[:, j] += eps
        zm[:, j] -= eps
        # differences: third derivatives are at most ~40 here, times eps^2 / 6, and 1e-16 / eps of rounding
        assert np.all(np.abs(got[:, j] - (f(zp) - f(zm)) / (2 * eps)) < 1e-5), j


def teacher(T, V, K, seed, padded=True, kind="f32"):
    rng = np.random.default_rng(seed)
    tok = np.stack([rng.permutation(max(V, K))[:K] for _ in range(T)]).astype(np.int64) if K else np.zeros((T, 0), np.int64)
    tok[tok >= V] = -1
    val = rng.normal(size=(T, K)) * 3
    if padded and K > 1:
        tok[0, K // 2:] = -1
        val[0, K // 2:] = np.nan              # not used
    if padded and T > 1:
        tok[1] = -1
        val[1] = np.inf
    dv = torch.from_numpy(val).to(TYPES[kind]).cuda()
    return torch.from_numpy(tok).cuda(), dv, tok, dv.double().cpu().numpy()


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("T,V", [(3, 1), (3, 9), (2, 511), (3, 4103), (2, 50001), (2, 262147)], ids=lambda v: str(v))
@pytest.mark.parametrize("K", [0, 1, 8, 65, 300, 1024])
def test_distill(tc, kind, T, V, K):
    if K > 2 * V:
        pytest.skip("fewer tokens than teacher entries")
    view, z = make(T, V, kind, seed=K, pad=1, shift=3)
    tt, tv, tok, val = teacher(T, V, K, V + K, kind=kind)
    t = 1.4
    w = np.random.default_rng(3).normal(size=T).astype(np.float32)
    loss, lse = tc.distill_topk(view, tt, tv, temperature=t)
    loss2, d = tc.distill_topk_grad(view, tt, tv, torch.from_numpy(w).cuda(), temperature=t)
    torch.cuda.synchronize()
    want, size, ref_lse = ref_distill(z, tok, val, t)
    near(lse, ref_lse, bound_log(z, t, ref_lse, ref_lse), "lse")
    # the teacher's own softmax has at most 1024 terms of the same kind, and the loss sums K of them
    tol = (t * t * bound_log(z, t, ref_lse, ref_lse) + t * t * err_log_sum(1024 * 16)
           + 2.0 ** -22 * (40 + -(-K // 32)) * size)
    near(loss, want, tol, "loss")
    near(loss2, want, tol, "loss")
    dref, G = ref_distill_grad(z, tok, val, w.astype(np.float64), t)
    check_grad(d, dref, G, kind, z, t, ref_lse)
    # in place, and the same bits
    _, d2 = tc.distill_topk_grad(view, tt, tv, torch.from_numpy(w).cuda(), temperature=t, dlogits=view)
    assert torch.equal(d2, d)


@pytest.mark.parametrize("mask", ["banned", "empty", "one", "lowest", "few", "equal"])
def test_distill_masks(tc, mask):
    T, V, K = 6, 9001, 17
    view, z = make(T, V, "bf16", mask, seed=3)
    tt, tv, tok, val = teacher(T, V, K, 5)
    val[3, 4:] = -np.inf
    tv.copy_(torch.from_numpy(val))
    w = np.random.default_rng(3).normal(size=T).astype(np.float32)
    loss, d = tc.distill_topk_grad(view, tt, tv, torch.from_numpy(w).cuda())
    want, size, ref_lse = ref_distill(z, tok, val, 1.0)
    near(loss, want, bound_log(z, 1.0, ref_lse, ref_lse) + err_log_sum(1024 * 16) + 2.0 ** -22 * 41 * np.nan_to_num(size, posinf=0.0),
         "loss")
    dref, G = ref_distill_grad(z, tok, val, w.astype(np.float64), 1.0)
    check_grad(d, dref, G, "bf16", z, 1.0, ref_lse)


def test_distill_repeated_tokens(tc):
    """A token given twice counts as two terms."""
    T, V, K = 3, 700, 12
    view, z = make(T, V, "f32", seed=3)
    tt, tv, tok, val = teacher(T, V, K, 5, padded=False)
    tok[:, 5], tok[:, 7], tok[:, 11] = tok[:, 0], tok[:, 0], tok[:, 1]
    tt.copy_(torch.from_numpy(tok))
    w = np.ones(T, np.float32)
    loss, d = tc.distill_topk_grad(view, tt, tv, torch.from_numpy(w).cuda())
    want, size, ref_lse = ref_distill(z, tok, val, 1.0)
    near(loss, want, bound_log(z, 1.0, ref_lse, ref_lse) + err_log_sum(1024 * 16) + 2.0 ** -22 * 41 * size, "loss")
    dref, G = ref_distill_grad(z, tok, val, w.astype(np.float64), 1.0)
    check_grad(d, dref, G, "f32", z, 1.0, ref_lse)


def test_distill_differences(tc):
    T, V, K, t = 3, 40, 6, 1.3
    view, z = make(T, V, "f32", seed=21)
    tt, tv, tok, val = teacher(T, V, K, 6)
    w = np.array([1.0, 2.0, -0.5])
    _, d = tc.distill_topk_grad(view, tt, tv, torch.from_numpy(w).float().cuda(), temperature=t)
    got, eps = d.double().cpu().numpy(), 1e-5
    for j in range(V):
        zp, zm = z.copy(), z.copy()
        zp[:, j] += eps
        zm[:, j] -= eps
        diff = w * (ref_distill(zp, tok, val, t)[0] - ref_distill(zm, tok, val, t)[0]) / (2 * eps)
        assert np.all(np.abs(got[:, j] - diff) < 1e-5), j


def test_other_stream_and_graph(tc):
    """On a stream of its own and from a captured graph: the same bits."""
    view, z = make(7, 30011, "bf16", seed=2)
    tokens = torch.arange(7, device="cuda") * 100
    g = torch.ones(7, device="cuda")
    want = tc.token_logprobs(view, tokens, 9)
    want_d = tc.token_logprobs_grad(view, tokens, g, g).dlogits
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = tc.token_logprobs(view, tokens, 9)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    out = torch.empty_like(view)
    with torch.cuda.graph(graph):
        got = tc.token_logprobs(view, tokens, 9)
        tc.token_logprobs_grad(view, tokens, g, g, dlogits=out)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(out, want_d)


def test_offsets_past_32_bits(tc):
    """Rows more than 2^31 elements apart."""
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB of device memory")
    ld, V = (1 << 31) + 24, 1000
    buf = torch.empty((2 * ld,), dtype=torch.float16, device="cuda")
    view = torch.as_strided(buf, (2, V), (ld, 1), 8)
    z = np.random.default_rng(1).normal(size=(2, V))
    view.copy_(torch.from_numpy(z))
    z = view.double().cpu().numpy()
    tokens = np.array([5, 999])
    check_logprobs(tc, view, z, tokens, 4, 1.0)
    one = np.ones(2)
    r = tc.token_logprobs_grad(view, torch.from_numpy(tokens).cuda(), torch.ones(2, device="cuda"),
                               torch.ones(2, device="cuda"), dlogits=view)
    d, G = ref_logprobs_grad(z, tokens, one, one, 1.0)
    check_grad(r.dlogits, d, G, "f16", z, 1.0, ref_logprobs(z, tokens, 1.0)[2])


def test_empty_calls(tc):
    z = torch.empty((0, 100), dtype=torch.float32, device="cuda")
    r = tc.token_logprobs(z, torch.empty(0, dtype=torch.int64, device="cuda"), 3)
    assert r.top_token.shape == (0, 3)
    z = torch.empty((2, 0), dtype=torch.float32, device="cuda")
    r = tc.token_logprobs(z, torch.zeros(2, dtype=torch.int64, device="cuda"), 2)
    assert r.lse.tolist() == [-np.inf] * 2 and r.logprob.tolist() == [0.0] * 2 and r.entropy.tolist() == [0.0] * 2
    assert r.top_token.tolist() == [[-1, -1]] * 2


def test_refusals(tc):
    z = torch.zeros((4, 64), device="cuda")
    i = torch.zeros(4, dtype=torch.int64, device="cuda")
    f = torch.zeros(4, device="cuda")
    for bad in (dict(logits=z.double()), dict(logits=z.t()), dict(logits=z[0]), dict(logits=z.cpu()),
                dict(tokens=i.int()), dict(tokens=i[:3]), dict(tokens=i.cpu()), dict(top=129), dict(top=-1)):
        a = dict(logits=z, tokens=i, top=2)
        a.update(bad)
        with pytest.raises(ValueError):
            tc.token_logprobs(a["logits"], a["tokens"], a["top"])
    for t in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(tc.GemmError):
            tc.token_logprobs(z, i, temperature=t)
    for kw in (dict(grad_logprob=f[:2]), dict(dlogits=z.half()), dict(dlogits=z[:, :60]), dict(grad_entropy=f.half())):
        with pytest.raises(ValueError):
            tc.token_logprobs_grad(z, i, **kw)
    with pytest.raises(ValueError):
        tc.token_logprobs_grad(z, None, f)
    tt, tv = torch.zeros((4, 5), dtype=torch.int64, device="cuda"), torch.zeros((4, 5), device="cuda")
    for a in ((tt.int(), tv), (tt[:, :4], tv), (tt[:3], tv[:3]), (tt, tv.double()), (tt, tv.cpu())):
        with pytest.raises(ValueError):
            tc.distill_topk(z, *a)
    big = torch.zeros((4, 1025), dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError):
        tc.distill_topk(z, big, big.float())
    with pytest.raises(ValueError):
        tc.distill_topk_grad(z, tt, tv, None)
