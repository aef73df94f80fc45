"""The operators on logits at sizes whose rows are scheduled as in training:
two rows one after another in a CTA, one CTA a row with more chunks than its
ring holds, and clusters of as many CTAs as the logits in flight leave to a row
(2, 3, 5, 6 and 7).  Against the definitions in 64 bits on the GPU, every row, with
the tolerances of test_gpu_logits.py.
"""
import numpy as np
import pytest
import torch

from test_gpu_logits import HALF_ULP, SMALLEST, TYPES, err_log_sum

pytestmark = pytest.mark.gpu

# two rows a CTA (an odd number of rows: the last CTA has one), also of one chunk each; one CTA a row, chunks copied in
# again; clusters of 2 to 7 (about 456 rows or their clusters are in flight at once)
SHORT = [(9001, 8200, "bf16"), (9001, 8192, "f16"), (7999, 4100, "f32"), (9001, 1000, "bf16")]
LONG = [(400, 50001, "bf16"), (520, 33000, "f32"), (500, 131072, "bf16"), (777, 100003, "f32"), (460, 181001, "f32"),
        (459, 210000, "f32"), (458, 250007, "f32")]
IDS = dict(ids=lambda v: str(v))


@pytest.fixture(scope="module")
def tc():
    from tensor_core_dense_tma_gb300 import build as tcbuild
    tcbuild.build()
    import tensor_core_dense_tma_gb300 as tc
    return tc


def logits(T, V, kind, pad, seed):
    """Rows `pad` elements apart (NaN there), one in seven with a mask, one in
    eleven with nothing but one."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.full((T, V + pad), float("nan"), dtype=TYPES[kind], device="cuda")
    view = buf[:, :V]
    for r in range(0, T, 512):
        z = torch.randn((min(512, T - r), V), generator=g, device="cuda") * 3
        z[::7][torch.rand(z[::7].shape, generator=g, device="cuda") < 0.5] = -float("inf")
        z[3::11] = -float("inf")
        view[r:r + 512] = z
    return buf, view


def close(got, want, tol, what):
    ok = (got.double() == want) | ((got.double() - want).abs() <= tol)
    bad = torch.nonzero(~ok)
    assert bad.numel() == 0, (f"{what}: {len(bad)} outside tolerance, first at {bad[0].tolist()}: "
                              f"{got[tuple(bad[0])].item()!r}, want {want[tuple(bad[0])].item()!r}")


class Rows:
    """lse and log p of a slice of rows in 64 bits."""

    def __init__(self, view, r, n, t):
        x = view[r:r + n].double() / t
        top = x.amax(1, keepdim=True)
        self.nothing = torch.isneginf(top[:, 0])
        top = torch.where(torch.isneginf(top), torch.zeros_like(top), top)
        log_sum = torch.log(torch.exp(x - top).sum(1))
        self.lse = top[:, 0] + log_sum
        self.logp = torch.where(torch.isneginf(x), x, x - top - torch.where(self.nothing, 0.0, log_sum)[:, None])
        self.p = torch.exp(self.logp)
        self.plogp = torch.where(self.p > 0, self.p * self.logp, 0.0)
        self.entropy = -self.plogp.sum(1)
        self.size = torch.where(torch.isneginf(x), 0.0, x).abs().amax(1)
        self.log_tol = err_log_sum(x.shape[1]) + 2.0 ** -22 * (self.size + self.lse.nan_to_num(neginf=0.0).abs())

    def gradient_tol(self, d, G, kind):
        rel = 2 * err_log_sum(d.shape[1]) + 2.0 ** -22 * (64 + self.size.clamp(max=200))
        return HALF_ULP[kind] * d.abs() * (1 + 1e-6) + SMALLEST[kind] + G * rel[:, None]


def tokens_of(T, V, seed):
    tok = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(seed))
    tok[::5] = -1
    return tok.cuda()


def slices(T, V):
    step = max(1, (1 << 24) // V)
    return [(r, min(step, T - r)) for r in range(0, T, step)]


@pytest.mark.parametrize("T,V,kind", SHORT + [(5000, 20011, "bf16")], **IDS)
@pytest.mark.parametrize("top", [0, 20])
def test_logprobs(tc, T, V, kind, top):
    t = 0.9
    _, view = logits(T, V, kind, 3, V)
    tok = tokens_of(T, V, 1)
    r = tc.token_logprobs(view, tok, top, temperature=t)
    for a, n in slices(T, V):
        ref = Rows(view, a, n, t)
        y = tok[a:a + n]
        lp = torch.where(y >= 0, ref.logp.gather(1, y.clamp(min=0)[:, None])[:, 0], 0.0)
        close(r.lse[a:a + n], ref.lse, ref.log_tol, "lse")
        close(r.logprob[a:a + n], lp, ref.log_tol + 2.0 ** -22 * lp.nan_to_num(neginf=0.0).abs(), "logprob")
        close(r.entropy[a:a + n], ref.entropy, (2 * err_log_sum(V) + 2.0 ** -22) * (1 + ref.entropy), "entropy")
        if top:
            # a stable order of the logits themselves: equal ones by the lowest token
            z, at = torch.sort(view[a:a + n].float(), dim=1, descending=True, stable=True)
            at = torch.where(torch.isneginf(z[:, :top]), -1, at[:, :top])
            assert torch.equal(r.top_token[a:a + n], at)
            val = torch.where(at >= 0, ref.logp.gather(1, at.clamp(min=0)), -float("inf"))
            close(r.top_logprob[a:a + n], val,
                  ref.log_tol[:, None] + 2.0 ** -22 * val.nan_to_num(neginf=0.0).abs(), "top_logprob")


@pytest.mark.parametrize("T,V,kind", SHORT + LONG, **IDS)
@pytest.mark.parametrize("inplace", [False, True], ids=["apart", "inplace"])
def test_logprobs_grad(tc, T, V, kind, inplace):
    t = 1.2
    _, view = logits(T, V, kind, 5, V)
    tok = tokens_of(T, V, 2)
    g = torch.Generator(device="cuda").manual_seed(3)
    gl, gh = (torch.randn(T, generator=g, device="cuda") for _ in range(2))
    keep = view.clone() if inplace else view
    out = view if inplace else torch.full((T, V + 9), 7.0, dtype=TYPES[kind], device="cuda")[:, 1:V + 1]
    r = tc.token_logprobs_grad(view, tok, gl, gh, temperature=t, dlogits=out)
    for a, n in slices(T, V):
        ref = Rows(keep, a, n, t)
        y = tok[a:a + n]
        close(r.lse[a:a + n], ref.lse, ref.log_tol, "lse")
        close(r.entropy[a:a + n], ref.entropy, (2 * err_log_sum(V) + 2.0 ** -22) * (1 + ref.entropy), "entropy")
        u = torch.where((y >= 0) & ~ref.nothing, gl[a:a + n].double(), 0.0)[:, None]
        h, ent = gh[a:a + n].double()[:, None], ref.entropy[:, None]
        d = -u * ref.p - h * (ref.plogp + ref.p * ent)
        G = u.abs() * ref.p + h.abs() * (ref.plogp.abs() + ref.p * ent)
        d.scatter_add_(1, y.clamp(min=0)[:, None], u)
        G.scatter_add_(1, y.clamp(min=0)[:, None], u.abs())
        d, G = d / t, G / t
        close(out[a:a + n], d, ref.gradient_tol(d, G, kind), "gradient")
    if not inplace:
        whole = torch.as_strided(out, (T, V + 9), (V + 9, 1), 0)
        assert bool((whole[:, 0] == 7).all()) and bool((whole[:, V + 1:] == 7).all())


@pytest.mark.parametrize("T,V,kind", SHORT + LONG, **IDS)
def test_distill(tc, T, V, kind):
    t, K = 1.5, 37
    buf, view = logits(T, V, kind, 1, V + 1)
    g = torch.Generator(device="cuda").manual_seed(4)
    span = V // K
    tt = torch.randint(0, span, (T, K), generator=g, device="cuda") + torch.arange(K, device="cuda") * span
    tv = torch.randn((T, K), generator=g, device="cuda") * 3
    tt[torch.rand((T, K), generator=g, device="cuda") < 0.2] = -1
    w = torch.randn(T, generator=g, device="cuda")
    loss, lse = tc.distill_topk(view, tt, tv, temperature=t)
    loss2, dz = tc.distill_topk_grad(view, tt, tv, w, temperature=t)      # its rows on whole 16 bytes, the logits' not
    for a, n in slices(T, V):
        ref = Rows(view, a, n, t)
        real = tt[a:a + n] >= 0
        at = tt[a:a + n].clamp(min=0)
        logP = torch.log_softmax((tv[a:a + n].double() / t).masked_fill(~real, -float("inf")), dim=1)
        P = torch.where(real, torch.exp(logP), 0.0)
        lq = ref.logp.gather(1, at)
        want = t * t * torch.where(P > 0, P * (logP - lq), 0.0).sum(1)
        size = t * t * torch.where(P > 0, P * (logP.abs() + lq.abs()), 0.0).sum(1)
        tol = t * t * (ref.log_tol + err_log_sum(1024 * 16)) + 2.0 ** -22 * 42 * size.nan_to_num(posinf=0.0)
        close(lse[a:a + n], ref.lse, ref.log_tol, "lse")
        close(loss[a:a + n], want, tol, "loss")
        close(loss2[a:a + n], want, tol, "loss")
        wt = (w[a:a + n].double() * t)[:, None]
        d = ref.p * wt * P.sum(1, keepdim=True)
        G = d.abs()
        P = torch.where(ref.nothing[:, None], 0.0, P)
        d.scatter_add_(1, at, -wt * P)
        G.scatter_add_(1, at, wt.abs() * P)
        close(dz[a:a + n], d, ref.gradient_tol(d, G, kind), "gradient")
    got = tc.distill_topk_grad(view, tt, tv, w, temperature=t, dlogits=view)[1]
    assert torch.equal(got, dz)
