"""Measured operators: the 8-bit integer product with a scale for each token
and channel, log-probabilities of given tokens with entropy and the top
alternatives (and their gradient), and distillation from a teacher's top
logits, forward and backward.

Together they are the output head of a language model next to the dense
product: a frozen (teacher's) head held in 8 bits gives logits, the
log-probability operator turns logits into the teacher's top tokens, and the
distillation loss turns those and the student's logits into the gradient that
goes back through the dense product.

``run`` computes the plain form (torch, 32 bits, rounded once at the end), or
with ``own`` set makes the package's calls.  Definitions:

* product     D = act(rs[i] * cs[j] * sum_k A[i,k] B[k,j] + bias[j]), A and B int8;
* linear      the same with A and rs made from rows X[i,:] of 16- or 32-bit floats:
              rs[i] = max_k |X[i,k]| / 127, A[i,k] = round(X[i,k] / rs[i]) (half to
              even; a row of zeros gives zeros);
* logprobs    x = logits / temperature; lse = log sum_j e^x_j; logprob = x_token - lse
              (0 for a token of -1), entropy = -sum_j p_j log p_j with p = e^(x - lse),
              and the n largest log p with their tokens, equal ones by the lowest
              token; tokens whose logit is -inf are no alternatives (token -1,
              log-probability -inf in the places that are left);
* logprobs_grad  logprob, entropy and lse, and the gradient of
              sum_i (g_i logprob_i + h_i entropy_i) for the logits:
              (g (1[j = token] - p_j) - h p_j (log p_j + entropy)) / temperature,
              without the first term where the token is -1;
* distill     a row's loss is t^2 sum_k P_k (log P_k - log Q_k), t the temperature,
              P the softmax of the teacher's K given logits / t (tokens of -1 are
              padding), Q the softmax of the student's logits / t over the whole
              vocabulary; a row without teacher tokens has loss 0;
* distill_grad   that and the gradient of sum_i w_i loss_i for the logits,
              w t (Q_j - sum of P_k over k with token j).
"""
import functools
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one token of a small layer: the weights are read once, latency counts
        dict(name="product one token", op="product", M=1, N=4096, K=4096, out="bf16", bias=False, act="none"),
        # a decoding batch through a wide layer (the memory-bound shape of the benchmark's bf16 product),
        # activations quantised in the call
        dict(name="linear decode", op="linear", M=16, N=8192, K=8192, x="bf16", out="bf16", bias=True, act="none"),
        # odd extents in every direction, fp32 output (the benchmark's ragged product)
        dict(name="product ragged", op="product", M=4097, N=2055, K=1000, out="f32", bias=True, act="none"),
        # a long prompt through a wide layer: compute-bound
        dict(name="linear prefill", op="linear", M=8192, N=8192, K=8192, x="bf16", out="bf16", bias=False, act="gelu"),
        # sampling one sequence: one row of logits, its token's log-probability and 20 alternatives
        dict(name="logprobs one row", op="logprobs", T=1, V=131072, x="f32", top=20, temperature=1.0, banned=0.0),
        # a decoding batch under a vocabulary mask, odd vocabulary
        dict(name="logprobs decode", op="logprobs", T=61, V=50001, x="f16", top=5, temperature=0.7, banned=0.3),
        # scoring a long batch: the teacher's top 64 at every position
        dict(name="logprobs scoring", op="logprobs", T=4096, V=131072, x="bf16", top=64, temperature=1.0, banned=0.0),
        # a policy-gradient step: log-probability and entropy with the gradient for the logits
        dict(name="logprobs gradient", op="logprobs_grad", T=2048, V=65537, x="bf16", temperature=1.0, banned=0.0),
        # a small distillation step
        dict(name="distill small", op="distill_grad", T=16, V=32768, K=8, x="f32", temperature=2.0, padded=False),
        # evaluation only: loss without gradient, ragged, teacher rows of different lengths
        dict(name="distill evaluation", op="distill", T=1000, V=50001, K=50, x="bf16", temperature=1.0, padded=True),
        # a training step over an odd vocabulary in fp32
        dict(name="distill odd", op="distill_grad", T=777, V=100003, K=33, x="f32", temperature=1.5, padded=True),
        # a large training step
        dict(name="distill training", op="distill_grad", T=4096, V=131072, K=64, x="bf16", temperature=1.0, padded=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["product", "linear", "logprobs", "logprobs_grad", "distill", "distill_grad"])
    if op in ("product", "linear"):
        M, N, K = _log(rng, 1, 8192), _log(rng, 256, 8192), _log(rng, 256, 8192)
        if rng.random() < 0.5:      # layer widths are mostly multiples of 64
            N, K = -(-N // 64) * 64, -(-K // 64) * 64
        case = dict(op=op, M=M, N=N, K=K, out=rng.choice(["f32", "f16", "bf16"]), bias=rng.random() < 0.5,
                    act=rng.choice(["none", "none", "relu", "gelu"]))
        if op == "linear":
            case["x"] = rng.choice(["f32", "f16", "bf16"])
        return case
    V = _log(rng, 8192, 262144)
    if rng.random() < 0.5:
        V = -(-V // 128) * 128
    x = rng.choice(["f32", "f16", "bf16"])
    # at most as many logits as the largest listed case
    T = _log(rng, 1, min(8192, max(1, (1 << 28) // V)))
    case = dict(op=op, T=T, V=V, x=x, temperature=rng.choice([0.6, 1.0, 1.0, 2.0]))
    if op == "logprobs":
        case.update(top=rng.choice([0, 1, 5, 20, 64, 128]), banned=rng.choice([0.0, 0.0, 0.5]))
    elif op == "logprobs_grad":
        case.update(banned=rng.choice([0.0, 0.0, 0.5]))
    else:
        case.update(K=_log(rng, 1, 256), padded=rng.random() < 0.5)
    return case


def work(case):
    op = case["op"]
    if op in ("product", "linear"):
        M, N, K = case["M"], case["N"], case["K"]
        a = M * K * BYTES[case["x"]] if op == "linear" else M * K + 4 * M
        return {"bytes": a + N * K + M * N * BYTES[case["out"]] + 4 * N * (2 if case["bias"] else 1),
                "flops": 2 * M * N * K}
    T, V, e = case["T"], case["V"], BYTES[case["x"]]
    if op == "logprobs":
        return {"bytes": T * V * e + T * (8 + 12 + 12 * case["top"]), "flops": 6 * T * V}
    if op == "logprobs_grad":
        return {"bytes": 2 * T * V * e + T * (8 + 8 + 12), "flops": 12 * T * V}
    if op == "distill":
        return {"bytes": T * V * e + T * (12 * case["K"] + 8), "flops": 4 * T * V}
    return {"bytes": 2 * T * V * e + T * (12 * case["K"] + 8), "flops": 8 * T * V}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _up(n, q):
    return -(-n // q) * q


def _rows(values, unit):
    """A matrix whose rows start on whole units of `unit` elements (the row
    stride the package's tensor loads ask for)."""
    r, c = values.shape
    if c % unit == 0:
        return values
    m = torch.zeros((r, _up(c, unit)), dtype=values.dtype, device=values.device)
    m[:, :c] = values
    return m[:, :c]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = torch.device("cuda")
    s = dict(case)
    op = case["op"]
    if op in ("product", "linear"):
        M, N, K = case["M"], case["N"], case["K"]
        # weights: rows of normal values quantised to the full int8 range
        w = torch.randn((N, K), generator=g, device=dev)
        top = w.abs().amax(1, keepdim=True)
        s["W"] = _rows(torch.round(w / top * 127).to(torch.int8), 16)
        s["col_scale"] = (top[:, 0] / 127 * K ** -0.5).contiguous()
        del w, top
        x = torch.randn((M, K), generator=g, device=dev)
        # tokens of different sizes, a few large channels as activations have
        x *= torch.exp(torch.randn((M, 1), generator=g, device=dev) * 0.5)
        x[:, :: max(1, K // 7)] *= 8.0
        if op == "product":
            top = x.abs().amax(1, keepdim=True)
            s["A"] = _rows(torch.round(x / top * 127).to(torch.int8), 16)
            s["row_scale"] = (top[:, 0] / 127).contiguous()
        else:
            s["X"] = x.to(DTYPES[case["x"]])
        s["bias_v"] = torch.randn((N,), generator=g, device=dev) if case["bias"] else None
        s["D"] = torch.empty((M, N), dtype=DTYPES[case["out"]], device=dev)
        return s
    T, V = case["T"], case["V"]
    z = torch.randn((T, V), generator=g, device=dev) * 2.5
    if op.startswith("logprobs"):
        s["tokens"] = torch.randint(0, V, (T,), generator=g, device=dev)
        # the row's own token is a likely one
        z.scatter_(1, s["tokens"][:, None], 8.0 + 2.0 * torch.randn((T, 1), generator=g, device=dev))
        if case["banned"] > 0:
            ban = torch.rand((T, V), generator=g, device=dev) < case["banned"]
            ban.scatter_(1, s["tokens"][:, None], False)
            z.masked_fill_(ban, -math.inf)
            del ban
        if T > 8:
            s["tokens"][::8] = -1       # positions of a prompt: nothing is scored
        if op == "logprobs_grad":
            s["g"] = torch.randn((T,), generator=g, device=dev)
            s["h"] = torch.randn((T,), generator=g, device=dev) * 0.01
    else:
        K = case["K"]
        # K different tokens a row, one from each of K ranges of the vocabulary
        span = V // K
        tok = torch.randint(0, span, (T, K), generator=g, device=dev) + torch.arange(K, device=dev) * span
        val, order = torch.sort(torch.randn((T, K), generator=g, device=dev) * 2.0 + 8.0, dim=1, descending=True)
        tok = torch.gather(tok, 1, order)
        # the student has learnt some of it
        z.scatter_(1, tok, val + torch.randn((T, K), generator=g, device=dev))
        if case["padded"]:
            n = torch.randint(0, K + 1, (T, 1), generator=g, device=dev)
            tok = torch.where(torch.arange(K, device=dev)[None, :] < n, tok, -1)
        s["teacher_tokens"], s["teacher_logits"] = tok.contiguous(), val.contiguous()
        if op == "distill_grad":
            s["w"] = torch.rand((T,), generator=g, device=dev) / T
    s["logits"] = z.to(DTYPES[case["x"]])
    del z
    if op.endswith("_grad"):
        s["dlogits"] = torch.empty_like(s["logits"])
    return s


# ---------------------------------------------------------------------------
# the package's calls
# ---------------------------------------------------------------------------
@functools.lru_cache(maxsize=None)
def _package():
    import tensor_core_dense_tma_gb300 as tc
    return tc, tc.Plan("f16")


def _run_own(s):
    tc, plan = _package()
    op = s["op"]
    if op == "product":
        return plan.gemm_i8(s["A"], s["W"].t(), s["D"], row_scale=s["row_scale"], col_scale=s["col_scale"],
                            bias=s["bias_v"], act=s["act"])
    if op == "linear":
        return plan.linear_i8(s["X"], s["W"].t(), s["D"], col_scale=s["col_scale"], bias=s["bias_v"], act=s["act"])
    if op == "logprobs":
        r = tc.token_logprobs(s["logits"], s["tokens"], top=s["top"], temperature=s["temperature"])
        return {"logprob": r.logprob, "entropy": r.entropy, "lse": r.lse, "top_logprob": r.top_logprob,
                "top_token": r.top_token}
    if op == "logprobs_grad":
        r = tc.token_logprobs_grad(s["logits"], s["tokens"], s["g"], s["h"], temperature=s["temperature"],
                                   dlogits=s["dlogits"])
        return {"logprob": r.logprob, "entropy": r.entropy, "lse": r.lse, "dlogits": r.dlogits}
    if op == "distill":
        loss, lse = tc.distill_topk(s["logits"], s["teacher_tokens"], s["teacher_logits"],
                                    temperature=s["temperature"])
        return {"loss": loss, "lse": lse}
    loss, dlogits = tc.distill_topk_grad(s["logits"], s["teacher_tokens"], s["teacher_logits"], s["w"],
                                         temperature=s["temperature"], dlogits=s["dlogits"])
    return {"loss": loss, "dlogits": dlogits}


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _act(u, act):
    if act == "relu":
        return torch.clamp(u, min=0)
    if act == "gelu":
        return 0.5 * u * (1 + torch.erf(u * 0.7071067811865476))
    return u


def _plain_product(s):
    if s["op"] == "linear":
        x = s["X"].float()
        top = x.abs().amax(1, keepdim=True)
        scale = top / torch.full_like(top, 127.0)
        a = torch.where(top > 0, torch.round(x / scale), torch.zeros_like(x))
        scale = scale[:, 0]
    else:
        a, scale = s["A"].float(), s["row_scale"]
    u = (a @ s["W"].float().t()) * scale[:, None] * s["col_scale"][None, :]
    if s["bias_v"] is not None:
        u = u + s["bias_v"]
    return _act(u, s["act"]).to(s["D"].dtype)


def _log_softmax(x):
    """(log p, lse) of the rows of x."""
    m = x.amax(1, keepdim=True)
    lse = m + torch.log(torch.exp(x - m).sum(1, keepdim=True))
    return x - lse, lse[:, 0]


def _top(logp, n):
    """The n largest of each row, equal ones by the lowest index: the values'
    bits as ordered integers above the complemented index."""
    V = logp.shape[1]
    bits = (logp + 0.0).view(torch.int32).to(torch.int64)
    key = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
    key = key * (1 << 31) + (V - 1 - torch.arange(V, device=logp.device))
    token = torch.topk(key, min(n, V), dim=1).indices
    value = torch.gather(logp, 1, token)
    return value, torch.where(value > -math.inf, token, -1)


def _plain_logprobs(s):
    x = s["logits"].float() / s["temperature"]
    logp, lse = _log_softmax(x)
    tok = s["tokens"]
    given = tok >= 0
    at = torch.gather(logp, 1, tok.clamp(min=0)[:, None])[:, 0]
    out = {"logprob": torch.where(given, at, torch.zeros_like(at))}
    p = torch.exp(logp)
    plogp = torch.where(p > 0, p * logp, torch.zeros_like(p))
    ent = -plogp.sum(1)
    out["entropy"], out["lse"] = ent, lse
    if s["op"] == "logprobs":
        # the order of the logits themselves: a shift by lse can make unequal ones equal
        value, token = _top(s["logits"].float(), s["top"])
        out["top_logprob"] = torch.where(token >= 0, value / s["temperature"] - lse[:, None],
                                         torch.full_like(value, -math.inf))
        out["top_token"] = token
        return out
    g, h = torch.where(given, s["g"], torch.zeros_like(s["g"]))[:, None], s["h"][:, None]
    d = -g * p - h * (plogp + p * ent[:, None])
    d.scatter_add_(1, tok.clamp(min=0)[:, None], g)
    out["dlogits"] = (d / s["temperature"]).to(s["logits"].dtype)
    return out


def _plain_distill(s):
    t = s["temperature"]
    logq, lse = _log_softmax(s["logits"].float() / t)
    tok = s["teacher_tokens"]
    real = tok >= 0
    v = torch.where(real, s["teacher_logits"].float() / t, torch.full_like(s["teacher_logits"], -math.inf))
    m = v.amax(1, keepdim=True).clamp(min=-1e30)
    e = torch.exp(v - m)
    total = e.sum(1, keepdim=True)
    total = torch.where(total > 0, total, torch.ones_like(total))
    P = e / total
    logP = v - m - torch.log(total)
    at = torch.gather(logq, 1, tok.clamp(min=0))
    loss = t * t * torch.where(P > 0, P * (logP - at), torch.zeros_like(P)).sum(1)
    if s["op"] == "distill":
        return {"loss": loss, "lse": lse}
    w = (s["w"] * real.any(1))[:, None]
    d = torch.exp(logq) * w * t
    d.scatter_add_(1, tok.clamp(min=0), -w * t * P)
    return {"loss": loss, "dlogits": d.to(s["logits"].dtype)}


def run(state):
    if own:
        return _run_own(state)
    op = state["op"]
    if op in ("product", "linear"):
        return _plain_product(state)
    if op.startswith("logprobs"):
        return _plain_logprobs(state)
    return _plain_distill(state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_product(s):
    if s["op"] == "linear":
        # the row's scale is the 32-bit number, by definition
        X = s["X"].double()
        top = X.abs().max(dim=1).values
        rs = (top / 127).float().double()
        A = torch.nan_to_num(torch.round(X / rs[:, None]), nan=0.0)
    else:
        A, rs = s["A"].double(), s["row_scale"].double()
    D = torch.matmul(A, s["W"].double().t())
    D.mul_(rs[:, None]).mul_(s["col_scale"].double()[None, :])
    if s["bias_v"] is not None:
        D.add_(s["bias_v"].double()[None, :])
    if s["act"] == "relu":
        D.clamp_(min=0)
    elif s["act"] == "gelu":
        D = D * 0.5 * torch.special.erfc(-D / math.sqrt(2.0))
    return D


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("product", "linear"):
        return _exact_product(s)
    T, V, t = case["T"], case["V"], case["temperature"]
    step = max(1, (1 << 27) // V)
    parts = {}

    def put(**kw):
        for k, v in kw.items():
            parts.setdefault(k, []).append(v)

    for r in range(0, T, step):
        x = s["logits"][r:r + step].double() / t
        lse = torch.logsumexp(x, dim=1)
        n = torch.arange(x.shape[0], device=x.device)
        if op.startswith("logprobs"):
            tok = s["tokens"][r:r + step]
            use = (tok >= 0).double()
            at = tok.clamp(min=0)
            put(logprob=(x[n, at] - lse) * use, lse=lse)
            logp = x - lse[:, None]
            del x
            ent = torch.special.entr(torch.exp(logp)).sum(1)
            put(entropy=ent)
            if op == "logprobs":
                put(top_logprob=torch.topk(logp, min(case["top"], V), dim=1).values)
                continue
            p = torch.exp(logp)
            g, h = s["g"][r:r + step].double() * use, s["h"][r:r + step].double()
            d = torch.special.entr(p) * h[:, None] - p * (g + h * ent)[:, None]
            d[n, at] += g
            put(dlogits=d / t)
        else:
            tok = s["teacher_tokens"][r:r + step]
            P = torch.softmax((s["teacher_logits"][r:r + step].double() / t).masked_fill(tok < 0, -math.inf), dim=1)
            P = torch.nan_to_num(P, nan=0.0)
            logq = x - lse[:, None]
            del x
            cross = (P * torch.gather(logq, 1, tok.clamp(min=0))).sum(1)
            put(loss=t * t * (-torch.special.entr(P).sum(1) - cross))
            if op == "distill":
                put(lse=lse)
                continue
            w = s["w"][r:r + step].double() * (tok >= 0).any(1)
            d = torch.exp(logq) * (w * t)[:, None]
            d.scatter_add_(1, tok.clamp(min=0), -P * (w * t)[:, None])
            put(dlogits=d)
    got = {k: torch.cat(v) for k, v in parts.items()}
    if op == "logprobs":
        got["top_token"] = None
    return got
