"""Measured operators: low-rank adapters of many requests beside a shared
projection, forward and backward, the clipped policy loss with a KL term and
the preference loss of paired sequences, each with the gradient for the logits.

Together they tune and serve adapters: the projection with adapters gives
hidden states or logits, one of the two losses turns logits into a gradient
(its reference model is the same projection without adapters), and the
adapters' backward pass turns what comes back into their gradients; rows of
many requests, each with its own adapter, are then served in one call.

``run`` computes the plain form (torch, 32 bits, rounded once at the end), or
with ``own`` set makes the package's calls.  Definitions:

* adapters    g = index[i] is row i's adapter (-1: none), s its scale, A = down[g]
              (R x K), U = up[g] (N x R):
              Y[i] = W X[i] + bias + U h[i],  h[i] = s A X[i];
* adapters_grad  of sum(dY * Y), with p[i] = s U^T dY[i]:  dX[i] = W^T dY[i] + A^T p[i],
              d_down[g] = sum of p[i] X[i]^T and d_up[g] = sum of dY[i] h[i]^T over the
              rows of g; an adapter without rows has gradients of zeros.  h is an input,
              as the forward pass leaves it: the sum of two numbers of X's type, the
              second one what the first one's rounding lost;
* policy_grad  x = logits / temperature, lp = x_token - log sum_j e^x_j, entropy =
              -sum_j p_j log p_j, r = e^(lp - old), k = e^(ref - lp) - (ref - lp) - 1,
              loss = -min(r a, clip(r, 1 - lo, 1 + hi) a) + c_k k - c_e entropy, a the
              row's advantage, and the gradient of sum_i w_i loss_i for the logits; a
              row with token -1 has results and gradient 0;
* preference_grad  sequence s has the rows offsets[s] .. offsets[s + 1] - 1, reward_s =
              beta * sum (lp - ref) over its rows with a token; pair q is the sequences
              2q (preferred) and 2q + 1, m = reward_2q - reward_2q+1, loss_q =
              -(1 - e) log sigma(m) - e log sigma(-m), and the gradient of
              sum_q w_q loss_q for the logits.
"""
import functools
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one token of one request through a small layer: the weights are read once, latency counts
        dict(name="adapters one token", op="adapters", M=1, N=4096, K=4096, R=16, G=8, x="bf16", out="bf16",
             bias=False, runs=1),
        # a decoding batch through a wide layer, every request with an adapter of its own or none
        dict(name="adapters decode", op="adapters", M=16, N=8192, K=8192, R=16, G=16, x="bf16", out="bf16", bias=False,
             runs=16),
        # odd extents in every direction, fp32 output and a bias: a batch of draft tokens, a few to a request
        dict(name="adapters ragged", op="adapters", M=61, N=2055, K=1000, R=24, G=5, x="f16", out="f32", bias=True,
             runs=17),
        # prompts of different lengths, packed
        dict(name="adapters prompts", op="adapters", M=2048, N=4096, K=4096, R=32, G=8, x="bf16", out="bf16",
             bias=False, runs=11),
        # long prompts through a wide layer: compute-bound
        dict(name="adapters prefill", op="adapters", M=8192, N=8192, K=8192, R=64, G=4, x="bf16", out="bf16",
             bias=False, runs=5),
        # a small training step of three adapters at once, odd extents
        dict(name="adapters training ragged", op="adapters_grad", M=1000, N=2055, K=1000, R=8, G=3, x="f16", runs=7),
        # a training step of one adapter
        dict(name="adapters training", op="adapters_grad", M=4096, N=4096, K=4096, R=16, G=1, x="bf16", runs=1),
        # a small policy step, without entropy bonus
        dict(name="policy small", op="policy_grad", T=16, V=32768, x="f32", temperature=1.0, kl=0.05, bonus=0.0,
             prompt=0.0),
        # a policy step over an odd vocabulary without a reference model, prompts not scored
        dict(name="policy odd", op="policy_grad", T=2048, V=65537, x="bf16", temperature=1.0, kl=0.0, bonus=0.0, prompt=0.25),
        # a large step with KL term and entropy bonus
        dict(name="policy training", op="policy_grad", T=4096, V=131072, x="bf16", temperature=1.0, kl=0.05, bonus=0.01,
             prompt=0.0),
        # two short pairs
        dict(name="preference small", op="preference_grad", T=120, V=50001, P=2, x="f16", temperature=1.0,
             smoothing=0.0, prompt=0.25),
        # eight pairs of long answers, every row scored
        dict(name="preference training", op="preference_grad", T=4096, V=131072, P=8, x="bf16", temperature=1.0,
             smoothing=0.1, prompt=0.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["adapters", "adapters", "adapters_grad", "policy_grad", "preference_grad"])
    if op.startswith("adapters"):
        M, N, K = _log(rng, 1, 8192), _log(rng, 256, 8192), _log(rng, 256, 8192)
        if op == "adapters_grad":
            M = max(M, rng.randint(32, 128))       # a training step has more than a few tokens
        if rng.random() < 0.5:      # layer widths are mostly multiples of 64
            N, K = -(-N // 64) * 64, -(-K // 64) * 64
        R = rng.choice([4, 8, 16, 16, 24, 32, 64, 100, 128])
        case = dict(op=op, M=M, N=N, K=K, R=R, G=_log(rng, 1, 32), x=rng.choice(["f16", "bf16"]),
                    runs=min(M, _log(rng, 1, 64)))
        if op == "adapters":
            case.update(out=rng.choice(["f32", case["x"], case["x"]]), bias=rng.random() < 0.3)
        # the whole step's work stays below the largest listed one's
        while 2 * M * (N * K + 4 * R * (N + K)) > 1.1e12:
            M = case["M"] = M // 2
            case["runs"] = min(case["runs"], M)
        return case
    V = _log(rng, 8192, 262144)
    if rng.random() < 0.5:
        V = -(-V // 128) * 128
    x = rng.choice(["f32", "f16", "bf16"])
    T = _log(rng, 4, min(8192, (1 << 29) // V // (BYTES[x] // 2)))
    case = dict(op=op, T=T, V=V, x=x, temperature=rng.choice([0.7, 1.0, 1.0]), prompt=rng.choice([0.0, 0.25, 0.5]))
    if op == "policy_grad":
        case.update(kl=rng.choice([0.0, 0.05]), bonus=rng.choice([0.0, 0.0, 0.01]))
    else:
        case.update(P=_log(rng, 1, max(1, min(32, T // 4))), smoothing=rng.choice([0.0, 0.1]))
    return case


CLIP = (0.2, 0.28)
BETA = 0.1


def _lengths(total, parts, minimum):
    """`parts` lengths of at least `minimum` that add up to `total`, different ones."""
    rng = random.Random(total * 1009 + parts)
    cuts = sorted(rng.randint(0, total - parts * minimum) for _ in range(parts - 1))
    edges = [0] + cuts + [total - parts * minimum]
    return [b - a + minimum for a, b in zip(edges, edges[1:])]


def _scored(case):
    """Which rows have a token: all but the first part of each sequence."""
    if case["op"] == "preference_grad":
        lengths = _lengths(case["T"], 2 * case["P"], 2)
    else:
        lengths = _lengths(case["T"], max(1, case["T"] // 256), 1)
    rows = []
    for n in lengths:
        skip = min(n - 1, int(n * case["prompt"]))
        rows += [False] * skip + [True] * (n - skip)
    return rows, lengths


def _rows_of(case):
    """The run of rows of each request: lengths and adapters."""
    lengths = _lengths(case["M"], case["runs"], 1)
    rng = random.Random(case["M"] * 31 + case["G"])
    # a request in eight has no adapter
    return lengths, [-1 if case["G"] > 1 and rng.random() < 0.125 else rng.randrange(case["G"]) for _ in lengths]


def work(case):
    op = case["op"]
    if op.startswith("adapters"):
        M, N, K, R, G, e = case["M"], case["N"], case["K"], case["R"], case["G"], BYTES[case["x"]]
        lengths, which = _rows_of(case)
        rows = sum(n for n, g in zip(lengths, which) if g >= 0)
        present = len(set(which) - {-1})
        weights = present * R * (N + K) * e
        if op == "adapters":
            out = M * N * BYTES[case["out"]] + (4 * N if case["bias"] else 0)
            return {"bytes": (M * K + N * K) * e + weights + out, "flops": 2 * M * N * K + 2 * rows * R * (N + K)}
        return {"bytes": (M * N + N * K + 2 * M * K + 2 * M * R) * e + weights + G * R * (N + K) * e,
                "flops": 2 * M * N * K + 4 * rows * R * (N + K)}
    rows, _ = _scored(case)
    T, V, e = case["T"], case["V"], BYTES[case["x"]]
    return {"bytes": (sum(rows) + T) * V * e + T * 36, "flops": 8 * sum(rows) * V}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _up(n, q):
    return -(-n // q) * q


def _aligned(values):
    """The tensor with rows that start on whole 16-byte units (the row stride
    the package's tensor loads ask for)."""
    c, unit = values.shape[-1], 16 // values.element_size()
    if c % unit == 0:
        return values.contiguous()
    m = torch.zeros((*values.shape[:-1], _up(c, unit)), dtype=values.dtype, device=values.device)
    m[..., :c] = values
    return m[..., :c]


def _part(R):
    """Columns of each of the two parts of h."""
    return 16 if R <= 16 else 32 if R <= 32 else 64 if R <= 64 else 128


def _hidden(s, dtype):
    P, R = _part(s["R"]), s["R"]
    return s["hidden"][:, :R].to(dtype) + s["hidden"][:, P:P + R].to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = torch.device("cuda")
    s = dict(case)
    op = case["op"]
    if op.startswith("adapters"):
        M, N, K, R, G, dt = case["M"], case["N"], case["K"], case["R"], case["G"], DTYPES[case["x"]]

        def normal(*shape, size):
            return torch.randn(shape, generator=g, device=dev) * size

        # tokens of different sizes, a few large channels as activations have
        x = normal(M, K, size=1.0) * torch.exp(normal(M, 1, size=0.5))
        x[:, :: max(1, K // 7)] *= 4.0
        s["X"] = _aligned(x.to(dt))
        s["W"] = _aligned(normal(N, K, size=K ** -0.5).to(dt))
        s["down"] = _aligned(normal(G, R, K, size=K ** -0.5).to(dt))
        s["up"] = _aligned(normal(G, N, R, size=0.3 * R ** -0.5).to(dt))
        s["scale"] = torch.exp2(torch.randint(-1, 2, (G,), generator=g, device=dev).float())
        lengths, which = _rows_of(case)
        # which adapter a request has: another assignment of the same numbers for another seed
        turn = random.Random(seed).randrange(G)
        which = [-1 if a < 0 else (a + turn) % G for a in which]
        s["index"] = torch.repeat_interleave(torch.tensor(which, dtype=torch.int32), torch.tensor(lengths)).to(dev)
        if op == "adapters":
            s["bias_v"] = normal(N, size=1.0) if case["bias"] else None
            s["D"] = torch.empty((M, N), dtype=DTYPES[case["out"]], device=dev)
        else:
            s["dY"] = _aligned(normal(M, N, size=0.02).to(dt))
            s["dX"] = torch.empty((M, _up(K, 8)), dtype=dt, device=dev)[:, :K]
            # the forward pass of the same step left it
            h = _low_rank(s["X"].float(), s["down"], s["up"][:, :1], s["index"], s["scale"])[1]
            P = _part(R)
            s["hidden"] = torch.zeros((M, 2 * P), dtype=dt, device=dev)
            s["hidden"][:, :R] = h
            s["hidden"][:, P:P + R] = h - s["hidden"][:, :R].float()
        return s
    T, V = case["T"], case["V"]
    z = torch.randn((T, V), generator=g, device=dev) * 2.5
    tok = torch.randint(0, V, (T,), generator=g, device=dev)
    # the row's own token is a likely one
    z.scatter_(1, tok[:, None], 8.0 + 2.0 * torch.randn((T, 1), generator=g, device=dev))
    rows, lengths = _scored(case)
    s["logits"] = z.to(DTYPES[case["x"]])
    del z
    s["dlogits"] = torch.empty_like(s["logits"])
    # log-probabilities of the tokens: what the sampler and the reference model gave is near them
    lp = torch.empty((T,), dtype=torch.float64, device=dev)
    step = max(1, (1 << 27) // V)
    for r in range(0, T, step):
        x = s["logits"][r:r + step].double() / case["temperature"]
        lp[r:r + step] = torch.gather(x, 1, tok[r:r + step, None])[:, 0] - torch.logsumexp(x, dim=1)
    del x
    scored = torch.tensor(rows, device=dev)
    s["tokens"] = torch.where(scored, tok, torch.full_like(tok, -1))

    def near(size):
        return lp + torch.randn((T,), generator=g, device=dev).double() * size

    if op == "policy_grad":
        old = near(0.2)
        # (a ratio next to a border of the clipped range falls on either side of it with the last
        # bit of the log-probability: none here is within 0.1 % of one)
        for border in (math.log(1 - CLIP[0]), math.log(1 + CLIP[1])):
            close = (lp - old - border).abs() < 1e-3
            old = torch.where(close, old - 0.01, old)
        s["old"] = old.float()
        s["advantage"] = torch.randn((T,), generator=g, device=dev)
        s["ref"] = near(0.3).float() if case["kl"] else None
        s["w"] = torch.where(scored, 1.0 / sum(rows), 0.0).float()
    else:
        s["ref"] = near(0.3).float()
        s["offsets"] = torch.tensor([0] + lengths, device=dev).cumsum(0)
        s["w"] = torch.full((case["P"],), 1.0 / case["P"], device=dev)
    return s


# ---------------------------------------------------------------------------
# the package's calls
# ---------------------------------------------------------------------------
@functools.lru_cache(maxsize=None)
def _package(kind="bf16"):
    import tensor_core_dense_tma_gb300 as tc
    return tc, tc.Plan(kind)


def _run_own(s):
    op = s["op"]
    if op == "adapters":
        _, plan = _package(s["x"])
        return plan.linear_adapters(s["X"], s["W"].t(), s["down"], s["up"], s["index"], s["scale"], s["D"],
                                    bias=s["bias_v"])[0]
    if op == "adapters_grad":
        _, plan = _package(s["x"])
        r = plan.linear_adapters_grad(s["dY"], s["W"].t(), s["X"], s["hidden"], s["down"], s["up"], s["index"],
                                      s["scale"], s["dX"])
        return {"dX": r.dX, "d_down": r.d_down, "d_up": r.d_up}
    tc, _ = _package()
    if op == "policy_grad":
        r = tc.policy_loss_grad(s["logits"], s["tokens"], s["old"], s["advantage"], s["w"], s["ref"], clip=CLIP,
                                kl=s["kl"], entropy_bonus=s["bonus"], temperature=s["temperature"],
                                dlogits=s["dlogits"])
        return {"loss": r.loss, "logprob": r.logprob, "kl": r.kl, "entropy": r.entropy, "dlogits": r.dlogits}
    r = tc.preference_loss_grad(s["logits"], s["tokens"], s["offsets"], s["w"], s["ref"], beta=BETA,
                                smoothing=s["smoothing"], temperature=s["temperature"], dlogits=s["dlogits"])
    return {"loss": r.loss, "reward": r.reward, "logprob": r.logprob, "dlogits": r.dlogits}


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _low_rank(x, first, second, index, scale):
    """second[g] (first[g] x) scale[g] of every row of x, g = index (0 for -1),
    and the middle: one adapter after another over all rows, or, for few rows,
    each row with its own copy of its adapter."""
    G, R = first.shape[0], first.shape[1]
    if x.shape[0] * R * max(first.shape[2], second.shape[1]) <= 1 << 26:
        at = index.clamp(min=0).long()
        h = (first[at].float() * x[:, None, :]).sum(2) * scale[at][:, None]
        h = torch.where((index >= 0)[:, None], h, torch.zeros_like(h))
        return (second[at].float() * h[:, None, :]).sum(2), h
    y = torch.zeros((x.shape[0], second.shape[1]), device=x.device)
    h = torch.zeros((x.shape[0], R), device=x.device)
    for a in range(G):
        mine = torch.where((index == a)[:, None], (x @ first[a].float().t()) * scale[a], torch.zeros_like(h))
        y += mine @ second[a].float().t()
        h += mine
    return y, h


def _plain_adapters(s):
    x = s["X"].float()
    y = x @ s["W"].float().t() + _low_rank(x, s["down"], s["up"], s["index"], s["scale"])[0]
    if s["bias_v"] is not None:
        y = y + s["bias_v"]
    return y.to(s["D"].dtype)


def _plain_adapters_grad(s):
    x, dy, h = s["X"].float(), s["dY"].float(), _hidden(s, torch.float32)
    dx, p = _low_rank(dy, s["up"].transpose(1, 2), s["down"].transpose(1, 2), s["index"], s["scale"])
    dx += dy @ s["W"].float()
    d_down, d_up = [], []
    for a in range(s["G"]):
        mine = (s["index"] == a)[:, None]
        d_down.append(torch.where(mine, p, torch.zeros_like(p)).t() @ x)
        d_up.append(dy.t() @ torch.where(mine, h, torch.zeros_like(h)))
    dt = s["X"].dtype
    return {"dX": dx.to(dt), "d_down": torch.stack(d_down).to(dt), "d_up": torch.stack(d_up).to(dt)}


def _plain_rows(s):
    """x, log p, p of all rows, log p of the rows' tokens and where there is one."""
    x = s["logits"].float() / s["temperature"]
    m = x.amax(1, keepdim=True)
    logp = x - (m + torch.log(torch.exp(x - m).sum(1, keepdim=True)))
    given = s["tokens"] >= 0
    at = torch.gather(logp, 1, s["tokens"].clamp(min=0)[:, None])[:, 0]
    return logp, torch.exp(logp), torch.where(given, at, torch.zeros_like(at)), given


def _plain_policy(s):
    logp, p, lp, given = _plain_rows(s)
    zero = torch.zeros_like(lp)
    ent = torch.where(given, -(p * logp).sum(1), zero)
    a, r = s["advantage"], torch.exp(lp - s["old"])
    clipped = r.clamp(1 - CLIP[0], 1 + CLIP[1])
    loss = -torch.minimum(r * a, clipped * a)
    slope = torch.where(r * a <= clipped * a, -r * a, zero)
    k = zero
    if s["ref"] is not None:
        d = s["ref"] - lp
        k = torch.exp(d) - d - 1
        loss = loss + s["kl"] * k
        slope = slope + s["kl"] * (1 - torch.exp(d))
    loss = torch.where(given, loss - s["bonus"] * ent, zero)
    k = torch.where(given, k, zero)
    w = torch.where(given, s["w"], zero)[:, None]
    dz = s["bonus"] * w * p * (logp + ent[:, None]) - w * slope[:, None] * p
    dz.scatter_add_(1, s["tokens"].clamp(min=0)[:, None], w * slope[:, None])
    return {"loss": loss, "logprob": lp, "kl": k, "entropy": ent,
            "dlogits": (dz / s["temperature"]).to(s["logits"].dtype)}


def _plain_preference(s):
    _, p, lp, given = _plain_rows(s)
    # long sums in 64 bits
    diff = torch.where(given, lp.double() - s["ref"].double(), torch.zeros_like(lp, dtype=torch.float64))
    total = torch.cat([torch.zeros_like(diff[:1]), diff.cumsum(0)])
    o = s["offsets"]
    reward = BETA * (total[o[1:]] - total[o[:-1]])
    m = reward[0::2] - reward[1::2]
    e = s["smoothing"]
    loss = (1 - e) * torch.log1p(torch.exp(-m)) + e * torch.log1p(torch.exp(m))
    slope = (e / (1 + torch.exp(-m)) - (1 - e) / (1 + torch.exp(m))) * s["w"] * BETA
    row = torch.bucketize(torch.arange(s["T"], device=o.device), o, right=True) - 1
    g = torch.where(given, torch.stack([slope, -slope], 1).reshape(-1)[row], torch.zeros_like(diff)).float()[:, None]
    dz = -g * p
    dz.scatter_add_(1, s["tokens"].clamp(min=0)[:, None], g)
    return {"loss": loss.float(), "reward": reward.float(), "logprob": lp,
            "dlogits": (dz / s["temperature"]).to(s["logits"].dtype)}


def run(state):
    if own:
        return _run_own(state)
    return {"adapters": _plain_adapters, "adapters_grad": _plain_adapters_grad, "policy_grad": _plain_policy,
            "preference_grad": _plain_preference}[state["op"]](state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_adapters(s):
    X, W, index = s["X"].double(), s["W"].double(), s["index"]
    backward = s["op"] == "adapters_grad"
    if backward:
        dY = s["dY"].double()
        out, d_down, d_up = torch.matmul(dY, W), [], []
    else:
        out = torch.matmul(X, W.t())
        if s["bias_v"] is not None:
            out += s["bias_v"].double()
    for a in range(s["G"]):
        rows = torch.nonzero(index == a)[:, 0]
        A, U = s["down"][a].double(), s["up"][a].double() * s["scale"][a].double()
        if not backward:
            out[rows] += X[rows] @ A.t() @ U.t()
            continue
        dh = dY[rows] @ U
        out[rows] += dh @ A
        d_down.append(dh.t() @ X[rows])
        d_up.append(dY[rows].t() @ _hidden(s, torch.float64)[rows])
    return {"dX": out, "d_down": torch.stack(d_down), "d_up": torch.stack(d_up)} if backward else out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("adapters"):
        return _exact_adapters(s)
    T, V, t = case["T"], case["V"], case["temperature"]
    step = max(1, (1 << 27) // V)
    use = (s["tokens"] >= 0).double()
    at = s["tokens"].clamp(min=0)

    def rows():
        for r in range(0, T, step):
            yield slice(r, r + step), torch.log_softmax(s["logits"][r:r + step].double() / t, dim=1)

    lp, ent = torch.zeros_like(use), torch.zeros_like(use)
    for part, logp in rows():
        lp[part] = logp[torch.arange(logp.shape[0], device=logp.device), at[part]] * use[part]
        ent[part] = torch.special.entr(torch.exp(logp)).sum(1) * use[part]
    if op == "policy_grad":
        r, a = torch.exp(lp - s["old"].double()), s["advantage"].double()
        bounded = torch.clamp(r, 1 - CLIP[0], 1 + CLIP[1])
        inside = ~(((a > 0) & (r > 1 + CLIP[1])) | ((a < 0) & (r < 1 - CLIP[0])))
        loss = torch.where(inside, -r * a, -bounded * a)
        slope = -r * a * inside
        kl = torch.zeros_like(lp)
        if s["ref"] is not None:
            d = (s["ref"].double() - lp) * use
            kl = torch.expm1(d) - d
            loss, slope = loss + case["kl"] * kl, slope - case["kl"] * torch.expm1(d)
        h = case["bonus"] * s["w"].double() * use
        g = slope * s["w"].double() * use
        got = {"loss": (loss - case["bonus"] * ent) * use, "logprob": lp, "kl": kl * use, "entropy": ent}
    else:
        o = s["offsets"].tolist()
        d = (lp - s["ref"].double()) * use
        reward = BETA * torch.stack([d[i:j].sum() for i, j in zip(o, o[1:])])
        m = reward[0::2] - reward[1::2]
        e = case["smoothing"]
        soft = torch.nn.functional.softplus
        slope = (e * torch.sigmoid(m) - (1 - e) * torch.sigmoid(-m)) * s["w"].double() * BETA
        g = torch.zeros_like(lp)
        for q in range(case["P"]):
            g[o[2 * q]:o[2 * q + 1]] = slope[q]
            g[o[2 * q + 1]:o[2 * q + 2]] = -slope[q]
        g, h = g * use, torch.zeros_like(g)
        got = {"loss": (1 - e) * soft(-m) + e * soft(m), "reward": reward, "logprob": lp}
    parts = []
    for part, logp in rows():
        p = torch.exp(logp)
        dz = p * (h[part, None] * (logp + ent[part, None]) - g[part, None])
        dz[torch.arange(p.shape[0], device=p.device), at[part]] += g[part]
        parts.append(dz / t)
    got["dlogits"] = torch.cat(parts)
    return got
