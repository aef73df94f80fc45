"""Adapters of many requests beside a shared product (include/adapters.h)
against a plain implementation in 64 bits, row by row from the definitions.

Tolerances.  A sum of K products in fp32, 16 at a step of the tensor cores (which
may truncate) or one by one in at least 32 lanes, then joined over at most 32
ranges, is off by at most a(K) = 2^-23 (K / 16 + 32) of the sum of the magnitudes.
h is off by a(K) of its own sum, and its two parts lose u^2 of it, u half a unit
of the plan's type relative (and 2^-25 for fp16, whose low part may be subnormal).
So D is off by a(K + 2 R) (|X| |W| + |bias| + |U| |h|) + |U| e_h, and by its own
rounding.  A gradient of a factor sums over the M rows: a(2 M) of its sum of
magnitudes plus |left| e_right.  Whole numbers small enough for every sum to be
exact are compared bit for bit.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_ULP = {k: torch.finfo(v).eps / 2 for k, v in TYPES.items()}      # of the rounding to the type, relative
SMALLEST = {"f32": 1e-37, "f16": 2.0 ** -25, "bf16": 1e-37}
F64 = torch.float64


@pytest.fixture(scope="module")
def tc():
    from tensor_core_dense_tma_gb300 import build as tcbuild
    tcbuild.build()
    import tensor_core_dense_tma_gb300 as tc
    return tc


@pytest.fixture(scope="module")
def plans(tc):
    p = {k: tc.Plan(k, 0) for k in ("f16", "bf16")}
    yield p
    torch.cuda.synchronize()
    for x in p.values():
        assert x.device_status() == 0
        x.close()


def acc(n):
    return 2.0 ** -23 * (n / 16 + 32)


def padded(values, kind, pad=8, swap=False):
    """A device tensor of the values with rows on 16-byte boundaries and NaN
    beside them; with swap the last two dimensions are stored the other way round."""
    v = values.transpose(-1, -2) if swap else values
    c = v.shape[-1]
    buf = torch.full((*v.shape[:-1], -(-max(c, 1) // 8) * 8 + pad), float("nan"), dtype=TYPES[kind], device="cuda")
    buf[..., :c] = v.to(TYPES[kind])
    view = buf[..., :c]
    return view.transpose(-1, -2) if swap else view


class Case:
    """Inputs in the plan's type and their values in 64 bits."""

    def __init__(self, M, N, K, R, G, kind, seed=0, index="runs", whole=False, w_row=False, down_col=False, up_col=False,
                 scale=True, bias=False, runs=5):
        g = torch.Generator(device="cuda").manual_seed(seed * 1000 + M + N + K + R)
        self.M, self.N, self.K, self.R, self.G, self.kind = M, N, K, R, G, kind

        def draw(*shape, size, top):
            if whole:
                return torch.randint(-top, top + 1, shape, generator=g, device="cuda").double()
            return torch.randn(shape, generator=g, device="cuda").double() * size

        self.X = padded(draw(M, K, size=1.0, top=2), kind)
        self.B = padded(draw(K, N, size=K ** -0.5, top=2), kind, swap=not w_row)
        self.down = padded(draw(G, R, K, size=K ** -0.5, top=1), kind, swap=down_col)
        self.up = padded(draw(G, N, R, size=0.5 * R ** -0.5, top=2), kind, swap=up_col)
        self.dY = padded(draw(M, N, size=0.1, top=1), kind)
        self.scale = torch.exp2(torch.randint(-1, 2, (G,), generator=g, device="cuda").float()) if scale else None
        if whole and scale:
            self.scale = self.scale.clamp(min=1)
        self.bias = draw(N, size=1.0, top=5).float() if bias else None
        rng = np.random.default_rng(seed + M)
        if index == "runs":
            cuts = np.sort(rng.integers(0, M + 1, runs))
            i = rng.integers(-1, G, runs + 1)[np.searchsorted(cuts, np.arange(M), side="right")]
        elif index == "mixed":
            i = rng.integers(-1, G, M)
        elif index == "none":
            i = rng.choice([-1, -7, G, 1 << 30, -(1 << 31)], M)
        elif index == "one":
            i = np.full(M, G - 1)
        elif index == "odd":
            i = np.where(rng.random(M) < 0.5, rng.choice([-1, -(1 << 31), G, (1 << 31) - 1], M), rng.integers(0, max(G, 1), M))
        self.index = torch.from_numpy(np.asarray(i).astype(np.int32)).cuda()

    def args(self):
        return self.B, self.down, self.up, self.index, self.scale

    def product(self, x, w, first, second, bias=None):
        """(out, size, h, e_h): x w + the rows' adapters, the sum of its magnitudes, the middle and its error."""
        x, w, first, second = x.to(F64), w.to(F64), first.to(F64), second.to(F64)
        out, size = x @ w, x.abs() @ w.abs()
        if bias is not None:
            out, size = out + bias.double(), size + bias.double().abs()
        h = torch.zeros((self.M, self.R), dtype=F64, device="cuda")
        e = torch.zeros_like(h)
        u = HALF_ULP[self.kind]
        n = x.shape[1]
        extra = torch.zeros_like(out)
        for a in range(self.G):
            rows = torch.nonzero(self.index == a)[:, 0]
            if len(rows) == 0:
                continue
            s = self.scale[a].double() if self.scale is not None else 1.0
            h[rows] = s * (x[rows] @ first[a].t())
            e[rows] = (s * (x[rows].abs() @ first[a].t().abs()) * acc(n) + h[rows].abs() * (u * u + 2.0 ** -23)
                       + (2.0 ** -24 if self.kind == "f16" else 0))
            out[rows] += h[rows] @ second[a].t()
            size[rows] += h[rows].abs() @ second[a].t().abs()
            extra[rows] = e[rows] @ second[a].t().abs()
        return out, size * acc(n + 2 * self.R) + extra, h, e

    def factor(self, left, e_left, right):
        """sum over each adapter's rows of left^T right and its error."""
        right = right.to(F64)
        out, tol = [], []
        for a in range(self.G):
            rows = torch.nonzero(self.index == a)[:, 0]
            l, r = left[rows], right[rows]
            out.append(l.t() @ r)
            tol.append(acc(2 * self.M) * (l.abs().t() @ r.abs()) + e_left[rows].t() @ r.abs())
        return torch.stack(out), torch.stack(tol)


def near(got, want, tol, kind, what):
    got = got.to(F64)
    tol = tol * (1 + HALF_ULP[kind]) + HALF_ULP[kind] * want.abs() + SMALLEST[kind]
    bad = ~((got - want).abs() <= tol)
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()}, first at {torch.nonzero(bad)[0].tolist()}: "
                                 f"{got[bad][0].item()!r}, want {want[bad][0].item()!r} +- {tol[bad][0].item():.3g}")


def hidden_value(hidden, R):
    P = hidden.shape[1] // 2
    assert not hidden[:, R:P].any() and not hidden[:, P + R:].any()
    return hidden[:, :R].double() + hidden[:, P:P + R].double()


def check_forward(plan, c, out=None, whole=False):
    want, tol, h, e = c.product(c.X, c.B, c.down, c.up, c.bias)
    D, hidden = plan.linear_adapters(c.X, *c.args(), bias=c.bias, out_dtype=out)
    torch.cuda.synchronize()
    out = out or c.kind
    if whole:
        assert torch.equal(hidden_value(hidden, c.R), h)
        assert torch.equal(D, want.to(TYPES[out]))
    else:
        near(hidden_value(hidden, c.R), h, e, "f32", "hidden")
        near(D, want, tol, out, "D")
    return D, hidden, h, e


def check_backward(plan, c, whole=False, out=None):
    _, hidden, h, e_h = check_forward(plan, c, whole=whole)
    kw = {}
    if out == "f32":
        kw = dict(d_down=torch.full((c.G, c.R, c.K), 7.0, device="cuda"), d_up=torch.full((c.G, c.N, c.R), 7.0, device="cuda"))
    r = plan.linear_adapters_grad(c.dY, c.B, c.X, hidden, c.down, c.up, c.index, c.scale, **kw)
    torch.cuda.synchronize()
    dX, t_x, p, e_p = c.product(c.dY, c.B.t(), c.up.transpose(1, 2), c.down.transpose(1, 2))
    d_down, t_down = c.factor(p, e_p, c.X)
    # h is given as its two parts: an input of this call
    d_up, t_up = c.factor(hidden_value(hidden, c.R), torch.zeros_like(h), c.dY)
    d_up, t_up = d_up.transpose(1, 2), t_up.transpose(1, 2)
    out = out or c.kind
    if whole:
        assert torch.equal(r.dX, dX.to(TYPES[c.kind]))
        assert torch.equal(r.d_down, d_down.to(TYPES[out])) and torch.equal(r.d_up, d_up.to(TYPES[out]))
        return
    near(r.dX, dX, t_x, c.kind, "dX")
    near(r.d_down, d_down, t_down, out, "d_down")
    near(r.d_up, d_up, t_up, out, "d_up")


SHAPES = [(1, 1, 1, 1, 1), (1, 300, 1000, 16, 3), (2, 129, 64, 4, 2), (5, 2055, 333, 24, 7), (16, 640, 520, 16, 16),
          (17, 257, 2048, 33, 4), (33, 8, 8, 128, 2), (61, 2055, 1000, 24, 5), (64, 72, 1040, 64, 3), (65, 300, 512, 8, 3),
          (100, 1, 200, 100, 2), (127, 511, 100, 17, 130), (129, 264, 640, 64, 3), (200, 255, 255, 1, 2),
          (256, 256, 256, 16, 1), (300, 520, 1000, 128, 4), (513, 1030, 77, 32, 9), (1024, 1000, 333, 48, 3),
          (1500, 640, 2055, 16, 2), (2300, 2290, 800, 65, 4)]


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(plans, kind, shape):
    check_forward(plans[kind], Case(*shape, kind))


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("index", ["runs", "mixed", "odd"])
def test_forward_whole_numbers(plans, shape, index):
    for kind, out in (("f16", "f32"), ("bf16", "bf16"), ("f16", "bf16"), ("bf16", "f32")):
        check_forward(plans[kind], Case(*shape, kind, seed=1, index=index, whole=True, bias=True), out, whole=True)


@pytest.mark.parametrize("w_row", [False, True])
@pytest.mark.parametrize("down_col", [False, True])
@pytest.mark.parametrize("up_col", [False, True])
@pytest.mark.parametrize("M,N,K,R,G", [(3, 520, 264, 24, 4), (40, 130, 136, 128, 3), (300, 520, 1000, 16, 4),
                                       (700, 1030, 200, 40, 3), (260, 300, 129, 100, 6)])
def test_layouts(plans, M, N, K, R, G, w_row, down_col, up_col):
    c = Case(M, N, K, R, G, "bf16", seed=2, index="mixed", whole=True, w_row=w_row, down_col=down_col, up_col=up_col,
             scale=False)
    check_forward(plans["bf16"], c, "f32", whole=True)


@pytest.mark.parametrize("index", ["none", "one", "mixed"])
@pytest.mark.parametrize("M", [7, 64, 130, 600])
def test_indices(plans, M, index):
    c = Case(M, 300, 264, 16, 40, "bf16", seed=3, index=index, bias=True)
    check_forward(plans["bf16"], c, "f32")


def test_many_adapters(plans):
    """Every row of a tile its own, in an order of no pattern."""
    for M in (64, 128, 300, 515):
        c = Case(M, 136, 200, 16, 600, "f16", seed=4, index="mixed", whole=True)
        c.index = torch.randperm(600, device="cuda")[:M].int()
        check_forward(plans["f16"], c, "f32", whole=True)


def test_no_adapters(plans):
    for M in (5, 200):
        c = Case(M, 136, 200, 16, 1, "bf16", seed=4, whole=True)
        c.down, c.up, c.scale, c.G = c.down[:0], c.up[:0], None, 0
        check_forward(plans["bf16"], c, "f32", whole=True)
        r = plans["bf16"].linear_adapters_grad(c.dY, c.B, c.X, None, c.down, c.up, c.index)
        assert r.d_down.shape == (0, 16, 200) and torch.equal(r.dX, (c.dY.double() @ c.B.t().double()).bfloat16())


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("shape", [s for s in SHAPES if s[0] > 1], ids=str)
def test_backward(plans, kind, shape):
    check_backward(plans[kind], Case(*shape, kind, seed=5), out="f32" if kind == "f16" else None)


@pytest.mark.parametrize("index", ["runs", "mixed", "odd", "one", "none"])
@pytest.mark.parametrize("shape", [(5, 140, 72, 24, 3), (130, 260, 300, 8, 3), (600, 520, 264, 64, 5), (1100, 129, 520, 100, 2),
                                   (777, 72, 1030, 16, 70)], ids=str)
def test_backward_whole_numbers(plans, shape, index):
    for kind in ("f16", "bf16"):
        c = Case(*shape, kind, seed=6, index=index, whole=True)
        check_backward(plans[kind], c, whole=True, out="f32")


def test_other_rows_do_not_matter(plans):
    """NaN and infinities in other rows, other adapters and beside the matrices."""
    for M in (6, 64, 200, 600):
        c = Case(M, 300, 264, 24, 6, "bf16", seed=7, index="mixed")
        plan = plans["bf16"]
        D, hidden = plan.linear_adapters(c.X, *c.args())
        g = plan.linear_adapters_grad(c.dY, c.B, c.X, hidden, c.down, c.up, c.index, c.scale)
        X, dY, down, up = c.X.clone(), c.dY.clone(), c.down.clone(), c.up.clone()
        down[1], up[2], down[4, :, ::3], up[4, 5] = float("nan"), float("inf"), float("inf"), float("nan")
        X[c.index == 3] = float("inf")
        dY[c.index == 3] = float("nan")
        X[(c.index == 1) | (c.index == 4)] = float("nan")
        X, dY, down, up = (padded(t.double(), "bf16") for t in (X, dY, down, up))
        D2, hidden2 = plan.linear_adapters(X, c.B, down, up, c.index, c.scale)
        same = (c.index == 0) | (c.index == 5) | (c.index == -1)
        assert torch.equal(D2[same], D[same]) and torch.equal(hidden2[same], hidden[same])
        assert torch.equal(hidden2[c.index == 2], hidden[c.index == 2])
        assert not torch.isfinite(D2[c.index == 2]).any() and torch.isnan(D2[c.index == 1]).all()
        g2 = plan.linear_adapters_grad(dY, c.B, X, hidden2, down, up, c.index, c.scale)
        assert torch.equal(g2.dX[same], g.dX[same])
        for a in (0, 5):
            assert torch.equal(g2.d_down[a], g.d_down[a]) and torch.equal(g2.d_up[a], g.d_up[a])
        assert torch.equal(g2.d_up[2], g.d_up[2])
        assert torch.isnan(g2.d_up[3]).all() or not bool((c.index == 3).any())


def test_infinite_hidden(plans):
    """A hidden value beyond the type's range is an infinity, not a NaN."""
    for M in (3, 200):
        X = torch.full((M, 64), 60000.0, dtype=torch.float16, device="cuda")
        down = torch.ones((1, 8, 64), dtype=torch.float16, device="cuda")
        up = torch.ones((1, 40, 8), dtype=torch.float16, device="cuda")
        B = torch.zeros((40, 64), dtype=torch.float16, device="cuda").t()
        D, hidden = plans["f16"].linear_adapters(X, B, down, up, torch.zeros(M, dtype=torch.int32, device="cuda"))
        assert torch.isposinf(D).all() and torch.isposinf(hidden[:, :8]).all() and not hidden[:, 8:].any()


def test_differences(plans):
    """The gradients against differences of the 64-bit definition."""
    c = Case(9, 16, 24, 4, 3, "f16", seed=8, index="mixed")
    _, hidden, _, _ = check_forward(plans["f16"], c)
    kw = dict(d_down=torch.empty((3, 4, 24), device="cuda"), d_up=torch.empty((3, 16, 4), device="cuda"))
    r = plans["f16"].linear_adapters_grad(c.dY, c.B, c.X, hidden, c.down, c.up, c.index, c.scale, **kw)
    for name, got in (("X", r.dX), ("down", r.d_down), ("up", r.d_up)):
        v = getattr(c, name).to(F64).contiguous().clone()
        flat, keep, num = v.view(-1), getattr(c, name), torch.zeros(v.numel(), dtype=F64, device="cuda")
        for j in range(0, v.numel(), 5):
            f = []
            for e in (0.5, -0.5):      # the sum is linear in each element: differences are exact
                flat[j] += e
                setattr(c, name, v)
                f.append((c.dY.to(F64) * c.product(c.X, c.B, c.down, c.up)[0]).sum())
                flat[j] -= e
            setattr(c, name, keep)
            num[j] = f[0] - f[1]
        at = torch.arange(0, v.numel(), 5, device="cuda")
        g = got.to(F64).reshape(-1)[at]
        # fp32 sums of a few tens of terms of size one, and the rounding of dX
        assert ((g - num[at]).abs() <= 2e-5 + HALF_ULP["f16"] * num[at].abs() * (name == "X")).all(), name


def test_given_outputs(plans):
    """Outputs with their own strides; nothing beside them is written."""
    plan = plans["bf16"]
    for M in (9, 300):
        c = Case(M, 133, 72, 24, 3, "bf16", seed=9, bias=True)
        D, hidden = plan.linear_adapters(c.X, *c.args(), bias=c.bias)
        Db = torch.full((M, 141), 7.0, dtype=torch.bfloat16, device="cuda")
        Hb = torch.full((M, 72), 7.0, dtype=torch.bfloat16, device="cuda")
        D2, H2 = plan.linear_adapters(c.X, *c.args(), Db[:, 3:136], bias=c.bias, hidden=Hb[:, :64])
        assert torch.equal(D2, D) and torch.equal(H2, hidden)
        assert bool((Db[:, :3] == 7).all()) and bool((Db[:, 136:] == 7).all()) and bool((Hb[:, 64:] == 7).all())
        g = plan.linear_adapters_grad(c.dY, c.B, c.X, hidden, c.down, c.up, c.index, c.scale)
        a = torch.full((4, 25, 75), 7.0, dtype=torch.bfloat16, device="cuda")
        b = torch.full((4, 134, 29), 7.0, dtype=torch.bfloat16, device="cuda")
        g2 = plan.linear_adapters_grad(c.dY, c.B, c.X, H2, c.down, c.up, c.index, c.scale, d_down=a[:3, :24, 1:73],
                                       d_up=b[:3, :133, 3:27])
        assert all(torch.equal(x, y) for x, y in zip(g, g2))
        a[:3, :24, 1:73] = 7
        b[:3, :133, 3:27] = 7
        assert bool((a == 7).all()) and bool((b == 7).all())


def test_streams_and_graphs(tc):
    """On a stream of its own and from graphs replayed together, a plan each: the same bits."""
    for M in (4, 40, 700):
        c = Case(M, 520, 264, 16, 5, "bf16", seed=10, index="mixed")

        def calls(plan):
            D, hidden = plan.linear_adapters(c.X, *c.args())
            return (D, hidden, *plan.linear_adapters_grad(c.dY, c.B, c.X, hidden, c.down, c.up, c.index, c.scale))

        p, q = tc.Plan("bf16", 0), tc.Plan("bf16", 0)
        want = [t.clone() for t in calls(p)]
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            got = calls(p)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        graphs = []
        for plan in (p, q):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                r = calls(plan)
            graphs.append((g, r, torch.cuda.Stream()))
        for _ in range(4):
            for g, _, s in graphs:
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for _, r, _ in graphs:
            assert all(torch.equal(a, b) for a, b in zip(r, want))
        assert p.device_status() == 0 and q.device_status() == 0
        p.close(), q.close()


def test_graph_after_other_work(plans):
    """A call captured behind a memset, a copy and kernels that make its inputs."""
    plan = plans["bf16"]
    for M in (9, 300):
        c = Case(M, 264, 520, 16, 3, "bf16", seed=11, index="mixed")
        src = c.X.clone()
        X, index = torch.empty((M, 520), dtype=torch.bfloat16, device="cuda"), c.index.clone()
        args = (c.B, c.down, c.up, index, c.scale)
        want = plan.linear_adapters(2 * src, *args)
        g, D = torch.cuda.CUDAGraph(), torch.empty((M, 264), dtype=torch.bfloat16, device="cuda")
        side = torch.zeros(1 << 20, device="cuda")
        with torch.cuda.graph(g):
            X.copy_(src)
            side.zero_()
            plan.linear_adapters(X, *args, D)
            X.copy_(src)
            X.mul_(2)
            D2, h2 = plan.linear_adapters(X, *args)
            X.zero_()
            side.zero_()
            D3, _ = plan.linear_adapters(X, *args)
        for _ in range(3):
            X.fill_(float("nan"))
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(D2, want[0]) and torch.equal(h2, want[1]) and not D3.any()
            assert torch.equal(D, plan.linear_adapters(src.contiguous(), *args)[0])


def test_pinned_and_tuned_configurations(tc):
    """A plan that is pinned to a configuration or division, or tuned, computes the same."""
    c = Case(700, 1030, 1000, 24, 5, "bf16", seed=12, index="mixed", whole=True, bias=True)
    few = Case(40, 1030, 1000, 24, 5, "bf16", seed=12, index="mixed", whole=True)
    with tc.Plan("bf16", 0) as plan:
        for config in ("single_128x256", "pair_256x256", "pair_256x224"):
            plan.force_config(config)
            check_forward(plan, c, whole=True)
            plan.force_config(config, 3)
            check_forward(plan, c, whole=True)
        plan.force_config("auto")
        plan.force_division("halves")
        check_forward(plan, c, whole=True)
        plan.force_division("auto")
        plan.autotune(c.X, c.B, out_dtype="bf16")
        check_forward(plan, c, whole=True)
        plan.clear_tuning()
        one = Case(11, 1030, 1000, 24, 5, "bf16", seed=12, index="mixed", whole=True)
        for config, x in (("single_128x64", few), ("single_128x64", one), ("single_128x16", one)):
            for splits in (0, 1, 2, 3):
                plan.force_config(config, splits)
                check_forward(plan, x, whole=True)
        plan.force_config("auto")
        for division in ("whole", "split", "pair_split", "halves"):
            plan.force_division(division)
            if division != "halves":
                check_forward(plan, one, whole=True)
            check_forward(plan, few, whole=True)
        torch.cuda.synchronize()
        assert plan.device_status() == 0


@pytest.mark.parametrize("division", ["early_split", "stream_k"])
def test_captured_early_partials(tc, division):
    """Divisions whose units leave partial sums for one another, captured: each replay uses its own."""
    c = Case(5200, 3840 if division == "early_split" else 5120, 520, 16, 5, "bf16", seed=13, index="runs", whole=True)
    with tc.Plan("bf16", 0) as plan:
        plan.force_division(division)
        want = check_forward(plan, c, whole=True)[0].clone()
        g, X, D = torch.cuda.CUDAGraph(), c.X.clone(), torch.empty_like(want)
        # (the stride of the clone's rows is the columns': whole 16-byte units here)
        with torch.cuda.graph(g):
            plan.linear_adapters(X, *c.args(), D)
        other = torch.randint(-2, 3, X.shape, device="cuda").to(X.dtype)
        for _ in range(3):
            X.copy_(other)
            g.replay()
            X.copy_(c.X)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(D, want)
        assert plan.device_status() == 0


def test_long_index(plans):
    """More rows than one look at the index takes (65536)."""
    c = Case(70001, 8, 24, 4, 3, "f16", seed=14, index="runs", whole=True, runs=9)
    check_backward(plans["f16"], c, whole=True, out="f32")


def test_unaligned_index(plans):
    """An index that starts anywhere on 4 bytes."""
    c = Case(700, 136, 264, 16, 3, "bf16", seed=15, index="runs", whole=True)
    for shift in (1, 2, 3):
        buf = torch.full((704 + shift,), 2, dtype=torch.int32, device="cuda")
        buf[shift:shift + 700] = c.index
        c.index = buf[shift:shift + 700]
        check_backward(plans["bf16"], c, whole=True, out="f32")


def test_offsets_past_32_bits(plans):
    """Factors, rows and gradients more than 2^31 elements apart."""
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of device memory")
    far = (1 << 31) + 64
    bufs = [torch.empty((2 * far + 4096,), dtype=torch.bfloat16, device="cuda") for _ in range(2)]

    def spread(t, buf, stride):
        v = torch.as_strided(buf, t.shape, stride, 8)
        v.copy_(t)
        return v

    c = Case(200, 136, 264, 16, 2, "bf16", seed=16, index="mixed", whole=True)
    c.down = spread(c.down, bufs[0], (far, 264, 1))
    c.up = spread(c.up, bufs[1], (far, 16, 1))
    check_forward(plans["bf16"], c, "f32", whole=True)
    check_backward(plans["bf16"], c, whole=True, out="f32")
    few = Case(3, 136, 264, 16, 2, "bf16", seed=16, index="mixed", whole=True)
    few.down, few.up = c.down, c.up
    check_forward(plans["bf16"], few, "f32", whole=True)
    # rows of X, of hidden, of D and of a gradient far apart
    near_X, few.down, few.up = few.X[:2].clone(), c.down.clone(), c.up.clone()
    few.M, few.X, few.index, few.dY = 2, spread(near_X, bufs[0], (far, 1)), few.index[:2].contiguous(), few.dY[:2]
    D = torch.as_strided(bufs[1], (2, 136), (far, 1), 1)
    hidden = torch.as_strided(bufs[1], (2, 32), (far, 1), 1024)
    want = plans["bf16"].linear_adapters(padded(near_X.double(), "bf16"), *few.args())
    got = plans["bf16"].linear_adapters(few.X, *few.args(), D, hidden=hidden)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    a = plans["bf16"].linear_adapters_grad(few.dY, few.B, few.X, hidden, few.down, few.up, few.index, few.scale)
    d_down = torch.as_strided(bufs[1], (2, 16, 264), (far, 264, 1), 2048)
    b = plans["bf16"].linear_adapters_grad(few.dY, few.B, few.X, hidden, few.down, few.up, few.index, few.scale, d_down=d_down)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_given_stream(plans):
    """`stream` another than the current one, which takes what memory it can get
    meanwhile: the call's own buffer is not among it."""
    plan = plans["bf16"]
    c = Case(300, 264, 520, 16, 3, "bf16", seed=18, index="mixed")
    _, hidden = plan.linear_adapters(c.X, *c.args())
    args = (c.dY, c.B, c.X, hidden, c.down, c.up, c.index, c.scale)
    want = plan.linear_adapters_grad(*args)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)
        got = plan.linear_adapters_grad(*args, stream=s.cuda_stream)
        for _ in range(8):
            torch.full((300, 32), float("nan"), dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_two_at_once(tc):
    """Two plans on two streams at the same time, time and again: the same bits as alone."""
    cases = [Case(M, 1032, 2056, 16, 7, "bf16", seed=17, index="mixed") for M in (33, 900)]
    ps = [tc.Plan("bf16", 0) for _ in cases]

    def calls(p, c):
        D, hidden = p.linear_adapters(c.X, *c.args())
        return (D, hidden, *p.linear_adapters_grad(c.dY, c.B, c.X, hidden, c.down, c.up, c.index, c.scale))

    want = [calls(p, c) for p, c in zip(ps, cases)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    for _ in range(5):
        got = []
        for p, c, s in zip(ps, cases, streams):
            with torch.cuda.stream(s):
                for _ in range(4):
                    r = calls(p, c)
                got.append(r)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for a, b in zip(got, want) for x, y in zip(a, b))
    for p in ps:
        assert p.device_status() == 0
        p.close()


def test_empty(plans):
    plan = plans["bf16"]
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")      # noqa: E731
    i = torch.zeros(0, dtype=torch.int32, device="cuda")
    D, h = plan.linear_adapters(z(0, 64), z(64, 32), z(2, 8, 64), z(2, 32, 8), i)
    assert D.shape == (0, 32) and h.shape == (0, 32)
    g = plan.linear_adapters_grad(z(0, 32), z(64, 32), z(0, 64), h, z(2, 8, 64), z(2, 32, 8), i)
    assert not g.d_down.any() and not g.d_up.any() and g.d_up.shape == (2, 32, 8)
    i = torch.zeros(5, dtype=torch.int32, device="cuda")
    bias = torch.arange(32, device="cuda").float()
    D, h = plan.linear_adapters(z(5, 0), z(0, 32), z(2, 8, 0), z(2, 32, 8), i, bias=bias)
    assert torch.equal(D, bias.bfloat16().expand(5, 32)) and not h.any()
    D, h = plan.linear_adapters(z(5, 64) + 1, z(64, 0), z(2, 8, 64) + 1, z(2, 0, 8), i)
    assert D.shape == (5, 0) and bool((h[:, :8] == 64).all())


def test_refusals(tc, plans):
    plan = plans["bf16"]
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")      # noqa: E731
    i = torch.zeros(4, dtype=torch.int32, device="cuda")
    ok = dict(X=z(4, 64), B=z(64, 32), down=z(2, 8, 64), up=z(2, 32, 8), index=i, scale=None)
    f = torch.ones(2, device="cuda")
    for kw in (dict(X=z(4, 64).half()), dict(X=z(4, 64).cpu()), dict(X=z(64, 4).t()), dict(X=z(64)), dict(B=z(63, 32)),
               dict(B=z(64, 32).float()), dict(down=z(2, 8, 65)), dict(down=z(8, 64)), dict(down=z(2, 129, 64)),
               dict(down=z(2, 0, 64)), dict(up=z(2, 32, 9)), dict(up=z(3, 32, 8)), dict(up=z(2, 33, 8)),
               dict(down=z(2, 8, 128)[:, :, ::2]), dict(index=i.long()), dict(index=i[:3]), dict(index=i.cpu()),
               dict(scale=f[:1]), dict(scale=f.double()), dict(bias=f), dict(D=z(4, 33)), dict(D=z(4, 32).double()),
               dict(hidden=z(4, 16)), dict(hidden=z(4, 32).half()), dict(D=z(4, 32), out_dtype="f32")):
        a = dict(ok, **kw)
        with pytest.raises(ValueError):
            plan.linear_adapters(a.pop("X"), a.pop("B"), a.pop("down"), a.pop("up"), a.pop("index"), a.pop("scale"), **a)
    for kw in (dict(X=z(4, 65)[:, 1:]), dict(B=z(64, 33)[:, :32]), dict(down=z(2, 8, 65)[:, :, :64]),
               dict(down=z(2, 8, 72)[:, :, 4:68]), dict(up=z(2, 32, 9)[:, :, :8])):
        a = dict(ok, **kw)
        with pytest.raises(tc.GemmError) as e:
            plan.linear_adapters(*[a[k] for k in ("X", "B", "down", "up", "index", "scale")])
        assert tc.STATUS[e.value.status] == "GEMM_ERR_MISALIGNED"
    with pytest.raises(tc.GemmError):
        plan.linear_adapters(*ok.values(), out_dtype="f16")
    with tc.Plan("e4m3", 0) as p8:
        with pytest.raises(ValueError):
            p8.linear_adapters(*ok.values())
    h = z(4, 32)
    for kw in (dict(dY=z(4, 31)), dict(dY=z(3, 32)), dict(dY=z(4, 32).half()), dict(hidden=z(4, 16)),
               dict(d_down=z(2, 8, 63)), dict(d_up=z(2, 32, 8).float()), dict(d_up=z(2, 32, 8).half()), dict(dX=z(4, 63))):
        a = dict(dY=z(4, 32), hidden=h, d_down=z(2, 8, 64), d_up=z(2, 32, 8), dX=None)
        a.update(kw)
        with pytest.raises(ValueError):
            plan.linear_adapters_grad(a["dY"], ok["B"], ok["X"], a["hidden"], ok["down"], ok["up"], i, dX=a["dX"],
                                      d_down=a["d_down"], d_up=a["d_up"])
