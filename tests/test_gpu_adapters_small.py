"""fp16 adapters whose h or p is small: the first steps of tuning (up near 0), gradients of a mean, small inputs.

Tolerances, with those of test_gpu_adapters.py.  A sum of n products in fp32 is off by a(n) of the sum of their
magnitudes.  p is high + 2^-11 rest: high is off by half a unit, 2^-11 of it, rest by 2^-11 of itself or,
subnormal, by 2^-25; so the pair by 2^-22 |p| + 2^-36, and twice 2^-24 |p| for the two subtractions and products
in fp32.  A gradient of a factor is off by a(2 M) of its sum of magnitudes, e_p of each row, and its own rounding.
dX sums high and low parts, which end at 2^-24: 2^-25 of the rows' sums of |A|.
"""
import pytest
import torch

from test_gpu_adapters import F64, HALF_ULP, SMALLEST, TYPES, Case, acc, near, padded, plans, tc      # noqa: F401

pytestmark = pytest.mark.gpu


def values(c, x, first):
    """The rows' values in the middle and their error."""
    h, e = torch.zeros((c.M, c.R), dtype=F64, device="cuda"), torch.zeros((c.M, c.R), dtype=F64, device="cuda")
    for a in range(c.G):
        rows, s = c.index == a, c.scale[a].double()
        h[rows] = s * (x[rows].double() @ first[a].double().t())
        size = s * (x[rows].double().abs() @ first[a].double().abs().t())
        e[rows] = size * acc(x.shape[1]) + h[rows].abs() * (2.0 ** -22 + 2.0 ** -23) + 2.0 ** -36
    return h, e


def small(M, N, K, R, G, dy, up, x=1.0, down=1.0, index="mixed"):
    c = Case(M, N, K, R, G, "f16", seed=50, index=index)
    c.dY = padded(c.dY.double() * 10 * dy, "f16")
    c.up = padded(c.up.double() * 2 * up, "f16")
    c.X = padded(c.X.double() * x, "f16")
    c.down = padded(c.down.double() * down, "f16")
    return c


# by the kernels that make p (up factors are rank-contiguous on the way back: tiles) and h, one or more parts
SHAPES = [(300, 264, 520, 16, 3), (1000, 2055, 264, 8, 3), (70, 1040, 264, 33, 2), (257, 520, 1032, 128, 5)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dy,up", [(6e-5, 1e-4), (2e-5, 1e-4), (1e-3, 1e-4), (1e-4, 1e-3), (1e-3, 6e-8)])
@pytest.mark.parametrize("out", ["f32", "f16"])
def test_first_steps(plans, shape, dy, up, out):      # noqa: F811
    c = small(*shape, dy, up)
    plan = plans["f16"]
    _, hidden = plan.linear_adapters(c.X, *c.args())
    kw = {}
    if out == "f32":
        kw = dict(d_down=torch.empty((c.G, c.R, c.K), device="cuda"), d_up=torch.empty((c.G, c.N, c.R), device="cuda"))
    g = plan.linear_adapters_grad(c.dY, c.B, c.X, hidden, c.down, c.up, c.index, c.scale, **kw)
    torch.cuda.synchronize()
    p, e = values(c, c.dY, c.up.transpose(1, 2))
    want, tol = c.factor(p, e, c.X)
    near(g.d_down, want, tol, out, "d_down")
    if out == "f32":
        # as a whole, far below what fp16 keeps of dY itself: e_p of p's root mean square, and fp32's 2^-18
        lost = (g.d_down.double() - want).norm().item()
        assert lost <= (2.0 ** -36 / max(p.square().mean().sqrt().item(), 1e-30) + 2.0 ** -18) * want.norm().item(), lost
    x, w = c.dY.double(), c.B.t().double()
    dX, size = x @ w, x.abs() @ w.abs()
    extra = torch.zeros_like(dX)
    for a in range(c.G):
        rows, A = c.index == a, c.down[a].double()
        dX[rows] += p[rows] @ A
        size[rows] += p[rows].abs() @ A.abs()
        extra[rows] = (e[rows] + 2.0 ** -25) @ A.abs()
    near(g.dX, dX, size * acc(c.N + 2 * c.R) + extra, "f16", "dX")


@pytest.mark.parametrize("M", [20, 300])
@pytest.mark.parametrize("R", [8, 40])
@pytest.mark.parametrize("down_col", [False, True])
def test_wide_hidden(plans, M, R, down_col):      # noqa: F811
    """hidden of 3 P columns, by either kernel: D as with 2 P, d_up of small inputs as exact as p's."""
    plan = plans["f16"]
    c = small(M, 264, 520, R, 3, 0.1, 0.5, x=1e-4, down=1e-2)
    if down_col:
        c.down = padded(c.down.double(), "f16", swap=True)
    D, hidden = plan.linear_adapters(c.X, *c.args())
    P = hidden.shape[1] // 2
    buf = torch.full((M, 3 * P + 16), 7.0, dtype=torch.float16, device="cuda")
    D3, wide = plan.linear_adapters(c.X, *c.args(), hidden=buf[:, 8:8 + 3 * P])
    assert torch.equal(D3, D) and bool((buf[:, :8] == 7).all()) and bool((buf[:, 8 + 3 * P:] == 7).all())
    assert torch.equal(wide[:, P:2 * P], hidden[:, :P]) and torch.equal(wide[:, :P], hidden[:, P:])
    h, e = values(c, c.X, c.down)
    got = wide[:, P:P + R].double() + wide[:, 2 * P:2 * P + R].double() * 2.0 ** -11
    near(got, h, e, "f32", "hidden")
    assert not wide[:, R:P].any() and not wide[:, P + R:2 * P].any() and not wide[:, 2 * P + R:].any()
    new = lambda: dict(d_down=torch.empty((3, R, 520), device="cuda"), d_up=torch.empty((3, 264, R), device="cuda"))  # noqa: E731
    args = (c.dY, c.B, c.X)
    rest = (c.down, c.up, c.index, c.scale)
    g = plan.linear_adapters_grad(*args, wide, *rest, **new())
    near(g.d_up, *[t.transpose(1, 2) for t in c.factor(h, e, c.dY)], "f32", "d_up")
    two = plan.linear_adapters_grad(*args, hidden, *rest, **new())
    assert torch.equal(g.d_down, two.d_down) and torch.equal(g.dX, two.dX)


def test_wide_extremes(plans):      # noqa: F811
    """The largest values, and those beyond the type: nothing but them is lost."""
    plan = plans["f16"]
    X = torch.zeros((4, 64), dtype=torch.float16, device="cuda")
    X[0, 0], X[1, 0], X[2, 0], X[3, 0] = 65504.0, 65504.0, -2.0, 1e-7
    down = torch.zeros((1, 8, 64), dtype=torch.float16, device="cuda")
    down[0, :, 0] = 1
    up = torch.ones((1, 32, 8), dtype=torch.float16, device="cuda")
    B = torch.zeros((32, 64), dtype=torch.float16, device="cuda").t()
    index = torch.tensor([0, -1, 0, 0], dtype=torch.int32, device="cuda")
    wide = torch.full((4, 48), 7.0, dtype=torch.float16, device="cuda")
    for scale, top in ((1.0, 65504.0), (65519.0 / 65504.0, 65519.0), (2.0, float("inf"))):
        s = torch.tensor([scale], device="cuda")
        plan.linear_adapters(X, B, down, up, index, s, hidden=wide)
        value = wide[:, 16:24].double() + wide[:, 32:40].double() / 2048
        assert not wide[1].any() and bool((wide[:, 8:16] == 0).all())
        # (65519 / 65504 in fp32, times 65504: half a unit of 2^-7 away, the rest in 11 bits of 15)
        assert value[0, 0].item() == top if top in (65504.0, float("inf")) else abs(value[0, 0].item() - top) <= 2 * 2.0 ** -7
        assert abs(value[2, 0].item() + 2 * scale) <= 2.0 ** -21
        assert abs(value[3, 0].item() - X[3, 0].item() * s.item()) <= 2.0 ** -36


def test_wide_is_fp16s(plans, tc):      # noqa: F811
    c = Case(40, 264, 520, 16, 3, "bf16", seed=51, index="mixed")
    with pytest.raises(ValueError):
        plans["bf16"].linear_adapters(c.X, *c.args(), hidden=torch.empty((40, 48), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        plans["f16"].linear_adapters(c.X.half(), c.B.half(), c.down.half(), c.up.half(), c.index, c.scale,
                                     hidden=torch.empty((40, 47), dtype=torch.float16, device="cuda"))
    lib, A = tc.load(), tc._adapters.Adapters
    a = A(3, 16, c.down.data_ptr(), c.down.stride(1), c.down.stride(0), 0, c.up.data_ptr(), c.up.stride(1),
          c.up.stride(0), 0, None, c.index.data_ptr(), 0, 1, 0)
    D, h = torch.empty((40, 264), dtype=torch.bfloat16, device="cuda"), torch.empty((40, 48), dtype=torch.bfloat16, device="cuda")
    st = lib.gemm_run_adapters(plans["bf16"].handle, c.X.data_ptr(), c.B.data_ptr(), D.data_ptr(), 40, 264, 520,
                               c.X.stride(0), c.B.stride(1), 264, 1, 1, None, tc._adapters.ctypes.byref(a), h.data_ptr(), 48,
                               torch.cuda.current_stream().cuda_stream)
    assert tc.STATUS[st] == "GEMM_ERR_UNSUPPORTED"
    # without adapters the rows are zeros, all of them
    z = Case(20, 264, 520, 16, 0, "f16", seed=52, index="none", scale=False)
    wide = torch.full((20, 56), 7.0, dtype=torch.float16, device="cuda")
    plans["f16"].linear_adapters(z.X, *z.args(), hidden=wide[:, :48])
    assert not wide[:, :48].any() and bool((wide[:, 48:] == 7).all())
