"""Calls of the adapters' entry points that the documentation refuses or leaves to the callee."""
import pytest
import torch

from test_gpu_adapters import Case, plans, tc      # noqa: F401

pytestmark = pytest.mark.gpu


def test_gradient_without_hidden(plans):      # noqa: F811
    """hidden is an input of the backward pass: without it there is nothing to make d_up of."""
    plan = plans["bf16"]
    c = Case(40, 264, 520, 16, 3, "bf16", seed=40, index="mixed")
    with pytest.raises(ValueError, match="hidden"):
        plan.linear_adapters_grad(c.dY, c.B, c.X, None, c.down, c.up, c.index, c.scale)
    z = Case(40, 264, 520, 16, 0, "bf16", seed=40, index="none", scale=False)
    g = plan.linear_adapters_grad(z.dY, z.B, z.X, None, z.down, z.up, z.index)
    want = plan.gemm(z.dY, z.B.t(), out_dtype="bf16")
    assert torch.equal(g.dX, want) and g.d_down.shape == (0, 16, 520) and g.d_up.shape == (0, 264, 16)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    g = plan.linear_adapters_grad(c.dY[:0], c.B, c.X[:0], None, c.down, c.up, none, c.scale)
    assert g.dX.shape == (0, 520) and not g.d_down.any() and not g.d_up.any()


def dropped(call, pick, want, fill):
    """call(stream) on a stream that is busy, all of its results dropped but pick's, the current stream's next
    allocations in the memory that this frees; pick's results as wanted, and what was allocated as filled."""
    s = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)
        got = pick(call(s.cuda_stream))
        later = [torch.full_like(t, 3) for t in fill for _ in range(3)]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        assert all(bool((t == 3).all()) for t in later)


@pytest.mark.parametrize("M", [4, 300])
def test_serving_on_a_given_stream(plans, M):      # noqa: F811
    """A caller that wants D alone drops the hidden rows while both kernels are still to run."""
    plan = plans["bf16"]
    c = Case(M, 264, 520, 16, 3, "bf16", seed=41, index="mixed")
    D, hidden = plan.linear_adapters(c.X, *c.args())
    dropped(lambda s: plan.linear_adapters(c.X, *c.args(), stream=s), lambda r: r[:1], [D], [hidden])
    dropped(lambda s: plan.linear_adapters(c.X, *c.args(), stream=s), lambda r: r[1:], [hidden], [D])


def test_gradient_on_a_given_stream(plans):      # noqa: F811
    """The same of a caller that does not want dX."""
    plan = plans["bf16"]
    c = Case(300, 264, 520, 16, 3, "bf16", seed=42, index="mixed")
    _, hidden = plan.linear_adapters(c.X, *c.args())
    args = (c.dY, c.B, c.X, hidden, c.down, c.up, c.index, c.scale)
    want = plan.linear_adapters_grad(*args)
    dropped(lambda s: plan.linear_adapters_grad(*args, stream=s), lambda r: r[1:], want[1:], [want.dX])


def test_losses_on_a_given_stream(tc):      # noqa: F811
    """One result of each operator on logits kept."""
    g = torch.Generator(device="cuda").manual_seed(43)
    z = torch.randn((64, 5000), generator=g, device="cuda")
    t = torch.randint(0, 5000, (64,), generator=g, device="cuda")
    old, adv = torch.randn((2, 64), generator=g, device="cuda").unbind()
    at, w = torch.tensor([0, 20, 64], device="cuda"), torch.ones(1, device="cuda")
    r = tc.token_logprobs(z, t, top=4)
    for name, args, kw in (("token_logprobs", (t,), dict(top=4)), ("token_logprobs_grad", (t, adv, old), {}),
                           ("distill_topk", (r.top_token, r.top_logprob), {}),
                           ("distill_topk_grad", (r.top_token, r.top_logprob, adv), {}),
                           ("policy_loss", (t, old, adv), {}), ("policy_loss_grad", (t, old, adv, adv), {}),
                           ("preference_loss", (t, at), {}), ("preference_loss_grad", (t, at, w), {})):
        call = lambda s=None: getattr(tc, name)(z, *args, stream=s, **kw)      # noqa: E731, B023
        want = call()
        for i in range(len(want)):
            dropped(call, lambda r, i=i: [r[i]], [want[i]], [t for k, t in enumerate(want) if k != i])


def test_gradients_that_overlap(tc, plans):      # noqa: F811
    """The C entry point on output stacks whose matrices share memory: refused before anything is launched; stacks
    of another order, where each element has a place of its own, are written."""
    plan = plans["bf16"]
    lib, Adapters = tc.load(), tc._adapters.Adapters
    c = Case(300, 264, 520, 16, 3, "bf16", seed=44, index="mixed")
    _, hidden = plan.linear_adapters(c.X, *c.args())
    want = plan.linear_adapters_grad(c.dY, c.B, c.X, hidden, c.down, c.up, c.index, c.scale)
    p = torch.empty_like(hidden)
    G, R, K, N = 3, 16, 520, 264
    a = Adapters(G, R, c.up.data_ptr(), c.up.stride(1), c.up.stride(0), 1, c.down.data_ptr(), c.down.stride(1),
                 c.down.stride(0), 1, c.scale.data_ptr(), c.index.data_ptr())      # the way back's: each in the other's place
    dX = torch.empty((300, K), dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    assert lib.gemm_run_adapters(plan.handle, c.dY.data_ptr(), c.B.data_ptr(), dX.data_ptr(), 300, K, N, c.dY.stride(0),
                                 c.B.stride(1), K, 0, 1, None, tc._adapters.ctypes.byref(a), p.data_ptr(), 32, s) == 0
    d_down = torch.full((G * R * K + 99,), 7.0, dtype=torch.bfloat16, device="cuda")
    d_up = torch.full((G * N * R + 99,), 7.0, dtype=torch.bfloat16, device="cuda")

    def grad(down_ld, down_stride, up_ld, up_stride, parts=3):
        return lib.gemm_adapters_grad(plan.handle, c.X.data_ptr(), c.dY.data_ptr(), 300, N, K, c.X.stride(0),
                                      c.dY.stride(0), tc._adapters.ctypes.byref(a), hidden.data_ptr(), p.data_ptr(), 32, 1,
                                      d_down.data_ptr() if parts & 1 else None, down_ld, down_stride,
                                      d_up.data_ptr() if parts & 2 else None, up_ld, up_stride, s)

    for bad in ((K, 0, R, N * R), (K, R * K - 1, R, N * R), (K, K, R, N * R), (G * K, K - 1, R, N * R),
                (G * K - 1, K, R, N * R), (K, R * K, R, 0), (K, R * K, R, N * R - 1), (K, R * K, G * R - 1, R)):
        assert tc.STATUS[grad(*bad)] == "GEMM_ERR_INVALID_ARG", bad
    torch.cuda.synchronize()
    assert bool((d_down == 7).all()) and bool((d_up == 7).all())
    assert grad(K, 0, R, N * R, 2) == 0                        # the other's strides count for nothing
    for down, up_ in (((K, R * K), (R, N * R)), ((G * K, K), (G * R, R)), ((G * K + 2, K), (R, N * R + 3))):
        d_down.fill_(7), d_up.fill_(7)
        assert grad(*down, *up_) == 0
        torch.cuda.synchronize()
        assert torch.equal(torch.as_strided(d_down, (G, R, K), (down[1], down[0], 1)), want.d_down)
        assert torch.equal(torch.as_strided(d_up, (G, N, R), (up_[1], up_[0], 1)), want.d_up)


@pytest.mark.parametrize("kind,R", [("bf16", 16), ("f16", 40)])
def test_hidden_in_a_wide_buffer(plans, kind, R):      # noqa: F811
    """hidden as a slice of a buffer for many layers: the call's own rows are not as wide, and results the same."""
    plan = plans[kind]
    c = Case(3000, 136, 264, R, 3, kind, seed=45, index="mixed")
    _, hidden = plan.linear_adapters(c.X, *c.args())
    args = (c.dY, c.B, c.X)
    rest = (c.down, c.up, c.index, c.scale)
    want = plan.linear_adapters_grad(*args, hidden, *rest)
    wide = torch.full((3000, 64 * hidden.shape[1]), float("nan"), dtype=c.X.dtype, device="cuda")
    part = wide[:, 8:8 + hidden.shape[1]]
    assert torch.equal(plan.linear_adapters(c.X, *c.args(), hidden=part)[1], hidden) and bool(wide[:, :8].isnan().all())
    out = [torch.empty_like(t) for t in want]
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    got = plan.linear_adapters_grad(*args, part, *rest, *out[:1], d_down=out[1], d_up=out[2])
    torch.cuda.synchronize()
    assert torch.cuda.max_memory_allocated() - before <= 2 * hidden.numel() * hidden.element_size() + (2 << 20)
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_plan_of_another_device(tc):      # noqa: F811
    """Tensors that are not on the plan's device: its kernels cannot read them (a plan that says it is on another)."""
    c = Case(40, 264, 520, 16, 3, "bf16", seed=46, index="mixed")
    with tc.Plan("bf16", 0) as plan:
        _, hidden = plan.linear_adapters(c.X, *c.args())
        plan.device = 1
        with pytest.raises(ValueError, match="device"):
            plan.linear_adapters(c.X, *c.args())
        with pytest.raises(ValueError, match="device"):
            plan.linear_adapters_grad(c.dY, c.B, c.X, hidden, c.down, c.up, c.index, c.scale)
        plan.device = 0
        plan.linear_adapters(c.X, *c.args())
        torch.cuda.synchronize()
        assert plan.device_status() == 0


@pytest.mark.parametrize("K,G", [(0, 2), (64, 0)])
def test_far_hidden_without_adapters(plans, K, G):      # noqa: F811
    """Rows of zeros 2^30 elements apart."""
    plan = plans["bf16"]
    far = 1 << 30
    buf = torch.full((2 * far + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    hidden = torch.as_strided(buf, (3, 32), (far, 1), 8)
    z = lambda *s: torch.ones(s, dtype=torch.bfloat16, device="cuda")      # noqa: E731
    bias = torch.arange(40, device="cuda").float()
    D, _ = plan.linear_adapters(z(3, K), z(K, 40), z(G, 8, K), z(G, 40, 8), torch.zeros(3, dtype=torch.int32, device="cuda"),
                                bias=bias, hidden=hidden)
    torch.cuda.synchronize()
    assert not hidden.any() and torch.equal(D, (bias + K).bfloat16().expand(3, 40))
    for i in range(3):
        assert bool((buf[i * far:i * far + 8] == 7).all()) and bool((buf[i * far + 40:i * far + 64] == 7).all())


@pytest.mark.parametrize("handle", [0, 1, 2], ids=["default", "legacy", "per_thread"])
def test_default_streams_by_handle(plans, tc, handle):      # noqa: F811
    """The runtime's default streams, by the handles that stand for them, while torch's current stream is another."""
    plan = plans["bf16"]
    c = Case(40, 264, 520, 16, 3, "bf16", seed=47, index="mixed")
    D, hidden = plan.linear_adapters(c.X, *c.args())
    args = (c.dY, c.B, c.X, hidden, c.down, c.up, c.index, c.scale)
    g = plan.linear_adapters_grad(*args)
    z = torch.randn((20, 300), device="cuda")
    t, at = torch.randint(0, 300, (20,), device="cuda"), torch.tensor([0, 9, 20], device="cuda")
    w = torch.ones(1, device="cuda")
    p = tc.preference_loss_grad(z, t, at, w)
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(torch.cuda.Stream()):
            got = (*plan.linear_adapters(c.X, *c.args(), stream=handle), *plan.linear_adapters_grad(*args, stream=handle),
                   *tc.preference_loss_grad(z, t, at, w, stream=handle))
            torch.full((4096, 32), float("nan"), device="cuda")
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, (D, hidden, *g, *p)))
        del got
