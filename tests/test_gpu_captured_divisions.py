"""Captured products whose units leave partial sums for one another (early partials, stream-K): a graph's
replays share one tag, and each has to wait for the partials of its own.  Whole numbers small enough for every sum
to be exact, so every result is compared bit for bit; inputs change from replay to replay.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

# (M, N, K) whose partial last wave can be divided so (the longer one has two whole waves)
SIZES = {"early_split": (5200, 3840, 520), "stream_k": (5200, 5120, 520)}


@pytest.fixture(scope="module")
def tc():
    from tensor_core_dense_tma_gb300 import build as tcbuild
    tcbuild.build()
    import tensor_core_dense_tma_gb300 as tc
    return tc


def whole(shape, top, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-top, top + 1, shape, generator=g, device="cuda")


def replayed(call, X, values, want):
    """call(), captured, with each of the values in X in turn."""
    X.copy_(values[0])
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        D = call()
    for _ in range(3):
        for v, w in zip(values, want):
            D.fill_(7)
            X.copy_(v)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(D, w)


@pytest.mark.parametrize("division", list(SIZES))
@pytest.mark.parametrize("kind", ["f16", "bf16", "e4m3", "tf32"])
@pytest.mark.parametrize("fused", [False, True], ids=["plain", "epilogue"])
def test_product(tc, kind, division, fused):
    M, N, K = SIZES[division]
    K = -(-K // 16) * 16 if kind == "e4m3" else K          # rows of whole 16-byte units
    dtype = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "tf32": torch.float32}[kind]
    values = [whole((M, K), 2, s) for s in (1, 2)]
    B = whole((N, K), 2, 3)
    bias = whole((N,), 5, 4).float()
    # (sums of some 500 products of at most 4: exact in fp32)
    want = [v.float() @ B.float().t() + (bias if fused else 0) for v in values]
    X, values, Bt = values[0].to(dtype), [v.to(dtype) for v in values], B.to(dtype).t()
    with tc.Plan(kind, 0) as plan:
        plan.force_division(division)
        name = {"early_split": "_esplitk", "stream_k": "_streamk"}[division]
        if name not in plan.describe(M, N, K, "row", "col", "f32", "f32"):
            pytest.skip("no such division of this type's tiles")
        replayed(lambda: plan.gemm(X, Bt, bias=bias if fused else None), X, values, want)
        assert plan.device_status() == 0


@pytest.mark.parametrize("division", list(SIZES))
@pytest.mark.parametrize("count", [0, 3])
def test_adapters(tc, division, count):
    """Without an adapter the call is a plain product; with some it is a kernel of its own."""
    M, N, K = SIZES[division]
    values = [whole((M, K), 2, s) for s in (5, 6)]
    B, down, up = whole((N, K), 1, 7), whole((count, 16, K), 1, 8), whole((count, N, 16), 1, 9)
    index = (torch.arange(M, device="cuda") // 700 % 4 - 1).int()
    want = []
    for v in values:
        y = v.double() @ B.double().t()
        for a in range(count):
            rows = index == a
            y[rows] += v[rows].double() @ down[a].double().t() @ up[a].double().t()
        want.append(y.float())                # (below 2^24: exact)
    bf = [t.bfloat16() for t in (values[0], B, down, up)]
    with tc.Plan("bf16", 0) as plan:
        plan.force_division(division)
        replayed(lambda: plan.linear_adapters(bf[0], bf[1].t(), bf[2], bf[3], index, out_dtype="f32")[0], bf[0],
                 [v.bfloat16() for v in values], want)
        assert plan.device_status() == 0


@pytest.mark.parametrize("division", list(SIZES))
@pytest.mark.parametrize("act", ["none", "relu"])
def test_codes(tc, division, act):
    """The 8-bit product on its 16-bit copies; its ReLU is a kernel of its own."""
    M, N, K = 5200, 5120, 2048
    values, B = [whole((M, K), 9, s).to(torch.int8) for s in (10, 11)], whole((N, K), 9, 12).to(torch.int8)
    scale = torch.exp2(whole((N,), 2, 13).float())
    want = [(v.float() @ B.float().t()) * scale for v in values]      # (below 2^24: exact)
    if act == "relu":
        want = [w.clamp(min=0) for w in want]
    X = values[0].clone()
    with tc.Plan("f16", 0) as plan:
        plan.force_division(division)
        replayed(lambda: plan.gemm_i8(X, B.t(), col_scale=scale, act=act), X, values, want)
        assert plan.device_status() == 0
