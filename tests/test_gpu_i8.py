"""The 8-bit product with token and channel scales (gemm_run_i8,
gemm_run_i8_dynamic) and the quantisation of rows (gemm_quantize_rows_i8)
against plain numpy in whole numbers and 64 bits.

Tolerances.  The codes' products are whole numbers and a sum is exact while
its partial sums stay below 2^24: such products are compared bit for bit
(without scales), or within three fp32 roundings of scaling and bias plus the
rounding to the output's type.  Sums beyond 2^24 round once per addition:
within K 2^-23 of the sum of the magnitudes.  The GELU is within 2e-7 of its
argument (its documented 1.5e-7 and roundings).
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_ULP = {k: torch.finfo(v).eps / 2 for k, v in TYPES.items()}      # of the rounding to the type, relative


@pytest.fixture(scope="module")
def tc():
    from tensor_core_dense_tma_gb300 import build as tcbuild
    tcbuild.build()
    import tensor_core_dense_tma_gb300 as tc
    return tc


@pytest.fixture(scope="module")
def plan(tc):
    p = tc.Plan("f16", 0)
    yield p
    torch.cuda.synchronize()
    assert p.device_status() == 0
    p.close()


def codes(rows, K, seed, pad=0, top=127):
    """int8 device matrix with rows on 16-byte boundaries; what lies beside the
    matrix is not zero."""
    g = np.random.default_rng(seed)
    ld = -(-max(K, 1) // 16) * 16 + pad
    buf = torch.full((rows, ld), 99, dtype=torch.int8, device="cuda")
    v = g.integers(-top, top + 1, (rows, K)).astype(np.int8)
    v.flat[0] = -128
    buf[:, :K] = torch.from_numpy(v).cuda()
    return buf[:, :K], v.astype(np.int64)


SHAPES = [(1, 1, 1), (1, 128, 16), (1, 300, 1000), (2, 129, 64), (3, 7, 33), (8, 512, 512), (16, 1104, 520),
          (17, 640, 2048), (33, 257, 129), (48, 600, 1040), (64, 128, 72), (65, 300, 512), (100, 1, 200),
          (127, 511, 100), (129, 264, 640), (255, 255, 255), (256, 256, 256), (300, 520, 1000), (513, 1030, 1017),
          (1024, 1000, 77), (2300, 2290, 800), (4097, 2055, 1000)]


@pytest.mark.parametrize("M,N,K", SHAPES, ids=lambda v: str(v))
def test_exact(plan, M, N, K):
    """K up to 1040 (and random codes beyond): every partial sum is exact, so
    the fp32 product equals the whole-number one."""
    A, a = codes(M, K, M + K, pad=16)
    W, w = codes(N, K, N + K)
    D = torch.full((M, N + 5), float("nan"), device="cuda")
    plan.gemm_i8(A, W.t(), D[:, 2:N + 2])
    torch.cuda.synchronize()
    got = D.cpu().numpy()
    assert np.array_equal(got[:, 2:N + 2].astype(np.int64), a @ w.T)
    assert np.isnan(got[:, :2]).all() and np.isnan(got[:, N + 2:]).all()


@pytest.mark.parametrize("M,N,K", [(1, 200, 8192), (5, 130, 5000), (16, 256, 16384), (40, 300, 9001), (200, 300, 8192),
                                   (1000, 700, 4099)], ids=lambda v: str(v))
def test_long_sums(plan, M, N, K):
    A, a = codes(M, K, 1)
    W, w = codes(N, K, 2)
    D = plan.gemm_i8(A, W.t())
    torch.cuda.synchronize()
    want = a @ w.T
    assert int(np.abs(want).max()) < 1 << 23
    assert np.array_equal(D.cpu().numpy().astype(np.int64), want)


@pytest.mark.parametrize("M,N,K", [(1, 64, 8192), (16, 100, 4099), (300, 130, 5000)], ids=lambda v: str(v))
def test_sums_past_24_bits(plan, M, N, K):
    """All codes of one sign: sums of up to 1.3e8 round as fp32 sums."""
    A, a = codes(M, K, 1)
    W, w = codes(N, K, 2)
    A.copy_(A.abs().clamp(100, 127))
    W.copy_(W.abs().clamp(100, 127))
    a, w = A.cpu().numpy().astype(np.int64), W.cpu().numpy().astype(np.int64)
    want = a @ w.T
    D = plan.gemm_i8(A, W.t()).double().cpu().numpy()
    assert np.all(np.abs(D - want) <= K * 2.0 ** -23 * want)


def gelu(x):
    return 0.5 * x * np.vectorize(math.erfc)(-x / math.sqrt(2.0)) if x.size else x


def finish(u, act):
    return np.maximum(u, 0) if act == "relu" else gelu(u) if act == "gelu" else u


@pytest.mark.parametrize("M,N,K", [(1, 300, 512), (7, 129, 100), (16, 520, 1000), (40, 300, 77), (130, 257, 640),
                                   (1025, 513, 129)], ids=lambda v: str(v))
@pytest.mark.parametrize("out", list(TYPES))
@pytest.mark.parametrize("act", ["none", "relu", "gelu"])
def test_scales_bias_activation(plan, M, N, K, out, act):
    g = np.random.default_rng(M + N)
    A, a = codes(M, K, 3)
    W, w = codes(N, K, 4)
    rs = (g.random(M) * 2e-2 / np.sqrt(K)).astype(np.float32)
    cs = (g.random(N) * 2e-2).astype(np.float32)
    bias = g.normal(size=N).astype(np.float32)
    d = [torch.from_numpy(v).cuda() for v in (rs, cs, bias)]
    for row, col, b in ((True, True, True), (True, False, False), (False, True, True), (False, False, True)):
        D = plan.gemm_i8(A, W.t(), row_scale=d[0] if row else None, col_scale=d[1] if col else None,
                         bias=d[2] if b else None, act=act, out_dtype=out)
        s = (a @ w.T) * (rs.astype(np.float64)[:, None] if row else 1.0) * (cs.astype(np.float64) if col else 1.0)
        u = s + (bias.astype(np.float64) if b else 0.0)
        got = D.double().cpu().numpy()
        if out == "f16":
            over = np.abs(u) > 60000          # beyond the type's range: infinities
            assert np.all(np.isinf(got[np.abs(u) > 65600]) | (act != "none"))
            got, u, s = np.where(over, 0, got), np.where(over, 0, u), np.where(over, 0, s)
        want = finish(u, act)
        tol = 2.0 ** -22 * (np.abs(s) + np.abs(u)) + HALF_ULP[out] * np.abs(want) + 2e-7 * np.abs(u) * (act == "gelu")
        if out == "f16":
            tol = tol + 2.0 ** -25
        bad = np.abs(got - want) > tol * (1 + 1e-6)
        assert not bad.any(), (row, col, b, int(bad.sum()), got[bad][:3], want[bad][:3])


def quantise(x):
    """The definition in fp32 (numpy's divisions and rounding are IEEE)."""
    top = np.abs(x).max(axis=1, initial=0.0).astype(np.float32)
    s = top / np.float32(127)
    with np.errstate(all="ignore"):
        q = np.rint(x / s[:, None])
    return np.where(s[:, None] > 0, q, 0).astype(np.int64), s


def values(M, K, kind, seed, pad=0, shift=0):
    g = np.random.default_rng(seed)
    x = g.normal(size=(M, K)) * np.exp(g.normal(size=(M, 1)))
    buf = torch.full((M * (K + pad) + shift + 8,), float("nan"), dtype=TYPES[kind], device="cuda")
    v = torch.as_strided(buf, (M, K), (K + pad, 1), shift)
    v.copy_(torch.from_numpy(x))
    if M > 2:
        v[2] = 0
    return v, v.float().cpu().numpy()


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("M,K", [(1, 1), (3, 17), (5, 1000), (4, 4096), (3, 8191), (2, 40000), (300, 64)],
                         ids=lambda v: str(v))
def test_quantize_rows(tc, kind, M, K):
    x, xn = values(M, K, kind, K, pad=3, shift=1)
    Q, s = tc.quantize_rows_i8(x)
    q, sn = quantise(xn)
    assert np.array_equal(s.cpu().numpy(), sn)
    assert np.array_equal(Q.cpu().numpy().astype(np.int64), q)
    assert Q.stride(0) % 16 == 0
    # into the caller's buffers, rows of any stride
    buf = torch.full((M, K + 3), 55, dtype=torch.int8, device="cuda")
    tc.quantize_rows_i8(x, buf[:, 1:K + 1], s)
    assert np.array_equal(buf[:, 1:K + 1].cpu().numpy().astype(np.int64), q)
    assert bool((buf[:, 0] == 55).all()) and bool((buf[:, K + 1:] == 55).all())


def test_quantize_rows_not_finite(tc):
    x = torch.ones((4, 100), device="cuda")
    x[0, 5], x[1, 99], x[2, 0] = float("nan"), float("inf"), -float("inf")
    s = tc.quantize_rows_i8(x)[1].tolist()
    assert math.isnan(s[0]) and s[1] == s[2] == math.inf and s[3] == float(np.float32(1) / np.float32(127))


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("M,N,K", [(1, 300, 1000), (3, 64, 17), (16, 520, 4096), (17, 129, 77), (70, 300, 1000),
                                   (300, 513, 515)], ids=lambda v: str(v))
def test_dynamic(plan, kind, M, N, K):
    """Quantised in the call: the codes are the definition's, so the sums are
    exact and two scalings are left."""
    x, xn = values(M, K, kind, K + M, pad=1, shift=1)
    W, w = codes(N, K, 4)
    cs = np.random.default_rng(1).random(N).astype(np.float32)
    D = plan.linear_i8(x, W.t(), col_scale=torch.from_numpy(cs).cuda(), out_dtype="f32")
    q, s = quantise(xn)
    want = (q @ w.T) * s.astype(np.float64)[:, None] * cs.astype(np.float64)
    got = D.double().cpu().numpy()
    assert np.all(np.abs(got - want) <= 2.0 ** -22 * np.abs(want))
    same = plan.linear_i8(x, W.t(), col_scale=torch.from_numpy(cs).cuda())
    assert same.dtype == x.dtype
    assert torch.equal(same, D.to(x.dtype))


def test_dynamic_not_finite_rows(plan):
    x = torch.ones((3, 64), device="cuda")
    x[1, 3] = float("nan")
    W, w = codes(40, 64, 4)
    D = plan.linear_i8(x, W.t())
    assert torch.isnan(D[1]).all() and torch.isfinite(D[0]).all() and torch.isfinite(D[2]).all()


def test_growing_and_streams(plan):
    """Problems of changing size one after another, on a stream of its own and
    from a graph captured after a call of its size."""
    s = torch.cuda.Stream()
    for M, N, K in ((5, 300, 100), (700, 2000, 3000), (9, 40, 64), (1500, 2500, 3200)):
        A, a = codes(M, K, M)
        W, w = codes(N, K, N)
        with torch.cuda.stream(s):
            s.wait_stream(torch.cuda.default_stream())
            D = plan.gemm_i8(A, W.t())
        s.synchronize()
        assert np.array_equal(D.cpu().numpy().astype(np.int64), a @ w.T)
    graph = torch.cuda.CUDAGraph()
    out = torch.empty_like(D)
    with torch.cuda.graph(graph):
        plan.gemm_i8(A, W.t(), out)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, D)


def test_empty(plan):
    W, _ = codes(20, 64, 1)
    A, _ = codes(4, 64, 1)
    assert plan.gemm_i8(A[:0], W.t()).shape == (0, 20)
    assert plan.gemm_i8(A, W[:0].t()).shape == (4, 0)
    D = plan.gemm_i8(A[:, :0], W[:, :0].t(), bias=torch.ones(20, device="cuda"))
    assert bool((D == 1).all())
    D = plan.linear_i8(A[:, :0].float(), W[:, :0].t())
    assert bool((D == 0).all())


def test_refusals(tc, plan):
    A, _ = codes(4, 64, 1)
    W, _ = codes(20, 64, 1)
    f = torch.zeros(20, device="cuda")
    for a, b, kw in ((A.float(), W.t(), {}), (A, W.float().t(), {}), (A, W, {}), (A[:, :32], W.t(), {}),
                     (A.cpu(), W.t(), {}), (A.t(), W[:4].t(), {}), (A, W.t(), dict(bias=f[:5])),
                     (A, W.t(), dict(col_scale=f.half())), (A, W.t(), dict(D=torch.zeros((4, 21), device="cuda"))),
                     (A, W.t(), dict(D=torch.zeros((4, 20), device="cuda"), out_dtype="f16"))):
        with pytest.raises(ValueError):
            plan.gemm_i8(a, b, **kw)
    wide = torch.zeros((4, 100), dtype=torch.int8, device="cuda")
    for a, b in ((wide[:, 1:65], W.t()), (wide[:, :64], W.t()), (A, torch.zeros((20, 72), dtype=torch.int8,
                                                                                device="cuda")[:, :64].t())):
        with pytest.raises(tc.GemmError) as e:
            plan.gemm_i8(a, b)
        assert e.value.status == 3
    with tc.Plan("bf16", 0) as other:
        with pytest.raises(tc.GemmError) as e:
            other.gemm_i8(A, W.t())
        assert e.value.status == 2
    with pytest.raises(ValueError):
        tc.quantize_rows_i8(A.float().t())
    with pytest.raises(ValueError):
        tc.quantize_rows_i8(A.float(), scale=f)


# CTA pairs: one wave and two, the second CTA's channels cut off or absent; few codes and many tokens
@pytest.mark.parametrize("M,N,K", [(1500, 2049, 2100), (1025, 3300, 70), (2100, 300, 130), (3000, 129, 64),
                                   (777, 4230, 2500), (5000, 1000, 1), (1025, 3300, 1000), (1300, 5633, 2100),
                                   (4100, 1000, 900), (9000, 300, 1101)], ids=lambda v: str(v))
@pytest.mark.parametrize("out", list(TYPES))
def test_many_tokens(plan, M, N, K, out):
    g = np.random.default_rng(K)
    A, a = codes(M, K, 1, top=60)
    W, w = codes(N, K, 2, top=60)
    rs = (g.random(M) * 0.1 / np.sqrt(K)).astype(np.float32)
    bias = g.normal(size=N).astype(np.float32)
    D = torch.full((M, N + 3), float("nan"), dtype=TYPES[out], device="cuda")
    plan.gemm_i8(A, W.t(), D[:, 1:N + 1], row_scale=torch.from_numpy(rs).cuda(), bias=torch.from_numpy(bias).cuda(),
                 act="relu")
    s = (a.astype(np.float64) @ w.T.astype(np.float64)) * rs.astype(np.float64)[:, None]
    u = s + bias.astype(np.float64)
    got = D.double().cpu().numpy()
    assert np.isnan(got[:, 0]).all() and np.isnan(got[:, N + 1:]).all()
    want = np.maximum(u, 0)
    tol = 2.0 ** -22 * (np.abs(s) + np.abs(u)) + HALF_ULP[out] * want + (2.0 ** -25 if out == "f16" else 0.0)
    assert np.all(np.abs(got[:, 1:N + 1] - want) <= tol * (1 + 1e-6))


def test_graph_outlives_a_grown_workspace(tc):
    """A graph captured before a larger call made the plan's workspace grow."""
    with tc.Plan("f16", 0) as plan:
        A, a = codes(40, 500, 1)
        W, w = codes(300, 500, 2)
        D = plan.gemm_i8(A, W.t())
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            plan.gemm_i8(A, W.t(), D)
        big, _ = codes(3000, 2000, 3)
        plan.gemm_i8(big, big.t())
        D.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(D.cpu().numpy().astype(np.int64), a @ w.T)
        assert plan.device_status() == 0
