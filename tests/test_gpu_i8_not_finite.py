"""The 8-bit product and the quantisation of rows on infinities and NaN.

A row with one has it as its scale (max |x| / 127), and x / scale is then no
number or 0: the row's codes are 0 and its results, 0 times the scale, NaN.
A NaN stays one through every activation.  No tolerance is needed there; the
rows beside are compared as in test_gpu_i8.py (exact codes and sums, two
scalings and the bias in fp32).
"""
import math

import numpy as np
import pytest
import torch

from test_gpu_i8 import HALF_ULP, TYPES, codes, finish, quantise

pytestmark = pytest.mark.gpu

# by the kernel that computes them, with the launches of a product of given codes: dot products, tiles on one CTA (K shared by a
# cluster and not), tiles on CTA pairs, 16-bit copies and the fp16 kernel
SIZES = [(1, 70, 100, 1), (2, 64, 96, 1), (4, 130, 64, 1), (16, 300, 2048, 2), (60, 129, 72, 2), (200, 520, 77, 2),
         (1000, 2100, 515, 2), (600, 4104, 4096, 2), (4100, 4096, 2048, 3)]
INF, NAN = math.inf, math.nan


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


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("K,pad", [(100, 0), (1024, 0), (1029, 3), (40000, 0)], ids=lambda v: str(v))
def test_quantize(tc, kind, K, pad):
    """Codes of 0 and the scale of the definition, in rows read eight elements
    at a time and one by one; the rows beside have theirs."""
    x = torch.randn((6, K + pad), device="cuda").to(TYPES[kind])[:, :K]
    x[0, K // 2], x[1, K - 1], x[3, 0], x[4, 3], x[4, 5] = INF, -INF, NAN, INF, NAN
    Q, s = tc.quantize_rows_i8(x)
    assert s[0].item() == s[1].item() == INF and math.isnan(s[3]) and math.isnan(s[4])
    assert not Q[[0, 1, 3, 4]].any()
    q, sn = quantise(x[[2, 5]].float().cpu().numpy())
    assert np.array_equal(Q[[2, 5]].cpu().numpy().astype(np.int64), q) and np.array_equal(s[[2, 5]].cpu().numpy(), sn)


@pytest.mark.parametrize("out", list(TYPES))
@pytest.mark.parametrize("M,N,K,launches", SIZES, ids=lambda v: str(v))
def test_dynamic(plan, M, N, K, launches, out):
    g = torch.Generator(device="cuda").manual_seed(M + K)
    x = torch.randn((M, K), generator=g, device="cuda").to(TYPES[out])
    bad = {0: INF, M // 3: -INF, M // 2: NAN} if M > 2 else {0: INF}
    for r, v in bad.items():
        x[r, (7 * r + 3) % K] = v
    W, w = codes(N, K, 4)
    cs = np.random.default_rng(1).random(N).astype(np.float32) / K
    D = plan.linear_i8(x, W.t(), col_scale=torch.from_numpy(cs).cuda())
    good = np.setdiff1d(np.arange(M), list(bad))
    assert torch.isnan(D[list(bad)]).all()
    q, s = quantise(x[good].float().cpu().numpy())
    want = (q.astype(np.float64) @ w.T.astype(np.float64)) * s.astype(np.float64)[:, None] * cs.astype(np.float64)
    tol = (2.0 ** -22 + HALF_ULP[out]) * np.abs(want) + (2.0 ** -25 if out == "f16" else 0.0)
    assert np.all(np.abs(D[good].double().cpu().numpy() - want) <= tol * (1 + 1e-6))


@pytest.mark.parametrize("M,N,K,launches", SIZES, ids=lambda v: str(v))
def test_scales_of_given_codes(plan, M, N, K, launches):
    """An infinite or NaN scale of a row or a channel: 0 times it is NaN."""
    A, a = codes(M, K, 3)
    W, w = codes(N, K, 4)
    rs, cs = np.ones(M, np.float32), np.ones(N, np.float32)
    rs[M // 2], cs[5], cs[N - 1] = INF, NAN, INF
    A[M // 2] = 0
    W[N - 1] = 0
    before = plan.launches
    D = plan.gemm_i8(A, W.t(), row_scale=torch.from_numpy(rs).cuda(), col_scale=torch.from_numpy(cs).cuda())
    assert (plan.launches - before >= 3) if launches == 3 else plan.launches - before == launches
    bad = torch.zeros((M, N), dtype=torch.bool, device="cuda")
    bad[M // 2], bad[:, 5], bad[:, N - 1] = True, True, True
    assert torch.equal(torch.isnan(D), bad)


@pytest.mark.parametrize("act", ["relu", "gelu"])
@pytest.mark.parametrize("M,N,K,launches", SIZES, ids=lambda v: str(v))
def test_activations_keep_a_nan(plan, M, N, K, launches, act):
    """A NaN sum is no negative number: it does not become 0."""
    x = torch.randn((M, K), device="cuda")
    x[M // 2, 3] = NAN
    W, _ = codes(N, K, 4)
    bias = torch.randn(N, device="cuda")
    bias[N // 2] = NAN
    cs = torch.full((N,), 1.0 / K, device="cuda")
    for out in TYPES:
        D = plan.linear_i8(x, W.t(), col_scale=cs, bias=bias, act=act, out_dtype=out)
        bad = torch.zeros((M, N), dtype=torch.bool, device="cuda")
        bad[M // 2], bad[:, N // 2] = True, True
        assert torch.equal(torch.isnan(D), bad)


@pytest.mark.parametrize("act", ["relu", "gelu"])
def test_activation_of_an_empty_sum_keeps_a_nan(plan, act):
    bias = torch.tensor([1.0, NAN, -1.0], device="cuda")
    A, W = torch.zeros((5, 0), dtype=torch.int8, device="cuda"), torch.zeros((3, 0), dtype=torch.int8, device="cuda")
    D = plan.gemm_i8(A, W.t(), bias=bias, act=act)
    assert torch.isnan(D[:, 1]).all() and not torch.isnan(D[:, [0, 2]]).any()


@pytest.mark.parametrize("M,N,K", [(4708, 8192, 2048), (4100, 4096, 2048), (1200, 16384, 4096)], ids=lambda v: str(v))
def test_relu_on_a_pinned_plan(tc, M, N, K):
    """Whatever a plan is pinned to, ReLU runs where no activation does."""
    A, _ = codes(M, K, 3)
    W, _ = codes(N, K, 4)
    scale = torch.full((M,), 1e-3, device="cuda")
    ran = 0
    with tc.Plan("f16", 0) as plan:
        for config in ("auto", "single_128x256", "pair_256x224", "pair_256x256"):
            for division in ("auto", "whole", "split", "early_split", "halves", "stream_k"):
                plan.force_config(config)
                plan.force_division(division)
                try:
                    want = plan.gemm_i8(A, W.t(), row_scale=scale)
                except tc.GemmError as e:
                    assert e.status == 2
                    continue
                ran += 1
                assert torch.equal(plan.gemm_i8(A, W.t(), row_scale=scale, act="relu"), want.clamp(min=0))
        torch.cuda.synchronize()
        assert plan.device_status() == 0
    assert ran > 8
