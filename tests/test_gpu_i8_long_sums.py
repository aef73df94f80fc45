"""The 8-bit product's sums at and past 2^24, where fp32 holds no longer every
whole number, on each of its kernels.

At most 2^24: exact, bit for bit (1024 products of -128 and -128 are 2^24, 1040
of 127 and 127 are below it).  Past it the accumulation of a step of 16 codes is
taken to drop at most one unit of 24 bits in each of two halves, less than
2 x 2^-23 of the sum, so K / 16 steps drop at most K 2^-26 of a sum of products
of one sign; joining up to eight ranges of K rounds by 8 x 2^-24 more.  Whole
numbers rounded once are within 2^-24.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

# dot products; tiles with K shared in clusters of eight and four, and not shared; tiles on CTA pairs; the fp16 kernel
ROWS = [(1, 300), (2, 256), (16, 200), (16, 20000), (60, 2100), (130, 4104), (700, 4104), (4100, 4096)]


@pytest.fixture(scope="module")
def plan():
    from tensor_core_dense_tma_gb300 import build as tcbuild
    tcbuild.build()
    import tensor_core_dense_tma_gb300 as tc
    p = tc.Plan("f16", 0)
    yield p
    torch.cuda.synchronize()
    assert p.device_status() == 0
    p.close()


def filled(rows, K, value):
    return torch.full((rows, -(-K // 16) * 16), value, dtype=torch.int8, device="cuda")[:, :K]


@pytest.mark.parametrize("M,N", ROWS, ids=lambda v: str(v))
@pytest.mark.parametrize("K,a,b", [(1024, -128, -128), (1040, 127, 127), (1040, -127, 127), (1023, -128, -128),
                                   (1000, -128, 127)], ids=lambda v: str(v))
def test_largest_exact_sums(plan, M, N, K, a, b):
    D = plan.gemm_i8(filled(M, K, a), filled(N, K, b).t())
    assert bool((D.double() == K * a * b).all())


@pytest.mark.parametrize("M,N", ROWS, ids=lambda v: str(v))
def test_one_product_past_the_bound(plan, M, N):
    """1024 products of -128 and -128 and one of 1 and 1: 2^24 + 1 is no fp32
    number."""
    A, W = filled(M, 1025, -128), filled(N, 1025, -128)
    A[:, 1024], W[:, 1024] = 1, 1
    D = plan.gemm_i8(A, W.t())
    assert bool((D == 2.0 ** 24).all())


@pytest.mark.parametrize("M,N", ROWS, ids=lambda v: str(v))
@pytest.mark.parametrize("K", [2048, 4100, 8192, 16384])
def test_sums_of_one_sign(plan, M, N, K):
    g = torch.Generator(device="cuda").manual_seed(K)
    A = torch.randint(90, 128, (M, -(-K // 16) * 16), generator=g, dtype=torch.int8, device="cuda")[:, :K]
    W = torch.randint(-128, -89, (N, -(-K // 16) * 16), generator=g, dtype=torch.int8, device="cuda")[:, :K]
    D = plan.gemm_i8(A, W.t()).double()
    want = A.double() @ W.double().t()
    rel = 2.0 ** -24 if M <= 2 else K * 2.0 ** -26 + 2.0 ** -21
    assert bool(((D - want).abs() <= rel * want.abs()).all())
