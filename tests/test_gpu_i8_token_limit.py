"""The 8-bit product of more tokens than a grid's second dimension has tiles
for (65535 of 128 or 256): sampled rows in whole numbers, every partial sum exact."""
import pytest
import torch

pytestmark = pytest.mark.gpu


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


def check(plan, M, N, K, row):
    if torch.cuda.mem_get_info()[0] < 4 * M * (3 * K + 4 * N) // 3:
        pytest.skip("needs more device memory")
    g = torch.Generator(device="cuda").manual_seed(M)
    A = torch.randint(-128, 128, (M, K), generator=g, dtype=torch.int8, device="cuda")
    W = torch.randint(-128, 128, (N, K), generator=g, dtype=torch.int8, device="cuda")
    D = torch.full((M, N), float("nan"), device="cuda")
    plan.gemm_i8(A, W.t(), D)
    rows = torch.cat([torch.randint(0, M, (5000,), generator=g, device="cuda"),
                      torch.arange(row - 300, min(row + 300, M), device="cuda"), torch.arange(M - 300, M, device="cuda")])
    assert torch.equal(D[rows].double(), A[rows].double() @ W.double().t())
    assert not torch.isnan(D.view(-1)[:: 997]).any()


@pytest.mark.parametrize("M,N,K", [(9_000_000, 16, 16), (8_388_480, 16, 32), (8_388_481, 130, 48), (16_900_001, 8, 16)],
                         ids=lambda v: str(v))
def test_many_tokens(plan, M, N, K):
    check(plan, M, N, K, 65535 * 128)


def test_many_tokens_on_cta_pairs():
    """Tiles of 256 tokens; 113 GB."""
    import tensor_core_dense_tma_gb300 as tc
    with tc.Plan("f16", 0) as plan:
        check(plan, 65535 * 256 + 301, 144, 2048, 65535 * 256)
        torch.cuda.synchronize()
        assert plan.device_status() == 0
