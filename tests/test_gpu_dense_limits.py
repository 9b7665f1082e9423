"""Dense entry points at the largest extents they accept: products whose operands are
zero but for a few elements, so that every value is exact."""
import pytest
import torch

from bit_ptq_looped_b200 import lq

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def release():
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("M,N", [(1, 1), (9, 2)])
def test_few_rows_over_the_longest_contraction(M, N):
    """K = 2^31 - 264: the steps past the last block stay past it."""
    K = 2 ** 31 - 264
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((N, K), dtype=torch.bfloat16, device="cuda")
    want = torch.zeros((M, N))
    for i, k in enumerate((0, 8, 1535, K // 2 + 1, K - 1536, K - 255, K - 9, K - 1)):
        x[:, k] = torch.arange(1, M + 1, device="cuda") * 2.0 ** (i % 3)
        w[:, k] = torch.arange(1, N + 1, device="cuda") * 0.5
        want += 2.0 ** (i % 3) * 0.5 * torch.outer(torch.arange(1.0, M + 1),
                                                   torch.arange(1.0, N + 1))
    y, _ = lq.lq_dense_linear(x, w)
    assert torch.equal(y.cpu(), want.to(torch.bfloat16))
