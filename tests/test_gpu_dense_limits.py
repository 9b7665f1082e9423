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


def test_gated_weight_gradients_of_more_than_31_bits_of_rows():
    """N a little above 2^30: both factors' columns together pass 2^31.  dh = 1 but for
    marked columns, u = 2 and g = 3 with the rectifier, so dg = 2 dh and du = 3 dh."""
    N, K, M = 2 ** 30 + 72, 8, 5
    if torch.cuda.mem_get_info()[0] < 110 << 30:
        pytest.skip("needs 110 GB")
    bf = torch.bfloat16
    x = torch.arange(M * K, device="cuda").view(M, K).remainder(7).to(bf)
    dh = torch.ones((M, N), dtype=bf, device="cuda")
    at = torch.tensor([0, 1, 65, 2 ** 29 - 1, 2 ** 30 - 129, 2 ** 30 - 1, 2 ** 30, N - 70, N - 1],
                      device="cuda")
    dh[:, at] = torch.arange(1, 10, device="cuda").to(bf)
    g = torch.full((M, N), 3.0, dtype=bf, device="cuda")
    u = torch.full((M, N), 2.0, dtype=bf, device="cuda")
    _, dwg, dwu, _, _ = lq.lq_gated_linear_bwd(dh, g, u, x, None, None, act=lq.LQ_ACT_RELU,
                                               want_dx=False)
    sums = x.float().sum(0)
    for dw, by in ((dwg, 2.0), (dwu, 3.0)):
        marked = torch.arange(1, 10, device="cuda").view(-1, 1) * sums * by
        assert torch.equal(dw[at], marked.to(bf))
        dw[at] = (sums * by).to(bf)
        one = (sums * by).to(bf)
        for rows in dw.split(1 << 26):
            assert bool((rows == one).all())
