"""Host-side checks of the dense entry points and the distillation loss at the ends of
what they accept (no GPU needed)."""
import pytest

from bit_ptq_looped_b200 import build as B
from bit_ptq_looped_b200 import lq

X, W, Y, Z = ((i + 1) << 40 for i in range(4))  # never dereferenced


@pytest.fixture(scope="module")
def L():
    B.build()
    return lq.lib()


def test_temperatures_whose_exponent_factor_is_not_finite_are_refused(L):
    """log2(e) / temp scales every exponent; at 3.5e-39 one over the temperature is
    finite in float32 (2.86e38) and this factor is not."""
    def call(temp):
        return L.lq_distill_loss(X, lq.LQ_F32, 4, 100, W, lq.LQ_F32, Z, 8, 5, None, None, temp, Y,
                                 None, None)

    for temp in (3.5e-39, 4.2e-39):
        assert call(temp) == lq.LQ_ERR_ARG
        assert "temperature" in L.lq_last_error().decode()


def test_workspace_sizes_at_the_longest_contractions(L):
    """Contractions of up to 2^31: the block times that choose a tile shape are sums of
    64-bit terms (the sanitizer build reports an overflow)."""
    for M, N, K in ((8, 2 ** 31 - 256, 8), (16, 2 ** 30 + 8, 64), (2 ** 31 - 256, 64, 8),
                    (100, 8, 2 ** 31 - 256)):
        n = L.lq_dense_linear_bwd_workspace_bytes(M, N, K, lq.LQ_ACT_SILU)
        assert n >= 2 * M * N and n % 256 == 0
        n = L.lq_gated_linear_bwd_workspace_bytes(M, N, K)
        assert n >= 4 * M * N and n % 256 == 0


def test_selftest_rejects_bad_limits(L):
    for bad in (0, -5, 10 ** 8):
        assert L.lq_selftest_dense_wait(bad, None) == lq.LQ_ERR_ARG
