"""The weights' gradient refuses row counts whose tiles pass 32 bits (multiples of 16 all)."""
import pytest

from tests.test_fp8_host import L, M, wgrad  # noqa: F401


@pytest.mark.parametrize("R", [(1 << 31) - 112, (1 << 31) - 64, (1 << 31) - 16, 1 << 31, 1 << 40])
def test_wgrad_refuses_rows_that_tiles_count_past_32_bits(L, R):  # noqa: F811
    assert R % 16 == 0
    assert wgrad(L, R=R, M=8, N=8, G=1) == 2
    assert b"R" in L.mhc_last_error()


def test_wgrad_accepts_the_most_rows_without_gpu(L):  # noqa: F811
    assert wgrad(L, R=(1 << 31) - 128, M=8, N=8, G=1) in (7, 8)
