"""Host-side: the norm takes every finite eps >= 0 (calls without rows, which
launch nothing)."""
import pytest

from moe_grouped_gemm_ragged_amd import binding as gg

A = 0x10000       # 16-byte aligned, never read


@pytest.mark.parametrize("eps", [0.0, 1e-45, 1e-6, 1.0, 3.0e38, 3.2e38, 3.4028234e38])
def test_every_finite_eps(eps):
    assert gg.call_raw("gg_rmsnorm", None, None, A, None, None, None, None, 0, 64, eps, None) == 0, gg.last_error()
