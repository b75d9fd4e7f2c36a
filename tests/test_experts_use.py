"""Host-side queries and checks of the expert products and Newton-Schulz as programs use them (no GPU call is made)."""
import pytest

from fp64_gemm_emulation_gb300 import ozaki as oz


@pytest.mark.parametrize("batch", [1, 5])
@pytest.mark.parametrize("slices", [1, 2])
@pytest.mark.parametrize("m,n", [(4096, 200), (200, 4096), (301, 129), (129, 301), (1001, 999), (640, 640), (100, 90)])
def test_newton_schulz_workspace_serves_both_layouts(m, n, slices, batch):
    # a row-major (m, n) matrix is n x m in C, a column-major one m x n
    got = oz.ozaki_newton_schulz_workspace_bytes(m, n, batch, slices)
    assert got >= oz._lib.ozaki_newton_schulz_workspace_bytes(n, m, batch, slices)
    assert got >= oz._lib.ozaki_newton_schulz_workspace_bytes(m, n, batch, slices)
    assert got == oz.ozaki_newton_schulz_workspace_bytes(n, m, batch, slices)
