"""Expert products and Newton-Schulz as programs call them: workspaces, layouts, large values (GPU)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from fp64_gemm_emulation_gb300 import ozaki as oz


@pytest.fixture(autouse=True)
def clean_status():
    oz.ozaki_get_device_status()
    yield
    assert oz.ozaki_get_device_status() == oz.OZ_OK


def randn(*shape, dtype=torch.float32, seed=0):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


# ------------------------------------------------------------------ the norm's range
def test_newton_schulz_norm_of_many_large_values():
    # 2^28 values of 2^50: their squares add up to 2^128.  One step of the polynomial x leaves X_0, here exact.
    g = torch.randint(0, 2, (64, 1 << 22), device="cuda", dtype=torch.int8,
                      generator=torch.Generator(device="cuda").manual_seed(0)).to(torch.bfloat16)
    g.mul_(2.0 ** 51).sub_(2.0 ** 50)
    got = oz.ozaki_newton_schulz(g, steps=1, coeffs=(1.0, 0.0, 0.0), eps=0.0)
    assert torch.equal(got, g * 2.0 ** -64)


@pytest.mark.parametrize("m,n", [(90, 130), (300, 301)])
@pytest.mark.parametrize("power", [-120, -90, -50, 44, 45, 46, 50, 80, 120])
def test_newton_schulz_ranges_of_the_norm(m, n, power):
    # a power of two only moves values between the norm's ranges: the sums' rounding (2^-22) passes on at most 2^5 fold
    g = randn(m, n)
    want = oz.ozaki_newton_schulz(g, eps=0.0)
    got = oz.ozaki_newton_schulz(g * 2.0 ** power, eps=0.0)
    assert (got - want).norm() <= 2.0 ** -17 * want.norm()


# ------------------------------------------------------------------ workspaces
@pytest.mark.parametrize("slices", [1, 2])
@pytest.mark.parametrize("m,n", [(4096, 200), (200, 4096), (301, 129), (129, 301), (1001, 999)])
def test_newton_schulz_runs_in_the_workspace_that_its_shape_asks_for(m, n, slices):
    g = randn(m, n)
    ws = torch.empty(oz.ozaki_newton_schulz_workspace_bytes(m, n, 1, slices), dtype=torch.uint8, device="cuda")
    want = oz.ozaki_newton_schulz(g, num_slices=slices)
    assert torch.equal(oz.ozaki_newton_schulz_ws(g, ws, num_slices=slices), want)
    turned = g.t().contiguous().t()
    assert torch.equal(oz.ozaki_newton_schulz_ws(turned, ws, num_slices=slices), oz.ozaki_newton_schulz(turned, num_slices=slices))
    three = torch.stack([g, 2 * g, g])
    ws = torch.empty(oz.ozaki_newton_schulz_workspace_bytes(m, n, 3, slices), dtype=torch.uint8, device="cuda")
    assert torch.equal(oz.ozaki_newton_schulz_ws(three, ws, num_slices=slices), oz.ozaki_newton_schulz(three, num_slices=slices))


# ------------------------------------------------------------------ layouts
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [1, 7, 300])
def test_newton_schulz_one_row_of_a_column_major_matrix(n, dtype):
    # the norm's sum has another order: an ulp of bfloat16, and of FP32 after five steps a few
    ulp = {torch.bfloat16: 2.0 ** -7, torch.float32: 2.0 ** -19}[dtype]
    row = randn(n, 12, dtype=dtype)[:, 3:4].t()  # (1, n), its elements 12 apart
    want = oz.ozaki_newton_schulz(row.contiguous())
    assert ((oz.ozaki_newton_schulz(row) - want).abs() <= ulp * want.abs()).all()
    out = torch.zeros(n, 5, dtype=dtype, device="cuda")
    for g in (row, row.contiguous()):  # and into one
        out.zero_()
        oz.ozaki_newton_schulz(g, out=out[:, 2:3].t())
        assert ((out[:, 2:3].t() - want).abs() <= ulp * want.abs()).all() and (out[:, [0, 1, 3, 4]] == 0).all()
