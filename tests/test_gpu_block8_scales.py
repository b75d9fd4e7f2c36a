"""8-bit products with scales far from one (GPU).

Tolerance: rounding to bfloat16 (relative 2^-8, and half of its smallest step, 2^-134), and as in the products' own tests 2^-23 of the magnitudes
for each of the sum's additions, the scales' product and each block's addition.  Where a product of scales is below the normal range it is
off by up to 2^-150, times the unscaled magnitudes of the sum; FP32 sums below that range lose 2^-149 a block more.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from fp64_gemm_emulation_gb300 import ozaki as oz

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


@pytest.fixture(autouse=True)
def clean_status():
    oz.ozaki_get_device_status()
    yield
    assert oz.ozaki_get_device_status() == oz.OZ_OK


def check(got, ref, mag, raw, terms):
    """raw: the sum of the 8-bit values' magnitudes, without scales."""
    assert torch.isfinite(got).all()
    tol = 2.0 ** -8 * ref.abs() + (terms + terms / 32 + 4) * 2.0 ** -23 * mag * (1 + 2.0 ** -8) + 2.0 ** -134 + (terms / 128 + 1) * 2.0 ** -149
    tol = tol + 2.0 ** -150 * raw * (1 + 2.0 ** -7)
    bad = (got.double() - ref).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}"
    assert (ref.abs() > tol).any()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def eight_bit(rows, cols, size, dtype, seed):
    """Multiples of the type's smallest step about `size`, whole rows and columns of zeros among them."""
    t = torch.randn(rows, cols, generator=gen(seed), device="cuda") * size
    t[rows // 2] = 0
    t[:, cols // 3] = 0
    return t.clamp(-448, 448).to(dtype)


def scales(shape, power, spread, seed):
    e = torch.randint(power - spread, power + spread + 1, shape, generator=gen(seed), device="cuda")
    return torch.ldexp(1 + torch.rand(shape, generator=gen(seed + 1), device="cuda"), e)


def spread_out(s, block, rows, cols):
    if block in ("row", "matrix"):
        s = s.repeat_interleave(128, -1)[..., :cols]
    if block in ("column", "matrix"):
        s = s.repeat_interleave(128, -2)[..., :rows, :]
    return s.double()


# (size of the 8-bit values, powers of the two scales, their spread)
FAR = [(200.0, 60, -60, 2), (200.0, 100, -100, 2), (200.0, -100, 100, 2), (200.0, -100, -20, 2), (200.0, -50, -60, 10), (200.0, -126, 0, 0),  # normal products
       (2.0 ** -8, 60, 60, 2), (2.0 ** -8, 100, 20, 2), (2.0 ** -8, 127, -1, 0), (1.0, 0, 0, 58),
       (200.0, -70, -60, 1), (200.0, -90, -45, 2), (200.0, -60, -60, 20)]  # products below 2^-126, and some


@pytest.mark.parametrize("rows,n,k", [(300, 256, 384), (40, 208, 272), (513, 640, 128)])
@pytest.mark.parametrize("size,px,pw,spread", FAR)
@pytest.mark.parametrize("dtype", [E4M3, E5M2])
def test_products_of_scales_far_from_one(rows, n, k, size, px, pw, spread, dtype):
    # operands that are large where products are small, and the other way round: no result leaves the range of bfloat16
    w = eight_bit(n, k, size, E4M3, 1)
    ws = scales(((n + 127) // 128, (k + 127) // 128), pw, spread, 2)
    W = w.double() * spread_out(ws, "matrix", n, k)
    x = eight_bit(rows, k, size, dtype, 3)
    xs = scales(((k + 127) // 128, rows), px, spread, 4).t()
    X = x.double() * spread_out(xs, "row", rows, k)
    check(oz.ozaki_grouped_gemm_f8(x, xs, w, ws), X @ W.T, X.abs() @ W.T.abs(), x.double().abs() @ w.double().T.abs(), k)
    y = eight_bit(rows, n, size, dtype, 5)
    ys = scales(((n + 127) // 128, rows), px, spread, 6).t()
    Y = y.double() * spread_out(ys, "row", rows, n)
    check(oz.ozaki_grouped_gemm_f8_dgrad(y, ys, w, ws), Y @ W, Y.abs() @ W.abs(), y.double().abs() @ w.double().abs(), n)
    blocks = (rows + 127) // 128
    xc, yc = scales((blocks, k), px, spread, 7), scales((blocks, n), pw, spread, 8)
    X, Y = x.double() * spread_out(xc, "column", rows, k), y.double() * spread_out(yc, "column", rows, n)
    check(oz.ozaki_grouped_gemm_f8_wgrad(y, yc, x, xc)[0], Y.T @ X, Y.T.abs() @ X.abs(), y.double().T.abs() @ x.double().abs(), rows)


def test_scales_of_zero_and_inf_are_multiplied_as_they_are():
    x, w = torch.ones(200, 256, device="cuda").to(E4M3), torch.ones(256, 256, device="cuda").to(E4M3)
    xs, ws = torch.ones(2, 200, device="cuda").t(), torch.ones(2, 2, device="cuda")
    xs[3, 0], xs[5, 1], xs[7, 0], xs[9] = 0, float("inf"), float("nan"), 0
    y = oz.ozaki_grouped_gemm_f8(x, xs, w, ws)
    assert (y[3] == 128).all() and torch.isinf(y[5]).all() and torch.isnan(y[7]).all() and (y[9] == 0).all() and (y[10:] == 256).all()
    xc, wc = torch.ones(2, 256, device="cuda"), torch.ones(2, 256, device="cuda")
    xc[0, 3], xc[1, 5], xc[0, 7], xc[:, 9] = 0, float("inf"), float("nan"), 0
    d = oz.ozaki_grouped_gemm_f8_wgrad(x, wc, x, xc)[0]
    assert (d[:, 3] == 72).all() and torch.isinf(d[:, 5]).all() and torch.isnan(d[:, 7]).all() and (d[:, 9] == 0).all() and (d[:, 10:] == 200).all()
