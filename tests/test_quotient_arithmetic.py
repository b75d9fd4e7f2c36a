"""The quotient that is rounded to 8 bits, restated on the CPU: v a / b formed as v y + v rest.

For a 16-bit v (8 or 11 significant bits) and its block's largest magnitude, of as many bits, the 8-bit result must be that of the exact
quotient, ties included.  Only significands matter (no step leaves the range of FP32), so all pairs of them are tried, in every
binade of the 8-bit types.
"""
import numpy as np
import pytest
import torch

F, D = np.float32, np.float64
TYPES = [(torch.float8_e4m3fn, 448.0, 20), (torch.float8_e5m2, 57344.0, 34)]


def quotient(a, b, near):
    """a / b as y + rest, as the kernels form it; near: FP32 within 2^-23 of b / a."""
    y = F(1) / near
    for _ in range(3):
        y = np.nextafter(y, F(0))
    lost = (a - y.astype(D) * b).astype(F)  # (48 bits, next to a: exact in 64)
    return y, lost * (y * F(1 / a))


def times(v, y, rest):
    p, t = v.astype(D) * y, (v * rest).astype(D)  # exact: 11 + 24 bits
    s = p + t
    lost = (t - (s - p)) + (p - (s - (s - p)))
    q = s.astype(F)
    # Rounded twice: where the sum lies in the middle of two FP32 numbers, what the first rounding lost decides.
    tie = (lost != 0) & (np.abs(s - q) * 2 == np.spacing(np.abs(q)).astype(D))
    return np.where(tie, np.nextafter(s, s + np.sign(lost)), s).astype(F)


def eight(x, dtype):
    return torch.from_numpy(x.astype(F)).to(dtype).view(torch.uint8).numpy()


@pytest.mark.parametrize("dtype,largest,binades", TYPES)
@pytest.mark.parametrize("bits", [8, 11])
def test_all_significands_go_the_way_of_the_exact_quotient(bits, dtype, largest, binades):
    n = 1 << (bits - 1)
    grid = (n + np.arange(n)).astype(F)
    v = np.concatenate([grid * F(2.0 ** -b) for b in range(binades)])
    for amax in grid[::1 if bits == 8 else 5]:
        near = np.array([amax / F(largest)], F)  # the scale
        y, rest = quotient(D(largest), np.array([amax]), near)
        some = v[v <= amax]
        want = (some.astype(D) * largest / D(amax)).astype(F)  # (8 or 11 by 8 or 11 bits: no FP32 neighbour of a middle is met)
        assert np.array_equal(eight(times(some, y, rest), dtype), eight(want, dtype)), amax


@pytest.mark.parametrize("a", [1.0, 448.0, 57344.0])
def test_fp32_values_within_their_bound(a):
    rng = np.random.default_rng(0)
    v, b = (rng.uniform(1, 2, 1 << 20).astype(F) for _ in range(2))
    for near in (b / F(a), b * F(1 / a)):
        y, rest = quotient(D(a), b, near)
        assert (rest >= 0).all()  # so that a v of -0 stays one
        exact = v.astype(D) * a / b
        # rest is at most 6 steps of 2^-23 of y, and off by as much of itself and four roundings: 6^2 2^-46 + 4 * 6 * 2^-47 < 2^-40.
        # v y is left out of both sides where 64 bits would round it: y a + rest against a / b, and the rounding of v rest
        off = np.abs((a - y.astype(D) * b) / b - rest) / (a / b.astype(D)) + np.abs((v * rest).astype(D) - v.astype(D) * rest) / exact
        assert (off <= 2.0 ** -40).all()
