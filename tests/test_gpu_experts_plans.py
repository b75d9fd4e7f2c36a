"""Expert products and Newton-Schulz at the tile plans of large problems (GPU).

Grouped products: integer operands in [-2, 2], whose sums are exact in FP32 (below 2^24), so that the result
is the exact sum rounded once and has to be equal.

Newton-Schulz against the definition in 64 bits, over the whole matrix and over its worst row and column:
  one slice   rounding X, S and B to FP16 in every step, worked out in 64 bits on matrices of the same kind
              (130 x 300 to 1000 x 1000, both orientations), gives 1.4e-3 to 1.8e-3, worst row or column 4.7e-3.
              Twice that.
  two slices  twice the error of the iteration in plain FP32 on the same input, and what the tensor core truncates: the
              four large additions of a k-block lose half an ulp (2^-24) each, which counts 2.5 times a product for
              the partial sums it falls on, in 3 products a step.  Three times that for a row or column.  Matrices
              that one CTA holds take S^2, which decides the error, out of the tensor core after every step: as a
              whole they are allowed no more than twice plain FP32.
A result of fewer than 32 bits is rounded once more.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from fp64_gemm_emulation_gb300 import ozaki as oz

COEFFS = (3.4445, -4.7750, 2.0315)
STEPS = 5
HALF_ULP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


@pytest.fixture(autouse=True)
def clean_status():
    oz.ozaki_get_device_status()
    yield
    assert oz.ozaki_get_device_status() == oz.OZ_OK


# ------------------------------------------------------------------ grouped products
def integers(*shape, dtype, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-2, 3, shape, generator=gen, device="cuda", dtype=torch.int8).to(dtype)


def check_exact(counts, n, k, dtype, before=0, after=0, ops="fdw", seed=0):
    offsets = [before]
    for c in counts:
        offsets.append(offsets[-1] + c)
    rows = offsets[-1] + after
    o = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    x, w, dy = (integers(*s, dtype=dtype, seed=seed + i) for i, s in enumerate(((rows, k), (len(counts), n, k), (rows, n))))
    y, dx = (torch.zeros(rows, f, dtype=torch.float64, device="cuda") for f in (n, k))
    dw = torch.zeros(len(counts), n, k, dtype=torch.float64, device="cuda")
    for e, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        if "f" in ops:
            y[lo:hi] = x[lo:hi].double() @ w[e].double().T
        if "d" in ops:
            dx[lo:hi] = dy[lo:hi].double() @ w[e].double()
        if "w" in ops:
            dw[e] = dy[lo:hi].double().T @ x[lo:hi].double()
    if "f" in ops:
        assert torch.equal(oz.ozaki_grouped_gemm(x, w, o), y.to(dtype)), "forward"
    if "d" in ops:
        assert torch.equal(oz.ozaki_grouped_gemm_dgrad(dy, w, o), dx.to(dtype)), "dgrad"
    if "w" in ops:
        assert torch.equal(oz.ozaki_grouped_gemm_wgrad(dy, x, o), dw.to(dtype)), "wgrad"


# 96 tiles in all: one wave of 76 pairs, and 20 tiles in parts
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("counts,n,k,ops", [
    ([700, 0, 1900, 33, 3000], 1024, 8192, "f"),
    ([700, 0, 1900, 33, 3000], 8192, 1024, "d"),
    ([9000, 5, 7000], 256, 8192, "w"),       # more parts than the middle group has k-blocks
])
def test_grouped_full_waves_and_parts(counts, n, k, ops, dtype):
    check_exact(counts, n, k, dtype, ops=ops)


@pytest.mark.parametrize("counts,n,k", [
    ([9000], 128, 64), ([4097, 4095], 72, 200), ([12289, 0, 63], 136, 328),  # parts whose borders are the group's
    ([64, 65, 63, 1, 128, 127, 129], 640, 512),
    ([257, 511, 513, 255, 1025], 1000, 1001),                               # no 16-byte row stride
    ([8192], 2048, 2048),
    ([3] * 200, 320, 384),
])
def test_grouped_borders(counts, n, k):
    check_exact(counts, n, k, torch.bfloat16, before=3, after=70)


@pytest.mark.parametrize("seed", range(6))
def test_grouped_drawn(seed):
    gen = torch.Generator().manual_seed(seed)

    def size(lo, hi):
        return int(lo * (hi / lo) ** float(torch.rand((), generator=gen)))

    groups = size(1, 40)
    counts = [size(1, 600) if torch.rand((), generator=gen) < 0.8 else 0 for _ in range(groups)]
    check_exact(counts, size(8, 1500), size(8, 1500), torch.bfloat16 if seed % 2 else torch.float16, before=size(1, 9) - 1,
                after=size(1, 300) - 1, seed=10 * seed)


# ------------------------------------------------------------------ Newton-Schulz
def momentum(b, m, n, seed=0):
    f = {"generator": torch.Generator(device="cuda").manual_seed(seed), "device": "cuda"}
    noise = torch.randn(b, m, n, **f) * torch.exp(0.5 * torch.randn(b, 1, n, **f))
    low = torch.randn(b, m, 4, **f) @ torch.randn(b, 4, n, **f)
    return noise + low * (noise.norm(dim=(1, 2), keepdim=True) / low.norm(dim=(1, 2), keepdim=True))


def iterate(g, dtype):
    """The definition, product by product, in `dtype`."""
    a, b, c = (float(v) for v in torch.tensor(COEFFS, dtype=torch.float32))
    x = g.to(dtype)
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2)
    x = x / x.square().sum(dim=(1, 2), keepdim=True).sqrt()
    for _ in range(STEPS):
        gram = x @ x.transpose(1, 2)
        x = a * x + (b * gram + c * gram @ gram) @ x
    return x.transpose(1, 2) if tall else x


def errors(got, ref):
    """Relative errors: the whole batch's, the worst row's and the worst column's."""
    diff, out = got.double() - ref, []
    for dim in ((0, 1, 2), 2, 1):
        out.append((torch.linalg.vector_norm(diff, dim=dim) / torch.linalg.vector_norm(ref, dim=dim)).max().item())
    return out


def check_newton(g, *, slices, dtypes, truncated):
    for dtype in dtypes:
        given = g.to(dtype)
        want = iterate(given, torch.float64)
        plain = errors(iterate(given, torch.float32), want) if 2 in slices else None
        for s in slices:
            got = errors(oz.ozaki_newton_schulz(given, steps=STEPS, coeffs=COEFFS, eps=0.0, num_slices=s), want)
            if s == 1:
                limits = [3.5e-3, 9.4e-3, 9.4e-3]
            else:
                cut = STEPS * 3 * 2.5 * 2.0 ** -24
                limits = [2 * plain[0] + truncated * cut, 2 * plain[1] + 3 * cut, 2 * plain[2] + 3 * cut]
            limits = [v + HALF_ULP[dtype] for v in limits]
            assert all(e <= v for e, v in zip(got, limits)), f"{dtype}, {s} slices: {got} > {limits}"


# The plans are those of 76 CTA pairs; widths are of the tiles of X X^T, S S and B X, one slice / two.
@pytest.mark.parametrize("b,m,n", [
    (24, 1024, 512),   # 128 256 256 / 128 128 128: several units a pair, several matrices in a wave
    (24, 512, 1024),   # the same, wide
    (1, 2048, 2048),   # 128 128 256 / 128
    (1, 2048, 8192),   # 128 128 256 / 128: four waves, seven waves
    (1, 8192, 2048),   # 128 128 224 / 128, tall
    (1, 1023, 2777),   # 64 64 192 / 64 64 96, odd
    (1, 2777, 1023),   # 128 in three parts, 64, 160
    (1, 4500, 1100),   # 160 in three parts across the rows, 64, 160 / 128 in two parts, 64, 160
    (1, 2500, 2400),   # 192 / a wave of whole tiles and one in two parts, 96, 128
    (40, 130, 300),    # 160: one tile a matrix, two for B X
    (40, 300, 130),
    (5, 900, 700),     # 128 128 192 / 128 128 160
    (4, 2500, 640),    # 128 96 256 / 128 96 160
    (1, 96, 9000),     # 64 in nine or eleven parts
    (1, 9000, 96),
])
def test_newton_schulz_plans(b, m, n):
    check_newton(momentum(b, m, n), slices=(1, 2), dtypes=(torch.float32,), truncated=True)


@pytest.mark.parametrize("b,m,n", [(24, 1024, 512), (1, 1500, 3000), (1, 2601, 655)])
def test_newton_schulz_plans_of_16_bits(b, m, n):
    check_newton(momentum(b, m, n, seed=3), slices=(1, 2), dtypes=(torch.bfloat16, torch.float16), truncated=True)


# matrices that one CTA holds: S^2 leaves the tensor core after every step
@pytest.mark.parametrize("b,m,n", [(64, 128, 128), (64, 100, 100), (64, 128, 256), (64, 255, 127), (64, 65, 200)])
def test_newton_schulz_small_is_as_exact_as_plain_fp32(b, m, n):
    check_newton(momentum(b, m, n), slices=(2,), dtypes=(torch.float32,), truncated=False)


@pytest.mark.parametrize("b,m,n", [(64, 128, 128), (200, 100, 500), (64, 512, 70)])
def test_newton_schulz_small_one_slice(b, m, n):
    check_newton(momentum(b, m, n), slices=(1,), dtypes=(torch.float32,), truncated=False)
