"""What the 8-bit values of the quantiser and of the norm are rounded from (GPU): equal to the definition, not only within a step."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from fp64_gemm_emulation_gb300 import ozaki as oz

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


def each(s, block, rows, k):
    """Scales as one value an element, in 64 bits."""
    if block in ("row", "matrix"):
        s = s.repeat_interleave(128, -1)[..., :k]
    if block in ("column", "matrix"):
        s = s.repeat_interleave(128, -2)[..., :rows, :]
    return s.double()


def rounded(ratio, eight):
    """A quotient in 64 bits rounded to FP32 (twice rounded is as once: 53 >= 2 * 24 + 2 bits), then to 8 bits."""
    return ratio.float().to(eight).view(torch.uint8)


def quotients(x, block, eight):
    """x over its block's scale before that is rounded: largest value * x / amax, x * 2^126 where the scale is at its least."""
    rows, k = x.shape
    br, bk = {"row": (1, 128), "column": (128, 1), "matrix": (128, 128)}[block]
    p = torch.nn.functional.pad(x.double().abs(), (0, -k % bk, 0, -rows % br))
    amax = each(p.unflatten(-1, (-1, bk)).unflatten(-3, (-1, br)).amax(dim=(-3, -1)), block, rows, k)
    top = 448.0 if eight == E4M3 else 57344.0
    return torch.where(amax < top * 2.0 ** -126, x.double() * 2.0 ** 126, top * x.double() / amax.clamp(min=1e-300))


# multiples of a power of two meet the middle of two 8-bit values often; the others cover the range (1e-44 is below the normal one)
@pytest.mark.parametrize("dtype,size", [(torch.float16, 1.0)] + [(d, s) for d in (torch.bfloat16, torch.float32) for s in (1.0, 1e-44, 1e-36, 1e-20, 1e30, 1.5e38)])
@pytest.mark.parametrize("eight", [E4M3, E5M2])
def test_quantised_values_are_the_rounded_quotients(dtype, size, eight):
    gen = torch.Generator(device="cuda").manual_seed(3)
    rows, k = 300, 520
    for x in (torch.randint(-127, 128, (rows, k), generator=gen, device="cuda").float() / 128, torch.randn(rows, k, generator=gen, device="cuda").clamp(-2, 2)):
        for v in ((x * size).to(dtype), (x * size).to(dtype)[:, 3:518]):  # whole 16-byte pieces, and not
            for block in ("row", "column", "matrix"):
                q, s = oz.ozaki_quantize_f8(v, block, dtype=eight)
                want = rounded(quotients(v, block, eight), eight)
                assert torch.equal(q.contiguous().view(torch.uint8), want), (block, int((q.contiguous().view(torch.uint8) != want).sum()))
            for got, alone in zip(oz.ozaki_quantize_f8(v, "both", dtype=eight),
                                  (*oz.ozaki_quantize_f8(v, "row", dtype=eight), *oz.ozaki_quantize_f8(v, "column", dtype=eight))):
                assert torch.equal(got.float(), alone.float())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows,k", [(1, 4096), (7, 1001), (3000, 520), (5, 8200), (2, 32768)])
def test_normed_values_are_rounded_from_the_exact_ratio(rows, k, dtype):
    # h and h w are FP32 numbers here (small multiples of 2^-3), so q is the rounded 448 h w / (the block's largest), whatever
    # the roundings of the row's factor and of the scale: that ratio in 64 bits, rounded to FP32 and to 8 bits.
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, res = (torch.randint(-60, 61, (rows, k), generator=gen, device="cuda").to(dtype) / 8 for _ in range(2))
    w = torch.randint(1, 16, (k,), generator=gen, device="cuda").to(dtype) / 8
    x[0, :128], res[0, :128] = 0, 0
    q, s, _, rstd = oz.ozaki_rms_norm_f8(x, w, res)
    t = (x.double() + res.double()) * w.double()
    amax = torch.nn.functional.pad(t.abs(), (0, -k % 128)).unflatten(-1, (-1, 128)).amax(-1)
    ratio = 448 * t / each(torch.where(amax == 0, torch.ones_like(amax), amax), "row", rows, k)
    assert torch.equal(q.contiguous().view(torch.uint8) & 0x7F, rounded(ratio, E4M3) & 0x7F)
    # the scale: rstd as it was returned, a product and a quotient rounded
    want = torch.where(amax == 0, torch.ones_like(amax), amax * rstd.double()[:, None] / 448)
    assert ((s.double() - want).abs() <= 2 * 2.0 ** -24 * (1 + 2.0 ** -20) * want).all()


@pytest.mark.parametrize("size", [1e-30, 1e-18, 1e17])
def test_norm_of_rows_and_weights_far_from_one(size):
    # the row's sum: 16 squares a thread and 10 partial sums within 2^-18 (see the norm's own tests); h, y and the scale a rounding each
    x, w = torch.randn(40, 300, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)), torch.ones(300, device="cuda")
    for a, g in ((x * size, w), (x, w * size), (x / size ** 0.5, w * size), (x, w * 1e30)):
        eps = 0.0 if a.abs().max() > 1e-17 else 1e-38
        q, s, _, rstd = oz.ozaki_rms_norm_f8(a, g, eps=eps)
        r = 1 / torch.sqrt(a.double().square().mean(1, keepdim=True) + eps)
        if size == 1e-30 and a.abs().max() < 1e-20:  # the squares vanish: only eps is left
            r = torch.full_like(r, eps ** -0.5)
        y = a.double() * r * g.double()
        amax = torch.nn.functional.pad(y.abs(), (0, 84)).unflatten(-1, (-1, 128)).amax(-1)
        assert ((s.double() - amax / 448).abs() <= 2.0 ** -17 * amax / 448).all()
        back = q.double() * each(s, "row", 40, 300)
        assert ((back - y).abs() <= (2.0 ** -4 + 2.0 ** -16) * y.abs() + 2.0 ** -10 * each(s, "row", 40, 300)).all()
