"""8-bit quantisation and products, RMS norm and clipping against their definitions in 64 bits (GPU).

Tolerances.  Rounding to nearest is off by at most half a step: relative 2^-4 (e4m3), 2^-3 (e5m2), 2^-8 (bfloat16),
2^-11 (float16), 2^-24 (float32), and half of the smallest step below the normal range (2^-10, 2^-17 for the 8-bit types, 2^-25
for float16).  An FP32 sum of K terms that loses at most 2^-23 of the running sum of magnitudes at each addition is off
by less than K 2^-23 of the sum of magnitudes; a scale's product and the scaled addition of each block of 128 add three roundings.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from fp64_gemm_emulation_gb300 import ozaki as oz

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
LARGEST = {E4M3: 448.0, E5M2: 57344.0}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24, E4M3: 2.0 ** -4, E5M2: 2.0 ** -3}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0, E4M3: 2.0 ** -10, E5M2: 2.0 ** -17}


@pytest.fixture(autouse=True)
def clean_status():
    oz.ozaki_get_device_status()
    yield
    assert oz.ozaki_get_device_status() == oz.OZ_OK


def randn(*shape, dtype=torch.float32, seed=0, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


def offsets_of(counts, before=0):
    out = [before]
    for c in counts:
        out.append(out[-1] + c)
    return torch.tensor(out, dtype=torch.int32, device="cuda"), out


def per_block(s, block, rows, k):
    """Scales as one value an element."""
    if block in ("row", "matrix"):
        s = s.repeat_interleave(128, -1)[..., :k]
    if block in ("column", "matrix"):
        s = s.repeat_interleave(128, -2)[..., :rows, :]
    return s.double()


def block_max(x, block):
    rows, k = x.shape[-2:]
    br, bk = {"row": (1, 128), "column": (128, 1), "matrix": (128, 128)}[block]
    p = torch.nn.functional.pad(x.double().abs(), (0, -k % bk, 0, -rows % br))
    return p.unflatten(-1, (-1, bk)).unflatten(-3, (-1, br)).amax(dim=(-3, -1))


def check_quantised(q, s, x, block):
    amax = block_max(x, block)
    want = torch.where(amax == 0, torch.ones_like(amax), (amax / LARGEST[q.dtype]).clamp(min=2.0 ** -126)).float()
    assert torch.equal(s, want)
    ratio = x.double() / per_block(s, block, *x.shape[-2:])
    off = (q.double() - ratio).abs()
    tol = torch.maximum(HALF[q.dtype] * ratio.abs(), torch.full_like(ratio, TINY[q.dtype])) * (1 + 2.0 ** -20)
    assert (off <= tol).all(), f"{int((off > tol).sum())} of {off.numel()} off"


def by_group(x, offsets, fill=0):
    """x's rows where column blocks of each group start."""
    rows, groups = x.shape[0], len(offsets) - 1
    p = torch.full((128 * (rows // 128 + groups), x.shape[1]), fill, dtype=x.dtype, device=x.device)
    for e, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        at = 128 * (lo // 128 + e)
        p[at:at + hi - lo] = x[lo:hi]
    return p


# ------------------------------------------------------------------ quantisation
SHAPES = [(1, 1), (1, 128), (3, 129), (128, 128), (127, 16), (130, 2000), (500, 77), (257, 384), (64, 4104)]


@pytest.mark.parametrize("eight", [E4M3, E5M2])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows,k", SHAPES)
def test_quantise(rows, k, dtype, eight):
    x = randn(rows, k, dtype=dtype) * torch.exp2(torch.randint(-8, 8, (k,), generator=torch.Generator().manual_seed(1)).float()).cuda().to(dtype)
    for block in ("row", "column", "matrix"):
        q, s = oz.ozaki_quantize_f8(x, block, dtype=eight)
        assert q.dtype == eight and q.shape == x.shape
        check_quantised(q, s, x, block)
    q, s, qc, sc = oz.ozaki_quantize_f8(x, "both", dtype=eight)
    for got, want in zip((q, s, qc, sc), (*oz.ozaki_quantize_f8(x, "row", dtype=eight), *oz.ozaki_quantize_f8(x, "column", dtype=eight))):
        assert torch.equal(got.float(), want.float())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(3, 100, 200), (2, 2, 130, 129), (5, 1, 33)])
def test_quantise_batches_of_matrices(shape, dtype):
    x = randn(*shape, dtype=dtype)
    q, s = oz.ozaki_quantize_f8(x, "matrix")
    check_quantised(q, s, x, "matrix")


@pytest.mark.parametrize("counts,before,after", [([300], 0, 0), ([0, 0, 5], 0, 0), ([128, 1, 0, 127, 129, 256], 0, 0), ([33] * 40, 0, 0),
                                                 ([100, 0, 300], 37, 270), ([0], 130, 140), ([1] * 300, 0, 0)])
@pytest.mark.parametrize("k", [40, 257])
def test_quantise_by_group(counts, before, after, k):
    o, offsets = offsets_of(counts, before)
    x = randn(offsets[-1] + after, k, dtype=torch.bfloat16)
    q, s, qc, sc = oz.ozaki_quantize_f8(x, "both", o, E5M2)
    check_quantised(q, s, x, "row")
    laid = by_group(x, offsets)
    assert qc.shape == laid.shape and sc.shape == (oz.ozaki_f8_column_blocks(x.shape[0], len(counts)), k)
    check_quantised(qc, sc, laid, "column")
    q2, s2 = oz.ozaki_quantize_f8(x, "column", o, E5M2)
    assert torch.equal(q2.float(), qc.float()) and torch.equal(s2, sc)
    q2, s2 = oz.ozaki_quantize_f8(x, "row", o, E5M2)
    assert torch.equal(q2.float(), q.float()) and torch.equal(s2, s)


def test_quantise_strided_rows_and_extreme_values():
    big = randn(70, 300)
    x = big[:, 3:260]
    check_quantised(*oz.ozaki_quantize_f8(x, "row"), x, "row")
    check_quantised(*oz.ozaki_quantize_f8(x[::2], "column"), x[::2], "column")
    for v in (0.0, 1e-45, 1e-38, 3e-37, 3.3e38):
        x = torch.full((2, 130), v, device="cuda")
        for block in ("row", "column", "matrix"):
            check_quantised(*oz.ozaki_quantize_f8(x, block), x, block)


def test_quantise_inf_and_nan_stay_in_their_block():
    for bad in (float("inf"), float("-inf"), float("nan")):
        for block in ("row", "column", "matrix"):
            x = randn(256, 256)
            clean_q, clean_s = oz.ozaki_quantize_f8(x, block)
            x[5, 7] = bad
            q, s = oz.ozaki_quantize_f8(x, block)
            wrong = ~torch.isfinite(s)
            assert wrong.sum() == 1
            same = ~per_block(wrong.float(), block, 256, 256).bool()
            assert torch.equal(q.float()[same], clean_q.float()[same]) and torch.equal(s[~wrong], clean_s[~wrong])
            assert not torch.isfinite(q.float()[5, 7] * per_block(s, block, 256, 256)[5, 7])


# ------------------------------------------------------------------ products
def check(got, ref, mag, terms, what):
    tol = HALF[got.dtype] * ref.abs() + (terms + terms / 32 + 4) * 2.0 ** -23 * mag * (1 + HALF[got.dtype]) + 2.0 ** -25
    bad = (got.double() - ref).abs() > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}"


def values(q, s, block):
    return q.double() * per_block(s, block, *q.shape[-2:])


def check_products(counts, n, k, types=(E4M3, E4M3, E4M3), out=torch.bfloat16, before=0, after=0, dense=False, seed=0):
    """types: of x, w and dy."""
    o, offsets = offsets_of(counts, before)
    rows, groups = offsets[-1] + after, len(counts)
    if dense:
        o = None
    tx, tw, tdy = types
    x, w, dy = randn(rows, k, seed=seed), randn(groups, n, k, seed=seed + 1, scale=max(1, k) ** -0.5), randn(rows, n, seed=seed + 2, scale=0.1)
    xq, xs = oz.ozaki_quantize_f8(x, "row", dtype=tx)
    wq, ws = oz.ozaki_quantize_f8(w, "matrix", dtype=tw)
    dq, ds, dqc, dsc = oz.ozaki_quantize_f8(dy, "both", o, tdy)
    xqc, xsc = oz.ozaki_quantize_f8(x, "column", o, tx)
    X, W, D = values(xq, xs, "row"), values(wq, ws, "matrix"), values(dq, ds, "row")
    XC, DC = values(xqc, xsc, "column"), values(dqc, dsc, "column")
    y, my = torch.zeros(2, rows, n, dtype=torch.float64, device="cuda")
    dx, mdx = torch.zeros(2, rows, k, dtype=torch.float64, device="cuda")
    dw, mdw = torch.zeros(2, groups, n, k, dtype=torch.float64, device="cuda")
    for e, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        at = slice(lo, hi) if dense else slice(128 * (lo // 128 + e), 128 * (lo // 128 + e) + hi - lo)
        y[lo:hi], my[lo:hi] = X[lo:hi] @ W[e].T, X[lo:hi].abs() @ W[e].T.abs()
        dx[lo:hi], mdx[lo:hi] = D[lo:hi] @ W[e], D[lo:hi].abs() @ W[e].abs()
        dw[e], mdw[e] = DC[at].T @ XC[at], DC[at].T.abs() @ XC[at].abs()
    check(oz.ozaki_grouped_gemm_f8(xq, xs, wq, ws, o, dtype=out), y, my, k, "forward")
    check(oz.ozaki_grouped_gemm_f8_dgrad(dq, ds, wq, ws, o, dtype=out), dx, mdx, n, "dgrad")
    check(oz.ozaki_grouped_gemm_f8_wgrad(dqc, dsc, xqc, xsc, o, dtype=out), dw, mdw, max(counts, default=0), "wgrad")


@pytest.mark.parametrize("rows,n,k", [(1, 1, 1), (1, 16, 128), (1, 300, 1000), (7, 256, 128), (31, 129, 127), (32, 128, 4096), (33, 100, 264), (128, 128, 128),
                                      (129, 257, 385), (256, 256, 256), (257, 512, 96), (1000, 520, 520), (2048, 64, 2048)])
def test_dense_products(rows, n, k):
    check_products([rows], n, k, dense=True)


@pytest.mark.parametrize("counts,n,k", [
    ([1, 1, 1], 3, 5),
    ([255, 256, 257], 256, 128),
    ([0, 0, 0], 64, 64),
    ([0, 513, 0, 31, 1, 0], 320, 192),
    ([63, 64, 65, 127, 128, 129], 129, 127),
    ([300, 20], 1000, 264),
    ([33] * 40, 96, 72),
    ([5, 700, 1, 0, 33], 517, 1001),
    ([8] * 64, 300, 200),
])
def test_grouped_products(counts, n, k):
    check_products(counts, n, k)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("types", [(E4M3, E4M3, E5M2), (E5M2, E4M3, E4M3), (E4M3, E5M2, E5M2), (E5M2, E5M2, E5M2)])
def test_products_of_both_types(types, out):
    check_products([200, 0, 90], 264, 300, types, out)


def test_products_rows_outside_every_group():
    check_products([40, 0, 300], 192, 320, before=37, after=270)
    check_products([0, 0], 40, 50, before=300, after=1)


def test_products_most_groups():
    check_products([(e * 7) % 5 for e in range(oz.OZ_MAX_GROUPS)], 64, 96)


def test_products_of_many_tiles():
    check_products([3000, 1, 1500], 2000, 1400)


def test_products_take_any_scales():
    rows, n, k = 300, 200, 400
    xq, xs = oz.ozaki_quantize_f8(randn(rows, k), "row")
    wq, ws = oz.ozaki_quantize_f8(randn(n, k, seed=1), "matrix")
    gen = torch.Generator(device="cuda").manual_seed(2)
    xs = (torch.exp(3 * torch.randn(4, rows, device="cuda", generator=gen))).t()
    ws = -torch.exp(3 * torch.randn(2, 4, device="cuda", generator=gen))
    X, W = values(xq, xs, "row"), values(wq, ws, "matrix")
    check(oz.ozaki_grouped_gemm_f8(xq, xs, wq, ws), X @ W.T, X.abs() @ W.T.abs(), k, "forward")


def test_products_strided_operands_and_outputs_keep_their_padding():
    counts, n, k = [70, 0, 200, 33], 208, 144
    o, offsets = offsets_of(counts)
    rows = offsets[-1]
    x, w, dy = randn(rows, k), randn(4, n, k, seed=1), randn(rows, n, seed=2)
    xq, xs = oz.ozaki_quantize_f8(x, "row")
    wq, ws = oz.ozaki_quantize_f8(w, "matrix")
    dq, ds, dqc, dsc = oz.ozaki_quantize_f8(dy, "both", o)
    xqc, xsc = oz.ozaki_quantize_f8(x, "column", o)

    def strided(t, pad):  # the padding is NaN for operands, which must not be read
        big = torch.full((*t.shape[:-1], t.shape[-1] + pad), float("nan"), device="cuda").to(t.dtype)
        big[..., :t.shape[-1]] = t
        return big[..., :t.shape[-1]]

    def colmajor(s):
        return strided(s.t(), 5).t()

    for pad in (8, 3):
        outs = [torch.full(shape, 7.0, dtype=torch.bfloat16, device="cuda") for shape in ((rows, n + pad), (rows, k + pad), (4, n, k + pad))]
        y, dx, dw = outs[0][:, :n], outs[1][:, :k], outs[2][..., :k]
        oz.ozaki_grouped_gemm_f8(strided(xq, 16), colmajor(xs), strided(wq, 32), ws, o, Y=y)
        oz.ozaki_grouped_gemm_f8_dgrad(strided(dq, 48), colmajor(ds), strided(wq, 16), ws, o, dX=dx)
        oz.ozaki_grouped_gemm_f8_wgrad(strided(dqc, 16), strided(dsc, 3), strided(xqc, 64), strided(xsc, 1), o, dW=dw)
        assert torch.equal(y, oz.ozaki_grouped_gemm_f8(xq, xs, wq, ws, o))
        assert torch.equal(dx, oz.ozaki_grouped_gemm_f8_dgrad(dq, ds, wq, ws, o))
        assert torch.equal(dw, oz.ozaki_grouped_gemm_f8_wgrad(dqc, dsc, xqc, xsc, o))
        assert all((t[..., -pad:] == 7.0).all() for t in outs)


def test_products_empty_sums_give_zeros():
    q = torch.empty(5, 0, dtype=E4M3, device="cuda")
    w = torch.empty(2, 6, 0, dtype=E4M3, device="cuda")
    o, _ = offsets_of([3, 2])
    s, sw = torch.empty(5, 0, device="cuda"), torch.empty(2, 1, 0, device="cuda")
    assert (oz.ozaki_grouped_gemm_f8(q, s, w, sw, o, Y=torch.ones(5, 6, dtype=torch.bfloat16, device="cuda")) == 0).all()
    none = torch.empty(0, 32, dtype=E4M3, device="cuda")
    dw = oz.ozaki_grouped_gemm_f8_wgrad(none, torch.empty(0, 32, device="cuda"), none, torch.empty(0, 32, device="cuda"),
                                        dW=torch.ones(1, 32, 32, dtype=torch.bfloat16, device="cuda"))
    assert (dw == 0).all()
    assert oz.ozaki_grouped_gemm_f8(none, torch.empty(1, 0, device="cuda").t(), torch.empty(7, 32, dtype=E4M3, device="cuda"),
                                    torch.ones(1, 1, device="cuda")).shape == (0, 7)


def test_products_nan_stays_in_its_rows_group_and_block():
    counts, n, k = [100, 90], 300, 300
    o, offsets = offsets_of(counts)
    x, w = randn(190, k), randn(2, n, k, seed=1)
    clean = oz.ozaki_grouped_gemm_f8(*oz.ozaki_quantize_f8(x, "row"), *oz.ozaki_quantize_f8(w, "matrix"), o)
    x[99, 5] = float("nan")
    w[1, 130, 0] = float("inf")
    got = oz.ozaki_grouped_gemm_f8(*oz.ozaki_quantize_f8(x, "row"), *oz.ozaki_quantize_f8(w, "matrix"), o)
    hit = torch.zeros(190, n, dtype=torch.bool, device="cuda")
    hit[99] = True
    hit[100:, 128:256] = True
    assert not torch.isfinite(got[hit]).any() and torch.equal(got[~hit], clean[~hit])
    dy = randn(190, n, seed=2)
    xc = oz.ozaki_quantize_f8(x, "column", o)
    dw = oz.ozaki_grouped_gemm_f8_wgrad(*oz.ozaki_quantize_f8(dy, "column", o), *xc, o)
    assert not torch.isfinite(dw[0, :, 5]).any()
    keep = torch.ones(2, n, k, dtype=torch.bool, device="cuda")
    keep[0, :, 5] = False
    assert torch.isfinite(dw[keep]).all()


def test_bad_offsets_are_clamped_and_reported():
    x, w = oz.ozaki_quantize_f8(randn(100, 64), "row"), oz.ozaki_quantize_f8(randn(3, 32, 64, seed=1), "matrix")
    bad, good = torch.tensor([-5, 60, 40, 1000], dtype=torch.int32, device="cuda"), torch.tensor([0, 60, 60, 100], dtype=torch.int32, device="cuda")
    got = oz.ozaki_grouped_gemm_f8(*x, *w, bad)
    assert oz.ozaki_get_device_status() == oz.OZ_EINVAL
    assert torch.equal(got, oz.ozaki_grouped_gemm_f8(*x, *w, good))
    got = oz.ozaki_quantize_f8(randn(100, 64), "both", bad)
    assert oz.ozaki_get_device_status() == oz.OZ_EINVAL
    for a, b in zip(got, oz.ozaki_quantize_f8(randn(100, 64), "both", good)):
        assert torch.equal(a.float(), b.float())


# ------------------------------------------------------------------ norm
WIDTHS = [(1, 1), (5, 8), (3, 100), (9, 129), (4, 256), (300, 264), (7, 1001), (2, 2048), (700, 520), (3, 8192), (5, 8200), (2, 16391), (3, 32768), (2, 32761)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows,k", WIDTHS)
@pytest.mark.parametrize("with_residual", [True, False])
def test_norm(rows, k, dtype, with_residual):
    # a thread adds at most 32 squares and 10 partial sums follow: the sum is within 42 * 2^-24, rstd within half of that and 3 more,
    # y within 4 roundings more: 2^-18 covers all of them
    x, w = randn(rows, k, dtype=dtype), (1 + randn(k, seed=1, scale=0.2)).to(dtype)
    res = randn(rows, k, dtype=dtype, seed=2, scale=3.0) if with_residual else None
    y_out = torch.empty_like(x)
    q, s, h_out, rstd = oz.ozaki_rms_norm_f8(x, w, res, 1e-5, Y=y_out)
    h = x.double() + (res.double() if with_residual else 0)
    r = 1 / torch.sqrt(h.square().mean(1) + 1e-5)
    y = h * r[:, None] * w.double()
    near = 2.0 ** -18
    assert ((rstd.double() - r).abs() <= near * r).all()
    assert ((h_out.double() - h).abs() <= (HALF[dtype] + 2.0 ** -23) * h.abs() + TINY[dtype]).all()
    assert ((y_out.double() - y).abs() <= (HALF[dtype] + near) * y.abs() + TINY[dtype]).all()
    amax = block_max(y, "row")
    assert ((s.double() - amax / 448).abs() <= 2 * near * amax / 448).all()
    ratio = y / per_block(s, "row", rows, k)
    tol = torch.maximum(HALF[E4M3] * ratio.abs(), torch.full_like(ratio, TINY[E4M3])) + 2 * near * ratio.abs()
    assert ((q.double() - ratio).abs() <= tol).all()
    assert h_out is x if not with_residual else True


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows,k", WIDTHS + [(2000, 64), (1500, 1000)])
@pytest.mark.parametrize("with_dh", [True, False])
def test_norm_backward(rows, k, dtype, with_dh):
    # dot: as the norm's sum; dw: any order of rows' sums is within (rows - 1) 2^-24 of the magnitudes
    h, w, dy = randn(rows, k, dtype=dtype, scale=2.0), (1 + randn(k, seed=1, scale=0.2)).to(dtype), randn(rows, k, dtype=dtype, seed=2)
    dh = randn(rows, k, dtype=dtype, seed=3) if with_dh else None
    rstd = (1 / torch.sqrt(h.double().square().mean(1) + 1e-5)).float()
    dx, dw = oz.ozaki_rms_norm_backward(dy, h, w, rstd, dh)
    H, W, D, r = h.double(), w.double(), dy.double(), rstd.double()[:, None]
    g = D * W
    want = r * (g - H * r.square() * (g * H).mean(1, keepdim=True)) + (dh.double() if with_dh else 0)
    mag = r * (g.abs() + H.abs() * r.square() * (g * H).abs().mean(1, keepdim=True)) + (dh.double().abs() if with_dh else 0)
    assert ((dx.double() - want).abs() <= HALF[dtype] * want.abs() + 2.0 ** -17 * mag + TINY[dtype]).all()
    z = D * H * r
    assert ((dw.double() - z.sum(0)).abs() <= HALF[dtype] * z.sum(0).abs() + (rows + 4) * 2.0 ** -24 * (1 + HALF[dtype]) * z.abs().sum(0) + TINY[dtype]).all()


# many rows a CTA (they are fetched ahead): whole pieces, rows that start anywhere, one and two runs a thread, several rows in 16 bytes
@pytest.mark.parametrize("rows, k, pad", [(2600, 520, 0), (2600, 513, 0), (5000, 3, 0), (5000, 1, 0), (1500, 4096, 8), (1500, 4095, 3), (500, 8200, 0), (500, 8193, 1), (400, 16384, 0)])
def test_norm_backward_of_many_rows(rows, k, pad):
    dtype = torch.bfloat16
    dy, h, dh = (torch.full((rows * (k + pad) + 9,), float("nan"), dtype=dtype, device="cuda")[1:1 + rows * (k + pad)].view(rows, k + pad)[:, :k] if k % 8 else
                 torch.full((rows, k + pad), float("nan"), dtype=dtype, device="cuda")[:, :k] for _ in range(3))
    for i, t in enumerate((dy, h, dh)):
        t.copy_(randn(rows, k, dtype=dtype, seed=i))
        t[5::7] = float("nan")  # each row's neighbours
    w = (1 + randn(k, seed=4, scale=0.2)).to(dtype)
    rstd = 1 + torch.rand(rows, generator=torch.Generator().manual_seed(1)).cuda()
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[5::7] = False
    H, W, D, r = h[keep].double(), w.double(), dy[keep].double(), rstd[keep].double()[:, None]
    g = D * W
    want = r * (g - H * r.square() * (g * H).mean(1, keepdim=True)) + dh[keep].double()
    mag = r * (g.abs() + H.abs() * r.square() * (g * H).abs().mean(1, keepdim=True)) + dh[keep].double().abs()
    for to in (None, dh):  # into dH itself at last
        dx, _ = oz.ozaki_rms_norm_backward(dy, h, w, rstd, dh, dX=to)
        assert ((dx[keep].double() - want).abs() <= HALF[dtype] * want.abs() + 2.0 ** -17 * mag + TINY[dtype]).all()
        assert torch.isnan(dx[~keep]).all()
    for t in (dy, h):
        t[5::7] = 0
    _, dw = oz.ozaki_rms_norm_backward(dy, h, w, rstd)
    z = dy.double() * h.double() * rstd.double()[:, None]
    assert ((dw.double() - z.sum(0)).abs() <= HALF[dtype] * z.sum(0).abs() + (rows + 4) * 2.0 ** -24 * (1 + HALF[dtype]) * z.abs().sum(0) + TINY[dtype]).all()


def test_norm_backward_is_the_derivative():
    # differences of the loss sum(c y) + sum(d h) in 64 bits
    rows, k = 6, 200
    x, w, c, d = (randn(*s, seed=i).double() for i, s in enumerate([(rows, k), (k,), (rows, k), (rows, k)]))
    x, w = x.float().double().requires_grad_(), w.float().double().requires_grad_()
    c, d = c.float().double(), d.float().double()

    def loss(x, w):
        return (c * x * (x.square().mean(1, keepdim=True) + 1e-6).rsqrt() * w).sum() + (d * x).sum()

    _, _, h, rstd = oz.ozaki_rms_norm_f8(x.detach().float(), w.detach().float())
    dx, dw = oz.ozaki_rms_norm_backward(c.float(), h, w.detach().float(), rstd, d.float())
    step = 1e-5
    for t, grad in ((x, dx), (w, dw)):
        for at in [(0,) * t.dim(), tuple(s - 1 for s in t.shape), tuple(s // 2 for s in t.shape)]:
            with torch.no_grad():
                v = t[at].item()
                t[at] = v + step
                up = loss(x, w)
                t[at] = v - step
                down = loss(x, w)
                t[at] = v
            # a central difference's error is step^2 / 6 of the third derivative (below 1e3 here), and 1e-16 * |loss| / step
            assert abs((up - down).item() / (2 * step) - grad[at].item()) <= 1e-6 + 2.0 ** -17 * (abs(grad[at].item()) + 10)


def test_norm_in_place_and_strided():
    for k, pad in ((520, 8), (333, 5)):
        x, res, w = randn(40, k + pad, dtype=torch.bfloat16)[:, :k], randn(40, k, dtype=torch.bfloat16, seed=1), randn(k, dtype=torch.bfloat16, seed=2)
        want = oz.ozaki_rms_norm_f8(x.contiguous(), w, res)
        buf = res.clone()
        got = oz.ozaki_rms_norm_f8(x, w, buf, H=buf)
        assert got[2] is buf and all(torch.equal(a.float(), b.float()) for a, b in zip(got, want))
        dy, dh = randn(40, k, dtype=torch.bfloat16, seed=3), randn(40, k, dtype=torch.bfloat16, seed=4)
        dx, dw = oz.ozaki_rms_norm_backward(dy, want[2], w, want[3], dh)
        for which in range(3):
            ops = [dy.clone(), want[2].clone(), dh.clone()]
            dx2, dw2 = oz.ozaki_rms_norm_backward(ops[0], ops[1], w, want[3], ops[2], dX=ops[which])
            assert torch.equal(dx2, dx) and torch.equal(dw2, dw) and dx2 is ops[which]


def test_norm_of_zero_and_nan_rows():
    x, w = randn(5, 300), randn(300, seed=1)
    clean = oz.ozaki_rms_norm_f8(x, w)
    x[1] = 0
    x[3, 7] = float("nan")
    q, s, _, rstd = oz.ozaki_rms_norm_f8(x, w)
    assert (q[1].float() == 0).all() and (s[1] == 1).all() and abs(rstd[1].item() - 1000) < 1e-3
    assert torch.isnan(s[3]).all() and torch.isnan(rstd[3])
    for r in (0, 2, 4):
        assert torch.equal(q[r].float(), clean[0][r].float()) and torch.equal(s[r], clean[1][r])


# ------------------------------------------------------------------ clipping
def check_clip(grads, limit, out=None):
    # 32 squares at a time in FP32: within 33 * 2^-24, half of it for the norm; the factor three roundings more
    before = [g.double() for g in grads]
    norm = torch.sqrt(sum((b.square().sum() for b in before), torch.zeros((), dtype=torch.float64, device="cuda")))
    factor = torch.clamp(limit / (norm + 1e-6), max=1.0)
    got = oz.ozaki_clip_grad_norm(grads, limit, out=out)
    assert got.shape == () and got.dtype == torch.float32
    assert abs(got.item() - norm.item()) <= 2.0 ** -18 * norm.item()
    for g, b in zip(grads if out is None else out, before):
        want = b * factor
        assert ((g.double() - want).abs() <= (HALF[g.dtype] + 2.0 ** -17) * want.abs() + TINY[g.dtype]).all()
    return got


DTYPES = (torch.float32, torch.bfloat16, torch.float16)


@pytest.mark.parametrize("limit", [1.0, 1e9, 0.0])
@pytest.mark.parametrize("sizes", [[1], [0, 7, 0], [5, 8, 16384, 16385], [100] * 64, [33] * 65, [1000, 3, 200000, 17], [9] * 1500, [3000001]])
def test_clip(sizes, limit):
    grads = [randn(n, dtype=DTYPES[i % 3], seed=i) for i, n in enumerate(sizes)]
    out = [torch.full_like(g, 7.0) for g in grads]
    keep = [g.clone() for g in grads]
    a = check_clip(grads, limit, out)
    assert all(torch.equal(g, k) for g, k in zip(grads, keep))
    b = check_clip(grads, limit)
    assert torch.equal(a, b) and all(torch.equal(g, o) for g, o in zip(grads, out))


def test_clip_unaligned_tensors_keep_their_neighbours():
    for dtype in DTYPES:
        big = randn(70000, dtype=dtype)
        keep = big.clone()
        at = [(1, 3), (11, 20000), (20013, 40001)]
        check_clip([big[a:a + n] for a, n in at], 0.5)
        inside = torch.zeros(70000, dtype=torch.bool, device="cuda")
        for a, n in at:
            inside[a:a + n] = True
        assert torch.equal(big[~inside], keep[~inside])


@pytest.mark.parametrize("power", [-140, -100, -60, -40, 40, 60, 100, 120])
def test_clip_large_and_small_values(power):
    g = (torch.randint(-3, 4, (5000,), generator=torch.Generator().manual_seed(0)).double() * 2.0 ** power).float().cuda()
    want = g.double().square().sum().sqrt().item()
    got = oz.ozaki_clip_grad_norm([g.clone()], 1.0, eps=0.0).item()
    assert abs(got - want) <= 2.0 ** -18 * want + 2.0 ** -150


def test_clip_inf_and_nan():
    g = randn(1000)
    g[3] = float("inf")
    norm = oz.ozaki_clip_grad_norm([g], 1.0)
    assert torch.isinf(norm) and torch.isnan(g[3]) and (g[:3] == 0).all()
    g = randn(1000)
    g[3] = float("nan")
    h = randn(50, dtype=torch.bfloat16)
    assert torch.isnan(oz.ozaki_clip_grad_norm([g, h], 1.0)) and torch.isnan(h).all()


def test_clip_zeros_and_no_limit():
    inf = float("inf")
    for limit, eps in ((0.0, 0.0), (1.0, 0.0), (inf, 0.0), (inf, 1e-6)):  # 0 / 0 among them
        g, out = [torch.zeros(1000, device="cuda")], [torch.full((1000,), 7.0, device="cuda")]
        assert oz.ozaki_clip_grad_norm(g, limit, eps, out=out).item() == 0 and (out[0] == 0).all()
    g = randn(1000)
    g[3] = inf
    keep = g.clone()
    assert oz.ozaki_clip_grad_norm([g], inf).item() == inf and torch.equal(g, keep)  # Inf / Inf
    g[4] = float("nan")
    assert torch.isnan(oz.ozaki_clip_grad_norm([g], inf)) and torch.isnan(g).all()


@pytest.mark.parametrize("workspace", [True, False])
def test_clip_repeated_calls_agree(workspace):
    # back to back on one stream, their launches overlapping, each with its own tensors
    sets = [[randn(n, seed=10 * j + i, scale=0.5 ** j) for i, n in enumerate([100, 30000, 7, 65536])] for j in range(8)]
    want = [torch.sqrt(sum(g.double().square().sum() for g in s)) for s in sets]
    outs = [[torch.empty_like(g) for g in s] for s in sets]
    ws = torch.empty(oz.ozaki_clip_grad_norm_workspace_bytes(), dtype=torch.uint8, device="cuda") if workspace else None
    norms = [oz.ozaki_clip_grad_norm(sets[i % 8], 1.0, out=outs[i % 8], workspace=ws) for i in range(400)]
    for i, n in enumerate(norms):
        assert abs(n.item() - want[i % 8].item()) <= 2.0 ** -18 * want[i % 8].item(), i
