"""Grouped expert products and Newton-Schulz against their definitions in 64 bits (GPU).

Tolerances.  A product of 16-bit operands is summed in FP32: a sum of K terms that loses at most
2^-23 of the running sum of magnitudes at each addition is off by less than (K + 2) 2^-23 |x| |w|, and
the result is rounded once (half an ulp: 2^-8 of it in bfloat16, 2^-11 in float16, 2^-25 below the
normal float16 range).  Newton-Schulz stores three matrices a step, each rounded to 11 s bits
(s slices: 2^-11s relative) and, with two slices, summed with at most 12 + sqrt(K / 64) roundings of
2^-24; a step's polynomial passes an error on at most fourfold (its derivative at 0 is 3.44).
"""
import math

import numpy as np
import pytest
import torch

gpu = pytest.mark.gpu
pytestmark = gpu

if torch.cuda.is_available():
    from fp64_gemm_emulation_gb300 import ozaki as oz

HALF_ULP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


@pytest.fixture(autouse=True)
def clean_status():
    oz.ozaki_get_device_status()
    yield
    assert oz.ozaki_get_device_status() == oz.OZ_OK


def randn(*shape, dtype=torch.bfloat16, seed=0, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


def make(counts, n, k, dtype, before=0, after=0, seed=0):
    offsets = [before]
    for c in counts:
        offsets.append(offsets[-1] + c)
    rows = offsets[-1] + after
    o = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    return (randn(rows, k, dtype=dtype, seed=seed), randn(len(counts), n, k, dtype=dtype, seed=seed + 1, scale=max(1, k) ** -0.5),
            randn(rows, n, dtype=dtype, seed=seed + 2), o, offsets)


def reference(x, w, dy, offsets):
    """(y, dx, dw) and the same of the magnitudes, in 64 bits; zeros outside the groups."""
    def run(x, w, dy):
        y = torch.zeros(x.shape[0], w.shape[1], dtype=torch.float64, device=x.device)
        dx = torch.zeros(x.shape[0], w.shape[2], dtype=torch.float64, device=x.device)
        dw = torch.zeros(w.shape, dtype=torch.float64, device=x.device)
        for e, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
            y[lo:hi] = x[lo:hi] @ w[e].T
            dx[lo:hi] = dy[lo:hi] @ w[e]
            dw[e] = dy[lo:hi].T @ x[lo:hi]
        return y, dx, dw

    x, w, dy = x.double(), w.double(), dy.double()
    return run(x, w, dy), run(x.abs(), w.abs(), dy.abs())


def check(got, ref, mag, terms, what):
    tol = HALF_ULP[got.dtype] * ref.abs() + (terms + 2) * 2.0 ** -23 * mag * (1 + HALF_ULP[got.dtype]) + 2.0 ** -25
    bad = (got.double() - ref).abs() > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}"


def check_all(counts, n, k, dtype, **kw):
    x, w, dy, o, offsets = make(counts, n, k, dtype, **kw)
    (y, dx, dw), (my, mdx, mdw) = reference(x, w, dy, offsets)
    check(oz.ozaki_grouped_gemm(x, w, o), y, my, k, "forward")
    check(oz.ozaki_grouped_gemm_dgrad(dy, w, o), dx, mdx, n, "dgrad")
    check(oz.ozaki_grouped_gemm_wgrad(dy, x, o), dw, mdw, max(counts, default=0), "wgrad")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("counts,n,k", [
    ([1], 1, 1),                          # one of everything
    ([1, 1, 1], 3, 5),
    ([7], 8, 64),
    ([255, 256, 257], 256, 128),          # around a tile
    ([0, 0, 0], 64, 64),                  # nobody
    ([0, 513, 0, 31, 1, 0], 320, 192),    # empty groups between
    ([63, 64, 65, 127, 129], 129, 127),   # around a k-block of the weight gradient, odd widths
    ([300, 20], 1000, 264),               # n not a multiple of 32
    ([33] * 40, 96, 72),
    ([5, 700, 1, 0, 33], 517, 1001),      # no 16-byte row stride
])
def test_grouped_products(counts, n, k, dtype):
    check_all(counts, n, k, dtype)


def test_grouped_rows_outside_every_group_are_zero():
    check_all([40, 0, 300], 192, 320, torch.bfloat16, before=37, after=270)


@pytest.mark.parametrize("counts,n,k", [([1], 4096, 8192), ([2, 0, 3], 8192, 2048), ([4000], 128, 64), ([1] * 8, 1024, 2048), ([9000], 128, 64), ([40, 0, 300], 700, 8192)])
def test_grouped_long_sums_are_split(counts, n, k):
    check_all(counts, n, k, torch.bfloat16)


@pytest.mark.parametrize("groups", [oz.OZ_MAX_GROUPS if torch.cuda.is_available() else 1])
def test_grouped_most_groups(groups):
    counts = [(e * 7) % 5 for e in range(groups)]
    check_all(counts, 64, 96, torch.bfloat16)


def test_grouped_strided_operands_and_outputs_keep_their_padding():
    counts, n, k = [70, 0, 200, 33], 200, 136
    x, w, dy, o, offsets = make(counts, n, k, torch.bfloat16)
    rows = x.shape[0]
    for pad in (8, 3):  # a multiple of 16 bytes, and not
        def strided(t):
            big = torch.full((*t.shape[:-1], t.shape[-1] + pad), 7.0, dtype=t.dtype, device="cuda")
            big[..., :t.shape[-1]] = t
            return big, big[..., :t.shape[-1]]

        (_, xs), (_, ws), (_, dys) = strided(x), strided(w), strided(dy)
        (yb, ys), (dxb, dxs), (dwb, dws) = strided(torch.zeros(rows, n).cuda().bfloat16()), \
            strided(torch.zeros(rows, k).cuda().bfloat16()), strided(torch.zeros(4, n, k).cuda().bfloat16())
        oz.ozaki_grouped_gemm(xs, ws, o, ys)
        oz.ozaki_grouped_gemm_dgrad(dys, ws, o, dxs)
        oz.ozaki_grouped_gemm_wgrad(dys, xs, o, dws)
        assert torch.equal(ys, oz.ozaki_grouped_gemm(x, w, o))
        assert torch.equal(dxs, oz.ozaki_grouped_gemm_dgrad(dy, w, o))
        assert torch.equal(dws, oz.ozaki_grouped_gemm_wgrad(dy, x, o))
        for big, t in ((yb, n), (dxb, k), (dwb, k)):
            assert (big[..., t:] == 7.0).all()


def test_grouped_misaligned_addresses():
    counts, n, k = [30, 100], 64, 80
    x, w, dy, o, offsets = make(counts, n, k, torch.float16)

    def shifted(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        flat[1:] = t.reshape(-1)
        return flat[1:].view(t.shape)

    assert torch.equal(oz.ozaki_grouped_gemm(shifted(x), shifted(w), o, shifted(torch.zeros_like(dy))), oz.ozaki_grouped_gemm(x, w, o))
    assert torch.equal(oz.ozaki_grouped_gemm_dgrad(shifted(dy), shifted(w), o), oz.ozaki_grouped_gemm_dgrad(dy, w, o))
    assert torch.equal(oz.ozaki_grouped_gemm_wgrad(shifted(dy), shifted(x), o), oz.ozaki_grouped_gemm_wgrad(dy, x, o))


def test_grouped_nan_and_inf_stay_in_their_group():
    counts, n, k = [50, 70, 64, 10], 160, 96
    x, w, dy, o, offsets = make(counts, n, k, torch.bfloat16, before=5, after=9)
    clean = [oz.ozaki_grouped_gemm(x, w, o), oz.ozaki_grouped_gemm_dgrad(dy, w, o), oz.ozaki_grouped_gemm_wgrad(dy, x, o)]
    lo, hi = offsets[1], offsets[2]
    x2, w2, dy2 = x.clone(), w.clone(), dy.clone()
    for t in (x2, dy2):  # group 1, and the rows outside every group
        t[lo:hi:2] = float("nan")
        t[lo + 1:hi:2] = float("inf")
        t[:5] = float("nan")
        t[offsets[-1]:] = float("inf")
    w2[1] = float("nan")
    y, dx, dw = oz.ozaki_grouped_gemm(x2, w2, o), oz.ozaki_grouped_gemm_dgrad(dy2, w2, o), oz.ozaki_grouped_gemm_wgrad(dy2, x2, o)
    keep = [r for r in range(x.shape[0]) if not lo <= r < hi]
    assert torch.equal(y[keep], clean[0][keep]) and torch.equal(dx[keep], clean[1][keep])
    assert torch.equal(dw[[0, 2, 3]], clean[2][[0, 2, 3]])
    assert y[lo:hi].isnan().all() and dx[lo:hi].isnan().all() and dw[1].isnan().all()


@pytest.mark.parametrize("offsets", [[0, 60, 40, 100], [-5, 30, 60, 100], [0, 50, 80, 1000], [90, 80, 70, 60]])
def test_grouped_bad_offsets_are_clamped_and_reported(offsets):
    x, w, dy, _, _ = make([100], 64, 72, torch.bfloat16)
    w = randn(3, 64, 72, seed=5)
    o = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    fixed, low = [], 0
    for v in offsets:
        low = max(low, min(max(v, 0), 100))
        fixed.append(low)
    for call in (lambda o: oz.ozaki_grouped_gemm(x, w, o), lambda o: oz.ozaki_grouped_gemm_dgrad(dy, w, o),
                 lambda o: oz.ozaki_grouped_gemm_wgrad(dy, x, o)):
        got = call(o)
        assert oz.ozaki_get_device_status() == oz.OZ_EINVAL
        assert torch.equal(got, call(torch.tensor(fixed, dtype=torch.int32, device="cuda")))


# the last two split their sums: the forward product's and the weight gradient's, the input gradient's
@pytest.mark.parametrize("counts,n,k", [([3, 0, 40, 300], 384, 2048), ([5000, 40, 9000], 320, 8192), ([3, 0, 70], 8192, 320)])
def test_grouped_results_repeat_on_any_stream_workspace_and_in_a_graph(counts, n, k):
    x, w, dy, o, _ = make(counts, n, k, torch.bfloat16)
    calls = {"f": lambda **kw: oz.ozaki_grouped_gemm(x, w, o, **kw), "d": lambda **kw: oz.ozaki_grouped_gemm_dgrad(dy, w, o, **kw),
             "w": lambda **kw: oz.ozaki_grouped_gemm_wgrad(dy, x, o, **kw)}
    sizes = {"f": oz.ozaki_grouped_gemm_workspace_bytes(x, w), "d": oz.ozaki_grouped_gemm_dgrad_workspace_bytes(dy, w),
             "w": oz.ozaki_grouped_gemm_wgrad_workspace_bytes(dy, x, len(counts))}
    side = torch.cuda.Stream()
    for name, call in calls.items():
        first = call()
        for _ in range(3):
            assert torch.equal(call(), first)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            other = call()
        side.synchronize()
        assert torch.equal(other.cpu(), first.cpu())
        assert torch.equal(call(stream=torch.cuda.current_stream()), first)
        ws = torch.full((sizes[name],), 255, dtype=torch.uint8, device="cuda")
        out = torch.empty_like(first)
        kw = {"f": "Y", "d": "dX", "w": "dW"}[name]
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            call(workspace=ws, **{kw: out})
        for _ in range(3):
            out.fill_(9.0)
            graph.replay()
            assert torch.equal(out, first)


def test_grouped_gradients_match_differences():
    # L = <c, y(x, w)> is linear in x and in w: the difference quotient of the 64-bit product is exact
    counts, n, k = [20, 0, 45], 48, 56
    x, w, c, o, offsets = make(counts, n, k, torch.float16)
    dx, dw = oz.ozaki_grouped_gemm_dgrad(c, w, o).double(), oz.ozaki_grouped_gemm_wgrad(c, x, o).double()

    def loss(x, w):
        return sum((c[lo:hi].double() * (x[lo:hi] @ w[e].T)).sum() for e, (lo, hi) in enumerate(zip(offsets, offsets[1:])))

    x64, w64 = x.double(), w.double()
    for seed in range(3):
        ex, ew = randn(*x.shape, dtype=torch.float64, seed=seed), randn(*w.shape, dtype=torch.float64, seed=seed + 9)
        for got, diff, mag in ((dx * ex, loss(x64 + ex, w64) - loss(x64 - ex, w64), dx.abs() * ex.abs()),
                               (dw * ew, loss(x64, w64 + ew) - loss(x64, w64 - ew), dw.abs() * ew.abs())):
            # each gradient entry is within 2 half-ulps of float16 (sum and rounding) of the exact one
            assert abs(got.sum() - diff / 2) <= 2 * 2.0 ** -11 * mag.sum() + 1e-9


# ------------------------------------------------------------------ Newton-Schulz
def newton64(g, steps=5, coeffs=None, eps=1e-7):
    coeffs = np.asarray(coeffs if coeffs is not None else oz.NEWTON_SCHULZ_COEFFS, dtype=np.float64).reshape(-1, 3)
    x = g.double()
    tall = x.shape[-2] > x.shape[-1]
    if tall:
        x = x.transpose(-1, -2)
    x = x / (torch.linalg.matrix_norm(x)[..., None, None] + eps)
    for i in range(steps):
        a, b, c = np.float32(coeffs[i % len(coeffs)]).astype(np.float64)
        A = x @ x.transpose(-1, -2)
        x = a * x + (b * A + c * A @ A) @ x
    return x.transpose(-1, -2) if tall else x


def newton_tolerance(m, n, dtype, slices, steps=5):
    stored = 2.0 ** (-11 * slices) + ((12 + math.sqrt(max(m, n) / 64)) * 2.0 ** -24 if slices == 2 else 0.0)
    return steps * 3 * 4 * stored + 2 * HALF_ULP[dtype]


def momentum(b, m, n, dtype, seed=0):
    noise = randn(b, m, n, dtype=torch.float32, seed=seed) * torch.exp(0.5 * randn(b, 1, n, dtype=torch.float32, seed=seed + 1))
    r = min(4, m, n)
    low = randn(b, m, r, dtype=torch.float32, seed=seed + 2) @ randn(b, r, n, dtype=torch.float32, seed=seed + 3)
    return (noise + low * (noise.norm() / low.norm())).to(dtype)


def check_newton(g, got, tol, **kw):
    ref = newton64(g, **kw)
    err = torch.linalg.matrix_norm(got.double() - ref) / torch.linalg.matrix_norm(ref).clamp_min(1e-300)
    assert (err <= tol).all(), f"{err.max().item():.2e} > {tol:.2e}"


@pytest.mark.parametrize("m,n", [(1, 1), (1, 9), (9, 1), (16, 16), (65, 129), (129, 65), (128, 128), (256, 512), (512, 256),
                                 (300, 301), (257, 1000), (1000, 257), (640, 640), (96, 4096), (4096, 96)])
@pytest.mark.parametrize("dtype,slices", [(torch.bfloat16, 1), (torch.float32, 2), (torch.float16, 2), (torch.bfloat16, 2)])
def test_newton_schulz(m, n, dtype, slices):
    g = momentum(1, m, n, dtype)[0]
    check_newton(g, oz.ozaki_newton_schulz(g, num_slices=slices), newton_tolerance(m, n, dtype, slices))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("b,m,n", [(3, 200, 72), (40, 64, 96), (2, 1024, 512)])
def test_newton_schulz_batches(b, m, n, dtype):
    g = momentum(b, m, n, dtype)
    got = oz.ozaki_newton_schulz(g)
    check_newton(g, got, newton_tolerance(m, n, dtype, 1 if dtype == torch.bfloat16 else 2))
    assert torch.equal(got[b - 1], oz.ozaki_newton_schulz(g[b - 1].clone())) or b > 3 or m * n > 200 * 72
    four = oz.ozaki_newton_schulz(g.view(1, b, m, n))
    assert four.shape == (1, b, m, n) and torch.equal(four[0], got)


@pytest.mark.parametrize("coeffs,steps", [((1.5, -0.5, 0.0), 6), ((1.875, -1.25, 0.375), 6),
                                          ([(3.4445, -4.775, 2.0315), (1.5, -0.5, 0.0), (1.875, -1.25, 0.375)], 3), ((2.0, -1.5, 0.5), 1)])
def test_newton_schulz_other_polynomials(coeffs, steps):
    g = momentum(1, 150, 220, torch.float32)[0]
    got = oz.ozaki_newton_schulz(g, steps=steps, coeffs=coeffs)
    check_newton(g, got, newton_tolerance(150, 220, torch.float32, 2, steps), steps=steps, coeffs=coeffs)


def test_newton_schulz_orthogonalises():
    g = randn(96, 400, dtype=torch.float32)
    x = oz.ozaki_newton_schulz(g, steps=30, coeffs=(1.5, -0.5, 0.0)).double()
    assert (x @ x.T - torch.eye(96, device="cuda")).abs().max() < 30 * 3 * 2.0 ** -21


@pytest.mark.parametrize("scale", [1e-36, 1e-20, 1e-3, 1e18, 1e30])
def test_newton_schulz_ignores_the_scale(scale):
    g = momentum(1, 90, 130, torch.float32)[0]
    check_newton(g * scale, oz.ozaki_newton_schulz(g * scale, eps=0.0), newton_tolerance(90, 130, torch.float32, 2), eps=0.0)


@pytest.mark.parametrize("norm", [1e-9, 1e-12, 1e-20])
def test_newton_schulz_below_eps(norm):
    # eps dominates the norm: the iteration stays linear and tiny, and keeps its bits
    g = momentum(1, 60, 80, torch.float32)[0]
    g = g * (norm / g.norm())
    check_newton(g, oz.ozaki_newton_schulz(g), newton_tolerance(60, 80, torch.float32, 2))


def test_newton_schulz_zero_nan_and_inf_matrices():
    g = momentum(4, 72, 100, torch.float32)
    clean = oz.ozaki_newton_schulz(g)
    g[1] = 0
    g[2, 5, 7] = float("nan")
    g[3, 0, 0] = float("-inf")
    got = oz.ozaki_newton_schulz(g)
    assert torch.equal(got[0], clean[0]) and (got[1] == 0).all() and got[2].isnan().all() and got[3].isnan().all()


def test_newton_schulz_strides():
    g = momentum(3, 70, 90, torch.bfloat16)
    want = oz.ozaki_newton_schulz(g)
    wide = torch.full((3, 80, 101), 5.0, dtype=g.dtype, device="cuda")
    wide[:, :70, :90] = g
    out = torch.full((3, 75, 99), 6.0, dtype=g.dtype, device="cuda")
    oz.ozaki_newton_schulz(wide[:, :70, :90], out=out[:, :70, :90])
    assert torch.equal(out[:, :70, :90], want) and (out[:, 70:] == 6).all() and (out[:, :, 90:] == 6).all()
    turned = g[0].t().contiguous().t()  # column-major in, column-major out
    got = oz.ozaki_newton_schulz(turned)
    assert got.stride() == turned.stride()
    check_newton(g[0], got, newton_tolerance(70, 90, torch.bfloat16, 1))


def test_newton_schulz_repeats_on_any_stream_workspace_and_in_a_graph():
    g = momentum(2, 300, 700, torch.bfloat16)
    for slices in (1, 2):
        first = oz.ozaki_newton_schulz(g, num_slices=slices)
        for _ in range(3):
            assert torch.equal(oz.ozaki_newton_schulz(g, num_slices=slices), first)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            other = oz.ozaki_newton_schulz(g, num_slices=slices)
        side.synchronize()
        assert torch.equal(other.cpu(), first.cpu())
        ws = torch.full((oz.ozaki_newton_schulz_workspace_bytes(700, 300, 2, slices),), 255, dtype=torch.uint8, device="cuda")
        out = torch.empty_like(g)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            oz.ozaki_newton_schulz_ws(g, ws, num_slices=slices, out=out)
        for _ in range(3):
            out.fill_(9.0)
            graph.replay()
            assert torch.equal(out, first)
        with pytest.raises(oz.OzakiError):
            oz.ozaki_newton_schulz_ws(g, ws[:1024], num_slices=slices, out=out)


def test_expired_waits_are_reported_and_leave_the_library_usable():
    # sums long enough that the first accumulator is not there when the epilogue looks for it
    x, w, dy, o, _ = make([4000, 3000], 2048, 8192, torch.bfloat16)
    g = momentum(1, 2048, 8192, torch.bfloat16)
    want = oz.ozaki_grouped_gemm(x, w, o), oz.ozaki_newton_schulz(g)
    lib = oz._lib
    assert lib.ozaki_set_epilogue_wait_ns(0) == oz.OZ_OK
    try:
        for call in (lambda: oz.ozaki_grouped_gemm(x, w, o), lambda: oz.ozaki_newton_schulz(g)):
            call()
            assert oz.ozaki_get_device_status() == oz.OZ_ETIMEOUT
    finally:
        lib.ozaki_set_epilogue_wait_ns(-1)
    assert torch.equal(oz.ozaki_grouped_gemm(x, w, o), want[0]) and torch.equal(oz.ozaki_newton_schulz(g), want[1])


def test_training_step_example():
    from fp64_gemm_emulation_gb300.run_experts import train

    losses = train(tokens=700, experts=5, k=96, n=160, steps=12)
    assert all(b < a for a, b in zip(losses, losses[1:]))
