"""Training steps of the expert layers against plain restatements, and refusals by address (GPU)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from fp64_gemm_emulation_gb300 import ozaki as oz
    from fp64_gemm_emulation_gb300 import run_experts

E4M3 = torch.float8_e4m3fn


def randn(*shape, seed, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda") * scale).to(dtype)


def problem(rows=260, experts=3, k=128, n=96):
    _, o = run_experts.route(torch.randint(experts, (rows,), generator=torch.Generator(device="cuda").manual_seed(9), device="cuda"), experts)
    return randn(rows, k, seed=1), randn(experts, n, k, seed=2, scale=k ** -0.5), o, randn(rows, n, seed=3)


def ulps(t):
    """One rounding to t's type, and a little for FP32's before it."""
    return (torch.finfo(t.dtype).eps / 2 + 2.0 ** -20) * t.double().abs()


def test_eight_bit_step_is_the_clipped_momentum_step():
    x, w, o, target = problem()
    gain, clip, lr, momentum = (1 + randn(128, seed=4, scale=0.1, dtype=torch.float32)).to(torch.bfloat16), 0.05, 0.02, 0.9
    layer = run_experts.EightBitExpertLayer(w.clone(), gain.clone(), lr, momentum, clip)
    M = torch.zeros_like(w)
    for _ in range(3):
        before_w, before_gain = layer.W.clone(), layer.gain.clone()
        loss, dx, dw, dgain = layer.gradients(x, o, target)
        norm = torch.sqrt(dw.double().square().sum() + dgain.double().square().sum())
        assert norm > 2 * clip  # the limit binds
        factor = clip / (norm + 1e-6)
        got, got_dx = layer.step(x, o, target)
        assert torch.equal(got, loss) and torch.equal(got_dx, dx)
        dw, dgain = dw.double() * factor, dgain.double() * factor
        # Three roundings to bfloat16, each of at most 2^-8 of what it gives: the clipped gradient (its factor's FP32 roundings: 2^-17, as in
        # the clipping's own tests), M * momentum (M.mul_ stores it in bfloat16), and their sum.
        off = (2.0 ** -8 + 2.0 ** -17) * dw.abs()
        want = M.double() * momentum
        assert ((layer.M.double() - (want + dw)).abs() <= off + 2.0 ** -8 * want.abs() + ulps(layer.M) + 2.0 ** -20 * (want.abs() + dw.abs())).all()
        M = layer.M.clone()
        step = oz.ozaki_newton_schulz(M).double() * lr  # bfloat16, rounded once more by the factor
        assert ((layer.W.double() - (before_w.double() - step)).abs() <= 2.0 ** -8 * step.abs() + ulps(layer.W)).all()
        off = (2 * 2.0 ** -8 + 2.0 ** -16) * lr * dgain.abs()
        assert ((layer.gain.double() - (before_gain.double() - lr * dgain)).abs() <= off + ulps(layer.gain)).all()


def test_sixteen_bit_step_is_the_plain_one():
    x, w, o, target = problem()
    layer = run_experts.ExpertLayer(w.clone(), 0.02, 0.9)
    loss, dx = layer.step(x, o, target)
    at, X, W = o.tolist(), x.double(), w.double()
    y = torch.cat([X[lo:hi] @ W[e].T for e, (lo, hi) in enumerate(zip(at, at[1:]))])
    my = torch.cat([X[lo:hi].abs() @ W[e].T.abs() for e, (lo, hi) in enumerate(zip(at, at[1:]))])
    rows, near = x.shape[0], 2.0 ** -8 + 2.0 ** -16
    diff = y - target.double()
    ey = near * y.abs() + 128 * 2.0 ** -23 * my                       # y, rounded to bfloat16
    assert abs(loss.item() - 0.5 * diff.square().sum().item() / rows) <= ((diff.abs() * ey + ey.square()).sum() / rows).item() * (1 + 2.0 ** -8)
    dy, edy = diff / rows, (ey + near * (diff.abs() + ey)) / rows     # and dy
    for e, (lo, hi) in enumerate(zip(at, at[1:])):
        want, off = dy[lo:hi] @ W[e], edy[lo:hi] @ W[e].abs()
        mag = (dy[lo:hi].abs() + edy[lo:hi]) @ W[e].abs()
        assert ((dx[lo:hi].double() - want).abs() <= off + near * (want.abs() + off) + 96 * 2.0 ** -23 * mag).all()
        want, off = dy[lo:hi].T @ X[lo:hi], edy[lo:hi].T @ X[lo:hi].abs()
        mag = (dy[lo:hi].abs() + edy[lo:hi]).T @ X[lo:hi].abs()
        assert ((layer.M[e].double() - want).abs() <= off + near * (want.abs() + off) + rows * 2.0 ** -23 * mag).all()  # the first momentum is dW
    step = oz.ozaki_newton_schulz(layer.M).double() * 0.02
    assert ((layer.W.double() - (w.double() - step)).abs() <= 2.0 ** -8 * step.abs() + ulps(layer.W)).all()


def test_operands_whose_rows_start_at_odd_addresses_are_refused():
    rows, n, k = 40, 48, 64
    x, w, dy = (randn(*s, seed=i, dtype=torch.float32).to(E4M3) for i, s in enumerate([(rows, k), (n, k), (rows, n)]))
    xs, ws, ys = torch.ones(1, rows, device="cuda").t(), torch.ones(1, 1, device="cuda"), torch.ones(1, rows, device="cuda").t()
    xc, yc = torch.ones(1, k, device="cuda"), torch.ones(1, n, device="cuda")

    def moved(t, pad, at):
        """t with rows `pad` elements further apart, `at` bytes behind a multiple of 16."""
        flat = torch.zeros(t.shape[0] * (t.shape[1] + pad) + 16, dtype=t.dtype, device="cuda")
        v = flat[at:at + t.shape[0] * (t.shape[1] + pad)].view(t.shape[0], t.shape[1] + pad)[:, :t.shape[1]]
        v.copy_(t)
        return v

    calls = [lambda f: oz.ozaki_grouped_gemm_f8(f(x), xs, w, ws), lambda f: oz.ozaki_grouped_gemm_f8(x, xs, f(w), ws),
             lambda f: oz.ozaki_grouped_gemm_f8_dgrad(f(dy), ys, w, ws), lambda f: oz.ozaki_grouped_gemm_f8_dgrad(dy, ys, f(w), ws),
             lambda f: oz.ozaki_grouped_gemm_f8_wgrad(f(dy), yc, x, xc), lambda f: oz.ozaki_grouped_gemm_f8_wgrad(dy, yc, f(x), xc)]
    for call in calls:
        want = call(lambda t: t)
        assert torch.equal(call(lambda t: moved(t, 16, 0)), want)
        for pad, at in ((0, 8), (8, 0), (1, 0), (16, 4)):
            with pytest.raises(ValueError, match="multiples of 16 bytes"):
                call(lambda t: moved(t, pad, at))
