"""Expert products and Newton-Schulz as programs call them: streams, workspaces, layouts, large values (GPU)."""
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


def test_workspaces_that_the_device_cannot_use_are_refused():
    x, w, o = randn(8, 8192, dtype=torch.bfloat16), randn(1, 64, 8192, dtype=torch.bfloat16), torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    need = max(oz.ozaki_grouped_gemm_workspace_bytes(x, w), oz.ozaki_newton_schulz_workspace_bytes(300, 300))
    assert need > 0
    for ws in (torch.empty(need, dtype=torch.uint8), torch.empty(1, dtype=torch.uint8, device="cuda").expand(need),
               torch.empty(2 * need, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError, match="workspace"):
            oz.ozaki_grouped_gemm_ws(x, w, o, ws)
        with pytest.raises(ValueError, match="workspace"):
            oz.ozaki_newton_schulz_ws(randn(300, 300), ws)


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


# ------------------------------------------------------------------ streams other than the current one
def operators():
    """name -> (operands, call); results of a few MB, so that the allocator's blocks are theirs alone."""
    rows, n, k = 1900, 1500, 1100
    x, w, dy = (randn(*s, dtype=torch.bfloat16, seed=i) for i, s in enumerate(((rows, k), (3, n, k), (rows, n))))
    o = torch.tensor([0, 700, 700, 1900], dtype=torch.int32, device="cuda")
    a, b = (oz.colmajor(randn(700, 900, dtype=torch.float64, seed=5)), oz.colmajor(randn(900, 800, dtype=torch.float64, seed=6)))
    return {
        "forward": ([x, w, o], oz.ozaki_grouped_gemm),
        "dgrad": ([dy, w, o], oz.ozaki_grouped_gemm_dgrad),
        "wgrad": ([dy, x, o], oz.ozaki_grouped_gemm_wgrad),
        "newton": ([x], oz.ozaki_newton_schulz),
        "newton small": ([randn(300, 100, 100)], oz.ozaki_newton_schulz),
        "scheme 2": ([a, b], lambda a, b, **kw: oz.ozaki2_dgemm(a, b, 14, **kw)),
        "scheme 2 scaled": ([a, b], lambda a, b, **kw: oz.ozaki2_dgemm_ex(a, b, 14, "accu", **kw)),
        "scheme 1": ([a, b], lambda a, b, **kw: oz.ozaki1_dgemm(a, b, 7, **kw)),
    }


NAMES = ["forward", "dgrad", "wgrad", "newton", "newton small", "scheme 2", "scheme 2 scaled", "scheme 1"]


def handles(side):
    return {"stream": side, "handle": side.cuda_stream}


@pytest.mark.parametrize("form", ["stream", "handle"])
@pytest.mark.parametrize("name", NAMES)
def test_results_for_another_stream_are_not_the_current_streams_memory(name, form):
    # the block that a result of this size would get on the current stream, where work may still use it
    operands, call = operators()[name]
    first = call(*operands)
    want, block = first.clone(), first.data_ptr()
    torch.cuda.synchronize()
    del first
    side = torch.cuda.Stream()
    got = call(*operands, stream=handles(side)[form])
    side.synchronize()
    assert torch.equal(got, want)
    assert got.data_ptr() != block


@pytest.mark.parametrize("form", ["stream", "handle"])
@pytest.mark.parametrize("name", NAMES)
def test_operands_are_kept_until_another_stream_is_done(name, form):
    operands, call = operators()[name]
    want = call(*operands)
    copies = [t.clone() if t.stride(-1) == 1 or t.dim() != 2 else oz.colmajor(t.t().clone().t()) for t in operands]
    blocks = {t.data_ptr() for t in copies if t.numel() > 1 << 16}
    sizes = [t.numel() * t.element_size() for t in copies if t.numel() > 1 << 16]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(1_000_000_000)  # about half a second
    got = call(*copies, stream=handles(side)[form])
    del copies
    again = [torch.empty(s, dtype=torch.uint8, device="cuda") for s in sizes]  # never written
    reused = blocks & {t.data_ptr() for t in again}
    side.synchronize()
    assert not reused
    assert torch.equal(got, want)


@pytest.mark.parametrize("name", NAMES)
def test_the_default_stream_named_from_another_one(name):
    operands, call = operators()[name]
    want = call(*operands)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = call(*operands, stream=0)
        named = call(*operands, stream=torch.cuda.default_stream())
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(named, want)


# ------------------------------------------------------------------ launches that overlap
def test_overlapping_launches_of_small_matrices():
    # more matrices than SMs, one launch after another, of kernels that each hold all tensor memory of their SM
    sets = [(randn(400, 64, 64, seed=1), s) for s in (1, 2)] + [(randn(500, 16, 40, seed=2), s) for s in (1, 2)]
    want = []
    for g, s in sets:
        want.append(oz.ozaki_newton_schulz(g, num_slices=s))
        torch.cuda.synchronize()
    got = [[oz.ozaki_newton_schulz(g, num_slices=s) for g, s in sets] for _ in range(10)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for row in got for a, b in zip(row, want))
