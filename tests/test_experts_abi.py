"""Grouped products and Newton-Schulz: argument checks and host-only queries (no GPU call is made)."""
import ctypes

import numpy as np
import pytest
import torch

from fp64_gemm_emulation_gb300 import ozaki as oz

lib = oz._lib
P = 4096  # an address that is never read: every call below returns before any CUDA call
FIVE_STEPS = np.tile(np.array(oz.NEWTON_SCHULZ_COEFFS, dtype=np.float32), 5)


def forward(n=8, k=8, rows=8, groups=2, dtype=oz.OZ_BF16, W=P, ldw=8, sw=64, X=P, ldx=8, off=P, Y=P, ldy=8):
    return lib.ozaki_grouped_gemm(n, k, rows, groups, dtype, W, ldw, sw, X, ldx, off, Y, ldy, None)


def dgrad(n=8, k=8, rows=8, groups=2, dtype=oz.OZ_BF16, W=P, ldw=8, sw=64, dY=P, lddy=8, off=P, dX=P, lddx=8):
    return lib.ozaki_grouped_gemm_dgrad(n, k, rows, groups, dtype, W, ldw, sw, dY, lddy, off, dX, lddx, None)


def wgrad(n=8, k=8, rows=8, groups=2, dtype=oz.OZ_BF16, dY=P, lddy=8, X=P, ldx=8, off=P, dW=P, ldw=8, sw=64):
    return lib.ozaki_grouped_gemm_wgrad(n, k, rows, groups, dtype, dY, lddy, X, ldx, off, dW, ldw, sw, None)


@pytest.mark.parametrize("call", [forward, dgrad, wgrad])
@pytest.mark.parametrize("bad", [dict(n=-1), dict(k=-1), dict(rows=-1), dict(rows=2**31 - 1), dict(groups=0), dict(groups=oz.OZ_MAX_GROUPS + 1),
                                 dict(dtype=oz.OZ_F32), dict(dtype=0), dict(ldw=7), dict(sw=63)])
def test_grouped_refuses_bad_arguments(call, bad):
    assert call(**bad) == oz.OZ_EINVAL


@pytest.mark.parametrize("call,bad", [
    (forward, dict(ldx=7)), (forward, dict(ldy=7)), (forward, dict(W=None)), (forward, dict(X=None)),
    (forward, dict(off=None)), (forward, dict(Y=None)),
    (dgrad, dict(lddy=7)), (dgrad, dict(lddx=7)), (dgrad, dict(W=None)), (dgrad, dict(dY=None)), (dgrad, dict(off=None)),
    (dgrad, dict(dX=None)),
    (wgrad, dict(lddy=7)), (wgrad, dict(ldx=7)), (wgrad, dict(dY=None)), (wgrad, dict(X=None)), (wgrad, dict(off=None)),
    (wgrad, dict(dW=None)),
])
def test_grouped_refuses_bad_strides_and_null_pointers(call, bad):
    assert call(**bad) == oz.OZ_EINVAL
    # null operands are found before anything is allocated, at sizes that need a workspace too
    big = dict(n=8192, k=8192, rows=16384, ldw=8192, sw=8192 * 8192)
    big.update({name: 8192 for name in call.__code__.co_varnames[:call.__code__.co_argcount] if name in ("ldx", "ldy", "lddx", "lddy")})
    assert call(**{**big, **bad}) == oz.OZ_EINVAL


def test_grouped_empty_problems_do_nothing():
    assert forward(n=0, ldy=1, sw=0, W=None, X=None, Y=None) == oz.OZ_OK
    assert forward(rows=0, X=None, Y=None) == oz.OZ_OK
    assert dgrad(k=0, ldw=1, lddx=1) == oz.OZ_OK
    assert dgrad(rows=0) == oz.OZ_OK
    assert wgrad(n=0, lddy=1) == oz.OZ_OK
    assert wgrad(k=0, ldx=1, ldw=1, sw=8) == oz.OZ_OK


def test_grouped_workspace():
    # a sum of few k-blocks and 16-byte aligned operands: nothing to split, nothing to lay out
    assert lib.ozaki_grouped_gemm_workspace_bytes(64, 64, 32, 2, oz.OZ_BF16, P, 64, 4096, P, 64) == 0
    assert lib.ozaki_grouped_gemm_workspace_bytes(64, 1024, 32, 2, oz.OZ_BF16, P, 1024, 65536, P, 1024) == 0
    long = lib.ozaki_grouped_gemm_workspace_bytes(64, 8192, 32, 2, oz.OZ_BF16, P, 8192, 524288, P, 8192)
    assert long > 0
    # an odd row stride of W or X, or an odd address, adds the room to lay it out
    odd = lib.ozaki_grouped_gemm_workspace_bytes(64, 8192, 32, 2, oz.OZ_BF16, P, 8193, 524400, P, 8192)
    assert odd >= long + 2 * 2 * 64 * 8192
    assert lib.ozaki_grouped_gemm_workspace_bytes(64, 8192, 32, 2, oz.OZ_BF16, P, 8192, 524288, P + 2, 8192) >= long + 2 * 32 * 8192
    assert lib.ozaki_grouped_gemm_workspace_bytes(64, -1, 32, 2, oz.OZ_BF16, P, 1024, 65536, P, 1024) == 0
    assert lib.ozaki_grouped_gemm_dgrad_workspace_bytes(8192, 64, 32, 2, oz.OZ_F16, P, 64, 524288, P, 8192) > 0
    assert lib.ozaki_grouped_gemm_wgrad_workspace_bytes(64, 64, 16384, 2, oz.OZ_F16, P, 64, P, 64) > 0
    # too small, or not aligned to 256 bytes
    args = (64, 8192, 32, 2, oz.OZ_BF16, P, 8192, 524288, P, 8192, P, P, 64)
    assert lib.ozaki_grouped_gemm_ws(*args, P, long - 1, None) == oz.OZ_ENOMEM
    assert lib.ozaki_grouped_gemm_ws(*args, P + 16, long, None) == oz.OZ_ENOMEM
    assert lib.ozaki_grouped_gemm_ws(*args, None, long, None) == oz.OZ_ENOMEM


def newton(m=300, n=300, batch=1, dtype=oz.OZ_F32, G=P, ldg=300, sg=90000, O=P, ldo=300, so=90000, steps=5, coeffs=FIVE_STEPS, eps=1e-7, slices=2):
    c = None if coeffs is None else np.ascontiguousarray(coeffs, dtype=np.float32)
    return lib.ozaki_newton_schulz_ws(m, n, batch, dtype, G, ldg, sg, O, ldo, so, steps, None if c is None else c.ctypes.data,
                                      ctypes.c_float(eps), slices, P, 16, None)


@pytest.mark.parametrize("bad", [dict(m=-1), dict(n=-1), dict(batch=-1), dict(batch=65536), dict(dtype=0), dict(dtype=4),
                                 dict(ldg=299), dict(ldo=299), dict(batch=2, sg=89999), dict(batch=2, so=89999), dict(steps=0),
                                 dict(steps=oz.OZ_MAX_NS_STEPS + 1), dict(coeffs=None), dict(eps=-1.0),
                                 dict(eps=float("nan")), dict(eps=float("inf")), dict(slices=0), dict(slices=3),
                                 dict(G=None), dict(O=None), dict(coeffs=[float("nan")] * 15)])
def test_newton_schulz_refuses_bad_arguments(bad):
    assert newton(**bad) == oz.OZ_EINVAL


def test_newton_schulz_refuses_polynomials_out_of_range():
    assert newton(steps=1, coeffs=[20.0, 0.0, 0.0]) == oz.OZ_ERANGE       # sigma = 1 goes to 20
    assert newton(steps=5, coeffs=[3.0, 0.0, 0.0] * 5) == oz.OZ_ERANGE    # 3^3 = 27 after three steps
    assert newton(steps=1, coeffs=[1.0, 1.0, 1e-4]) == oz.OZ_ERANGE       # b^2 / 4c = 2500 cancels against a
    assert newton(steps=1, coeffs=[0.0, 0.0, 0.0]) == oz.OZ_ERANGE
    # the usual ones are in range: what stops them here is the workspace
    for c in ([3.4445, -4.775, 2.0315], [1.5, -0.5, 0.0], [1.875, -1.25, 0.375]):
        assert newton(steps=1, coeffs=c) == oz.OZ_ENOMEM


def test_newton_schulz_empty_and_workspace():
    assert newton(m=0) == oz.OZ_OK
    assert newton(n=0) == oz.OZ_OK
    assert newton(batch=0) == oz.OZ_OK
    one, two = (oz.ozaki_newton_schulz_workspace_bytes(300, 500, 3, s) for s in (1, 2))
    assert one >= 2 * 2 * 3 * 300 * 512 and two >= 2 * 2 * 2 * 3 * 300 * 512
    assert oz.ozaki_newton_schulz_workspace_bytes(0, 5) == 0
    assert oz.ozaki_newton_schulz_workspace_bytes(128, 256, 7, 2) == 0  # small matrices need none
    assert oz.ozaki_newton_schulz_workspace_bytes(129, 129, 1, 1) > 0
    assert oz.ozaki_newton_schulz_workspace_bytes(5, 5, 1, 3) == 0


def test_binding_refuses_before_the_library():
    x, w, o = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(2, 6, 8, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        oz.ozaki_grouped_gemm(x, w, o)
    with pytest.raises(ValueError, match="shape"):
        oz.ozaki_grouped_gemm(x[:, :7], w, o)
    with pytest.raises(ValueError, match="row-major"):
        oz.ozaki_grouped_gemm(x.t().contiguous().t(), w, o)
    with pytest.raises(ValueError, match="row-major matrices"):
        oz.ozaki_grouped_gemm(x, w.transpose(1, 2).contiguous().transpose(1, 2), o)
    with pytest.raises(ValueError, match="CUDA"):
        oz.ozaki_newton_schulz(torch.zeros(4, 4))


def test_the_completed_square_is_the_polynomial():
    # B = c (A + b/2c)^2 + a - b^2/4c, which the kernel forms, against a + b A + c A^2
    rng = np.random.default_rng(0)
    for a, b, c in ((3.4445, -4.775, 2.0315), (1.875, -1.25, 0.375)):
        x = rng.standard_normal((6, 9))
        x /= np.linalg.norm(x)
        A = x @ x.T
        S = A + b / (2 * c) * np.eye(6)
        assert np.allclose(c * S @ S + (a - b * b / (4 * c)) * np.eye(6), a * np.eye(6) + b * A + c * A @ A, atol=1e-12)


def test_strides_beyond_an_int_are_refused():
    torch = pytest.importorskip("torch")
    far = 2**31
    assert oz._tokens(torch.empty_strided((1, 8), (far, 1), device="meta"), "X") == 8  # one row: its stride says nothing
    with pytest.raises(ValueError):
        oz._tokens(torch.empty_strided((2, 8), (far, 1), device="meta"), "X")
    with pytest.raises(ValueError):
        oz._tokens(torch.empty_strided((far, 8), (8, 1), device="meta"), "X")
    assert oz._experts(torch.empty_strided((2, 4, 8), (far, 8, 1), device="meta"), "W") == (8, far)  # between matrices: 64 bits
    with pytest.raises(ValueError):
        oz._experts(torch.empty_strided((2, 4, 8), (4 * far, far, 1), device="meta"), "W")
