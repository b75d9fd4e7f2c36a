"""8-bit products, quantisation, RMS norm and clipping: argument checks and host-only queries (no GPU call is made)."""
import ctypes

import pytest
import torch

from fp64_gemm_emulation_gb300 import ozaki as oz

lib = oz._lib
P = 4096  # an address that is never read: every call below returns before any CUDA call
E4M3 = torch.float8_e4m3fn


def forward(n=8, k=16, rows=8, groups=2, tw=oz.OZ_E4M3, W=P, ldw=16, sw=128, SW=P, tx=oz.OZ_E4M3, X=P, ldx=16, SX=P, ldsx=8, off=P,
            dtype=oz.OZ_BF16, Y=P, ldy=8):
    return lib.ozaki_grouped_gemm_f8(n, k, rows, groups, tw, W, ldw, sw, SW, tx, X, ldx, SX, ldsx, off, dtype, Y, ldy, None)


def dgrad(n=16, k=16, rows=8, groups=2, tw=oz.OZ_E4M3, W=P, ldw=16, sw=256, SW=P, tdy=oz.OZ_E5M2, dY=P, lddy=16, SdY=P, ldsdy=8, off=P,
          dtype=oz.OZ_BF16, dX=P, lddx=16):
    return lib.ozaki_grouped_gemm_f8_dgrad(n, k, rows, groups, tw, W, ldw, sw, SW, tdy, dY, lddy, SdY, ldsdy, off, dtype, dX, lddx, None)


def wgrad(n=16, k=16, rows=8, groups=2, tdy=oz.OZ_E5M2, dY=P, lddy=16, SdY=P, ldsdy=16, tx=oz.OZ_E4M3, X=P, ldx=16, SX=P, ldsx=16, off=P,
          dtype=oz.OZ_F16, dW=P, ldw=16, sw=256):
    return lib.ozaki_grouped_gemm_f8_wgrad(n, k, rows, groups, tdy, dY, lddy, SdY, ldsdy, tx, X, ldx, SX, ldsx, off, dtype, dW, ldw, sw, None)


PRODUCTS = [forward, dgrad, wgrad]


@pytest.mark.parametrize("call", PRODUCTS)
@pytest.mark.parametrize("bad", [dict(n=-1), dict(k=-1), dict(rows=-1), dict(rows=2**31 - 1), dict(k=2**31 - 1), dict(groups=0), dict(groups=oz.OZ_MAX_GROUPS + 1),
                                 dict(dtype=oz.OZ_F32), dict(dtype=oz.OZ_E4M3), dict(off=None), dict(ldw=15), dict(sw=127)])
def test_products_refuse_bad_arguments(call, bad):
    assert call(**bad) == oz.OZ_EINVAL


@pytest.mark.parametrize("call,bad", [
    (forward, dict(tw=oz.OZ_BF16)), (forward, dict(tx=0)), (forward, dict(W=None)), (forward, dict(SW=None)), (forward, dict(X=None)),
    (forward, dict(SX=None)), (forward, dict(Y=None)), (forward, dict(W=P + 8)), (forward, dict(X=P + 1)), (forward, dict(SX=P + 2)),
    (forward, dict(Y=P + 1)), (forward, dict(ldw=24)), (forward, dict(sw=136)), (forward, dict(ldx=15)), (forward, dict(ldx=17)),
    (forward, dict(ldsx=7)), (forward, dict(ldy=7)),
    (dgrad, dict(tdy=6)), (dgrad, dict(W=None)), (dgrad, dict(dY=None)), (dgrad, dict(SdY=None)), (dgrad, dict(dX=None)), (dgrad, dict(dY=P + 8)),
    (dgrad, dict(lddy=8)), (dgrad, dict(lddy=24)), (dgrad, dict(ldsdy=7)), (dgrad, dict(lddx=15)),
    (wgrad, dict(tdy=0)), (wgrad, dict(tx=oz.OZ_F16)), (wgrad, dict(dY=None)), (wgrad, dict(X=None)), (wgrad, dict(SX=None)), (wgrad, dict(SdY=None)),
    (wgrad, dict(dW=None)), (wgrad, dict(dW=P + 1)), (wgrad, dict(X=P + 4)), (wgrad, dict(ldx=20)), (wgrad, dict(lddy=15)), (wgrad, dict(ldsx=15)),
    (wgrad, dict(ldsdy=15)),
])
def test_products_refuse_bad_operands(call, bad):
    assert call(**bad) == oz.OZ_EINVAL


def test_empty_products_do_nothing():
    assert forward(n=0, W=None, Y=None) == oz.OZ_OK
    assert forward(rows=0, X=None, Y=None) == oz.OZ_OK
    assert dgrad(k=0, W=None, dX=None) == oz.OZ_OK
    assert dgrad(rows=0, dY=None, dX=None) == oz.OZ_OK
    assert wgrad(n=0, dY=None, dW=None) == oz.OZ_OK
    assert wgrad(k=0, X=None, dW=None) == oz.OZ_OK
    assert forward(groups=1, off=None, rows=0) == oz.OZ_OK


def quantize(block=oz.OZ_BLOCK_BOTH, k=16, rows=8, groups=2, dtype=oz.OZ_BF16, X=P, ldx=16, sx=0, off=P, t=oz.OZ_E4M3, Q=P, ldq=16, sq=0, S=P, lds=8,
             QC=P, ldqc=16, SC=P, ldsc=16):
    return lib.ozaki_quantize_f8(block, k, rows, groups, dtype, X, ldx, sx, off, t, Q, ldq, sq, S, lds, QC, ldqc, SC, ldsc, None)


MATRIX = dict(block=oz.OZ_BLOCK_MATRIX, off=None, sx=128, sq=128)


@pytest.mark.parametrize("bad", [
    dict(block=0), dict(block=5), dict(k=-1), dict(rows=-1), dict(rows=2**31 - 1), dict(groups=0), dict(groups=oz.OZ_MAX_GROUPS + 1), dict(dtype=0),
    dict(dtype=oz.OZ_E4M3), dict(t=oz.OZ_BF16), dict(ldx=15), dict(off=None), dict(X=None), dict(X=P + 1), dict(Q=None), dict(S=None), dict(QC=None),
    dict(SC=None), dict(Q=P + 8), dict(QC=P + 8), dict(S=P + 2), dict(SC=P + 1), dict(ldq=15), dict(ldq=24), dict(ldqc=17), dict(lds=7), dict(ldsc=15),
    dict(block=oz.OZ_BLOCK_ROW), dict(block=oz.OZ_BLOCK_ROW, off=None), dict(block=oz.OZ_BLOCK_ROW, groups=1),
    {**MATRIX, "off": P}, {**MATRIX, "sx": 127}, {**MATRIX, "sq": 127}, {**MATRIX, "sq": 136}, {**MATRIX, "Q": None},
])
def test_quantise_refuses_bad_arguments(bad):
    assert quantize(**bad) == oz.OZ_EINVAL


def test_empty_quantisations_do_nothing():
    assert quantize(k=0, X=None, Q=None) == oz.OZ_OK
    assert quantize(block=oz.OZ_BLOCK_ROW, rows=0, groups=1, off=None, X=None, Q=None, S=None) == oz.OZ_OK
    assert quantize(**MATRIX, rows=0, X=None, Q=None, S=None) == oz.OZ_OK


def test_column_blocks():
    assert [oz.ozaki_f8_column_blocks(r) for r in (0, 1, 128, 129)] == [0, 1, 1, 2]
    assert [oz.ozaki_f8_column_blocks(r, 5) for r in (0, 1, 128, 700)] == [5, 5, 6, 10]
    with pytest.raises(oz.OzakiError):
        oz.ozaki_f8_column_blocks(-1)
    # no two groups meet, and the last one fits
    for lengths in ([0] * 4, [1] * 300, [127, 128, 129, 0, 255, 1], [1000, 3, 0, 0, 200]):
        at, end = 0, 0
        for e, length in enumerate(lengths):
            first = at // 128 + e
            assert first >= end
            end = first + (length + 127) // 128
            at += length
        assert end <= oz.ozaki_f8_column_blocks(at, len(lengths))


def norm(k=16, rows=8, dtype=oz.OZ_BF16, X=P, ldx=16, R=P, ldr=16, W=P, eps=1e-6, Q=P, ldq=16, S=P, lds=8, H=P, ldh=16, rstd=P, Y=P, ldy=16):
    return lib.ozaki_rms_norm_f8(k, rows, dtype, X, ldx, R, ldr, W, eps, Q, ldq, S, lds, H, ldh, rstd, Y, ldy, None)


@pytest.mark.parametrize("bad", [dict(k=-1), dict(k=oz.OZ_MAX_NORM_WIDTH + 1), dict(rows=-1), dict(rows=2**31 - 1, lds=2**31 - 1), dict(dtype=0), dict(dtype=oz.OZ_E4M3), dict(eps=-1.0),
                                 dict(eps=float("nan")), dict(ldx=15), dict(ldr=15), dict(ldh=15), dict(ldy=15), dict(ldq=15), dict(ldq=24), dict(lds=7),
                                 dict(X=None), dict(W=None), dict(Q=None), dict(S=None), dict(rstd=None), dict(X=P + 1), dict(R=P + 1), dict(W=P + 1),
                                 dict(H=P + 1), dict(Y=P + 1), dict(Q=P + 8), dict(S=P + 2), dict(rstd=P + 2)])
def test_norm_refuses_bad_arguments(bad):
    assert norm(**bad) == oz.OZ_EINVAL


def back(k=16, rows=8, dtype=oz.OZ_BF16, dY=P, lddy=16, H=P, ldh=16, W=P, rstd=P, dH=P, lddh=16, dX=P, lddx=16, dW=P, ws=P, nbytes=1 << 20):
    args = (k, rows, dtype, dY, lddy, H, ldh, W, rstd, dH, lddh, dX, lddx, dW)
    a = lib.ozaki_rms_norm_backward_ws(*args, ws, nbytes, None)
    return a if ws is None or nbytes < 1 << 20 else (a, lib.ozaki_rms_norm_backward(*args, None))


@pytest.mark.parametrize("bad", [dict(k=-1), dict(k=oz.OZ_MAX_NORM_WIDTH + 1), dict(rows=-1), dict(rows=2**31 - 1), dict(dtype=0), dict(lddy=15), dict(ldh=15), dict(lddh=15),
                                 dict(lddx=15), dict(dY=None), dict(H=None), dict(W=None), dict(rstd=None), dict(dX=None), dict(dW=None), dict(dY=P + 1)])
def test_norm_backward_refuses_bad_arguments(bad):
    if "dY" in bad and bad["dY"]:
        assert lib.ozaki_rms_norm_backward_ws(16, 8, oz.OZ_BF16, P + 1, 16, P, 16, P, P, P, 16, P, 16, P, P, 1 << 20, None) == oz.OZ_EINVAL
    else:
        assert back(**bad) == (oz.OZ_EINVAL, oz.OZ_EINVAL)


def test_norm_backward_workspace():
    need = oz.ozaki_rms_norm_backward_workspace_bytes(16, 8)
    assert need > 0 and oz.ozaki_rms_norm_backward_workspace_bytes(16, -1) == 0
    assert back(ws=None) == oz.OZ_ENOMEM and back(nbytes=need - 1) == oz.OZ_ENOMEM
    assert norm(rows=0, X=None) == oz.OZ_OK and norm(k=0, X=None) == oz.OZ_OK


def clip(counts=(5, 0), dtypes=None, grads=None, outs=None, limit=1.0, eps=1e-6, result=P, count=None, ws=P, nbytes=1 << 20):
    n = len(counts)
    grads = [P] * n if grads is None else grads
    args = (n if count is None else count, (ctypes.c_int * n)(*(dtypes or [oz.OZ_F32] * n)), (ctypes.c_void_p * n)(*grads),
            (ctypes.c_void_p * n)(*(grads if outs is None else outs)), (ctypes.c_longlong * n)(*counts), limit, eps, result)
    return lib.ozaki_clip_grad_norm_ws(*args, ws, nbytes, None)


@pytest.mark.parametrize("bad", [dict(count=-1), dict(count=1 << 20), dict(dtypes=[oz.OZ_F32, 0]), dict(grads=[None, P]), dict(outs=[None, P]),
                                 dict(grads=[P + 2, P]), dict(counts=(5, -1)), dict(limit=-1.0), dict(limit=float("nan")), dict(eps=-1e-9),
                                 dict(result=None), dict(result=P + 1)])
def test_clip_refuses_bad_arguments(bad):
    assert clip(**bad) == oz.OZ_EINVAL


def test_clip_refuses_outputs_that_meet():
    f32, bf16 = oz.OZ_F32, oz.OZ_BF16
    assert clip(counts=(5, 5), grads=[P, P]) == oz.OZ_EINVAL                                    # one tensor twice
    assert clip(counts=(5, 5), grads=[P + 16, P]) == oz.OZ_EINVAL                               # its end in another's
    assert clip(counts=(5, 5), dtypes=[bf16, f32], grads=[P + 64, P + 128], outs=[P, P + 8]) == oz.OZ_EINVAL
    for fine in (dict(counts=(4, 5), grads=[P, P + 16]), dict(counts=(5, 4), grads=[P + 16, P]), dict(counts=(5, 0), grads=[P, P])):
        assert clip(**fine, ws=None) == oz.OZ_ENOMEM  # past the checks of the tensors


def test_clip_workspace():
    need = oz.ozaki_clip_grad_norm_workspace_bytes()
    assert clip(ws=None) == oz.OZ_ENOMEM and clip(nbytes=need - 1) == oz.OZ_ENOMEM and clip(ws=P + 8) == oz.OZ_ENOMEM


def test_binding_refuses_host_tensors_and_wrong_shapes():
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    q, s = torch.zeros(4, 32, dtype=E4M3), torch.zeros(4, 1)
    for call in (lambda: oz.ozaki_quantize_f8(x), lambda: oz.ozaki_rms_norm_f8(x, x[0]), lambda: oz.ozaki_rms_norm_backward(x, x, x[0], s[:, 0]),
                 lambda: oz.ozaki_clip_grad_norm([x], 1.0), lambda: oz.ozaki_grouped_gemm_f8(q, s, q, torch.zeros(1, 1)),
                 lambda: oz.ozaki_grouped_gemm_f8_dgrad(q, s, q, torch.zeros(1, 1)), lambda: oz.ozaki_grouped_gemm_f8_wgrad(q, s, q, s)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="block"):
        oz.ozaki_quantize_f8(x, "tile")
    with pytest.raises(ValueError, match="no gradients"):
        oz.ozaki_clip_grad_norm([], 1.0)


@pytest.mark.parametrize("lists, error", [
    (([torch.zeros(3)], [torch.zeros(3)]), ValueError),  # not on a GPU
    (([3], [3]), TypeError),
    (([torch.zeros(3, dtype=torch.float64)], [None]), ValueError),
    (((), ()), TypeError),                               # lists
    (([],), TypeError),
])
def test_facts_of_tensors_refuse(lists, error):
    with pytest.raises(error):
        oz._tensor_lists().pairs(*lists)


def test_facts_of_no_tensors():
    assert oz._tensor_lists().pairs([], []) == (-1, b"", b"", b"", b"")
