"""Python binding of libozaki (argument marshalling only; every step runs in the CUDA kernels).

The functions carry the C ABI's names (``include/ozaki.h``).  Device operands are
torch CUDA tensors; matrices are column-major float64 (a tensor ``X`` of shape
(rows, cols) with ``X.stride(0) == 1``; :func:`colmajor` makes one).  Calls are
ordered on the current torch CUDA stream unless ``stream`` (a torch stream or a raw handle) is
given.  Such a call is what it would be inside ``with torch.cuda.stream(stream)``: the caller
sees to it that the operands are ready there, and new results are memory of that stream.  The
operands' memory is kept until the stream has done the call's work, so the stream has to outlive them.

There is no fallback: if ``libozaki.so`` is missing or fails to load, importing
this module raises, and every call reports the library's status code as an
exception.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import sys

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libozaki.so")

OZ_OK, OZ_EINVAL, OZ_ERANGE, OZ_ECUDA, OZ_ENOMEM, OZ_ETIMEOUT, OZ_ENODEV = 0, -1, -2, -3, -4, -5, -6
OZ_EXP_EMPTY = np.int32(np.uint32(0x80808080).view(np.int32))
OZ_EXP_NONFINITE = np.int32(0x7FFFFFFF)
PAD_M, PAD_N, PAD_K = 256, 256, 64
OZ_NOALLOC_SCRATCH_BYTES = 64 << 20
OZ_SCALE_UNIFORM, OZ_SCALE_FAST, OZ_SCALE_ACCU = 0, 1, 2
OZ_OZAKI1_RN, OZ_OZAKI1_EF, OZ_OZAKI1_HYBRID = 0, 1, 2
OZ_BF16, OZ_F16, OZ_F32 = 1, 2, 3
OZ_E4M3, OZ_E5M2 = 4, 5
OZ_BLOCK_ROW, OZ_BLOCK_COLUMN, OZ_BLOCK_BOTH, OZ_BLOCK_MATRIX = 1, 2, 3, 4
OZ_MAX_GROUPS, OZ_MAX_NS_STEPS, OZ_MAX_NORM_WIDTH = 1024, 32, 32768
F8_BLOCK = 128
F8_BLOCKS = {"row": OZ_BLOCK_ROW, "column": OZ_BLOCK_COLUMN, "both": OZ_BLOCK_BOTH, "matrix": OZ_BLOCK_MATRIX}
OZAKI1_VARIANTS = {"rn": OZ_OZAKI1_RN, "ef": OZ_OZAKI1_EF, "hybrid": OZ_OZAKI1_HYBRID}
SCALINGS = {"uniform": OZ_SCALE_UNIFORM, "fast": OZ_SCALE_FAST, "accu": OZ_SCALE_ACCU}


class OzakiError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {_lib.ozaki_status_string(code).decode()}")


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m fp64_gemm_emulation_gb300.build_lib`")
    lib = ctypes.CDLL(LIB_PATH)
    I, L, P, S, F = ctypes.c_int, ctypes.c_longlong, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_float
    sig = {
        "ozaki2_moduli": (I, [I, P]),
        "ozaki2_choose_k": (I, [I, L, P]),
        "ozaki2_plane_dims": (I, [I, I, I, P, P, P]),
        "ozaki2_workspace_bytes": (S, [I, I, I, I]),
        "ozaki2_exponents": (I, [I, I, I, P, I, P, I, P, P, P]),
        "ozaki2_split": (I, [I, I, I, P, I, P, I, I, P, P, P, P, P]),
        "ozaki2_residue_gemm": (I, [I, I, I, I, P, P, P, P]),
        "ozaki2_scale_split": (I, [I, I, I, P, I, P, I, I, P, P, P, P, P]),
        "ozaki2_crt": (I, [I, I, I, I, P, P, P, P, I, P]),
        "ozaki2_dgemm_ws": (I, [I, I, I, P, I, P, I, P, I, I, P, S, P]),
        "ozaki2_dgemm": (I, [I, I, I, P, I, P, I, P, I, I, P]),
        "ozaki2_dgemm_host": (I, [I, I, I, P, I, P, I, P, I, I]),
        "ozaki2_dgemm_noalloc": (I, [I, I, I, P, I, P, I, P, I, I, P]),
        "ozaki2_scaling_k": (I, [I, L, I, P]),
        "ozaki2_exponents_workspace_bytes": (S, [I, I, I, I]),
        "ozaki2_exponents_ex": (I, [I, I, I, P, I, P, I, I, I, P, P, P, S, P]),
        "ozaki2_split_ex": (I, [I, I, I, P, I, P, I, I, I, P, P, P, P, P]),
        "ozaki2_crt_ex": (I, [I, I, I, I, I, P, P, P, P, I, P]),
        "ozaki2_workspace_bytes_ex": (S, [I, I, I, I, I]),
        "ozaki2_dgemm_ex_ws": (I, [I, I, I, P, I, P, I, P, I, I, I, P, S, P]),
        "ozaki2_dgemm_ex": (I, [I, I, I, P, I, P, I, P, I, I, I, P]),
        "ozaki1_beta": (I, [L, P]),
        "ozaki1_split_scratch_bytes": (S, [I, I, I]),
        "ozaki1_workspace_bytes": (S, [I, I, I, I]),
        "ozaki1_split": (I, [I, I, I, P, I, P, I, I, P, P, P, P, P, S, P]),
        "ozaki1_slice_gemm": (I, [I, I, I, I, P, P, P, P]),
        "ozaki1_accumulate": (I, [I, I, I, I, P, P, P, P, I, P]),
        "ozaki1_dgemm_ws": (I, [I, I, I, P, I, P, I, P, I, I, P, S, P]),
        "ozaki1_dgemm": (I, [I, I, I, P, I, P, I, P, I, I, P]),
        "ozaki1_group_r": (I, [L, P]),
        "ozaki1_num_batches": (I, [I, L, I, P]),
        "ozaki1_split_scratch_bytes_ex": (S, [I, I, I, I]),
        "ozaki1_workspace_bytes_ex": (S, [I, I, I, I, I]),
        "ozaki1_split_ex": (I, [I, I, I, P, I, P, I, I, I, P, P, P, P, P, S, P]),
        "ozaki1_slice_gemm_ex": (I, [I, I, I, I, I, P, P, P, P]),
        "ozaki1_accumulate_ex": (I, [I, I, I, I, I, P, P, P, P, I, P]),
        "ozaki1_dgemm_ex_ws": (I, [I, I, I, P, I, P, I, P, I, I, I, P, S, P]),
        "ozaki1_dgemm_ex": (I, [I, I, I, P, I, P, I, P, I, I, I, P]),
        "ozaki_grouped_gemm_workspace_bytes": (S, [I, I, I, I, I, P, I, L, P, I]),
        "ozaki_grouped_gemm_dgrad_workspace_bytes": (S, [I, I, I, I, I, P, I, L, P, I]),
        "ozaki_grouped_gemm_wgrad_workspace_bytes": (S, [I, I, I, I, I, P, I, P, I]),
        "ozaki_grouped_gemm_ws": (I, [I, I, I, I, I, P, I, L, P, I, P, P, I, P, S, P]),
        "ozaki_grouped_gemm_dgrad_ws": (I, [I, I, I, I, I, P, I, L, P, I, P, P, I, P, S, P]),
        "ozaki_grouped_gemm_wgrad_ws": (I, [I, I, I, I, I, P, I, P, I, P, P, I, L, P, S, P]),
        "ozaki_grouped_gemm": (I, [I, I, I, I, I, P, I, L, P, I, P, P, I, P]),
        "ozaki_grouped_gemm_dgrad": (I, [I, I, I, I, I, P, I, L, P, I, P, P, I, P]),
        "ozaki_grouped_gemm_wgrad": (I, [I, I, I, I, I, P, I, P, I, P, P, I, L, P]),
        "ozaki_newton_schulz_workspace_bytes": (S, [I, I, I, I]),
        "ozaki_newton_schulz_ws": (I, [I, I, I, I, P, I, L, P, I, L, I, P, ctypes.c_float, I, P, S, P]),
        "ozaki_newton_schulz": (I, [I, I, I, I, P, I, L, P, I, L, I, P, ctypes.c_float, I, P]),
        "ozaki_f8_column_blocks": (I, [I, I, I]),
        "ozaki_quantize_f8": (I, [I, I, I, I, I, P, I, L, P, I, P, I, L, P, I, P, I, P, I, P]),
        "ozaki_grouped_gemm_f8": (I, [I, I, I, I, I, P, I, L, P, I, P, I, P, I, P, I, P, I, P]),
        "ozaki_grouped_gemm_f8_dgrad": (I, [I, I, I, I, I, P, I, L, P, I, P, I, P, I, P, I, P, I, P]),
        "ozaki_grouped_gemm_f8_wgrad": (I, [I, I, I, I, I, P, I, P, I, I, P, I, P, I, P, I, P, I, L, P]),
        "ozaki_rms_norm_f8": (I, [I, I, I, P, I, P, I, P, F, P, I, P, I, P, I, P, P, I, P]),
        "ozaki_rms_norm_backward_workspace_bytes": (S, [I, I]),
        "ozaki_rms_norm_backward_ws": (I, [I, I, I, P, I, P, I, P, P, P, I, P, I, P, P, S, P]),
        "ozaki_rms_norm_backward": (I, [I, I, I, P, I, P, I, P, P, P, I, P, I, P, P]),
        "ozaki_clip_grad_norm_workspace_bytes": (S, []),
        "ozaki_clip_grad_norm_ws": (I, [I, P, P, P, P, F, F, P, P, S, P]),
        "ozaki_clip_grad_norm": (I, [I, P, P, P, P, F, F, P, P]),
        "ozaki_get_device_status": (I, [P]),
        "ozaki_status_string": (ctypes.c_char_p, [I]),
        "ozaki_set_epilogue_wait_ns": (I, [L]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = _load()


def _check(rc: int, where: str) -> None:
    if rc != OZ_OK:
        raise OzakiError(rc, where)


def _stream(stream):
    if stream is None:
        import torch

        return torch.cuda.current_stream().cuda_stream
    return int(getattr(stream, "cuda_stream", stream))


def _other_stream(stream, device):
    """`stream` as a torch stream, or None where it is (or stands for) the device's current one."""
    if stream is None or device.type != "cuda":
        return None
    torch = _torch()
    handle = int(getattr(stream, "cuda_stream", stream))
    if handle == torch._C._cuda_getCurrentRawStream(device.index):
        return None
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)


def _call_on(stream, fn, *operands, **named):
    """fn on another stream than the current one: what it allocates comes from that stream's memory (a block of the
    current stream's may still be in use there), and the operands' blocks are not handed out again before
    that stream has done with them."""
    torch = _torch()
    with torch.cuda.stream(stream):
        result = fn(*operands, **named)
    for t in (*operands, *named.values()):
        if isinstance(t, torch.Tensor) and t.is_cuda:
            t.record_stream(stream)
    return result


def _on_given_stream(fn):
    """A function whose last parameter is the stream, able to run on one that is not the current one."""
    last = fn.__code__.co_argcount - 1

    @functools.wraps(fn)
    def call(*args, **named):
        stream = args[last] if len(args) > last else named.get("stream")
        if stream is not None:
            device = next((t.device for t in (*args, *named.values()) if isinstance(t, _torch().Tensor)), None)
            other = device and _other_stream(stream, device)
            if other:
                named.pop("stream", None)
                return _call_on(other, fn, *args[:last], **named)
        return fn(*args, **named)

    return call


def _torch():
    """torch, which whoever passes tensors has imported (an import statement costs more than this lookup)."""
    return sys.modules["torch"]


def _ptr(t):
    return None if t is None else t.data_ptr()


def colmajor(x):
    """A column-major copy (or view) of a 2-D tensor: same shape, stride(0) == 1."""
    return x if (x.dim() == 2 and x.stride(0) == 1 and x.stride(1) >= max(1, x.shape[0])) else x.t().contiguous().t()


def _ld(x) -> int:
    assert x.dim() == 2 and x.stride(0) == 1, "operand must be column-major (stride(0) == 1)"
    return max(1, int(x.stride(1)), int(x.shape[0]))


# ------------------------------------------------------------------ host-only queries
def ozaki2_moduli(num_moduli: int) -> list[int]:
    out = (ctypes.c_int * max(1, num_moduli))()
    _check(_lib.ozaki2_moduli(num_moduli, out), "ozaki2_moduli")
    return list(out[:num_moduli])


def ozaki2_choose_k(num_moduli: int, k_inner: int) -> int:
    k = ctypes.c_int()
    _check(_lib.ozaki2_choose_k(num_moduli, k_inner, ctypes.byref(k)), "ozaki2_choose_k")
    return k.value


def ozaki2_plane_dims(m: int, n: int, k: int) -> tuple[int, int, int]:
    a, b, c = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    _check(_lib.ozaki2_plane_dims(m, n, k, ctypes.byref(a), ctypes.byref(b), ctypes.byref(c)), "ozaki2_plane_dims")
    return a.value, b.value, c.value


def ozaki2_workspace_bytes(m: int, n: int, k: int, num_moduli: int) -> int:
    return int(_lib.ozaki2_workspace_bytes(m, n, k, num_moduli))


# ------------------------------------------------------------------ steps
@_on_given_stream
def ozaki2_exponents(A, B, stream=None):
    """Step a1: (rowexp[m], colexp[n]) int32 tensors on A's device."""
    import torch

    m, k = A.shape
    n = B.shape[1]
    rowexp = torch.empty(m, dtype=torch.int32, device=A.device)
    colexp = torch.empty(n, dtype=torch.int32, device=A.device)
    _check(_lib.ozaki2_exponents(m, n, k, _ptr(A), _ld(A), _ptr(B), _ld(B), _ptr(rowexp), _ptr(colexp),
                                 _stream(stream)), "ozaki2_exponents")
    return rowexp, colexp


@_on_given_stream
def ozaki2_split(A, B, num_moduli: int, rowexp, colexp, stream=None):
    """Step a2: bf16-bit residue planes (uint16 views as int16 tensors) [s, Mp, Kp] and [s, Np, Kp]."""
    import torch

    m, k = A.shape
    n = B.shape[1]
    mp, np_, kp = ozaki2_plane_dims(m, n, k)
    Ap = torch.empty((num_moduli, mp, kp), dtype=torch.int16, device=A.device)
    Bp = torch.empty((num_moduli, np_, kp), dtype=torch.int16, device=A.device)
    _check(_lib.ozaki2_split(m, n, k, _ptr(A), _ld(A), _ptr(B), _ld(B), num_moduli, _ptr(rowexp), _ptr(colexp),
                             _ptr(Ap), _ptr(Bp), _stream(stream)), "ozaki2_split")
    return Ap, Bp


@_on_given_stream
def ozaki2_scale_split(A, B, num_moduli: int, stream=None):
    """Steps a1 + a2 in one call: (rowexp, colexp, A_planes, B_planes); either operand may be None."""
    import torch

    dev = (A if A is not None else B).device
    k = A.shape[1] if A is not None else B.shape[0]
    m = A.shape[0] if A is not None else 0
    n = B.shape[1] if B is not None else 0
    mp, np_, kp = ozaki2_plane_dims(m, n, k)
    rowexp = torch.empty(m, dtype=torch.int32, device=dev) if A is not None else None
    colexp = torch.empty(n, dtype=torch.int32, device=dev) if B is not None else None
    Ap = torch.empty((num_moduli, mp, kp), dtype=torch.int16, device=dev) if A is not None else None
    Bp = torch.empty((num_moduli, np_, kp), dtype=torch.int16, device=dev) if B is not None else None
    _check(_lib.ozaki2_scale_split(m, n, k, _ptr(A), _ld(A) if A is not None else 1, _ptr(B),
                                   _ld(B) if B is not None else 1, num_moduli, _ptr(rowexp), _ptr(colexp),
                                   _ptr(Ap), _ptr(Bp), _stream(stream)), "ozaki2_scale_split")
    return rowexp, colexp, Ap, Bp


@_on_given_stream
def ozaki2_residue_gemm(m: int, n: int, k: int, num_moduli: int, A_planes, B_planes, stream=None):
    """Steps a3+a4: C_res uint8 tensor [s, Np, Mp] with C''_t = (A'_t B'_t) mod m_t."""
    import torch

    mp, np_, kp = ozaki2_plane_dims(m, n, k)
    Cr = torch.empty((num_moduli, np_, mp), dtype=torch.uint8, device=A_planes.device)
    _check(_lib.ozaki2_residue_gemm(m, n, k, num_moduli, _ptr(A_planes), _ptr(B_planes), _ptr(Cr),
                                    _stream(stream)), "ozaki2_residue_gemm")
    return Cr


@_on_given_stream
def ozaki2_crt(m: int, n: int, k: int, num_moduli: int, C_res, rowexp, colexp, C=None, stream=None):
    """Steps a5+a6: C (m x n column-major float64)."""
    import torch

    if C is None:
        C = torch.empty((n, m), dtype=torch.float64, device=C_res.device).t()
    _check(_lib.ozaki2_crt(m, n, k, num_moduli, _ptr(C_res), _ptr(rowexp), _ptr(colexp), _ptr(C), _ld(C),
                           _stream(stream)), "ozaki2_crt")
    return C


# ------------------------------------------------------------------ composed
@_on_given_stream
def ozaki2_dgemm(A, B, num_moduli: int = 14, C=None, stream=None):
    """C = A B by Ozaki Scheme II (stream-ordered workspace allocation inside the library)."""
    import torch

    m, k = A.shape
    n = B.shape[1]
    if C is None:
        C = torch.empty((n, m), dtype=torch.float64, device=A.device).t()
    _check(_lib.ozaki2_dgemm(m, n, k, _ptr(A), _ld(A), _ptr(B), _ld(B), _ptr(C), _ld(C), num_moduli,
                             _stream(stream)), "ozaki2_dgemm")
    return C


@_on_given_stream
def ozaki2_dgemm_ws(A, B, num_moduli: int, workspace, C=None, stream=None):
    """C = A B using a caller-owned device workspace (a uint8 tensor of at least
    ozaki2_workspace_bytes(m, n, k, num_moduli) bytes)."""
    import torch

    m, k = A.shape
    n = B.shape[1]
    if C is None:
        C = torch.empty((n, m), dtype=torch.float64, device=A.device).t()
    _check(_lib.ozaki2_dgemm_ws(m, n, k, _ptr(A), _ld(A), _ptr(B), _ld(B), _ptr(C), _ld(C), num_moduli,
                                _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)),
           "ozaki2_dgemm_ws")
    return C


@_on_given_stream
def ozaki2_dgemm_noalloc(A, B, num_moduli: int = 14, C=None, stream=None):
    """C = A B without any device allocation: the library's fixed 64 MiB scratch buffer
    holds the workspace (for callers that cannot allocate; see include/ozaki.h)."""
    import torch

    m, k = A.shape
    n = B.shape[1]
    if C is None:
        C = torch.empty((n, m), dtype=torch.float64, device=A.device).t()
    _check(_lib.ozaki2_dgemm_noalloc(m, n, k, _ptr(A), _ld(A), _ptr(B), _ld(B), _ptr(C), _ld(C), num_moduli,
                                     _stream(stream)), "ozaki2_dgemm_noalloc")
    return C


def ozaki2_dgemm_host(A: np.ndarray, B: np.ndarray, num_moduli: int = 14, C: np.ndarray | None = None):
    """C = A B with HOST (numpy, column-major float64) operands; synchronous."""
    A = np.asfortranarray(A, dtype=np.float64)
    B = np.asfortranarray(B, dtype=np.float64)
    m, k = A.shape
    n = B.shape[1]
    if C is None:
        C = np.empty((m, n), dtype=np.float64, order="F")
    assert C.flags.f_contiguous and C.dtype == np.float64
    _check(_lib.ozaki2_dgemm_host(m, n, k, A.ctypes.data, max(1, m), B.ctypes.data, max(1, k), C.ctypes.data,
                                  max(1, m), num_moduli), "ozaki2_dgemm_host")
    return C


def ozaki2_dgemm_host_ptr(m, n, k, a_ptr, lda, b_ptr, ldb, c_ptr, ldc, num_moduli):
    """Raw-pointer form of ozaki2_dgemm_host (host pointers, e.g. pinned torch tensors)."""
    _check(_lib.ozaki2_dgemm_host(m, n, k, a_ptr, lda, b_ptr, ldb, c_ptr, ldc, num_moduli), "ozaki2_dgemm_host")


# ------------------------------------------------------------------ range estimation modes
def _scaling(scaling) -> int:
    return SCALINGS[scaling] if isinstance(scaling, str) else int(scaling)


def ozaki2_scaling_k(num_moduli: int, k_inner: int, scaling="uniform") -> int:
    k = ctypes.c_int()
    _check(_lib.ozaki2_scaling_k(num_moduli, k_inner, _scaling(scaling), ctypes.byref(k)), "ozaki2_scaling_k")
    return k.value


def ozaki2_exponents_workspace_bytes(m: int, n: int, k: int, scaling="uniform") -> int:
    return int(_lib.ozaki2_exponents_workspace_bytes(m, n, k, _scaling(scaling)))


def ozaki2_workspace_bytes_ex(m: int, n: int, k: int, num_moduli: int, scaling="uniform") -> int:
    return int(_lib.ozaki2_workspace_bytes_ex(m, n, k, num_moduli, _scaling(scaling)))


@_on_given_stream
def ozaki2_exponents_ex(A, B, num_moduli: int, scaling="uniform", stream=None):
    """Step a1 in a scaling mode: (rowexp[m], colexp[n]) int32 tensors."""
    import torch

    m, k = A.shape
    n = B.shape[1]
    sc = _scaling(scaling)
    rowexp = torch.empty(m, dtype=torch.int32, device=A.device)
    colexp = torch.empty(n, dtype=torch.int32, device=A.device)
    nbytes = ozaki2_exponents_workspace_bytes(m, n, k, sc)
    ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=A.device)
    _check(_lib.ozaki2_exponents_ex(m, n, k, _ptr(A), _ld(A), _ptr(B), _ld(B), num_moduli, sc, _ptr(rowexp),
                                    _ptr(colexp), _ptr(ws), nbytes, _stream(stream)), "ozaki2_exponents_ex")
    return rowexp, colexp


@_on_given_stream
def ozaki2_split_ex(A, B, num_moduli: int, rowexp, colexp, scaling="uniform", stream=None):
    """Step a2 for exponents of a scaling mode (planes as in ozaki2_split)."""
    import torch

    m, k = A.shape
    n = B.shape[1]
    mp, np_, kp = ozaki2_plane_dims(m, n, k)
    Ap = torch.empty((num_moduli, mp, kp), dtype=torch.int16, device=A.device)
    Bp = torch.empty((num_moduli, np_, kp), dtype=torch.int16, device=A.device)
    _check(_lib.ozaki2_split_ex(m, n, k, _ptr(A), _ld(A), _ptr(B), _ld(B), num_moduli, _scaling(scaling),
                                _ptr(rowexp), _ptr(colexp), _ptr(Ap), _ptr(Bp), _stream(stream)), "ozaki2_split_ex")
    return Ap, Bp


@_on_given_stream
def ozaki2_crt_ex(m: int, n: int, k: int, num_moduli: int, C_res, rowexp, colexp, scaling="uniform", C=None,
                  stream=None):
    """Steps a5+a6 for exponents of a scaling mode."""
    import torch

    if C is None:
        C = torch.empty((n, m), dtype=torch.float64, device=C_res.device).t()
    _check(_lib.ozaki2_crt_ex(m, n, k, num_moduli, _scaling(scaling), _ptr(C_res), _ptr(rowexp), _ptr(colexp),
                              _ptr(C), _ld(C), _stream(stream)), "ozaki2_crt_ex")
    return C


@_on_given_stream
def ozaki2_dgemm_ex(A, B, num_moduli: int = 14, scaling="uniform", C=None, workspace=None, stream=None):
    """C = A B by Ozaki Scheme II in a scaling mode ("uniform", "fast", "accu");
    with ``workspace`` (uint8 tensor of ozaki2_workspace_bytes_ex bytes) the _ws form."""
    import torch

    m, k = A.shape
    n = B.shape[1]
    if C is None:
        C = torch.empty((n, m), dtype=torch.float64, device=A.device).t()
    sc = _scaling(scaling)
    if workspace is None:
        rc = _lib.ozaki2_dgemm_ex(m, n, k, _ptr(A), _ld(A), _ptr(B), _ld(B), _ptr(C), _ld(C), num_moduli, sc,
                                  _stream(stream))
    else:
        rc = _lib.ozaki2_dgemm_ex_ws(m, n, k, _ptr(A), _ld(A), _ptr(B), _ld(B), _ptr(C), _ld(C), num_moduli, sc,
                                     _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    _check(rc, "ozaki2_dgemm_ex")
    return C


@_on_given_stream
def ozaki2_dgemm_ex_ws(A, B, num_moduli: int, scaling, workspace, C=None, stream=None):
    """C = A B in a scaling mode with a caller-owned workspace (ozaki2_workspace_bytes_ex bytes)."""
    return ozaki2_dgemm_ex(A, B, num_moduli, scaling, C=C, workspace=workspace, stream=stream)


# ------------------------------------------------------------------ Scheme I
def ozaki1_beta(k_inner: int) -> int:
    b = ctypes.c_int()
    _check(_lib.ozaki1_beta(k_inner, ctypes.byref(b)), "ozaki1_beta")
    return b.value


def ozaki1_split_scratch_bytes(m: int, n: int, k: int) -> int:
    return int(_lib.ozaki1_split_scratch_bytes(m, n, k))


def ozaki1_workspace_bytes(m: int, n: int, k: int, num_slices: int) -> int:
    return int(_lib.ozaki1_workspace_bytes(m, n, k, num_slices))


@_on_given_stream
def ozaki1_split(A, B, num_slices: int, stream=None):
    """RN split: (A_planes [s,Mp,Kp], B_planes [s,Np,Kp] as int16 bf16 bits, A_exps [s,m], B_exps [s,n])."""
    import torch

    m, k = A.shape
    n = B.shape[1]
    mp, np_, kp = ozaki2_plane_dims(m, n, k)
    Ap = torch.empty((num_slices, mp, kp), dtype=torch.int16, device=A.device)
    Bp = torch.empty((num_slices, np_, kp), dtype=torch.int16, device=A.device)
    Ae = torch.empty((num_slices, m), dtype=torch.int32, device=A.device)
    Be = torch.empty((num_slices, n), dtype=torch.int32, device=A.device)
    nbytes = ozaki1_split_scratch_bytes(m, n, k)
    scratch = torch.empty(nbytes + 256, dtype=torch.uint8, device=A.device)
    sp = (scratch.data_ptr() + 255) // 256 * 256
    _check(_lib.ozaki1_split(m, n, k, _ptr(A), _ld(A), _ptr(B), _ld(B), num_slices, _ptr(Ap), _ptr(Bp),
                             _ptr(Ae), _ptr(Be), sp, nbytes, _stream(stream)), "ozaki1_split")
    return Ap, Bp, Ae, Be


@_on_given_stream
def ozaki1_slice_gemm(m: int, n: int, k: int, num_slices: int, A_planes, B_planes, stream=None):
    """Exact INT32 products [s(s+1)/2, Np, Mp] of the slice pairs (i outer, j inner)."""
    import torch

    mp, np_, kp = ozaki2_plane_dims(m, n, k)
    P = torch.empty((num_slices * (num_slices + 1) // 2, np_, mp), dtype=torch.int32, device=A_planes.device)
    _check(_lib.ozaki1_slice_gemm(m, n, k, num_slices, _ptr(A_planes), _ptr(B_planes), _ptr(P), _stream(stream)),
           "ozaki1_slice_gemm")
    return P


@_on_given_stream
def ozaki1_accumulate(m: int, n: int, k: int, num_slices: int, products, A_exps, B_exps, C=None, stream=None):
    import torch

    if C is None:
        C = torch.empty((n, m), dtype=torch.float64, device=products.device).t()
    _check(_lib.ozaki1_accumulate(m, n, k, num_slices, _ptr(products), _ptr(A_exps), _ptr(B_exps), _ptr(C), _ld(C),
                                  _stream(stream)), "ozaki1_accumulate")
    return C


@_on_given_stream
def ozaki1_dgemm(A, B, num_slices: int = 7, C=None, stream=None):
    """C = A B by Ozaki Scheme I (stream-ordered workspace inside the library)."""
    import torch

    m, k = A.shape
    n = B.shape[1]
    if C is None:
        C = torch.empty((n, m), dtype=torch.float64, device=A.device).t()
    _check(_lib.ozaki1_dgemm(m, n, k, _ptr(A), _ld(A), _ptr(B), _ld(B), _ptr(C), _ld(C), num_slices,
                             _stream(stream)), "ozaki1_dgemm")
    return C


@_on_given_stream
def ozaki1_dgemm_ws(A, B, num_slices: int, workspace, C=None, stream=None):
    import torch

    m, k = A.shape
    n = B.shape[1]
    if C is None:
        C = torch.empty((n, m), dtype=torch.float64, device=A.device).t()
    _check(_lib.ozaki1_dgemm_ws(m, n, k, _ptr(A), _ld(A), _ptr(B), _ld(B), _ptr(C), _ld(C), num_slices,
                                _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)),
           "ozaki1_dgemm_ws")
    return C


# ------------------------------------------------------------------ grouped products (experts)
_DTYPE_CODES: dict = {}


_INT_MAX = 2**31 - 1


def _dtype(t) -> int:
    if not _DTYPE_CODES:
        import torch

        _DTYPE_CODES.update({torch.bfloat16: OZ_BF16, torch.float16: OZ_F16, torch.float32: OZ_F32})
    code = _DTYPE_CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"dtype must be bfloat16, float16 or float32: {t.dtype}")
    return code


def _tokens(t, what: str, features: int | None = None) -> int:
    """Leading dimension of a row-major (rows, features) matrix whose rows may be strided."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or (features is not None and shape[1] != features):
        raise ValueError(f"{what} must have shape (rows, {'features' if features is None else features}): {tuple(shape)}")
    cols = shape[1]
    if max(shape[0], cols, stride[0] if shape[0] > 1 else 0) > _INT_MAX:
        raise ValueError(f"{what} must have dimensions and a row stride below 2^31")
    if shape[0] <= 1:
        if cols > 1 and stride[1] != 1:
            raise ValueError(f"{what} must be row-major (stride(1) == 1)")
        return max(1, cols)
    if (cols > 1 and stride[1] != 1) or stride[0] < cols:
        raise ValueError(f"{what} must be row-major (stride(1) == 1, stride(0) >= {cols})")
    return max(1, stride[0])


def _experts(t, what: str) -> tuple[int, int]:
    """(leading dimension, stride between matrices) of a (groups, n, k) stack of row-major matrices."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 3:
        raise ValueError(f"{what} must have shape (groups, n, k): {tuple(shape)}")
    g, n, k = shape
    ld = max(1, k, stride[1] if n > 1 else 0)
    if max(ld, n) > _INT_MAX:
        raise ValueError(f"{what} must have dimensions and a row stride below 2^31")
    if (k > 1 and stride[2] != 1) or (n > 1 and stride[1] < k) or (g > 1 and stride[0] < ld * n):
        raise ValueError(f"{what} must hold row-major matrices that do not overlap")
    return ld, (stride[0] if g > 1 else ld * n)


def _offsets(offsets, groups: int | None, device):
    n = offsets.numel()
    if offsets.dtype != _torch().int32 or offsets.dim() != 1 or not offsets.is_contiguous() or offsets.device != device:
        raise ValueError("offsets must be a contiguous int32 vector on the operands' device")
    if n < 2 or (groups is not None and n != groups + 1):
        raise ValueError(f"offsets must hold groups + 1 entries: {n} for {groups} groups")


def _same(*tensors):
    dtype, device = tensors[0].dtype, tensors[0].device
    if device.type != "cuda":
        raise ValueError("operands must be CUDA tensors")
    for t in tensors[1:]:
        if t is not None and (t.dtype != dtype or t.device != device):
            raise ValueError("operands must share one dtype and one device")


def _result(out, what: str, rows: int, features: int, like):
    """(out, its leading dimension): checked, or new."""
    if out is None:
        return _torch().empty((rows, features), dtype=like.dtype, device=like.device), max(1, features)
    ld = _tokens(out, what, features)
    if out.shape[0] != rows:
        raise ValueError(f"{what} must have {rows} rows")
    return out, ld


def _stream_of(stream, device) -> int:
    """The raw handle of `stream`, or of the device's current stream."""
    if stream is None:
        return _torch()._C._cuda_getCurrentRawStream(device.index)
    return int(getattr(stream, "cuda_stream", stream))


def _run_on(name, args, workspace, stream, device):
    """Calls `name`, or its _ws form when a workspace (a uint8 tensor) is given, on the operands' device."""
    torch = _torch()
    st = _stream_of(stream, device)
    if workspace is not None:
        if workspace.device != device or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the operands' device")
        name += "_ws"
        args += (workspace.data_ptr(), workspace.numel() * workspace.element_size())
    if device.index == torch._C._cuda_getDevice():
        rc = getattr(_lib, name)(*args, st)
    else:
        with torch.cuda.device(device):
            rc = getattr(_lib, name)(*args, st)
    _check(rc, name)


def ozaki_grouped_gemm(X, W, offsets, Y=None, workspace=None, stream=None):
    """Y[r] = W[e] X[r] for the rows r of group e: X (rows, k), W (groups, n, k), offsets (groups + 1) int32.

    bfloat16 or float16; row-major (rows of X and Y, and the matrices of W, may be strided).
    Rows outside [offsets[0], offsets[-1]) give zero.  Like all functions here it records nothing for
    autograd: the gradients are ozaki_grouped_gemm_dgrad and ozaki_grouped_gemm_wgrad."""
    if stream is not None and (other := _other_stream(stream, X.device)):
        return _call_on(other, ozaki_grouped_gemm, X, W, offsets, Y, workspace)
    ldw, sw = _experts(W, "W")
    groups, n, k = W.shape
    ldx, rows, device = _tokens(X, "X", k), X.shape[0], X.device
    _same(X, W, Y)
    _offsets(offsets, groups, device)
    Y, ldy = _result(Y, "Y", rows, n, X)
    _run_on("ozaki_grouped_gemm", (n, k, rows, groups, _dtype(X), W.data_ptr(), ldw, sw, X.data_ptr(), ldx,
                                        offsets.data_ptr(), Y.data_ptr(), ldy), workspace, stream, device)
    return Y


def ozaki_grouped_gemm_ws(X, W, offsets, workspace, Y=None, stream=None):
    """ozaki_grouped_gemm with a caller-owned workspace (see ozaki_grouped_gemm_workspace_bytes)."""
    return ozaki_grouped_gemm(X, W, offsets, Y, workspace, stream)


def ozaki_grouped_gemm_dgrad(dY, W, offsets, dX=None, workspace=None, stream=None):
    """dX[r] = W[e]^T dY[r]: the gradient in X of a loss whose gradient in Y is dY (rows, n)."""
    if stream is not None and (other := _other_stream(stream, dY.device)):
        return _call_on(other, ozaki_grouped_gemm_dgrad, dY, W, offsets, dX, workspace)
    ldw, sw = _experts(W, "W")
    groups, n, k = W.shape
    lddy, rows, device = _tokens(dY, "dY", n), dY.shape[0], dY.device
    _same(dY, W, dX)
    _offsets(offsets, groups, device)
    dX, lddx = _result(dX, "dX", rows, k, dY)
    _run_on("ozaki_grouped_gemm_dgrad", (n, k, rows, groups, _dtype(dY), W.data_ptr(), ldw, sw, dY.data_ptr(), lddy,
                                              offsets.data_ptr(), dX.data_ptr(), lddx), workspace, stream, device)
    return dX


def ozaki_grouped_gemm_dgrad_ws(dY, W, offsets, workspace, dX=None, stream=None):
    """ozaki_grouped_gemm_dgrad with a caller-owned workspace."""
    return ozaki_grouped_gemm_dgrad(dY, W, offsets, dX, workspace, stream)


def ozaki_grouped_gemm_wgrad(dY, X, offsets, dW=None, workspace=None, stream=None):
    """dW[e] = sum over the rows r of group e of dY[r] X[r]^T: (groups, n, k)."""
    if stream is not None and (other := _other_stream(stream, dY.device)):
        return _call_on(other, ozaki_grouped_gemm_wgrad, dY, X, offsets, dW, workspace)
    lddy, ldx, device = _tokens(dY, "dY"), _tokens(X, "X"), dY.device
    if X.shape[0] != dY.shape[0]:
        raise ValueError("X and dY must have the same rows")
    _offsets(offsets, None, device)
    groups, n, k, rows = offsets.numel() - 1, dY.shape[1], X.shape[1], X.shape[0]
    if dW is None:
        dW = _torch().empty((groups, n, k), dtype=dY.dtype, device=device)
    _same(dY, X, dW)
    ldw, sw = _experts(dW, "dW")
    if tuple(dW.shape) != (groups, n, k):
        raise ValueError(f"dW must have shape {(groups, n, k)}: {tuple(dW.shape)}")
    _run_on("ozaki_grouped_gemm_wgrad", (n, k, rows, groups, _dtype(X), dY.data_ptr(), lddy, X.data_ptr(), ldx,
                                              offsets.data_ptr(), dW.data_ptr(), ldw, sw), workspace, stream, device)
    return dW


def ozaki_grouped_gemm_wgrad_ws(dY, X, offsets, workspace, dW=None, stream=None):
    """ozaki_grouped_gemm_wgrad with a caller-owned workspace."""
    return ozaki_grouped_gemm_wgrad(dY, X, offsets, dW, workspace, stream)


def ozaki_grouped_gemm_workspace_bytes(X, W) -> int:
    """Device workspace of ozaki_grouped_gemm_ws for these operands (alignment decides part of it)."""
    ldw, sw = _experts(W, "W")
    groups, n, k = W.shape
    ldx = _tokens(X, "X", k)
    return int(_lib.ozaki_grouped_gemm_workspace_bytes(n, k, X.shape[0], groups, _dtype(X), _ptr(W), ldw, sw, _ptr(X), ldx))


def ozaki_grouped_gemm_dgrad_workspace_bytes(dY, W) -> int:
    """Device workspace of ozaki_grouped_gemm_dgrad_ws for these operands."""
    ldw, sw = _experts(W, "W")
    groups, n, k = W.shape
    lddy = _tokens(dY, "dY", n)
    return int(_lib.ozaki_grouped_gemm_dgrad_workspace_bytes(n, k, dY.shape[0], groups, _dtype(dY), _ptr(W), ldw, sw,
                                                             _ptr(dY), lddy))


def ozaki_grouped_gemm_wgrad_workspace_bytes(dY, X, groups: int) -> int:
    """Device workspace of ozaki_grouped_gemm_wgrad_ws for these operands."""
    lddy, ldx = _tokens(dY, "dY"), _tokens(X, "X")
    return int(_lib.ozaki_grouped_gemm_wgrad_workspace_bytes(dY.shape[1], X.shape[1], X.shape[0], groups, _dtype(X),
                                                             _ptr(dY), lddy, _ptr(X), ldx))


# ------------------------------------------------------------------ Newton-Schulz orthogonalisation
NEWTON_SCHULZ_COEFFS = (3.4445, -4.7750, 2.0315)


def ozaki_newton_schulz_workspace_bytes(m: int, n: int, batch: int = 1, num_slices: int = 2) -> int:
    """Device workspace of ozaki_newton_schulz_ws for a G of shape (batch, m, n), or (m, n) in either layout.

    (The C query wants the contiguous extent first, whose rows are padded: the larger of both orders serves
    row-major and column-major matrices.)"""
    return max(int(_lib.ozaki_newton_schulz_workspace_bytes(a, b, batch, num_slices)) for a, b in ((m, n), (n, m)))


def ozaki_newton_schulz(G, steps: int = 5, coeffs=NEWTON_SCHULZ_COEFFS, eps: float = 1e-7, num_slices: int | None = None,
                        out=None, workspace=None, stream=None):
    """Newton-Schulz orthogonalisation of each matrix of G (..., m, n): X = G / (|G|_F + eps), then
    `steps` times X <- a X + (b A + c A^2) X with A = X X^T (on the smaller side).

    G is bfloat16, float16 or float32; its matrices are row-major (2-D and 3-D G may have strided
    rows, a 2-D G may be column-major if out is too).  coeffs: one (a, b, c) for every step, or one for each.
    num_slices: FP16 slices of the intermediate matrices; by default 1 for bfloat16 (11 bits kept: the
    result is off by 2.0e-3 to 2.3e-3, where rounding it alone costs 1.7e-3; 2 slices reach that in
    1.8 to 3.2 times the time) and 2 otherwise (22 bits).  `out` has G's shape and dtype; by default it is new and row-major
    (column-major for a column-major G)."""
    import torch

    if G.dim() < 2 or not G.is_cuda:
        raise ValueError("G must be a CUDA tensor of shape (..., m, n)")
    if stream is not None and (other := _other_stream(stream, G.device)):
        return _call_on(other, ozaki_newton_schulz, G, steps, coeffs, eps, num_slices, out, workspace)
    code = _dtype(G)
    try:
        flat = [float(c) for c in coeffs]
    except (TypeError, ValueError):  # a sequence of (a, b, c)
        flat = [float(c) for triple in coeffs for c in triple]
    if len(flat) == 3:
        flat *= max(1, steps)
    if steps < 1 or len(flat) != 3 * steps:
        raise ValueError("coeffs must be one (a, b, c), or one for each of the steps (at least 1)")
    if out is None:
        turned = G.dim() == 2 and G.stride(0) == 1 and G.stride(1) != 1
        out = torch.empty((G.shape[1], G.shape[0]), dtype=G.dtype, device=G.device).t() if turned else \
            torch.empty(G.shape, dtype=G.dtype, device=G.device)
    if out.shape != G.shape or out.dtype != G.dtype or out.device != G.device:
        raise ValueError("out must have G's shape, dtype and device")
    m, n = G.shape[-2:]
    lead, result = G.shape[:-2], out
    # The transposed problem is the same one.  (One row has no row stride to go by, only its elements'.)
    turn = (G.stride(0) == 1 and out.stride(0) == 1) if m > 1 else (G.stride(1) != 1 or out.stride(1) != 1)
    if G.dim() == 2 and n > 1 and turn:
        G, out, m, n = G.t(), out.t(), n, m
    batch = 1
    for d in lead:
        batch *= d
    if G.dim() != 3:  # leading dimensions as one (a view: they have to be contiguous)
        G, out = (G[None], out[None]) if G.dim() == 2 else (G.view(batch, m, n), out.view(batch, m, n))
    ldg, sg = _experts(G, "G")
    ldo, so = _experts(out, "out")
    ns = num_slices if num_slices is not None else (1 if code == OZ_BF16 else 2)
    args = (n, m, batch, code, G.data_ptr(), ldg, sg, out.data_ptr(), ldo, so, steps, (ctypes.c_float * len(flat))(*flat), float(eps), int(ns))
    _run_on("ozaki_newton_schulz", args, workspace, stream, G.device)
    return result


def ozaki_newton_schulz_ws(G, workspace, **kwargs):
    """ozaki_newton_schulz with a caller-owned workspace (see ozaki_newton_schulz_workspace_bytes)."""
    return ozaki_newton_schulz(G, workspace=workspace, **kwargs)


# ------------------------------------------------------------------ 8-bit operands with scales
_F8_CODES: dict = {}


def _f8(dtype) -> int:
    if not _F8_CODES:
        torch = _torch()
        _F8_CODES.update({torch.float8_e4m3fn: OZ_E4M3, torch.float8_e5m2: OZ_E5M2})
    code = _F8_CODES.get(dtype)
    if code is None:
        raise TypeError(f"8-bit type must be float8_e4m3fn or float8_e5m2: {dtype}")
    return code


def _new(shape, dtype, device, ld: int | None = None):
    """A new row-major tensor whose rows start ld elements apart (by default, without gaps)."""
    n = len(shape) - 1
    stride = [1] * (n + 1)
    if n:
        stride[n - 1] = step = shape[n] if ld is None else ld
        for i in range(n - 2, -1, -1):
            stride[i] = step = step * shape[i + 1]
    return _torch().empty_strided(shape, stride, dtype=dtype, device=device)


def _ld16(k: int) -> int:
    """The row stride of a new 8-bit tensor: rows start at multiples of 16 bytes."""
    return (k + 15) // 16 * 16 or 16


def _row_scales(S, what: str, rows: int, k: int, device) -> int:
    """Leading dimension of the scales of row blocks: (rows, blocks) with the rows of a block next to each other."""
    shape, stride, blocks = S.shape, S.stride(), (k + 127) // 128
    if S.dtype != _torch().float32 or S.device != device:
        raise ValueError(f"{what} must be float32 on the operands' device")
    if shape != (rows, blocks):
        raise ValueError(f"{what} must have shape ({rows}, {blocks}): {tuple(shape)}")
    if (rows > 1 and stride[0] != 1) or (blocks > 1 and not rows <= stride[1] <= _INT_MAX):
        raise ValueError(f"{what} must be column-major (stride(0) == 1): colmajor makes it so")
    return max(1, rows, stride[1] if blocks > 1 else 0)


def _column_scales(S, what: str, blocks: int, k: int, device) -> int:
    if S.dtype != _torch().float32 or S.device != device:
        raise ValueError(f"{what} must be float32 on the operands' device")
    if S.shape != (blocks, k):
        raise ValueError(f"{what} must have shape ({blocks}, {k}): {tuple(S.shape)}")
    return _tokens(S, what, k)


def _f8_rows(Q, what: str, features: int | None = None):
    """(rows, features, leading dimension, type) of an 8-bit operand, whose rows start at multiples of 16 bytes."""
    shape, stride, code = Q.shape, Q.stride(), _f8(Q.dtype)
    if len(shape) == 2 and 1 < shape[0] <= _INT_MAX and 0 < shape[1] <= stride[0] <= _INT_MAX and stride[1] == 1 and \
            features in (None, shape[1]) and not (stride[0] | Q.data_ptr()) & 15:
        return shape[0], shape[1], stride[0], code
    ld = _tokens(Q, what, features)  # (says what is wrong)
    if Q.numel() and (Q.data_ptr() & 15 or (shape[0] > 1 and ld & 15)):
        raise ValueError(f"{what} must have rows that start at multiples of 16 bytes")
    return shape[0], shape[1], ld, code


def _f8_experts(W, SW, device):
    """(groups, n, k, row stride, matrix stride) of 8-bit weights (groups, n, k), or (n, k) for one group."""
    if len(W.shape) == 2:
        W, SW = W[None], (SW[None] if SW.dim() == 2 else SW)
    groups, n, k = shape = W.shape
    stride = W.stride()
    if n > 1 and groups > 1 and 0 < k <= stride[1] <= _INT_MAX and stride[2] == 1 and stride[0] >= stride[1] * n and n <= _INT_MAX:
        ld, step = stride[1], stride[0]
    else:
        ld, step = _experts(W, "W")  # (says what is wrong)
    if n and k and (W.data_ptr() & 15 or (n > 1 and ld & 15) or (groups > 1 and step & 15)):
        raise ValueError("W must have rows and matrices that start at multiples of 16 bytes")
    if W.device != device or SW.device != device:
        raise ValueError("operands must share one device")
    want = (groups, (n + 127) // 128, (k + 127) // 128)
    if SW.dtype != _torch().float32 or SW.shape != want or not SW.is_contiguous():
        raise ValueError(f"the scales of W must be contiguous float32 of shape {want}: {tuple(SW.shape)}")
    return groups, n, k, ld, step


def _cuda(t, what: str):
    device = t.device
    if device.type != "cuda":
        raise ValueError(f"{what} must be a CUDA tensor")
    return device


def _product_offsets(offsets, groups: int | None, device):
    if offsets is None:
        if groups not in (None, 1):
            raise ValueError(f"{groups} groups need offsets")
        return None
    _offsets(offsets, groups, device)
    return offsets.data_ptr()


def _output(out, what: str, rows: int, features: int, dtype, device):
    """(output, its type's code, its leading dimension): new, 16-bit, or the given one, checked."""
    if out is None:
        if dtype is None:
            dtype = _torch().bfloat16
        out, ld = _torch().empty_strided((rows, features), (features, 1), dtype=dtype, device=device), features or 1
    else:
        if out.device != device or (dtype is not None and out.dtype != dtype):
            raise ValueError(f"{what} must be on the operands' device, with the dtype asked for")
        ld = _tokens(out, what, features)
        if out.shape[0] != rows:
            raise ValueError(f"{what} must have {rows} rows")
    return out, _16bit(out, what), ld


def _16bit(t, what: str) -> int:
    code = _dtype(t)
    if code == OZ_F32:
        raise TypeError(f"{what} must be bfloat16 or float16")
    return code


def ozaki_f8_column_blocks(rows: int, groups: int | None = None) -> int:
    """Blocks of 128 rows of one column: ceil(rows / 128), or with groups (offsets) rows // 128 + groups."""
    n = int(_lib.ozaki_f8_column_blocks(rows, 1 if groups is None else groups, groups is not None))
    if n < 0:
        _check(n, "ozaki_f8_column_blocks")
    return n


def ozaki_quantize_f8(X, block: str = "row", offsets=None, dtype=None, stream=None):
    """X (bfloat16, float16 or float32) in 8 bits (dtype: float8_e4m3fn, the default, or float8_e5m2), with a float32 scale for
    each block of 128: X = Q * scale.  Returns new tensors; Q's rows start at multiples of 16 bytes.

    block="row":    (Q, S)  128 neighbours of a row of X (rows, k): Q (rows, k), S (rows, ceil(k / 128)), column-major.
    block="column": (Q, S)  128 rows of a column: S (blocks, k).  With offsets (groups + 1, int32) blocks start anew with each
                    group: group e's rows lie from 128 * (offsets[e] // 128 + e) on, zeros behind its last one,
                    in 128 * (rows // 128 + groups) rows of Q.
    block="both":   (Q, S, Qc, Sc)  both of them in one pass (a gradient on its way into dgrad and wgrad).
    block="matrix": (Q, S)  128 x 128 of each matrix of X (..., n, k): S (..., ceil(n / 128), ceil(k / 128)).

    Row blocks do not depend on offsets.  A scale is the block's largest magnitude over the type's largest value, 1 for a
    block of zeros; a block with Inf or NaN gets an Inf or NaN scale."""
    if stream is not None and (other := _other_stream(stream, X.device)):
        return _call_on(other, ozaki_quantize_f8, X, block, offsets, dtype)
    torch = _torch()
    kind = F8_BLOCKS.get(block)
    if kind is None:
        raise ValueError(f"block must be one of {sorted(F8_BLOCKS)}: {block!r}")
    device, code = _cuda(X, "X"), _dtype(X)
    if dtype is None:
        dtype = torch.float8_e4m3fn
    eight = _f8(dtype)
    if kind == OZ_BLOCK_MATRIX:
        if offsets is not None:
            raise ValueError("matrix blocks have no offsets")
        if X.dim() < 2:
            raise ValueError("X must have shape (..., n, k)")
        n, k = X.shape[-2:]
        X3 = X if X.dim() == 3 else X[None] if X.dim() == 2 else X.view(math.prod(X.shape[:-2]), n, k)
        ldx, sx = _experts(X3, "X")
        mats, ldq = X3.shape[0], _ld16(k)
        Q = _new(X.shape, dtype, device, ldq)
        S = _new((*X.shape[:-2], (n + 127) // 128, (k + 127) // 128), torch.float32, device)
        if mats:
            _run_on("ozaki_quantize_f8", (kind, k, n, mats, code, X.data_ptr(), ldx, sx, None, eight, Q.data_ptr(), ldq, ldq * n,
                                          S.data_ptr(), 0, None, 0, None, 0), None, None, device)
        return Q, S
    ldx = _tokens(X, "X")
    rows, k = X.shape
    ldq = _ld16(k)
    groups, off, results, args = 1, None, [], []
    if offsets is not None:
        _offsets(offsets, None, device)
        if kind != OZ_BLOCK_ROW:
            groups, off = offsets.numel() - 1, offsets.data_ptr()
            if groups > OZ_MAX_GROUPS:
                raise ValueError(f"at most {OZ_MAX_GROUPS} groups: {groups}")
    if kind != OZ_BLOCK_COLUMN:
        Q = _new((rows, k), dtype, device, ldq)
        S = torch.empty_strided((rows, (k + 127) // 128), (1, max(1, rows)), dtype=torch.float32, device=device)
        results += [Q, S]
        args += [Q.data_ptr(), ldq, 0, S.data_ptr(), max(1, rows)]
    else:
        args += [None, 0, 0, None, 0]
    if kind != OZ_BLOCK_ROW:
        blocks = rows // 128 + groups if off else (rows + 127) // 128
        Q = _new((128 * blocks if off else rows, k), dtype, device, ldq)
        S = _new((blocks, k), torch.float32, device)
        results += [Q, S]
        args += [Q.data_ptr(), ldq, S.data_ptr(), max(1, k)]
    else:
        args += [None, 0, None, 0]
    _run_on("ozaki_quantize_f8", (kind, k, rows, groups, code, X.data_ptr(), ldx, 0, off, eight, *args), None, None, device)
    return tuple(results)


def ozaki_grouped_gemm_f8(X, SX, W, SW, offsets=None, Y=None, dtype=None, stream=None):
    """Y[r] = W[e] X[r] for the rows r of group e, from 8-bit operands and their scales (ozaki_quantize_f8).

    X (rows, k) with SX in row blocks, W (groups, n, k) with SW in matrix blocks; Y (rows, n) is bfloat16 (or float16: dtype, or
    a Y of that type).  offsets (groups + 1, int32) as in ozaki_grouped_gemm; None: one group of all rows, W (n, k) or (1, n, k).
    X and W may each be float8_e4m3fn or float8_e5m2; their rows start at multiples of 16 bytes."""
    if stream is not None and (other := _other_stream(stream, X.device)):
        return _call_on(other, ozaki_grouped_gemm_f8, X, SX, W, SW, offsets, Y, dtype)
    device = _cuda(X, "X")
    groups, n, k, ldw, sw = _f8_experts(W, SW, device)
    rows, _, ldx, tx = _f8_rows(X, "X", k)
    lds = _row_scales(SX, "the scales of X", rows, k, device)
    off = _product_offsets(offsets, groups, device)
    Y, code, ldy = _output(Y, "Y", rows, n, dtype, device)
    _run_on("ozaki_grouped_gemm_f8", (n, k, rows, groups, _f8(W.dtype), W.data_ptr(), ldw, sw, SW.data_ptr(), tx, X.data_ptr(),
                                      ldx, SX.data_ptr(), lds, off, code, Y.data_ptr(), ldy), None, None, device)
    return Y


def ozaki_grouped_gemm_f8_dgrad(dY, SdY, W, SW, offsets=None, dX=None, dtype=None, stream=None):
    """dX[r] = W[e]^T dY[r]: the gradient in X; dY (rows, n) with SdY in row blocks, W and SW as in the forward product."""
    if stream is not None and (other := _other_stream(stream, dY.device)):
        return _call_on(other, ozaki_grouped_gemm_f8_dgrad, dY, SdY, W, SW, offsets, dX, dtype)
    device = _cuda(dY, "dY")
    groups, n, k, ldw, sw = _f8_experts(W, SW, device)
    rows, _, lddy, tdy = _f8_rows(dY, "dY", n)
    lds = _row_scales(SdY, "the scales of dY", rows, n, device)
    off = _product_offsets(offsets, groups, device)
    dX, code, lddx = _output(dX, "dX", rows, k, dtype, device)
    _run_on("ozaki_grouped_gemm_f8_dgrad", (n, k, rows, groups, _f8(W.dtype), W.data_ptr(), ldw, sw, SW.data_ptr(), tdy, dY.data_ptr(),
                                            lddy, SdY.data_ptr(), lds, off, code, dX.data_ptr(), lddx), None, None, device)
    return dX


def ozaki_grouped_gemm_f8_wgrad(dY, SdY, X, SX, offsets=None, dW=None, dtype=None, rows: int | None = None, stream=None):
    """dW[e] = sum over the rows r of group e of dY[r] X[r]^T: (groups, n, k), or (1, n, k) without offsets.

    dY (laid, n) and X (laid, k) in column blocks with their scales (blocks, n) and (blocks, k).  With offsets they are laid
    out by group as ozaki_quantize_f8 does, in 128 * (rows // 128 + groups) rows; rows, the number of tokens, is only
    needed where offsets speak of other tokens than those (any number with the same rows // 128 serves)."""
    if stream is not None and (other := _other_stream(stream, dY.device)):
        return _call_on(other, ozaki_grouped_gemm_f8_wgrad, dY, SdY, X, SX, offsets, dW, dtype, rows)
    device = _cuda(dY, "dY")
    laid, n, lddy, tdy = _f8_rows(dY, "dY")
    laid_x, k, ldx, tx = _f8_rows(X, "X")
    if laid_x != laid or X.device != device:
        raise ValueError("X and dY must have the same rows, on one device")
    off = _product_offsets(offsets, None, device)
    if off is None:
        groups, blocks = 1, (laid + 127) // 128
        if rows not in (None, laid):
            raise ValueError(f"without offsets the rows are those of dY and X: {laid}")
        rows = laid
    else:
        groups, blocks = offsets.numel() - 1, laid // 128
        if rows is None:  # the most tokens that are laid out in so many blocks
            rows = max(0, 128 * (blocks - groups) + 127)
        if laid != 128 * (rows // 128 + groups):
            raise ValueError(f"with offsets X and dY must have 128 * (rows // 128 + groups) rows: {laid}")
    ldsy, ldsx = _column_scales(SdY, "the scales of dY", blocks, n, device), _column_scales(SX, "the scales of X", blocks, k, device)
    if dW is None:
        dW, ldw, sw = _new((groups, n, k), dtype or _torch().bfloat16, device), max(1, k), max(1, k) * n
    else:
        if dW.device != device or (dtype is not None and dW.dtype != dtype):
            raise ValueError("dW must be on the operands' device, with the dtype asked for")
        ldw, sw = _experts(dW, "dW")
        if dW.shape != (groups, n, k):
            raise ValueError(f"dW must have shape {(groups, n, k)}: {tuple(dW.shape)}")
    code = _16bit(dW, "dW")
    _run_on("ozaki_grouped_gemm_f8_wgrad", (n, k, rows, groups, tdy, dY.data_ptr(), lddy, SdY.data_ptr(), ldsy, tx,
                                            X.data_ptr(), ldx, SX.data_ptr(), ldsx, off, code, dW.data_ptr(), ldw, sw), None, None, device)
    return dW


# ------------------------------------------------------------------ root-mean-square norm
def _norm_rows(t, what: str, rows: int, k: int, like) -> int:
    if t.dtype != like.dtype or t.device != like.device:
        raise ValueError(f"{what} must have X's dtype and device")
    shape, stride = t.shape, t.stride()
    if shape == (rows, k) and k > 0 and stride[1] == 1 and k <= stride[0] <= _INT_MAX:
        return stride[0]
    ld = _tokens(t, what, k)  # (says what is wrong)
    if shape[0] != rows:
        raise ValueError(f"{what} must have {rows} rows")
    return ld


def _norm_weight(W, k: int, like):
    if W.dtype != like.dtype or W.device != like.device or W.shape != (k,) or not W.is_contiguous():
        raise ValueError(f"W must be a contiguous vector of {k} values with the operands' dtype and device")


def ozaki_rms_norm_f8(X, W, residual=None, eps: float = 1e-6, H=None, Y=None, stream=None):
    """h = X + residual, y = h / sqrt(mean(h^2) + eps) * W for each row of X (rows, k): (Q, S, H, rstd).

    Q (float8_e4m3fn) and S are y in row blocks, ready for ozaki_grouped_gemm_f8; H is h in X's dtype (X itself without a
    residual) and rstd (rows, float32) the rows' 1 / sqrt(...), which ozaki_rms_norm_backward needs.  H: where to write it (may
    be X or residual); Y: where to write y in X's dtype too.  X is bfloat16, float16 or float32, k <= OZ_MAX_NORM_WIDTH."""
    if stream is not None and (other := _other_stream(stream, X.device)):
        return _call_on(other, ozaki_rms_norm_f8, X, W, residual, eps, H, Y)
    torch = _torch()
    device, code = _cuda(X, "X"), _dtype(X)
    rows, k = X.shape if X.dim() == 2 else (0, 0)
    ldx = _norm_rows(X, "X", rows, k, X)
    if k > OZ_MAX_NORM_WIDTH:
        raise ValueError(f"at most {OZ_MAX_NORM_WIDTH} features: {k}")
    _norm_weight(W, k, X)
    least = max(1, k)
    ldr = ldh = ldy = least
    if residual is not None:
        ldr = _norm_rows(residual, "residual", rows, k, X)
        if H is None:
            H = torch.empty_strided((rows, k), (k, 1), dtype=X.dtype, device=device)
        else:
            ldh = _norm_rows(H, "H", rows, k, X)
    elif H is not None:
        ldh = _norm_rows(H, "H", rows, k, X)
    if Y is not None:
        ldy = _norm_rows(Y, "Y", rows, k, X)
    ldq, lds = _ld16(k), max(1, rows)
    Q = torch.empty_strided((rows, k), (ldq, 1), dtype=torch.float8_e4m3fn, device=device)
    S = torch.empty_strided((rows, (k + 127) // 128), (1, lds), dtype=torch.float32, device=device)
    rstd = torch.empty_strided((rows,), (1,), dtype=torch.float32, device=device)
    _run_on("ozaki_rms_norm_f8", (k, rows, code, X.data_ptr(), ldx, _ptr(residual), ldr, W.data_ptr(), float(eps), Q.data_ptr(),
                                  ldq, S.data_ptr(), lds, _ptr(H), ldh, rstd.data_ptr(), _ptr(Y), ldy), None, None, device)
    return Q, S, X if H is None else H, rstd


def ozaki_rms_norm_backward(dY, H, W, rstd, dH=None, dX=None, workspace=None, stream=None):
    """The gradients of a loss in X (and the residual, the same) and in W: (dX, dW).

    dY (rows, k): its gradient in y; H and rstd: the forward's; dH: its gradient in h by other paths (the residual stream).  dX
    may be dY, H or dH.  Sums are float32; dX and dW have dY's dtype."""
    if stream is not None and (other := _other_stream(stream, dY.device)):
        return _call_on(other, ozaki_rms_norm_backward, dY, H, W, rstd, dH, dX, workspace)
    torch = _torch()
    device, code = _cuda(dY, "dY"), _dtype(dY)
    lddy = _tokens(dY, "dY")
    rows, k = dY.shape
    if k > OZ_MAX_NORM_WIDTH:
        raise ValueError(f"at most {OZ_MAX_NORM_WIDTH} features: {k}")
    ldh = _norm_rows(H, "H", rows, k, dY)
    _norm_weight(W, k, dY)
    if rstd.dtype != torch.float32 or rstd.device != device or rstd.shape != (rows,) or not rstd.is_contiguous():
        raise ValueError(f"rstd must be a contiguous float32 vector of {rows} values on the operands' device")
    lddh = _norm_rows(dH, "dH", rows, k, dY) if dH is not None else max(1, k)
    if dX is None:
        dX, lddx = torch.empty_strided((rows, k), (k, 1), dtype=dY.dtype, device=device), max(1, k)
    else:
        lddx = _norm_rows(dX, "dX", rows, k, dY)
    dW = torch.empty_strided((k,), (1,), dtype=dY.dtype, device=device)
    _run_on("ozaki_rms_norm_backward", (k, rows, code, dY.data_ptr(), lddy, H.data_ptr(), ldh, W.data_ptr(), rstd.data_ptr(), _ptr(dH), lddh,
                                        dX.data_ptr(), lddx, dW.data_ptr()), workspace, None, device)
    return dX, dW


def ozaki_rms_norm_backward_ws(dY, H, W, rstd, workspace, dH=None, dX=None, stream=None):
    """ozaki_rms_norm_backward with a caller-owned workspace (see ozaki_rms_norm_backward_workspace_bytes)."""
    return ozaki_rms_norm_backward(dY, H, W, rstd, dH, dX, workspace, stream)


def ozaki_rms_norm_backward_workspace_bytes(k: int, rows: int) -> int:
    """Device workspace of ozaki_rms_norm_backward_ws."""
    return int(_lib.ozaki_rms_norm_backward_workspace_bytes(k, rows))


# ------------------------------------------------------------------ clipping by the global norm
def _tensor_lists():
    """The module that gathers what the library wants to know of many tensors (built beside it; it needs torch)."""
    try:
        from . import _tensor_lists
    except ImportError as e:
        there = os.path.exists(os.path.join(_PKG, "_tensor_lists.so"))
        what = f"does not load ({e}): build it for this torch and Python" if there else "is missing: build it"
        raise ImportError(f"_tensor_lists.so {what} with `python -m fp64_gemm_emulation_gb300.build_lib`") from e
    return _tensor_lists


def ozaki_clip_grad_norm(grads, max_norm: float, eps: float = 1e-6, out=None, workspace=None, stream=None):
    """The 2-norm over all tensors of grads (a float32 scalar on the device), each of which is multiplied by
    min(1, max_norm / (norm + eps)): in place, or into the tensors of out.

    Tensors are contiguous, bfloat16, float16 or float32 (each its own), on one device; out has their dtypes and numbers of
    elements, and each of its tensors is its gradient itself or does not overlap any; no tensor is listed twice.  A norm of Inf
    makes the factor 0, one of NaN makes it NaN; max_norm = inf only takes the norm."""
    torch = _torch()
    grads = list(grads)
    outs = grads if out is None else list(out)
    if not grads:
        raise ValueError("no gradients")
    device = _cuda(grads[0], "gradients")
    if stream is not None and (other := _other_stream(stream, device)):
        result = _call_on(other, ozaki_clip_grad_norm, grads, max_norm, eps, out, workspace)
        for t in (*grads, *outs):
            t.record_stream(other)
        return result
    n = len(grads)
    if len(outs) != n:
        raise ValueError(f"out must hold {n} tensors: {len(outs)}")
    _, codes, pointers, to, counts = _tensor_lists().pairs(grads, outs)
    norm = torch.empty_strided((), (), dtype=torch.float32, device=device)
    _run_on("ozaki_clip_grad_norm", (n, codes, pointers, to, counts, float(max_norm), float(eps), norm.data_ptr()), workspace, None, device)
    return norm


def ozaki_clip_grad_norm_ws(grads, max_norm: float, workspace, eps: float = 1e-6, out=None, stream=None):
    """ozaki_clip_grad_norm with a caller-owned workspace (see ozaki_clip_grad_norm_workspace_bytes)."""
    return ozaki_clip_grad_norm(grads, max_norm, eps, out, workspace, stream)


def ozaki_clip_grad_norm_workspace_bytes() -> int:
    """Device workspace of ozaki_clip_grad_norm_ws."""
    return int(_lib.ozaki_clip_grad_norm_workspace_bytes())


# ------------------------------------------------------------------ Scheme I variants
def _variant(v) -> int:
    return OZAKI1_VARIANTS[v] if isinstance(v, str) else int(v)


def ozaki1_group_r(k_inner: int) -> int:
    r = ctypes.c_int()
    _check(_lib.ozaki1_group_r(k_inner, ctypes.byref(r)), "ozaki1_group_r")
    return r.value


def ozaki1_num_batches(num_slices: int, k_inner: int, variant="rn") -> int:
    c = ctypes.c_int()
    _check(_lib.ozaki1_num_batches(num_slices, k_inner, _variant(variant), ctypes.byref(c)), "ozaki1_num_batches")
    return c.value


def ozaki1_split_scratch_bytes_ex(m: int, n: int, k: int, variant="rn") -> int:
    return int(_lib.ozaki1_split_scratch_bytes_ex(m, n, k, _variant(variant)))


def ozaki1_workspace_bytes_ex(m: int, n: int, k: int, num_slices: int, variant="rn") -> int:
    return int(_lib.ozaki1_workspace_bytes_ex(m, n, k, num_slices, _variant(variant)))


@_on_given_stream
def ozaki1_split_ex(A, B, num_slices: int, variant="rn", stream=None):
    """Split of a variant: (A_planes, B_planes, A_exps, B_exps) as ozaki1_split."""
    import torch

    m, k = A.shape
    n = B.shape[1]
    v = _variant(variant)
    mp, np_, kp = ozaki2_plane_dims(m, n, k)
    Ap = torch.empty((num_slices, mp, kp), dtype=torch.int16, device=A.device)
    Bp = torch.empty((num_slices, np_, kp), dtype=torch.int16, device=A.device)
    Ae = torch.empty((num_slices, m), dtype=torch.int32, device=A.device)
    Be = torch.empty((num_slices, n), dtype=torch.int32, device=A.device)
    nbytes = ozaki1_split_scratch_bytes_ex(m, n, k, v)
    scratch = torch.empty(nbytes + 256, dtype=torch.uint8, device=A.device)
    sp = (scratch.data_ptr() + 255) // 256 * 256
    _check(_lib.ozaki1_split_ex(m, n, k, _ptr(A), _ld(A), _ptr(B), _ld(B), num_slices, v, _ptr(Ap), _ptr(Bp),
                                _ptr(Ae), _ptr(Be), sp, nbytes, _stream(stream)), "ozaki1_split_ex")
    return Ap, Bp, Ae, Be


@_on_given_stream
def ozaki1_slice_gemm_ex(m: int, n: int, k: int, num_slices: int, variant, A_planes, B_planes, stream=None):
    """Exact INT32 pair products of a variant, in its order: [s(s+1)/2, Np, Mp]."""
    import torch

    v = _variant(variant)
    mp, np_, kp = ozaki2_plane_dims(m, n, k)
    P = torch.empty((num_slices * (num_slices + 1) // 2, np_, mp), dtype=torch.int32, device=A_planes.device)
    _check(_lib.ozaki1_slice_gemm_ex(m, n, k, num_slices, v, _ptr(A_planes), _ptr(B_planes), _ptr(P),
                                     _stream(stream)), "ozaki1_slice_gemm_ex")
    return P


@_on_given_stream
def ozaki1_accumulate_ex(m: int, n: int, k: int, num_slices: int, variant, products, A_exps, B_exps, C=None,
                         stream=None):
    import torch

    if C is None:
        C = torch.empty((n, m), dtype=torch.float64, device=products.device).t()
    _check(_lib.ozaki1_accumulate_ex(m, n, k, num_slices, _variant(variant), _ptr(products), _ptr(A_exps),
                                     _ptr(B_exps), _ptr(C), _ld(C), _stream(stream)), "ozaki1_accumulate_ex")
    return C


@_on_given_stream
def ozaki1_dgemm_ex(A, B, num_slices: int = 7, variant="rn", C=None, workspace=None, stream=None):
    """C = A B by Scheme I in a variant ("rn", "ef", "hybrid"); with ``workspace`` the _ws form."""
    import torch

    m, k = A.shape
    n = B.shape[1]
    v = _variant(variant)
    if C is None:
        C = torch.empty((n, m), dtype=torch.float64, device=A.device).t()
    if workspace is None:
        rc = _lib.ozaki1_dgemm_ex(m, n, k, _ptr(A), _ld(A), _ptr(B), _ld(B), _ptr(C), _ld(C), num_slices, v,
                                  _stream(stream))
    else:
        rc = _lib.ozaki1_dgemm_ex_ws(m, n, k, _ptr(A), _ld(A), _ptr(B), _ld(B), _ptr(C), _ld(C), num_slices, v,
                                     _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    _check(rc, "ozaki1_dgemm_ex")
    return C


@_on_given_stream
def ozaki1_dgemm_ex_ws(A, B, num_slices: int, variant, workspace, C=None, stream=None):
    return ozaki1_dgemm_ex(A, B, num_slices, variant, C=C, workspace=workspace, stream=stream)


def ozaki_get_device_status(stream=None) -> int:
    """Status word of the current device after the work on ``stream`` (default: the current
    torch stream) has finished; cleared by the read."""
    return int(_lib.ozaki_get_device_status(_stream(stream)))


def ozaki_set_epilogue_wait_ns(ns: int) -> None:
    """Time limit of the GEMM epilogue's accumulator wait for later launches (-1: default 4 s)."""
    _check(_lib.ozaki_set_epilogue_wait_ns(int(ns)), "ozaki_set_epilogue_wait_ns")


def ozaki_status_string(code: int) -> str:
    return _lib.ozaki_status_string(code).decode()


def exported_symbols() -> list[str]:
    """Names the loaded library exports among those ``include/ozaki.h`` declares."""
    return [name for name in _declared_names() if hasattr(_lib, name)]


def _declared_names() -> list[str]:
    import re

    hdr = os.path.join(os.path.dirname(_PKG), "include", "ozaki.h")
    with open(hdr) as f:
        text = f.read()
    return re.findall(r"^(?:int|size_t|const char\*)\s+(\w+)\s*\(", text, flags=re.M)
