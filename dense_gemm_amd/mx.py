"""Block-scaled (MX) matrices: the C ABI's functions one to one, and the
torch conveniences over them.

An `MxMatrix` holds rows x cols values in blocks of 32 along a row, with one
power-of-two scale per block and elements of 4 or 8 bits (include/dense_gemm.h,
"Block-scaled (MX) matrices").  Like the rest of the package, these functions
only marshal arguments: every step runs in the library's HIP kernels, on the
current torch stream of the tensors' device unless `stream` (a torch stream of
that device) is given, without waiting.
"""
from __future__ import annotations

import ctypes

import torch

from . import DG_EPI_GELU, DG_EPI_RELU, DG_EPI_RELU_POSITIVE, DG_ERR_HIP, DG_KERNEL_AUTO, DG_OK, EPILOGUES, GemmError, _lib
from . import dg_gemm_splitk_workspace_size, dg_last_hip_error, dg_status_string, hip_error_name

DG_ELEM_F32, DG_ELEM_F16, DG_ELEM_BF16 = 0, 1, 2
DG_MXFP4, DG_MXFP8, DG_MXINT8 = 0, 1, 2
MX_FORMATS = {"mxfp4": DG_MXFP4, "mxfp8": DG_MXFP8, "mxint8": DG_MXINT8}
_ELEM = {torch.float32: DG_ELEM_F32, torch.float16: DG_ELEM_F16, torch.bfloat16: DG_ELEM_BF16}
_ACTIVATIONS = {"relu": DG_EPI_RELU, "gelu": DG_EPI_GELU}
GROUP = 256          # columns of a scale group

_i64, _f32, _vp, _ci, _sz = ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
_MX = [_ci, _vp, _i64, _vp, _i64]                      # format, Q, ldq, S, lds
_GEMM_MX = [_i64, _i64, _i64, _f32] + _MX + _MX + [_f32, _vp, _i64, _ci, _vp, _ci, _vp]
_GEMM_DQ = [_ci, _i64, _i64, _i64, _f32, _vp, _i64, _ci] + _MX + [_f32, _vp, _i64, _ci, _ci, _vp, _sz, _vp]
_GEMM_DQ_NAMES = ("transA M N K alpha A lda typeA formatB B ldb SB ldsb beta C ldc typeC splits workspace "
                  "workspace_bytes stream")
# name: (result, argument types, argument names in position order)
_SIGNATURES = {
    "dg_mx_row_bytes": (_i64, [_ci, _i64], "format cols"),
    "dg_mx_scale_bytes": (_i64, [_i64, _i64], "lds cols"),
    "dg_mx_quantize": (_ci, [_ci, _i64, _i64, _vp, _i64, _ci, _ci, _vp, _i64, _vp, _i64, _vp],
                       "transX rows cols X ldx type format Q ldq S lds stream"),
    "dg_mx_dequantize": (_ci, [_i64, _i64] + _MX + [_vp, _i64, _ci, _vp],
                         "rows cols format Q ldq S lds X ldx type stream"),
    "dg_gemm_mx": (_ci, _GEMM_MX, "M N K alpha formatA A lda SA ldsa formatB B ldb SB ldsb beta C ldc type bias "
                                  "epilogue stream"),
    "dg_gemm_mx_with_kernel": (_ci, _GEMM_MX + [_ci], "M N K alpha formatA A lda SA ldsa formatB B ldb SB ldsb beta C "
                                                      "ldc type bias epilogue stream kernel"),
    "dg_gemm_mx_select": (_ci, [_ci, _i64, _i64, _i64], "formatA M N K"),
    "dg_gemm_mx_kernel_name": (ctypes.c_char_p, [_ci], "kernel"),
    "dg_gemm_dq": (_ci, _GEMM_DQ, _GEMM_DQ_NAMES),
    "dg_gemm_dq_with_kernel": (_ci, _GEMM_DQ + [_ci], _GEMM_DQ_NAMES + " kernel"),
    "dg_gemm_dq_select": (_ci, [_i64, _i64, _i64], "M N K"),
    "dg_gemm_dq_kernel_name": (ctypes.c_char_p, [_ci], "kernel"),
    "dg_gemm_dq_choose": (_ci, [_i64, _i64, _i64], "M N K"),
    "dg_act_checkpoint": (_ci, [_i64, _i64, _vp, _i64, _vp, _i64, _ci, _ci] + _MX + [_vp],
                          "rows cols Z ldz H ldh type activation format Q ldq S lds stream"),
    "dg_act_backward": (_ci, [_i64, _i64, _vp, _i64] + _MX + [_vp, _i64, _ci, _ci, _vp, _vp, _sz, _vp],
                        "rows cols dH ldh format Q ldq S lds dZ ldz type activation dbias workspace workspace_bytes "
                        "stream"),
    "dg_act_backward_workspace_size": (_sz, [_i64, _i64], "rows cols"),
}
EXPORTED = sorted(_SIGNATURES)
__all__ = EXPORTED + ["MxMatrix", "MxError", "MX_FORMATS", "DG_ELEM_F32", "DG_ELEM_F16", "DG_ELEM_BF16", "DG_MXFP4",
                      "DG_MXFP8", "DG_MXINT8", "quantize_mx", "dequantize_mx", "gemm_mx", "gemm_dq", "act_checkpoint",
                      "act_backward", "mx_kernel_names", "dq_kernel_names"]
_functions = {}
for _name, (_res, _args, _) in _SIGNATURES.items():
    _f = getattr(_lib, _name)
    _f.restype, _f.argtypes = _res, _args
    _functions[_name] = globals()[_name] = _f


def _kernel_names(name_of) -> list[str]:
    names = []
    while (n := name_of(len(names))) is not None:
        names.append(n.decode())
    return names


def mx_kernel_names() -> list[str]:
    """The kernels of dg_gemm_mx, by index."""
    return _kernel_names(dg_gemm_mx_kernel_name)  # noqa: F821


def dq_kernel_names() -> list[str]:
    """The kernels of dg_gemm_dq, by index."""
    return _kernel_names(dg_gemm_dq_kernel_name)  # noqa: F821


class MxError(GemmError):
    """A failed MX call, with the name of an invalid argument."""

    def __init__(self, function: str, status: int):
        names = _SIGNATURES[function][2].split()
        if -len(names) <= status < 0:
            msg = f"invalid argument {-status} ({names[-status - 1]})"
        else:
            msg = dg_status_string(status)
            if status == DG_ERR_HIP:
                e = dg_last_hip_error()
                msg += f" (hipError_t {e} {hip_error_name(e)})"
        RuntimeError.__init__(self, f"{function} failed: {status} ({msg})")
        self.status = status


class MxMatrix:
    """rows x cols values in an MX format: `q` (uint8 [rows, bytes], rows of
    whole 256-column groups) and `s` (uint8 [groups, rows, 8], the scale bytes
    of each row's group).  Both may be views: unit stride along the bytes, and
    the rows of a group of `s` 8 bytes apart.  Elements of the last group past
    `cols` must be zero (every function here writes them so): a matrix of a
    stored one's first columns ends at a multiple of 256."""

    __slots__ = ("format", "rows", "cols", "q", "s", "code", "ldq", "lds")

    def __init__(self, format: str, rows: int, cols: int, q: torch.Tensor, s: torch.Tensor):
        code = MX_FORMATS.get(format)
        if code is None:
            raise ValueError(f"format must be one of {sorted(MX_FORMATS)}")
        groups = -(-cols // GROUP)
        nb = groups * (GROUP // 2 if code == DG_MXFP4 else GROUP)
        if q.dtype != torch.uint8 or s.dtype != torch.uint8 or q.get_device() != s.get_device():
            raise TypeError("q and s must be uint8 tensors on one device")
        qs, qt, st = q.shape, q.stride(), s.stride()
        if len(qs) != 2 or qs[0] != rows or qs[1] < nb or (qt[1] != 1 and qs[1] > 1):
            raise ValueError(f"q must be [{rows}, {nb}] bytes or wider, with unit column stride")
        if s.shape != (groups, rows, 8) or (groups and rows and (st[2] != 1 or (rows > 1 and st[1] != 8))):
            raise ValueError(f"s must be [{groups}, {rows}, 8] with rows 8 bytes apart")
        self.format, self.rows, self.cols, self.q, self.s, self.code = format, rows, cols, q, s, code
        # a single row or group gives no stride: any valid one will do
        self.ldq = qt[0] if rows > 1 and nb > 0 else nb
        if groups > 1:
            if st[0] % 8:
                raise ValueError("the groups of s must be a multiple of 8 bytes apart")
            self.lds = st[0] // 8
        else:
            self.lds = rows

    @classmethod
    def empty(cls, format: str, rows: int, cols: int, device, stream=None) -> "MxMatrix":
        """Uninitialised storage (`stream`: the one it is first used on, when it
        is not the current one)."""
        code = MX_FORMATS.get(format)
        if code is None:
            raise ValueError(f"format must be one of {sorted(MX_FORMATS)}")
        return cls(format, rows, cols, _empty((rows, dg_mx_row_bytes(code, cols)), torch.uint8, device, stream),  # noqa: F821
                   _empty((-(-cols // GROUP), rows, 8), torch.uint8, device, stream))

    @property
    def device(self):
        return self.q.device

    def __repr__(self):
        return f"MxMatrix({self.format}, {self.rows} x {self.cols}, {self.device})"


def _plain(t, name, rows, cols):
    """The row stride of a plain 2-D matrix of that shape."""
    if t.shape != (rows, cols):
        raise ValueError(f"{name} must be [{rows}, {cols}]")
    ld, one = t.stride()
    if one != 1 and cols > 1:
        raise ValueError(f"{name} must have unit column stride (row-major rows)")
    if rows <= 1:
        return max(cols, 1)
    if ld < cols:
        raise ValueError(f"{name} has overlapping rows (a row stride below {cols})")
    return max(ld, 1)


def _elem(t, name):
    code = _ELEM.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, float16 or bfloat16")
    return code


# A device's current stream and the current device without building torch's
# objects for them (a microsecond and a half a call); the public way where
# torch lacks these.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream_of(stream, tensors):
    """The handle of the caller's stream, or of the current one, on the device
    of the tensors (None among them: not given).  Tensors handed to a stream of
    the caller's stay allocated until that stream has passed them."""
    index = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError("all matrices must be on one device")
    if index < 0:
        raise ValueError("the matrices must be on a GPU")
    if stream is None:
        return index, _raw_stream(index)
    if stream.device.index != index:
        raise ValueError("stream belongs to another device than the matrices")
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    return index, stream.cuda_stream


def _empty(shape, dtype, device, stream):
    """Uninitialised memory that belongs to the stream the call runs on (the
    allocator reuses freed blocks in the order of their own stream)."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _workspace(workspace):
    """Address and size of a caller's workspace (0 of None)."""
    if workspace is None:
        return None, 0
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _call(function, index, *args):
    """One library call with device `index` current."""
    f = _functions[function]
    if index == _current_device():
        rc = f(*args)
    else:
        with torch.cuda.device(index):
            rc = f(*args)
    if rc != DG_OK:
        raise MxError(function, rc)


def quantize_mx(X, format="mxfp4", trans=False, out=None, stream=None) -> MxMatrix:
    """X (or its transpose) rounded to an MX format, blocks of 32 along the
    result's rows.  X is 2-D float32, float16 or bfloat16 with unit column
    stride.  `out` (an MxMatrix) is written when given, and sets the format."""
    shape = X.shape
    if len(shape) != 2:
        raise ValueError("X must be 2-D")
    rows, cols = shape[::-1] if trans else shape
    if out is None:
        out = MxMatrix.empty(format, rows, cols, X.device, stream)
    elif out.rows != rows or out.cols != cols:
        raise ValueError(f"out must be {rows} x {cols}")
    ldx, code = _plain(X, "X", *shape), _elem(X, "X")
    index, handle = _stream_of(stream, (X, out.q, out.s))
    _call("dg_mx_quantize", index, bool(trans), rows, cols, X.data_ptr(), ldx, code, out.code, out.q.data_ptr(),
          out.ldq, out.s.data_ptr(), out.lds, handle)
    return out


def dequantize_mx(m: MxMatrix, dtype=torch.float32, out=None, stream=None):
    """The values of an MX matrix as a plain one, of `dtype` or out's."""
    if out is None:
        out = _empty((m.rows, m.cols), dtype, m.device, stream)
    ldx = _plain(out, "out", m.rows, m.cols)
    index, handle = _stream_of(stream, (out, m.q, m.s))
    _call("dg_mx_dequantize", index, m.rows, m.cols, m.code, m.q.data_ptr(), m.ldq, m.s.data_ptr(), m.lds, out.data_ptr(),
          ldx, _elem(out, "out"), handle)
    return out


def gemm_mx(A: MxMatrix, B: MxMatrix, C=None, alpha=1.0, beta=0.0, bias=None, activation="none",
            out_dtype=torch.bfloat16, kernel=DG_KERNEL_AUTO, stream=None):
    """C = act(alpha * A @ B^T + beta * C + bias): A [M, K] in mxfp4 or mxfp8,
    B [N, K] in mxfp4.  C (allocated with `out_dtype` when None, beta 0 then)
    is [M, N]; bias has N elements of C's dtype; activation is "none", "relu"
    or "gelu".  Sums are fp32; with an mxfp8 A, more than a few rows and a 16-bit
    C, products far below their neighbours' largest are cut (1e-5 of the result by
    norm, see include/dense_gemm.h), which an fp32 C avoids at up to twice the
    time."""
    M, K, N = A.rows, A.cols, B.rows
    if B.cols != K:
        raise ValueError(f"inner dimensions differ: {K} vs {B.cols}")
    if C is None:
        if beta != 0.0:
            raise ValueError("beta != 0 needs C")
        C = _empty((M, N), out_dtype, A.device, stream)
    if activation not in EPILOGUES:
        raise ValueError(f"activation must be one of {sorted(EPILOGUES)}")
    if bias is not None and (bias.dtype != C.dtype or bias.dim() != 1 or bias.shape[0] != N or (N > 1 and bias.stride(0) != 1)):
        raise ValueError(f"bias must be a contiguous 1-D tensor of {N} elements of C's dtype")
    ldc = _plain(C, "C", M, N)
    index, handle = _stream_of(stream, (A.q, A.s, B.q, B.s, C, bias))
    _call("dg_gemm_mx_with_kernel", index, M, N, K, alpha, A.code, A.q.data_ptr(), A.ldq, A.s.data_ptr(), A.lds, B.code,
          B.q.data_ptr(), B.ldq, B.s.data_ptr(), B.lds, beta, C.data_ptr(), ldc, _elem(C, "C"),
          None if bias is None else bias.data_ptr(), EPILOGUES[activation], handle, kernel)
    return C


def gemm_dq(A, B: MxMatrix, C=None, transA=False, alpha=1.0, beta=0.0, out_dtype=None, splits=0, workspace=None,
            stream=None, kernel=DG_KERNEL_AUTO):
    """C = alpha * op(A) @ B + beta * C: A float16 or bfloat16, [M, K] or (with
    transA) [K, M]; B [K, N] in any MX format.  C (allocated when None, with
    `out_dtype` or A's dtype) has A's dtype or float32.  `splits` cuts K into
    ranges (0: the library's choice); their fp32 partials go to `workspace`, a
    16-byte aligned tensor of dg_gemm_splitk_workspace_size(M, N, splits)
    bytes, or to one allocated here."""
    if A.dim() != 2:
        raise ValueError("A must be 2-D")
    M, K = (A.shape[1], A.shape[0]) if transA else (A.shape[0], A.shape[1])
    N = B.cols
    if B.rows != K:
        raise ValueError(f"inner dimensions differ: {K} vs {B.rows}")
    if A.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError("A must be float16 or bfloat16")
    if C is None:
        if beta != 0.0:
            raise ValueError("beta != 0 needs C")
        C = _empty((M, N), out_dtype or A.dtype, A.device, stream)
    if C.dtype not in (A.dtype, torch.float32):
        raise TypeError("C must have A's dtype or float32")
    lda, ldc = _plain(A, "A", A.shape[0], A.shape[1]), _plain(C, "C", M, N)
    if splits == 0:
        splits = dg_gemm_dq_choose(M, N, K)  # noqa: F821
    if workspace is None and splits > 1:
        workspace = _empty(dg_gemm_splitk_workspace_size(M, N, splits), torch.uint8, A.device, stream)
    ws, wsb = _workspace(workspace)
    index, handle = _stream_of(stream, (A, B.q, B.s, C, workspace))
    _call("dg_gemm_dq_with_kernel", index, bool(transA), M, N, K, alpha, A.data_ptr(), lda, _ELEM[A.dtype], B.code, B.q.data_ptr(),
          B.ldq, B.s.data_ptr(), B.lds, beta, C.data_ptr(), ldc, _ELEM[C.dtype], splits, ws, wsb, handle,
          kernel)
    return C


def act_checkpoint(Z, activation="gelu", H=None, out=None, format="mxint8", stream=None, keep_positive=False):
    """(H, kept): H = act(Z) ("relu" or "gelu") and Z in 8 bits ("mxfp8" or
    "mxint8") for act_backward, in one pass.  H may be Z itself; `out` (an
    MxMatrix) sets the format when given.

    With relu, a positive Z that rounds to zero loses its gradient (1.1% of the
    positive elements of normal data in mxint8, 0.0005% in mxfp8).
    `keep_positive` rounds those to the format's least positive element, so that
    act_backward's mask is that of Z itself; nothing else changes."""
    if Z.dim() != 2:
        raise ValueError("Z must be 2-D")
    rows, cols = Z.shape
    if activation not in _ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(_ACTIVATIONS)}")
    if keep_positive and activation != "relu":
        raise ValueError("keep_positive goes with relu")
    if H is None:
        H = _empty((rows, cols), Z.dtype, Z.device, stream)
    elif H.dtype != Z.dtype:
        raise TypeError("H must have Z's dtype")
    if out is None:
        out = MxMatrix.empty(format, rows, cols, Z.device, stream)
    elif out.rows != rows or out.cols != cols:
        raise ValueError(f"out must be {rows} x {cols}")
    ldz, ldh = _plain(Z, "Z", rows, cols), _plain(H, "H", rows, cols)
    index, handle = _stream_of(stream, (Z, H, out.q, out.s))
    _call("dg_act_checkpoint", index, rows, cols, Z.data_ptr(), ldz, H.data_ptr(), ldh, _elem(Z, "Z"),
          DG_EPI_RELU_POSITIVE if keep_positive else _ACTIVATIONS[activation], out.code, out.q.data_ptr(), out.ldq,
          out.s.data_ptr(), out.lds, handle)
    return H, out


def act_backward(dH, kept: MxMatrix, activation="gelu", dZ=None, dbias=None, workspace=None, stream=None):
    """dZ = dH * act'(kept).  dZ (allocated when None) may be dH itself.
    `dbias`, a float32 tensor of cols elements, receives the column sums of dZ
    when given; the partial sums go to `workspace` (a 16-byte aligned tensor of
    dg_act_backward_workspace_size(rows, cols) bytes) or to one allocated here."""
    rows, cols = kept.rows, kept.cols
    if activation not in _ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(_ACTIVATIONS)}")
    if dZ is None:
        dZ = _empty((rows, cols), dH.dtype, dH.device, stream)
    elif dZ.dtype != dH.dtype:
        raise TypeError("dZ must have dH's dtype")
    ldh, ldz = _plain(dH, "dH", rows, cols), _plain(dZ, "dZ", rows, cols)
    if dbias is not None:
        if dbias.dtype != torch.float32 or dbias.dim() != 1 or dbias.shape[0] != cols or (cols > 1 and dbias.stride(0) != 1):
            raise ValueError(f"dbias must be a contiguous float32 tensor of {cols} elements")
        if workspace is None:
            workspace = _empty(dg_act_backward_workspace_size(rows, cols), torch.uint8, dH.device, stream)  # noqa: F821
    ws, wsb = _workspace(workspace)
    index, handle = _stream_of(stream, (dH, kept.q, kept.s, dZ, dbias, workspace))
    _call("dg_act_backward", index, rows, cols, dH.data_ptr(), ldh, kept.code, kept.q.data_ptr(), kept.ldq,
          kept.s.data_ptr(), kept.lds, dZ.data_ptr(), ldz, _elem(dH, "dH"), _ACTIVATIONS[activation],
          None if dbias is None else dbias.data_ptr(), ws, wsb, handle)
    return dZ
