"""A layer's products: the C ABI's functions one to one, and the torch
conveniences over them (include/dense_gemm.h, "A layer's products").

    gemm_fused, gemm_grouped                 C = act(alpha A op(B) + bias) + beta R
    gemm_act_grad, gemm_grouped_act_grad     C = (alpha A op(B) + beta R) * act'(Z)
    gemm_dw                                  C = alpha A^T B + beta C, and A's column sums

The grouped forms take rows that lie sorted by group (an expert's tokens, one
after the other) and a matrix B for each group.  Like the rest of the package,
these functions only marshal arguments: every step runs in the library's HIP
kernels, on the current torch stream of the tensors' device unless `stream` (a
torch stream of that device) is given, without waiting.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import DG_BF16_F32ACC, DG_BF16_F32OUT, DG_EPI_GELU, DG_EPI_RELU, DG_ERR_HIP, DG_F16_F32ACC, DG_F16_F32OUT, DG_F32
from . import DG_KERNEL_AUTO, DG_OK, EPILOGUES, GemmError, _dtype_code, _lib
from . import dg_last_hip_error, dg_status_string, hip_error_name
from .mx import _current_device, _empty, _kernel_names, _plain, _stream_of, _workspace

_i64, _f32, _vp, _ci, _sz = ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
_ACT_GRADS = {"relu": DG_EPI_RELU, "gelu": DG_EPI_GELU}
_ROWS = [_ci, _i64, _vp, _i64, _i64, _i64, _f32, _vp, _i64, _vp, _i64, _i64]
_ROWS_NAMES = "transB groups offsets M N K alpha A lda B ldb strideB "
_END = [_vp, _i64, _ci, _ci, _vp, _sz, _vp]
_END_NAMES = " C ldc dtype splits workspace workspace_bytes stream"
_FUSED = _ROWS + [_vp, _i64, _ci, _vp, _i64, _f32, _vp, _i64] + _END
_FUSED_NAMES = _ROWS_NAMES + "bias strideBias epilogue Z ldz beta R ldr" + _END_NAMES
_GRAD = _ROWS + [_f32, _vp, _i64, _vp, _i64, _ci, _vp, _i64] + _END
_GRAD_NAMES = _ROWS_NAMES + "beta R ldr H ldh activation Z ldz" + _END_NAMES
_DW = [_i64, _vp, _i64, _i64, _i64, _f32, _vp, _i64, _vp, _i64, _f32, _vp, _i64, _i64, _vp, _ci, _ci, _vp, _sz, _vp]
_DW_NAMES = ("groups offsets rows M N alpha A lda B ldb beta C ldc strideC dbias dtype splits workspace workspace_bytes "
             "stream")
# name: (result, argument types, argument names in position order)
_SIGNATURES = {
    "dg_gemm_fused": (_ci, _FUSED, _FUSED_NAMES),
    "dg_gemm_fused_with_kernel": (_ci, _FUSED + [_ci], _FUSED_NAMES + " kernel"),
    "dg_gemm_fused_choose": (_ci, [_i64, _i64, _i64, _ci, _ci], "M N K transB dtype"),
    "dg_gemm_fused_choose_for": (_ci, [_i64, _i64, _i64, _ci, _ci, _vp, _i64, _vp, _i64], "M N K transB dtype A lda B ldb"),
    "dg_gemm_act_grad": (_ci, _GRAD, _GRAD_NAMES),
    "dg_gemm_act_grad_with_kernel": (_ci, _GRAD + [_ci], _GRAD_NAMES + " kernel"),
    "dg_gemm_dw": (_ci, _DW, _DW_NAMES),
    "dg_gemm_dw_with_kernel": (_ci, _DW + [_ci], _DW_NAMES + " kernel"),
    "dg_gemm_dw_choose": (_ci, [_i64, _i64, _i64, _i64, _ci], "groups rows M N dtype"),
    "dg_gemm_dw_choose_for": (_ci, [_i64, _i64, _i64, _i64, _ci, _vp, _i64, _vp, _i64], "groups rows M N dtype A lda B ldb"),
    "dg_gemm_fused_select": (_ci, [_i64, _i64, _i64, _ci, _ci, _i64, _ci], "M N K transB dtype groups splits"),
    "dg_gemm_dw_select": (_ci, [_i64, _i64, _i64, _i64, _ci, _ci], "groups rows M N dtype splits"),
    "dg_layer_workspace_size": (_sz, [_i64, _i64, _i64, _ci], "groups M N splits"),
    "dg_layer_kernel_name": (ctypes.c_char_p, [_ci], "kernel"),
}
EXPORTED = sorted(_SIGNATURES)
__all__ = EXPORTED + ["LayerError", "gemm_fused", "gemm_grouped", "gemm_act_grad", "gemm_grouped_act_grad", "gemm_dw",
                      "layer_kernel_names"]
_functions = {}
for _name, (_res, _args, _) in _SIGNATURES.items():
    _f = getattr(_lib, _name)
    _f.restype, _f.argtypes = _res, _args
    _functions[_name] = globals()[_name] = _f


def layer_kernel_names() -> list[str]:
    """The kernels of a layer's products, by index."""
    return _kernel_names(dg_layer_kernel_name)  # noqa: F821


class LayerError(GemmError):
    """A failed call of a layer's product, with the name of an invalid argument."""

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


def _run(function, index, args):
    """One library call with device `index` current."""
    f = _functions[function]
    if index == _current_device():
        rc = f(*args)
    else:
        with torch.cuda.device(index):
            rc = f(*args)
    if rc != DG_OK:
        raise LayerError(function, rc)


@functools.lru_cache(1024)
def _fused_splits(M, N, K, transB, dtype, A=0, lda=0, B=0, ldb=0):
    """The library's choice of K ranges by shape and alignment, A and B being addresses modulo
    4 (1 where the call itself will refuse it)."""
    return max(dg_gemm_fused_choose_for(M, N, K, transB, dtype, A, lda, B, ldb), 1)  # noqa: F821


@functools.lru_cache(1024)
def _dw_splits(groups, rows, M, N, dtype, A=0, lda=0, B=0, ldb=0):
    return max(dg_gemm_dw_choose_for(groups, rows, M, N, dtype, A, lda, B, ldb), 1)  # noqa: F821


# (operand, output) -> the library's dtype
_DTYPES = {(torch.float32, torch.float32): DG_F32, (torch.float16, torch.float16): DG_F16_F32ACC,
           (torch.bfloat16, torch.bfloat16): DG_BF16_F32ACC, (torch.float16, torch.float32): DG_F16_F32OUT,
           (torch.bfloat16, torch.float32): DG_BF16_F32OUT}


def _groups(offsets):
    """(groups, address) of a tensor of row offsets."""
    if offsets.dtype != torch.int32:
        raise TypeError("offsets must be int32")
    if offsets.dim() != 1 or offsets.shape[0] < 1 or (offsets.shape[0] > 1 and offsets.stride(0) != 1):
        raise ValueError("offsets must be a contiguous 1-D tensor of groups + 1 elements")
    return offsets.shape[0] - 1, offsets.data_ptr()


def _rows(t, name, shape, dtype):
    """(address, row stride) of a matrix of rows."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must have C's dtype")
    return t.data_ptr(), _plain(t, name, *shape)


def _matrices(B, groups, rows, cols, name="B"):
    """(row stride, stride between the matrices) of [groups, rows, cols]."""
    if B.shape != (groups, rows, cols):
        raise ValueError(f"{name} must be [{groups}, {rows}, {cols}]")
    if groups == 0:
        return max(cols, 1), 0
    return _plain(B[0], name, rows, cols), B.stride(0) if groups > 1 else 0


def _product(grad, A, B, offsets, C, transB, alpha, bias, activation, Z, R, beta, keep, out_dtype, splits, workspace, kernel,
             stream):
    """One product over rows.  `keep`: what the epilogue stores beside C (Z of the
    forward, H of the gradient); Z: the gradient's."""
    sb = B.shape
    if len(A.shape) != 2:
        raise ValueError("A must be 2-D")
    if B.dtype != A.dtype:
        raise TypeError("A and B must share one dtype")
    M, K = A.shape
    if len(sb) != (2 if offsets is None else 3):
        raise ValueError("B must be 2-D" if offsets is None else "B must be 3-D, a matrix for each group")
    N, inner = (sb[-2], sb[-1]) if transB else (sb[-1], sb[-2])
    if inner != K:
        raise ValueError(f"inner dimensions differ: {K} vs {inner}")
    if offsets is None:
        groups, address, ldb, strideB = 1, None, _plain(B, "B", *sb), 0
    else:
        groups, address = _groups(offsets)
        ldb, strideB = _matrices(B, groups, sb[-2], sb[-1])
    shape = (M, N)
    if C is None:
        C = _empty(shape, out_dtype or A.dtype, A.device, stream)
    cd = C.dtype
    dtype = _DTYPES.get((A.dtype, cd))
    if dtype is None:
        raise TypeError(f"unsupported operand/output dtypes {A.dtype}/{cd} (float32, float16 or bfloat16 operands; an "
                        "output of the operand dtype, or float32)")
    lda, ldc, a, b = _plain(A, "A", M, K), _plain(C, "C", M, N), A.data_ptr(), B.data_ptr()
    k, ldk = (None, N or 1) if keep is None else _rows(keep, "H" if grad else "Z", shape, cd)
    r, ldr = (None, N or 1) if R is None else _rows(R, "R", shape, cd)
    if offsets is not None:
        splits = 1
    # more than one range by the library's choice: left to the call, whose kernel belongs to it
    elif splits == 0 and workspace is None and (n := _fused_splits(M, N, K, transB, dtype, a & 3, lda, b & 3, ldb)) == 1:
        splits = 1
    if splits != 1 and workspace is None:
        workspace = _empty(dg_layer_workspace_size(1, M, N, splits or n), torch.uint8, A.device, stream)  # noqa: F821
    ws, wsb = (None, 0) if workspace is None else _workspace(workspace)
    if grad:
        z, ldz = _rows(Z, "Z", shape, cd)
    bias_at, stride_bias = None, 0
    if bias is not None:
        if bias.dtype != cd:
            raise TypeError("bias must have C's dtype")
        if offsets is None:
            if bias.shape != (N,) or (N > 1 and bias.stride(0) != 1):
                raise ValueError(f"bias must be [{N}], contiguous")
        else:
            if bias.shape != (groups, N) or (N > 1 and bias.stride(1) != 1):
                raise ValueError(f"bias must be [{groups}, {N}], its rows contiguous")
            stride_bias = bias.stride(0) if groups > 1 else 0
        bias_at = bias.data_ptr()
    index, handle = _stream_of(stream, (A, B, C, offsets, workspace, bias, Z, R, keep))
    if grad:
        _run("dg_gemm_act_grad_with_kernel", index,
             (transB, groups, address, M, N, K, alpha, a, lda, b, ldb, strideB, beta, r, ldr, k, ldk,
              activation, z, ldz, C.data_ptr(), ldc, dtype, splits, ws, wsb, handle, kernel))
        return C
    _run("dg_gemm_fused_with_kernel", index,
         (transB, groups, address, M, N, K, alpha, a, lda, b, ldb, strideB, bias_at, stride_bias, activation,
          k, ldk, beta, r, ldr, C.data_ptr(), ldc, dtype, splits, ws, wsb, handle, kernel))
    return C


def _activation(codes, name):
    code = codes.get(name)
    if code is None:
        raise ValueError(f"activation must be one of {sorted(codes)}")
    return code


def gemm_fused(A, B, C=None, transB=False, alpha=1.0, bias=None, activation="none", R=None, beta=1.0, Z=None, out_dtype=None,
               splits=0, workspace=None, kernel=DG_KERNEL_AUTO, stream=None):
    """C = act(alpha * A @ op(B) + bias) + beta * R, a layer with its residual.

    A is [M, K]; B [K, N] or (transB) [N, K], of A's dtype; C (allocated when
    None, with `out_dtype` or A's dtype) has A's dtype or, for 16-bit operands,
    float32.  bias (N elements) and the matrices R and Z ([M, N]) have C's dtype
    and may be left out.  Z receives the activation's input, for gemm_act_grad.
    R may be C itself.  activation: "none", "relu" or "gelu".  Sums are fp32, and
    each output is rounded once.

    `splits` cuts K into ranges (0: the library's choice, among those that a given
    workspace holds) whose fp32 sums go to `workspace`, a 16-byte aligned tensor of
    dg_layer_workspace_size(1, M, N, splits) bytes, or to one allocated here."""
    return _product(False, A, B, None, C, transB, alpha, bias, _activation(EPILOGUES, activation), None, R, beta, Z, out_dtype,
                    splits, workspace, kernel, stream)


def gemm_grouped(A, B, offsets, C=None, transB=False, alpha=1.0, bias=None, activation="none", R=None, beta=1.0, Z=None,
                 out_dtype=None, kernel=DG_KERNEL_AUTO, stream=None):
    """gemm_fused with a matrix for each group of rows: rows offsets[g] ..
    offsets[g + 1] - 1 of A, C, R and Z belong to group g, with B[g] and bias[g].

    offsets is an int32 tensor of groups + 1 ascending elements on the device (a
    group may be empty); B is [groups, K, N] or (transB) [groups, N, K]; bias is
    [groups, N].  Rows before offsets[0] and from offsets[-1] on are left as
    they were, in every output (in a C allocated here: uninitialised memory)."""
    return _product(False, A, B, offsets, C, transB, alpha, bias, _activation(EPILOGUES, activation), None, R, beta, Z,
                    out_dtype, 1, None, kernel, stream)


def gemm_act_grad(A, B, Z, C=None, transB=False, alpha=1.0, activation="gelu", R=None, beta=1.0, H=None, out_dtype=None,
                  splits=0, workspace=None, kernel=DG_KERNEL_AUTO, stream=None):
    """C = H * act'(Z) with H = alpha * A @ op(B) + beta * R: the gradient that a
    layer hands to the activation below it.

    Z is the activation's input as gemm_fused keeps it, R a gradient that joins
    (a residual's), and H, where given, receives the sum before act'.  All are
    [M, N] of C's dtype (C: allocated when None, with Z's dtype).  relu chooses H
    or 0; activation is "relu" or "gelu".  The rest as gemm_fused."""
    return _product(True, A, B, None, C, transB, alpha, None, _activation(_ACT_GRADS, activation), Z, R, beta, H,
                    out_dtype or Z.dtype, splits, workspace, kernel, stream)


def gemm_grouped_act_grad(A, B, offsets, Z, C=None, transB=False, alpha=1.0, activation="gelu", R=None, beta=1.0, H=None,
                          out_dtype=None, kernel=DG_KERNEL_AUTO, stream=None):
    """gemm_act_grad with a matrix for each group of rows, as gemm_grouped."""
    return _product(True, A, B, offsets, C, transB, alpha, None, _activation(_ACT_GRADS, activation), Z, R, beta, H,
                    out_dtype or Z.dtype, 1, None, kernel, stream)


def gemm_dw(A, B, C=None, offsets=None, alpha=1.0, beta=0.0, dbias=None, out_dtype=None, splits=0, workspace=None,
            kernel=DG_KERNEL_AUTO, stream=None):
    """C = alpha * A^T @ B + beta * C, a layer's weight gradient from its rows: A
    [rows, M] (the output's gradient), B [rows, N] (the layer's input), C [M, N] of
    their dtype or float32 (allocated when None; beta must be 0 then).

    With offsets (as gemm_grouped) C is [groups, M, N], each over its group's rows
    (a group without rows: beta * C).  dbias, a float32 tensor of M elements (or
    [groups, M], contiguous), receives A's column sums, + beta * dbias; alpha does
    not scale it.

    `splits` cuts every group's rows into ranges (0: the library's choice, among
    those that a given workspace holds) whose fp32 sums go to `workspace`
    (dg_layer_workspace_size(groups, M, N, splits) bytes, 16-byte aligned) or to one
    allocated here."""
    if A.dim() != 2 or B.dim() != 2:
        raise ValueError("A and B must be 2-D")
    if B.dtype != A.dtype:
        raise TypeError("A and B must share one dtype")
    rows, M = A.shape
    if B.shape[0] != rows:
        raise ValueError(f"A and B differ in rows: {rows} vs {B.shape[0]}")
    N = B.shape[1]
    groups, address = (None, None) if offsets is None else _groups(offsets)
    count = 1 if groups is None else groups
    if C is None:
        if beta != 0.0:
            raise ValueError("beta != 0 needs C")
        C = _empty((M, N) if groups is None else (groups, M, N), out_dtype or A.dtype, A.device, stream)
    dtype = _dtype_code(A.dtype, C.dtype)
    ldc, strideC = (_plain(C, "C", M, N), 0) if groups is None else _matrices(C, groups, M, N, "C")
    if dbias is not None and (dbias.dtype != torch.float32 or dbias.shape != ((M,) if groups is None else (groups, M))
                              or not dbias.is_contiguous()):
        raise ValueError("dbias must be a contiguous float32 tensor of " + (f"[{M}]" if groups is None else f"[{groups}, {M}]"))
    lda, ldb, a, b = _plain(A, "A", rows, M), _plain(B, "B", rows, N), A.data_ptr(), B.data_ptr()
    # (more than one range by the library's choice, as in _product)
    if splits == 0 and workspace is None and (n := _dw_splits(count, rows, M, N, dtype, a & 3, lda, b & 3, ldb)) == 1:
        splits = 1
    if splits != 1 and workspace is None:
        workspace = _empty(dg_layer_workspace_size(count, M, N, splits or n), torch.uint8, A.device, stream)  # noqa: F821
    ws, wsb = (None, 0) if workspace is None else _workspace(workspace)
    index, handle = _stream_of(stream, (A, B, C, offsets, dbias, workspace))
    _run("dg_gemm_dw_with_kernel", index,
         (count, address, rows, M, N, alpha, a, lda, b, ldb, beta, C.data_ptr(), ldc, strideC,
          None if dbias is None else dbias.data_ptr(), dtype, splits, ws, wsb, handle, kernel))
    return C
