"""Block-scaled (MX) operators on the CPU: the reference's own pins, the
storage arithmetic, and every refusal (invalid calls return before any HIP
call)."""
import numpy as np
import pytest
import torch

import dense_gemm_amd as dg
import mx_ref
import oracle

NULL = None


# ---- the reference ---------------------------------------------------------------
def test_reference_tables():
    assert list(mx_ref.FP4[:8]) == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    e4m3 = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(mx_ref.FP8, e4m3, equal_nan=True)
    assert mx_ref.INT8[127] == 127 / 64 and mx_ref.INT8[255] == -1 / 64


def test_reference_rounding():
    # block maximum 5: e = floor(log2 5) - 2 = 0; ties to even, saturation at 6
    x = np.zeros((1, 32))
    x[0, :9] = [5.0, 0.25, 0.75, 1.25, 2.5, 3.5, -1.75, 4.999, -0.2]
    code, byte = mx_ref.quantize(x, "mxfp4")
    assert byte[0, 0] == 127 and not byte[0, 1:].any()
    v = mx_ref.values(mx_ref.pack(code, "mxfp4"), mx_ref.scales_to_s(byte), "mxfp4", 32)
    assert list(v[0, :9]) == [4, 0, 1, 1, 2, 4, -2, 4, -0.0]
    x[0, 0] = 7.9                                    # same e: saturates
    v = mx_ref.values(*(lambda c, b: (mx_ref.pack(c, "mxfp4"), mx_ref.scales_to_s(b)))(*mx_ref.quantize(x, "mxfp4")), "mxfp4", 32)
    assert v[0, 0] == 6
    # values that a block holds under the scale of its largest element are kept
    rng = np.random.default_rng(1)
    for fmt, top in (("mxfp4", 6.0), ("mxfp8", 448.0), ("mxint8", 127 / 64)):
        q, s = mx_ref.random_stored(rng, 3, 70, fmt, spread=1)
        s[:] = 127
        w = mx_ref.values(q, s, fmt, 70)
        w[:, 0::32] = top
        code, byte = mx_ref.quantize(w, fmt)
        assert (byte[:, :3] == 127).all()
        assert np.array_equal(mx_ref.values(mx_ref.pack(code, fmt), mx_ref.scales_to_s(byte), fmt, 70), w)


def test_oracle_agrees_with_the_reference():
    """The library's triple-loop oracle on the decoded operands gives the
    reference products that these tests compare with."""
    rng = np.random.default_rng(54)
    q, s = mx_ref.random_stored(rng, 6, 90, "mxfp8", whole=True)
    p, t = mx_ref.random_stored(rng, 5, 90, "mxfp4", whole=True)
    a, b = mx_ref.values(q, s, "mxfp8", 90), mx_ref.values(p, t, "mxfp4", 90)
    ref, _ = oracle.gemm(False, True, 6, 5, 90, 1.0, a.astype(np.float32), 90, b.astype(np.float32), 90, 0.0, None, 5)
    assert np.array_equal(np.asarray(ref).reshape(6, -1)[:, :5], a @ b.T)


# ---- storage -----------------------------------------------------------------------
def test_storage_arithmetic():
    for cols, fp4, b8 in ((0, 0, 0), (1, 128, 256), (256, 128, 256), (257, 256, 512), (2048, 1024, 2048)):
        assert dg.dg_mx_row_bytes(dg.DG_MXFP4, cols) == fp4
        assert dg.dg_mx_row_bytes(dg.DG_MXFP8, cols) == dg.dg_mx_row_bytes(dg.DG_MXINT8, cols) == b8
    assert dg.dg_mx_row_bytes(3, 1) == -1 and dg.dg_mx_row_bytes(0, -1) == -2 and dg.dg_mx_row_bytes(0, 2 ** 31) == -2
    assert dg.dg_mx_scale_bytes(5, 257) == 80 and dg.dg_mx_scale_bytes(-1, 1) == -1 and dg.dg_mx_scale_bytes(1, -1) == -2


def _mx(fmt, rows, cols, extra=0, lds=None):
    q = torch.zeros(rows, mx_ref.row_bytes(fmt, cols) + extra, dtype=torch.uint8)
    s = torch.zeros(mx_ref.groups(cols), lds or rows, 8, dtype=torch.uint8)[:, :rows]
    return dg.MxMatrix(fmt, rows, cols, q, s)


def test_matrix_strides():
    m = _mx("mxfp4", 5, 600, extra=32, lds=9)
    assert (m.ldq, m.lds, m.code) == (3 * 128 + 32, 9, dg.DG_MXFP4)
    m = _mx("mxfp8", 1, 10)
    assert (m.ldq, m.lds) == (256, 1)
    assert "mxfp8, 1 x 10" in repr(m)


@pytest.mark.parametrize("fmt,rows,cols,q,s,err", [
    ("fp4", 1, 1, (1, 128), (1, 1, 8), ValueError),
    ("mxfp4", 2, 1, (1, 128), (1, 2, 8), ValueError),
    ("mxfp4", 1, 257, (1, 128), (2, 1, 8), ValueError),
    ("mxfp4", 1, 257, (1, 256), (1, 1, 8), ValueError),
    ("mxfp4", 3, 1, (3, 128), (1, 2, 8), ValueError),
])
def test_matrix_refusals(fmt, rows, cols, q, s, err):
    with pytest.raises(err):
        dg.MxMatrix(fmt, rows, cols, torch.zeros(q, dtype=torch.uint8), torch.zeros(s, dtype=torch.uint8))


def test_matrix_refuses_types_and_strides():
    q, s = torch.zeros(2, 128, dtype=torch.uint8), torch.zeros(1, 2, 8, dtype=torch.uint8)
    with pytest.raises(TypeError):
        dg.MxMatrix("mxfp4", 2, 4, q.to(torch.int8), s)
    with pytest.raises(ValueError):
        dg.MxMatrix("mxfp4", 2, 4, torch.zeros(128, 2, dtype=torch.uint8).t(), s)
    with pytest.raises(ValueError):
        dg.MxMatrix("mxfp4", 2, 4, q, torch.zeros(1, 8, 2, dtype=torch.uint8).transpose(1, 2))
    with pytest.raises(ValueError):
        dg.MxMatrix("mxfp4", 1, 300, torch.zeros(1, 256, dtype=torch.uint8), torch.zeros(20, dtype=torch.uint8).as_strided((2, 1, 8), (12, 8, 1)))


# ---- refusals of the C calls: (argument changes, position) -------------------------
QUANT = dict(transX=0, rows=4, cols=40, X=0x1000, ldx=40, type=0, format=0, Q=0x2000, ldq=128, S=0x3000, lds=4, stream=NULL)
DEQ = dict(rows=4, cols=40, format=0, Q=0x2000, ldq=128, S=0x3000, lds=4, X=0x1000, ldx=40, type=0, stream=NULL)
MX = dict(M=4, N=5, K=40, alpha=1.0, formatA=1, A=0x1000, lda=256, SA=0x2000, ldsa=4, formatB=0, B=0x3000, ldb=128,
          SB=0x4000, ldsb=5, beta=0.0, C=0x5000, ldc=5, type=2, bias=0x6000, epilogue=0, stream=NULL)
DQ = dict(transA=0, M=4, N=40, K=64, alpha=1.0, A=0x1000, lda=64, typeA=1, formatB=0, B=0x2000, ldb=128, SB=0x3000,
          ldsb=64, beta=0.0, C=0x4000, ldc=40, typeC=1, splits=1, workspace=NULL, workspace_bytes=0, stream=NULL)
CKPT = dict(rows=4, cols=40, Z=0x1000, ldz=40, H=0x2000, ldh=40, type=1, activation=2, format=1, Q=0x3000, ldq=256,
            S=0x4000, lds=4, stream=NULL)
BWD = dict(rows=4, cols=40, dH=0x1000, ldh=40, format=1, Q=0x3000, ldq=256, S=0x4000, lds=4, dZ=0x5000, ldz=40, type=1,
           activation=2, dbias=NULL, workspace=NULL, workspace_bytes=0, stream=NULL)
BIG = 2 ** 31

REFUSED = (
    [("dg_mx_quantize", QUANT, kw, c) for kw, c in [
        (dict(transX=2), 1), (dict(rows=-1), 2), (dict(rows=BIG), 2), (dict(cols=-1), 3), (dict(cols=BIG), 3),
        (dict(X=NULL), 4), (dict(X=0x1002), 4), (dict(type=1, X=0x1001), 4), (dict(ldx=39), 5),
        (dict(transX=1, ldx=3), 5), (dict(type=3), 6), (dict(type=-1), 6), (dict(format=3), 7), (dict(Q=NULL), 8),
        (dict(Q=0x2008), 8), (dict(ldq=64), 9), (dict(ldq=136), 9), (dict(format=1), 9), (dict(cols=257, ldx=257), 9),
        (dict(S=NULL), 10), (dict(S=0x3004), 10), (dict(lds=3), 11)]] +
    [("dg_mx_dequantize", DEQ, kw, c) for kw, c in [
        (dict(rows=-1), 1), (dict(cols=-1), 2), (dict(format=-1), 3), (dict(Q=NULL), 4), (dict(Q=0x2001), 4),
        (dict(ldq=127), 5), (dict(S=NULL), 6), (dict(S=0x3001), 6), (dict(lds=3), 7), (dict(X=NULL), 8),
        (dict(X=0x1002), 8), (dict(ldx=39), 9), (dict(type=7), 10)]] +
    [("dg_gemm_mx", MX, kw, c) for kw, c in [
        (dict(M=-1), 1), (dict(N=-1), 2), (dict(K=-1), 3), (dict(K=BIG - 1), 3), (dict(formatA=2), 5), (dict(formatA=9), 5),
        (dict(A=NULL), 6), (dict(A=0x1008), 6), (dict(lda=128), 7), (dict(lda=264), 7), (dict(SA=NULL), 8),
        (dict(SA=0x2002), 8), (dict(ldsa=3), 9), (dict(formatB=1), 10), (dict(B=NULL), 11), (dict(B=0x3004), 11),
        (dict(ldb=127), 12), (dict(SB=NULL), 13), (dict(SB=0x4004), 13), (dict(ldsb=4), 14), (dict(C=NULL), 16),
        (dict(C=0x5001), 16), (dict(ldc=4), 17), (dict(type=3), 18), (dict(bias=0x6001), 19), (dict(epilogue=3), 20)]] +
    [("dg_gemm_dq", DQ, kw, c) for kw, c in [
        (dict(transA=5), 1), (dict(M=-1), 2), (dict(N=BIG), 3), (dict(K=-1), 4), (dict(A=NULL), 6), (dict(A=0x1001), 6),
        (dict(lda=63), 7), (dict(transA=1, lda=3), 7), (dict(typeA=0), 8), (dict(typeA=3), 8), (dict(formatB=4), 9),
        (dict(B=NULL), 10), (dict(B=0x2008), 10), (dict(ldb=64), 11), (dict(formatB=2), 11), (dict(SB=NULL), 12),
        (dict(SB=0x3001), 12), (dict(ldsb=63), 13), (dict(C=NULL), 15), (dict(C=0x4001), 15), (dict(ldc=39), 16),
        (dict(typeC=2), 17), (dict(typeC=-1), 17), (dict(splits=-1), 18), (dict(splits=4097), 18),
        (dict(K=640, lda=640, ldsb=640, splits=2), 19),
        (dict(K=640, lda=640, ldsb=640, splits=2, workspace=0x9004, workspace_bytes=1 << 20), 19),
        (dict(K=640, lda=640, ldsb=640, splits=2, workspace=0x9000, workspace_bytes=2 * 4 * 40 * 4 - 1), 20)]] +
    [("dg_act_checkpoint", CKPT, kw, c) for kw, c in [
        (dict(rows=-1), 1), (dict(cols=-1), 2), (dict(Z=NULL), 3), (dict(Z=0x1001), 3), (dict(ldz=39), 4),
        (dict(H=NULL), 5), (dict(H=0x2001), 5), (dict(ldh=39), 6), (dict(H=0x1000, ldh=48), 6), (dict(type=5), 7),
        (dict(activation=0), 8), (dict(activation=3), 8), (dict(format=0), 9), (dict(Q=NULL), 10), (dict(Q=0x3001), 10),
        (dict(ldq=128), 11), (dict(S=NULL), 12), (dict(lds=3), 13)]] +
    [("dg_act_backward", BWD, kw, c) for kw, c in [
        (dict(rows=-1), 1), (dict(cols=-1), 2), (dict(dH=NULL), 3), (dict(dH=0x1001), 3), (dict(ldh=39), 4),
        (dict(format=0), 5), (dict(Q=NULL), 6), (dict(ldq=100), 7), (dict(S=NULL), 8), (dict(lds=0), 9),
        (dict(dZ=NULL), 10), (dict(dZ=0x5001), 10), (dict(ldz=39), 11), (dict(dZ=0x1000, ldz=48), 11), (dict(type=3), 12),
        (dict(activation=0), 13), (dict(dbias=0x7002), 14), (dict(dbias=0x7000), 15),
        (dict(dbias=0x7000, workspace=0x8004, workspace_bytes=1 << 20), 15),
        (dict(dbias=0x7000, workspace=0x8000, workspace_bytes=39 * 4), 16)]]
)


@pytest.mark.parametrize("name,good,change,position", REFUSED)
def test_refusals(name, good, change, position):
    args = dict(good, **change)
    assert getattr(dg, name)(*args.values()) == -position
    named = list(good)[position - 1]
    assert f"invalid argument {position} ({named})" in str(dg.MxError(name, -position))


def test_empty_problems_do_nothing():
    for name, good in (("dg_mx_quantize", QUANT), ("dg_mx_dequantize", DEQ), ("dg_act_checkpoint", CKPT), ("dg_act_backward", BWD)):
        for kw in (dict(rows=0), dict(cols=0)):
            none = {k: NULL for k in good if isinstance(good[k], int) and good[k] >= 0x1000}
            assert getattr(dg, name)(*dict(good, **kw, **none).values()) == 0, (name, kw)
    for name, good in (("dg_gemm_mx", MX), ("dg_gemm_dq", DQ)):
        for kw in (dict(M=0), dict(N=0)):
            none = {k: NULL for k in good if isinstance(good[k], int) and good[k] >= 0x1000}
            assert getattr(dg, name)(*dict(good, **kw, **none).values()) == 0, (name, kw)


def test_kernel_choice():
    names = dg.mx_kernel_names()
    assert len(names) == len(set(names)) and dg.dg_gemm_mx_kernel_name(-1) is None
    pick = lambda M, N, K, fa=dg.DG_MXFP8: names[dg.dg_gemm_mx_select(fa, M, N, K)]  # noqa: E731
    for fa in (dg.DG_MXFP4, dg.DG_MXFP8):
        # single tokens: the kernel that reads the weights once
        for N, K in ((64, 64), (5632, 2048), (8192, 8192)):
            assert pick(1, N, K, fa) == "mx_16x16_rows"
        assert pick(8192, 8192, 8192, fa) == "mx_256x256_tile"
    # the faster kernel when measured on either side
    assert pick(16, 8192, 8192) == "mx_16x16_rows" and pick(64, 2048, 2048) == "mx_32x16_rows"
    assert pick(32, 8192, 8192) == "mx_64x64_tile" and pick(128, 5632, 2048) == "mx_64x64_tile"
    assert pick(1024, 8192, 8192) == "mx_128x128_tile"
    assert pick(2048, 8192, 4096, dg.DG_MXFP4) == "mx_256x256_tile"
    assert [dg.dg_gemm_mx_select(*a) for a in ((2, 1, 1, 1), (1, -1, 1, 1), (1, 1, -1, 1), (1, 1, 1, -1))] == [-1, -2, -3, -4]
    assert dg.dg_gemm_mx_with_kernel(*MX.values(), len(names)) == dg.DG_ERR_UNSUPPORTED
    # rows too long for the tiled kernels' 32-bit offsets: refused when forced
    far = dict(MX, lda=1 << 23, M=100, ldsa=100)
    assert dg.dg_gemm_mx_with_kernel(*far.values(), len(names) - 1) == dg.DG_ERR_UNSUPPORTED
    big = 2 ** 30
    assert dg.dg_gemm_dq(*dict(DQ, M=big, N=big, lda=64, ldb=big, ldc=big).values()) == dg.DG_ERR_UNSUPPORTED


def test_split_choice():
    assert dg.dg_gemm_dq_choose(5632, 2048, 16384) == 1
    assert dg.dg_gemm_dq_choose(32, 2048, 4096) > 1
    assert dg.dg_gemm_dq_choose(32, 2048, 64) == 1
    assert dg.dg_gemm_dq_choose(0, 5, 5) == 1
    assert [dg.dg_gemm_dq_choose(*a) for a in ((-1, 1, 1), (1, -1, 1), (1, 1, -1))] == [-1, -2, -3]
    assert dg.dg_act_backward_workspace_size(0, 5) == 0
    for r, c in ((1, 1), (511, 5631), (32768, 5632), (3, 2 ** 20)):
        n = dg.dg_act_backward_workspace_size(r, c)
        assert n % (4 * c) == 0 and 1 <= n // (4 * c) <= min(2048, (r + 3) // 4)


# ---- refusals of the torch functions (CPU tensors never reach the library) ----------
def test_torch_functions_refuse():
    x = torch.zeros(4, 40)
    w = _mx("mxfp4", 5, 40)
    a8 = _mx("mxfp8", 4, 40)
    for call in (
        lambda: dg.quantize_mx(x),                                       # not on a GPU
        lambda: dg.quantize_mx(x[0]),
        lambda: dg.quantize_mx(x[:1].expand(4, 40)),                     # rows on top of each other
        lambda: dg.quantize_mx(x, out=_mx("mxfp4", 4, 41)),
        lambda: dg.quantize_mx(torch.zeros(40, 4).t(), out=a8),
        lambda: dg.quantize_mx(x, format="fp4"),
        lambda: dg.dequantize_mx(a8, out=torch.zeros(4, 41)),
        lambda: dg.dequantize_mx(a8),
        lambda: dg.gemm_mx(a8, _mx("mxfp4", 5, 41)),
        lambda: dg.gemm_mx(a8, w, beta=1.0),
        lambda: dg.gemm_mx(a8, w, activation="tanh"),
        lambda: dg.gemm_mx(a8, w, bias=torch.zeros(5)),
        lambda: dg.gemm_mx(a8, w, C=torch.zeros(5, 4)),
        lambda: dg.gemm_mx(a8, w),
        lambda: dg.gemm_dq(torch.zeros(3, 7, dtype=torch.float16), w),
        lambda: dg.gemm_dq(torch.zeros(3, 5, dtype=torch.float16), w, beta=1.0),
        lambda: dg.gemm_dq(torch.zeros(3, 5, dtype=torch.float16), w),
        lambda: dg.gemm_dq(torch.zeros(3, 5, dtype=torch.float16), w, workspace=torch.zeros(64, 2)[:, 0]),
        lambda: dg.act_checkpoint(x, "none"),
        lambda: dg.act_checkpoint(x, "gelu", out=_mx("mxfp8", 4, 39)),
        lambda: dg.act_checkpoint(x, "gelu"),
        lambda: dg.act_backward(x, a8, "none"),
        lambda: dg.act_backward(torch.zeros(4, 41), a8, "gelu"),
        lambda: dg.act_backward(x, a8, "gelu", dbias=torch.zeros(41)),
        lambda: dg.act_backward(x, a8, "gelu"),
    ):
        with pytest.raises(ValueError):
            call()
    for call in (
        lambda: dg.quantize_mx(x.double(), out=a8),
        lambda: dg.gemm_dq(torch.zeros(3, 5), w),
        lambda: dg.gemm_dq(torch.zeros(3, 5, dtype=torch.float16), w, C=torch.zeros(3, 40, dtype=torch.bfloat16)),
        lambda: dg.act_checkpoint(x, "gelu", H=x.half()),
        lambda: dg.act_backward(x, a8, "gelu", dZ=x.half()),
    ):
        with pytest.raises(TypeError):
            call()


def test_keep_positive_goes_with_relu_in_the_checkpoint():
    """The checkpoint's own activation value is refused everywhere else."""
    assert dg.dg_act_backward(*dict(BWD, activation=dg.DG_EPI_RELU_POSITIVE).values()) == -13
    assert dg.dg_gemm_mx(*dict(MX, epilogue=dg.DG_EPI_RELU_POSITIVE).values()) == -20
    assert dg.dg_act_checkpoint(*dict(CKPT, activation=dg.DG_EPI_RELU_POSITIVE, Q=NULL).values()) == -10
    with pytest.raises(ValueError, match="relu"):
        dg.act_checkpoint(torch.zeros(4, 40), "gelu", keep_positive=True)


def test_dq_kernel_choice():
    names = dg.dq_kernel_names()
    assert len(names) == len(set(names)) and dg.dg_gemm_dq_kernel_name(-1) is None
    pick = lambda *mnk: (names[dg.dg_gemm_dq_select(*mnk)], dg.dg_gemm_dq_choose(*mnk))  # noqa: E731
    # each tile serves a shape: dW of an adapter, dX of a step and of a batch, large products
    assert pick(32, 2048, 4096)[0] == "dq_32x128_tile" and pick(32, 2048, 4096)[1] > 1
    assert pick(512, 2048, 5632) == ("dq_64x128_tile", 4)
    assert pick(1024, 2048, 8192) == ("dq_128x128_tile", 3)
    assert pick(4096, 4096, 4096) == ("dq_256x256_tile", 1)
    assert pick(5632, 2048, 16384) == ("dq_256x256_tile", 1)
    assert [dg.dg_gemm_dq_select(*a) for a in ((-1, 1, 1), (1, -1, 1), (1, 1, -1))] == [-1, -2, -3]
    forced = lambda kernel, **kw: dg.dg_gemm_dq_with_kernel(*dict(DQ, **kw).values(), kernel)  # noqa: E731
    assert forced(len(names)) == forced(-2) == dg.DG_ERR_UNSUPPORTED
    # the 256 x 256 tile takes A by direct loads: 4-byte aligned rows, whole pieces of a transposed A
    for kw in (dict(A=0x1002), dict(lda=65), dict(transA=1, lda=64), dict(lda=1 << 22)):
        assert forced(3, **kw) == dg.DG_ERR_UNSUPPORTED, kw
    assert forced(3, A=NULL) == -6


@pytest.mark.parametrize("rows,cols", [(1, 1), (8, 9), (33, 8), (511, 5631), (512, 5632), (2048, 2048), (32768, 5632),
                                       (32773, 24), (131072 + 37, 8), (2 ** 31 - 1, 1), (3, 2 ** 20), (40, 2 ** 31 - 1),
                                       (2 ** 20, 2 ** 21)])
def test_backward_workspace(rows, cols):
    """One row of partial sums per slice: a band of rows each (32 rows where that
    leaves 1024 workgroups of 512 columns, else 16 where that leaves 256, else 8), 4096
    at most and no more than 2^22 workgroups."""
    chunks = -(-cols // 512)
    band = 32 if -(-rows // 32) * chunks >= 1024 else 16 if -(-rows // 16) * chunks >= 256 else 8
    slices = max(1, min(-(-rows // band), 4096, 2 ** 22 // chunks))
    assert dg.dg_act_backward_workspace_size(rows, cols) == slices * cols * 4
    assert slices * chunks <= 2 ** 22


def test_select_names_what_no_kernel_runs():
    """More tiles than a launch holds: the products' own status, not that of an
    invalid argument."""
    big = 2 ** 31 - 1
    for fa in (dg.DG_MXFP4, dg.DG_MXFP8):
        for M, N, K in ((big, big, 1), (big, 1, 1), (1, big, 1), (2 ** 21, 2 ** 21, 256)):
            assert dg.dg_gemm_mx_select(fa, M, N, K) == dg.DG_ERR_UNSUPPORTED, (M, N, K)
            args = dict(MX, M=M, N=N, K=K, formatA=fa, lda=256, ldb=256, ldsa=M, ldsb=N, ldc=N)
            assert dg.dg_gemm_mx(*args.values()) == dg.DG_ERR_UNSUPPORTED
        names = dg.mx_kernel_names()
        assert names[dg.dg_gemm_mx_select(fa, 2 ** 30 - 256, 256, 256)] == "mx_256x256_tile"


def test_status_texts_say_whose_argument_they_name():
    """A position means another argument in every family of calls: a text that
    names one says for which call."""
    for i in range(1, 23):
        text = dg.dg_status_string(-i)
        assert text.startswith(f"invalid argument {i}")
        names = text[len(f"invalid argument {i}"):].strip(" ()")
        assert not names or all(n.strip().startswith("dg_gemm") for n in names.split(";")), text


def test_dq_ranges_of_large_partials():
    """Partials of 46 MB and more a range: two ranges where they fill the last
    round of tiles, one where they would add a round."""
    names = dg.dq_kernel_names()
    for shape, tile, ranges in (((4096, 2048, 16384), "dq_256x256_tile", 2), ((5632, 4096, 16384), "dq_256x256_tile", 2),
                                ((3584, 2048, 16384), "dq_256x256_tile", 2), ((5632, 2048, 16384), "dq_256x256_tile", 1),
                                ((4608, 3584, 16384), "dq_256x256_tile", 1), ((256, 1024, 1024), "dq_32x128_tile", 1)):
        assert (names[dg.dg_gemm_dq_select(*shape)], dg.dg_gemm_dq_choose(*shape)) == (tile, ranges), shape
