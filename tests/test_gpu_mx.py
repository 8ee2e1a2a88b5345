"""Block-scaled (MX) operators on an MI355X, against the fp64 definition of
mx_ref: rounding bit for bit, the products exactly on data whose sums are
exact and within derived bounds on others, the activations' two passes, and
the calls as a program makes them (views, streams, graphs, a chain of all)."""
import math

import numpy as np
import pytest
import torch

import dense_gemm_amd as dg
import mx_ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
FORMATS = ("mxfp4", "mxfp8", "mxint8")
#: half a step of a type, relative to the value, and its least step halved
HALF = {t: torch.finfo(t).eps / 2 for t in T.values()}
TINY = {t: torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2 for t in T.values()}


def np64(t):
    return t.detach().double().cpu().numpy()


def plain(rng, rows, cols, dtype, pad=0, std=1.0):
    """A random matrix on the GPU with `pad` NaN columns behind its rows."""
    x = torch.full((rows, cols + pad), math.nan, dtype=dtype)
    x[:, :cols] = torch.from_numpy(rng.standard_normal((rows, cols)) * std).to(dtype)
    return x.to(DEV)[:, :cols]


def stored(rng, rows, cols, fmt, extra=0, lds=None, **kw):
    """A random MX matrix on the GPU, its rows `extra` bytes and its groups
    lds rows apart, and its fp64 values."""
    q, s = mx_ref.random_stored(rng, rows, cols, fmt, **kw)
    qt = torch.full((rows, q.shape[1] + extra), 0xA5, dtype=torch.uint8)
    qt[:, :q.shape[1]] = torch.from_numpy(q)
    st = torch.full((s.shape[0], lds or rows, 8), 0xA5, dtype=torch.uint8)
    st[:, :rows] = torch.from_numpy(s)
    m = dg.MxMatrix(fmt, rows, cols, qt.to(DEV), st.to(DEV)[:, :rows])
    return m, mx_ref.values(q, s, fmt, cols)


def rounded(x, fmt):
    code, byte = mx_ref.quantize(x, fmt)
    return mx_ref.pack(code, fmt), mx_ref.scales_to_s(byte)


# ---- rounding ------------------------------------------------------------------------
SHAPES = [(1, 1), (1, 31), (3, 32), (5, 33), (2, 255), (7, 256), (4, 257), (33, 1000), (65, 513), (300, 70)]


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("ty", list(T))
def test_quantize_bit_for_bit(ty, fmt, trans):
    rng = np.random.default_rng(10)
    for rows, cols in SHAPES:
        for pad in (0, 1, 8):
            x = plain(rng, *((cols, rows) if trans else (rows, cols)), T[ty], pad, std=0.3)
            extra, lds = 32, rows + 3
            q = torch.full((rows, mx_ref.row_bytes(fmt, cols) + extra), 0xA5, dtype=torch.uint8, device=DEV)
            s = torch.full((mx_ref.groups(cols), lds, 8), 0xA5, dtype=torch.uint8, device=DEV)
            m = dg.quantize_mx(x, trans=trans, out=dg.MxMatrix(fmt, rows, cols, q, s[:, :rows]))
            wq, ws = rounded(np64(x).T if trans else np64(x), fmt)
            nb = wq.shape[1]
            assert np.array_equal(q[:, :nb].cpu().numpy(), wq), (rows, cols, pad)
            assert np.array_equal(s[:, :rows].cpu().numpy(), ws), (rows, cols, pad)
            assert (q[:, nb:] == 0xA5).all() and (s[:, rows:] == 0xA5).all()      # nothing else is written
            back = dg.dequantize_mx(m)
            assert np.array_equal(np64(back), mx_ref.values(wq, ws, fmt, cols))


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("fmt", FORMATS)
def test_quantize_special_values(fmt, trans):
    """Zeros, signed zeros, ties, saturation, the ends of the range, subnormals,
    NaN and infinities: one block each, with a block of ordinary values behind."""
    x = np.zeros((14, 64), np.float32)
    x[:, 32:] = np.linspace(-3, 3, 32)
    x[1, :32] = -0.0
    x[2, :32] = np.arange(32) * 0.25 - 4               # ties of mxfp4
    x[3, :32] = np.linspace(7.0, 7.99, 32)             # saturates in mxfp4
    x[4, :32] = np.linspace(448, 511.9, 32)            # saturates in mxfp8
    x[5, :32] = np.linspace(1.9, 1.9999999, 32)        # saturates in mxint8
    x[6, :32] = 3.4028235e38
    x[7, :32] = 2.0 ** -149
    x[8, :32] = np.arange(32) * 2.0 ** -130
    x[9, :32] = 2.0 ** -126 * np.linspace(1, 1.9, 32)
    x[10, 5] = np.nan
    x[11, 6] = np.inf
    x[12, 31] = -np.inf
    x[13, :32] = np.float32(2.0) ** np.arange(-16, 16)
    X = torch.from_numpy(np.ascontiguousarray(x.T) if trans else x).to(DEV)
    m = dg.quantize_mx(X, format=fmt, trans=trans)
    wq, ws = rounded(x.astype(np.float64), fmt)
    assert np.array_equal(m.q.cpu().numpy(), wq) and np.array_equal(m.s.cpu().numpy(), ws)
    want = mx_ref.values(wq, ws, fmt, 64)
    got = np64(dg.dequantize_mx(m))
    assert np.isnan(want[10:13, :32]).all() and np.array_equal(got, want.astype(np.float32).astype(np.float64), equal_nan=True)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("ty", ["f16", "bf16"])
def test_rounding_from_16_bits_is_exact_in_16_bits(ty, fmt):
    """A matrix rounded from a 16-bit type has values that the type holds, down
    to the type's least step and up to its largest value."""
    rng = np.random.default_rng(11)
    info = torch.finfo(T[ty])
    x = torch.from_numpy(rng.standard_normal((40, 300))).to(T[ty])
    x[0, :] = torch.from_numpy(rng.uniform(-1, 1, 300)).to(T[ty]) * info.max
    if ty == "f16":
        x[1, :] = torch.from_numpy(rng.integers(-40, 40, 300) * 2.0 ** -24).to(T[ty])
    m = dg.quantize_mx(x.to(DEV), format=fmt)
    exact = np64(dg.dequantize_mx(m))
    for pad in (0, 1, 8):
        out = torch.full((40, 300 + pad), math.nan, dtype=T[ty], device=DEV)
        dg.dequantize_mx(m, out=out[:, :300])
        assert np.array_equal(np64(out[:, :300]), exact) and torch.isnan(out[:, 300:]).all()


def test_views_of_rows_and_groups():
    """Row ranges and column groups of a stored matrix are matrices of their own."""
    rng = np.random.default_rng(12)
    m, v = stored(rng, 50, 700, "mxfp4")
    part = dg.MxMatrix("mxfp4", 13, 700, m.q[7:20], m.s[:, 7:20])
    assert np.array_equal(np64(dg.dequantize_mx(part)), v[7:20])
    part = dg.MxMatrix("mxfp4", 50, 444, m.q[:, 128:], m.s[1:])
    assert np.array_equal(np64(dg.dequantize_mx(part)), v[:, 256:])
    x = plain(rng, 9, 37, torch.float16)
    part, _ = stored(rng, 50, 700, "mxfp4")
    before = part.q.clone()
    dg.quantize_mx(x, out=dg.MxMatrix("mxfp4", 9, 37, part.q[3:12], part.s[:1, 3:12]))
    assert torch.equal(part.q[:3], before[:3]) and torch.equal(part.q[12:], before[12:])
    assert torch.equal(part.q[3:12, 128:], before[3:12, 128:])


# ---- products of two MX matrices -------------------------------------------------------
def erfc(x):
    return torch.special.erfc(torch.from_numpy(np.ascontiguousarray(x))).numpy()


def act64(x, act):
    if act == "relu":
        return np.maximum(x, 0)
    if act == "gelu":
        return 0.5 * x * erfc(-x / math.sqrt(2))
    return x


@pytest.mark.parametrize("fa", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("kernel", range(len(dg.mx_kernel_names())))
def test_product_exact(kernel, fa):
    """Elements of a few bits and scales within 2^-1 .. 2^1: every product is a
    multiple of 2^-4 (2^-2 scales, halves by halves at the least) and a row's sum
    stays below 2^20, so the fp32 sums are exact in any order; an mxfp8 operand's
    products span 2^11, within the 2^13 that the instruction keeps."""
    rng = np.random.default_rng(20)
    for M, N, K in ((1, 1, 1), (1, 40, 256), (5, 17, 33), (16, 64, 700), (31, 33, 2048), (33, 65, 257), (70, 130, 513),
                    (129, 127, 1030), (300, 270, 300), (257, 513, 1280)):
        A, a = stored(rng, M, K, fa, extra=16, lds=M + 1, spread=1, whole=True)
        B, b = stored(rng, N, K, "mxfp4", extra=48, lds=N + 2, spread=1, whole=True)
        C = torch.full((M + 1, N + 3), math.nan, device=DEV)
        dg.gemm_mx(A, B, C=C[:M, :N], kernel=kernel)
        assert np.array_equal(np64(C[:M, :N]), a @ b.T), (M, N, K)
        assert torch.isnan(C[M:]).all() and torch.isnan(C[:, N:]).all()


@pytest.mark.parametrize("ty", list(T))
@pytest.mark.parametrize("fa", ["mxfp4", "mxfp8"])
def test_product_epilogue(fa, ty):
    """alpha, beta, bias, activation, odd row strides and every output type, on
    exact sums.  The epilogue is three fp32 operations, then gelu (1e-6 |x| and
    slope at most 1.13), then half a step of the output type."""
    rng = np.random.default_rng(21)
    for M, N, K in ((3, 50, 300), (40, 75, 300), (200, 131, 512)):
        A, a = stored(rng, M, K, fa, spread=1, whole=True)
        B, b = stored(rng, N, K, "mxfp4", spread=1, whole=True)
        s = a @ b.T
        alpha, beta = 1.0 / 64, -0.5
        for act in ("none", "relu", "gelu"):
            for pad in (0, 1):
                c0 = plain(rng, M, N, T[ty], pad)
                bias = plain(rng, 1, N, T[ty])[0]
                base = np64(c0)
                full = c0.as_strided((M, N + pad), (N + pad, 1))
                dg.gemm_mx(A, B, C=c0, alpha=alpha, beta=beta, bias=bias, activation=act)
                pre = alpha * s + beta * base + np64(bias)
                mag = np.abs(alpha * s) + np.abs(beta * base) + np.abs(np64(bias))
                want = act64(pre, act)
                tol = 1.13 * 4 * 2.0 ** -24 * mag + (1e-6 * np.abs(pre) if act == "gelu" else 0)
                tol = tol * (1 + HALF[T[ty]]) + HALF[T[ty]] * np.abs(want) + TINY[T[ty]]
                assert (np.abs(np64(c0) - want) <= tol).all(), (M, N, act, pad)
                if pad:
                    assert torch.isnan(full[:, N:]).all()


@pytest.mark.parametrize("fa,rel", [("mxfp4", 2.0 ** -21), ("mxfp8", 2.0 ** -16)])
@pytest.mark.parametrize("kernel", range(len(dg.mx_kernel_names())))
def test_product_normal_data(kernel, fa, rel):
    """Normal data rounded to MX, fp32 output, by norm.  Two mxfp4 operands: at
    most K/64 + 8 = 40 fp32 roundings of 2^-24 each, relative to sums that random
    signs leave at least 1/8 of the largest partial sum on average: 2^-24 * 40 / 8
    < 2^-21.  An mxfp8 operand drops what lies 2^-13 below a step's largest
    product: each of the 64 products of a step loses at most one unit of 2^-13 of
    it, at random, so a step is off by 8 units of 2^-13 / sqrt(12), against a
    step's norm of about 8 products at a third to a quarter of the largest:
    2^-13 / 3.5 * 4 < 2^-12 per product pair that is hit; products of normal data
    have at least 2^4 of their bits above that line: 2^-16."""
    rng = np.random.default_rng(22)
    M, N, K = 150, 170, 2048
    A = dg.quantize_mx(plain(rng, M, K, torch.float32), format=fa)
    B = dg.quantize_mx(plain(rng, N, K, torch.float32), format="mxfp4")
    a, b = np64(dg.dequantize_mx(A)), np64(dg.dequantize_mx(B))
    got = np64(dg.gemm_mx(A, B, out_dtype=torch.float32, kernel=kernel))
    want = a @ b.T
    assert np.linalg.norm(got - want) <= rel * np.linalg.norm(want)


def test_product_special_values():
    """A NaN scale reaches its row (or column) of C only; beta = 0 ignores C's
    NaN; alpha = 0 and K = 0 do not read A and B; the largest and least scales."""
    rng = np.random.default_rng(23)
    for M in (4, 100):
        A, a = stored(rng, M, 512, "mxfp8", spread=1, whole=True)
        B, b = stored(rng, 90, 512, "mxfp4", spread=1, whole=True)
        A.s[1, 2, 5] = 255
        B.s[0, 7, 0] = 255
        C = np64(dg.gemm_mx(A, B, out_dtype=torch.float32))
        bad = np.zeros((M, 90), bool)
        bad[2], bad[:, 7] = True, True
        assert np.isnan(C[bad]).all() and np.array_equal(C[~bad], (a @ b.T)[~bad])
        c0 = plain(rng, M, 90, torch.float32)
        want = 0.5 * np64(c0)
        dg.gemm_mx(A, B, C=c0, alpha=0.0, beta=0.5)
        assert np.array_equal(np64(c0), want)
        none = dg.MxMatrix.empty("mxfp8", M, 0, DEV), dg.MxMatrix.empty("mxfp4", 90, 0, DEV)
        bias = plain(rng, 1, 90, torch.float32)[0]
        assert np.array_equal(np64(dg.gemm_mx(*none, bias=bias, out_dtype=torch.float32)), np.tile(np64(bias), (M, 1)))
        A, a = stored(rng, M, 64, "mxfp4", whole=True)
        B, b = stored(rng, 90, 64, "mxfp4", whole=True)
        A.s.fill_(0)                                     # 2^-127 times 2^100
        B.s.fill_(227)
        q, s = A.q.cpu().numpy(), A.s.cpu().numpy()
        av = mx_ref.values(q, s, "mxfp4", 64)
        bv = mx_ref.values(B.q.cpu().numpy(), B.s.cpu().numpy(), "mxfp4", 64)
        assert np.array_equal(np64(dg.gemm_mx(A, B, out_dtype=torch.float32)), av @ bv.T)


# ---- a 16-bit matrix times an MX matrix ------------------------------------------------
DQ_SHAPES = [(1, 1, 1), (3, 40, 5), (32, 256, 64), (33, 129, 65), (31, 300, 200), (128, 128, 192), (130, 270, 130),
             (257, 391, 321), (8, 2048, 640), (300, 130, 1000)]


@pytest.mark.parametrize("transA", [False, True])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("ty", ["f16", "bf16"])
def test_dq_product_exact(ty, fmt, transA):
    """Whole A of at most 8 and B as in the exact products above: all sums are
    exact in fp32.  Padded, odd and misaligned rows of A, every K tail."""
    rng = np.random.default_rng(30)
    for M, N, K in DQ_SHAPES:
        B, b = stored(rng, K, N, fmt, extra=16, lds=K + 1, spread=1, whole=True)
        for pad, shift in ((0, 0), (1, 0), (2, 2), (8, 1)):
            r, c = (K, M) if transA else (M, K)
            flat = torch.full((r * (c + pad) + shift,), math.nan, dtype=T[ty])
            a = rng.integers(-8, 9, (r, c)).astype(np.float64)
            flat[shift:].view(r, c + pad)[:, :c] = torch.from_numpy(a).to(T[ty])
            A = flat.to(DEV)[shift:].view(r, c + pad)[:, :c]
            C = torch.full((M, N + 1), math.nan, device=DEV)
            dg.gemm_dq(A, B, C=C[:, :N], transA=transA)
            assert np.array_equal(np64(C[:, :N]), (a.T if transA else a) @ b), (M, N, K, pad, shift)
            assert torch.isnan(C[:, N:]).all()


@pytest.mark.parametrize("M,N,K", [(3, 50, 700), (140, 200, 700), (1800, 1801, 300), (2100, 4000, 200), (6000, 2500, 100)])
def test_dq_product_large_tiles_and_types(M, N, K):
    """Each tile of the library, 16-bit outputs, alpha and beta: fp32 epilogue, half a step."""
    rng = np.random.default_rng(31)
    for ty in ("f16", "bf16"):
        B, b = stored(rng, K, N, "mxfp8", spread=1, whole=True)
        a = rng.integers(-4, 5, (K, M)).astype(np.float64)
        c0 = plain(rng, M, N, T[ty])
        base = np64(c0)
        if ty == "f16":
            A = torch.from_numpy(a).to(T[ty]).to(DEV)
            dg.gemm_dq(A, B, C=c0, transA=True, alpha=0.25, beta=2.0)
        else:
            A = torch.from_numpy(np.ascontiguousarray(a.T)).to(T[ty]).to(DEV)
            dg.gemm_dq(A, B, C=c0, alpha=0.25, beta=2.0)
        s = a.T @ b
        want = 0.25 * s + 2.0 * base
        tol = 3 * 2.0 ** -24 * (np.abs(0.25 * s) + np.abs(2 * base))
        assert (np.abs(np64(c0) - want) <= tol * 2 + HALF[T[ty]] * np.abs(want) + TINY[T[ty]]).all()


@pytest.mark.parametrize("transA", [False, True])
@pytest.mark.parametrize("splits", [1, 2, 3, 7, 0])
def test_dq_product_splits(splits, transA):
    rng = np.random.default_rng(32)
    for M, N, K in ((32, 260, 900), (64, 257, 1111), (5, 128, 64)):
        B, b = stored(rng, K, N, "mxint8", spread=1, whole=True)
        a = rng.integers(-8, 9, (M, K)).astype(np.float64)
        A = torch.from_numpy(np.ascontiguousarray(a.T) if transA else a).half().to(DEV)
        C = dg.gemm_dq(A, B, transA=transA, splits=splits, out_dtype=torch.float32)
        assert np.array_equal(np64(C), a @ b), (M, N, K)
    ws = torch.empty(dg.dg_gemm_splitk_workspace_size(5, 128, 2), dtype=torch.uint8, device=DEV)
    B, b = stored(rng, 640, 128, "mxint8", spread=1, whole=True)
    A = torch.ones((640, 5) if transA else (5, 640), dtype=torch.float16, device=DEV)
    C = dg.gemm_dq(A, B, transA=transA, splits=2, workspace=ws, out_dtype=torch.float32)
    assert np.array_equal(np64(C), np.tile(b.sum(0), (5, 1)))
    with pytest.raises(dg.MxError, match="workspace_bytes"):
        dg.gemm_dq(A, B, transA=transA, splits=3, workspace=ws)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("ty", ["f16", "bf16"])
def test_dq_product_normal_data(ty, fmt):
    """Every value of B is exact in A's type (B was rounded from it): K roundings
    of fp32 at most, each 2^-24 of the sum of magnitudes."""
    rng = np.random.default_rng(33)
    M, N, K = 140, 300, 777
    B = dg.quantize_mx(plain(rng, K, N, T[ty]), format=fmt)
    A = plain(rng, M, K, T[ty], pad=8)
    b = np64(dg.dequantize_mx(B))
    got = np64(dg.gemm_dq(A, B, out_dtype=torch.float32))
    assert (np.abs(got - np64(A) @ b) <= K * 2.0 ** -24 * (np.abs(np64(A)) @ np.abs(b))).all()
    b2 = B.s.clone()
    B.s[0, 5, 2] = 255                                   # NaN in columns 64 .. 95 of every row of C
    c = np64(dg.gemm_dq(A, B, out_dtype=torch.float32))
    assert np.isnan(c[:, 64:96]).all() and np.array_equal(np.delete(c, range(64, 96), 1), np.delete(got, range(64, 96), 1))
    B.s.copy_(b2)
    c0 = plain(rng, M, N, T[ty])
    want = (c0.double() * 0.5).to(T[ty])                 # one rounding (of halved subnormals)
    dg.gemm_dq(A, B, C=c0, alpha=0.0, beta=0.5)
    assert torch.equal(c0, want)
    none = dg.MxMatrix.empty(fmt, 0, N, DEV)
    assert not np64(dg.gemm_dq(torch.empty(M, 0, dtype=T[ty], device=DEV), none)).any()


# ---- activations ----------------------------------------------------------------------
def slope64(z, act):
    if act == "relu":
        return (z > 0).astype(np.float64)
    cdf = 0.5 * erfc(-z / math.sqrt(2))
    return cdf + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)


ACT_SHAPES = [(1, 1), (3, 33), (4, 512), (5, 513), (70, 300), (257, 1030)]


@pytest.mark.parametrize("act", ["relu", "gelu"])
@pytest.mark.parametrize("fmt", ["mxfp8", "mxint8"])
@pytest.mark.parametrize("ty", list(T))
def test_act_checkpoint(ty, fmt, act):
    rng = np.random.default_rng(40)
    for rows, cols in ACT_SHAPES:
        for pz, ph in ((0, 0), (1, 0), (0, 3), (8, 8)):
            z = plain(rng, rows, cols, T[ty], pz, std=2.0)
            h = torch.full((rows, cols + ph), math.nan, dtype=T[ty], device=DEV)
            _, m = dg.act_checkpoint(z, act, H=h[:, :cols], format=fmt)
            x = np64(z)
            wq, ws = rounded(x, fmt)
            assert np.array_equal(m.q.cpu().numpy(), wq) and np.array_equal(m.s.cpu().numpy(), ws), (rows, cols)
            want = act64(x, act)
            tol = 1e-6 * np.abs(x) * (act == "gelu") + HALF[T[ty]] * np.abs(want) + TINY[T[ty]]
            assert (np.abs(np64(h[:, :cols]) - want) <= tol).all(), (rows, cols)
            assert torch.isnan(h[:, cols:]).all()
    z = plain(rng, 9, 100, T[ty])                        # in place
    want_h, want_m = dg.act_checkpoint(z, act, format=fmt)
    _, m = dg.act_checkpoint(z, act, H=z, format=fmt)
    assert torch.equal(z, want_h) and torch.equal(m.q, want_m.q) and torch.equal(m.s, want_m.s)


@pytest.mark.parametrize("act", ["relu", "gelu"])
@pytest.mark.parametrize("fmt", ["mxfp8", "mxint8"])
@pytest.mark.parametrize("ty", list(T))
def test_act_backward(ty, fmt, act):
    """dZ: the slope is off by at most 2e-6 (the erfc approximation's 1.5e-7, the
    exponential's and the reciprocal's few units), then half a step.  dbias: the
    same per element and one fp32 rounding of the sum of magnitudes per row."""
    rng = np.random.default_rng(41)
    for rows, cols in ACT_SHAPES + [(3000, 40)]:
        m, z = stored(rng, rows, cols, fmt, extra=16, lds=rows + 1, spread=2)
        if fmt == "mxfp8":
            m.s.sub_(6)                                  # values of about 100 down to about 1.6
            z = z * 2.0 ** -6
        for ph, pz in ((0, 0), (1, 0), (0, 3)):
            d = plain(rng, rows, cols, T[ty], ph)
            dz = torch.full((rows, cols + pz), math.nan, dtype=T[ty], device=DEV)
            db = torch.full((cols,), math.nan, device=DEV)
            dg.act_backward(d, m, act, dZ=dz[:, :cols], dbias=db)
            want = np64(d) * slope64(z, act)
            err = 2e-6 * np.abs(np64(d)) * (act == "gelu")
            tol = err + HALF[T[ty]] * np.abs(want) + TINY[T[ty]]
            assert (np.abs(np64(dz[:, :cols]) - want) <= tol).all(), (rows, cols)
            assert torch.isnan(dz[:, cols:]).all()
            tol = err.sum(0) + (rows + 1) * 2.0 ** -24 * np.abs(want).sum(0) + 1e-30
            assert (np.abs(np64(db) - want.sum(0)) <= tol).all(), (rows, cols)
            other = dg.act_backward(d, m, act)
            assert torch.equal(other, dz[:, :cols])      # without the sums
            again = torch.empty(cols, device=DEV)
            dg.act_backward(d, m, act, dZ=other, dbias=again)
            assert torch.equal(again, db)                # in the same order
    d = plain(rng, 9, 100, T[ty])
    m, _ = stored(rng, 9, 100, fmt)
    want = dg.act_backward(d, m, act)
    assert torch.equal(dg.act_backward(d, m, act, dZ=d), want) and torch.equal(d, want)       # in place
    db = torch.full((7,), math.nan, device=DEV)          # no rows: the sums are zero
    dg.act_backward(torch.empty(0, 7, device=DEV), dg.MxMatrix.empty(fmt, 0, 7, DEV), act, dbias=db)
    assert not db.any()


def test_gelu_gradient_by_differences():
    """gelu'(z) of the kernel against central differences of gelu in fp64 (step
    1e-5: the difference quotient is off by less than 1e-9)."""
    z = torch.linspace(-9, 9, 4096).view(4, 1024)
    z[0, :6] = torch.tensor([0.0, 100.0, -100.0, 14.0, -14.0, 1e-30])
    m = dg.quantize_mx(z.to(DEV), format="mxint8")
    v = np64(dg.dequantize_mx(m))
    got = np64(dg.act_backward(torch.ones(4, 1024, device=DEV), m, "gelu"))
    step = 1e-5
    diff = (act64(v + step, "gelu") - act64(v - step, "gelu")) / (2 * step)
    assert (np.abs(got - diff) <= 2e-6 + 1e-9 * np.abs(v)).all()


def test_act_special_values():
    """A NaN block gives NaN, its neighbours keep their values; huge values of z
    have slope 1 and 0; relu's slope at zero of either sign is 0."""
    z = torch.zeros(2, 96, device=DEV)
    z[0, 3] = math.inf
    z[0, 32:64] = 1e30
    z[0, 64:] = -1e30
    z[1, 32:64] = -0.0
    z[1, 64:] = 2.0
    ones = torch.ones(2, 96, device=DEV)
    for fmt in ("mxfp8", "mxint8"):
        m = dg.quantize_mx(z, format=fmt)
        for act, at2 in (("relu", 1.0), ("gelu", float(slope64(np.array([2.0]), "gelu")[0]))):
            got = np64(dg.act_backward(ones, m, act))
            assert np.isnan(got[0, :32]).all()
            assert (got[0, 32:64] == 1).all() and (got[0, 64:] == 0).all()
            assert (np.abs(got[1, :64] - (0.5 if act == "gelu" else 0)) <= 2e-6).all() and np.allclose(got[1, 64:], at2, atol=2e-6)
        h, _ = dg.act_checkpoint(z, "relu", format=fmt)
        assert torch.equal(h[0, 32:], z[0, 32:].clamp(min=0)) and h[0, 3] == math.inf


# ---- as a program uses them ---------------------------------------------------------
def _mlp(x, w1, w2, dy, bias):
    """Forward and backward of y = gelu(x W1^T + bias) W2^T with W1, W2 kept in
    mxfp4 and the two saved inputs in 8 bits; returns every gradient."""
    m, f = x.shape[0], w1.rows
    a = dg.quantize_mx(x, format="mxfp8")
    z = dg.gemm_mx(a, w1, bias=bias, out_dtype=x.dtype)
    h, kept = dg.act_checkpoint(z, "gelu", format="mxint8")
    h8 = dg.quantize_mx(h, format="mxfp8")
    y = dg.gemm_mx(h8, w2, out_dtype=x.dtype)
    dw2 = dg.gemm_dq(dy, h8, transA=True, out_dtype=torch.float32)
    dh = dg.gemm_dq(dy, w2)
    db = torch.empty(f, device=x.device)
    dz = dg.act_backward(dh, kept, "gelu", dbias=db)
    dw1 = dg.gemm_dq(dz, a, transA=True, out_dtype=torch.float32)
    dx = dg.gemm_dq(dz, w1)
    return {"z": z, "h": h, "y": y, "dw2": dw2, "dh": dh, "dz": dz, "db": db, "dw1": dw1, "dx": dx,
            "a": dg.dequantize_mx(a), "kept": dg.dequantize_mx(kept), "h8": dg.dequantize_mx(h8)}


def _mlp_inputs(rng, m, d, f, ty):
    x, dy = plain(rng, m, d, T[ty]), plain(rng, m, d, T[ty], std=0.1)
    w1 = dg.quantize_mx(plain(rng, f, d, T[ty], std=0.1), format="mxfp4")
    w2 = dg.quantize_mx(plain(rng, d, f, T[ty], std=0.1), format="mxfp4")
    return x, w1, w2, dy, plain(rng, 1, f, T[ty])[0]


@pytest.mark.parametrize("ty", ["f16", "bf16"])
def test_mlp_forward_and_backward(ty):
    """Every step against fp64 on that step's own inputs: sums of n products are
    off by n 2^-24 of the magnitudes (plus 2^-13 of the largest product of a
    step, per product, with an mxfp8 operand), then half a step of the type."""
    rng = np.random.default_rng(50)
    x, w1, w2, dy, bias = _mlp_inputs(rng, 70, 300, 520, ty)
    r = {k: np64(v) for k, v in _mlp(x, w1, w2, dy, bias).items()}
    v1, v2 = np64(dg.dequantize_mx(w1)), np64(dg.dequantize_mx(w2))
    half, tiny = HALF[T[ty]], TINY[T[ty]]

    def near(got, p, q, extra=0.0, out_half=half, add=0.0):
        want, mag = p @ q + add, np.abs(p) @ np.abs(q)
        big = np.abs(p).max(1)[:, None] * np.abs(q).max(0)[None, :]
        n = p.shape[1]
        tol = n * 2.0 ** -24 * (mag + np.abs(add)) + extra * n * big
        assert (np.abs(got - want) <= tol * (1 + out_half) + out_half * np.abs(want) + tiny).all()

    assert np.array_equal(r["a"], mx_ref.values(*rounded(np64(x), "mxfp8"), "mxfp8", 300))
    near(r["z"], r["a"], v1.T, 2.0 ** -13, add=np64(bias))
    assert np.array_equal(r["kept"], mx_ref.values(*rounded(r["z"], "mxint8"), "mxint8", 520))
    assert np.array_equal(r["h8"], mx_ref.values(*rounded(r["h"], "mxfp8"), "mxfp8", 520))
    near(r["y"], r["h8"], v2.T, 2.0 ** -13)
    near(r["dw2"], np64(dy).T, r["h8"], out_half=0.0)
    near(r["dh"], np64(dy), v2)
    want = r["dh"] * slope64(r["kept"], "gelu")
    assert (np.abs(r["dz"] - want) <= 2e-6 * np.abs(r["dh"]) + half * np.abs(want) + tiny).all()
    near(r["dw1"], r["dz"].T, r["a"], out_half=0.0)
    near(r["dx"], r["dz"], v1)


def test_streams():
    """A side stream of the caller's, and two streams at once."""
    rng = np.random.default_rng(51)
    args = [_mlp_inputs(rng, 64, 256, 512, "bf16") for _ in range(2)]
    want = [_mlp(*a) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in args]
    for _ in range(3):
        got = []
        for s, a in zip(streams, args):
            with torch.cuda.stream(s):
                got.append(_mlp(*a))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(g[k], w[k]) for k in w)
    s = streams[0]
    x, w1, w2, dy, bias = args[0]
    s.wait_stream(torch.cuda.current_stream())
    m = dg.quantize_mx(x, format="mxfp8", stream=s)
    z = dg.gemm_mx(m, w1, bias=bias, stream=s)
    h, kept = dg.act_checkpoint(z, "gelu", stream=s)
    db = torch.empty(512, device=DEV)
    dz = dg.act_backward(want[0]["dh"], kept, "gelu", dbias=db, stream=s)
    dw = dg.gemm_dq(dz, m, transA=True, out_dtype=torch.float32, splits=2, stream=s)
    v = dg.dequantize_mx(m, stream=s)
    s.synchronize()
    assert torch.equal(z, want[0]["z"]) and torch.equal(h, want[0]["h"]) and torch.equal(dz, want[0]["dz"])
    assert torch.equal(db, want[0]["db"]) and torch.equal(v, want[0]["a"])
    assert torch.allclose(dw, want[0]["dw1"], rtol=1e-4, atol=1e-4)


def test_captured_graphs():
    """The chain captured once and replayed on new inputs, with eager work in
    between, equals the eager chain; two graphs with workspaces of their own."""
    rng = np.random.default_rng(52)
    sets = [_mlp_inputs(rng, 40, 256, 512, "f16") for _ in range(3)]
    held = [[t.clone() if isinstance(t, torch.Tensor) else t for t in sets[0]] for _ in range(2)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _mlp(*held[0])
    torch.cuda.current_stream().wait_stream(s)
    graphs, outs = [], []
    for h in held:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_mlp(*h))
        graphs.append(g)
    for k in (1, 2, 0, 1):
        x, w1, w2, dy, bias = sets[k]
        want = _mlp(held[0][0].copy_(x), held[0][1], held[0][2], held[0][3].copy_(dy), held[0][4])
        want = {n: t.clone() for n, t in want.items()}
        held[1][0].copy_(x), held[1][3].copy_(dy)
        for g, o in zip(graphs, outs):
            g.replay()
        torch.cuda.synchronize()
        for o in outs:
            assert all(torch.equal(o[n], want[n]) for n in want), k


def test_no_allocation_and_guard():
    """With its outputs and workspace given, a call allocates nothing; tensors of
    another device are refused."""
    rng = np.random.default_rng(53)
    x = plain(rng, 32, 700, torch.float16)
    m = dg.MxMatrix.empty("mxfp8", 32, 700, DEV)
    w, _ = stored(rng, 65, 700, "mxfp4")
    c = torch.empty(32, 65, dtype=torch.float16, device=DEV)
    out = torch.empty(32, 700, device=DEV)
    ws = torch.empty(dg.dg_gemm_splitk_workspace_size(65, 700, 2) + dg.dg_act_backward_workspace_size(32, 700), dtype=torch.uint8, device=DEV)
    dw = torch.empty(65, 700, device=DEV)
    h, dz, db = torch.empty_like(x), torch.empty_like(x), torch.empty(700, device=DEV)
    before = torch.cuda.memory_stats()["allocation.all.allocated"]
    dg.quantize_mx(x, out=m)
    dg.dequantize_mx(m, out=out)
    dg.gemm_mx(m, w, C=c)
    dg.gemm_dq(c, m, C=dw, transA=True, splits=2, workspace=ws)
    dg.act_checkpoint(x, "gelu", H=h, out=m)
    dg.act_backward(x, m, "gelu", dZ=dz, dbias=db, workspace=ws)
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == before
    with pytest.raises(ValueError):
        dg.gemm_mx(m, w, C=torch.empty(32, 65, dtype=torch.float16))


def test_long_rows_and_many_rows():
    """Offsets past 32 bits: a stored matrix of more than 4 GiB, rounded, read
    back in places, and multiplied through its last rows."""
    rows, cols = 9000, 500_000
    free, _ = torch.cuda.mem_get_info()
    if free < 40 << 30:
        pytest.skip("needs 40 GiB of free GPU memory")
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV)
    for i in range(0, rows, 1000):
        x[i:i + 1000] = torch.randn(1000, cols, generator=g, device=DEV).to(torch.bfloat16)
    m = dg.quantize_mx(x, format="mxfp8")
    assert m.q.numel() > 1 << 32
    for r in (0, 4321, rows - 1):
        wq, ws = rounded(np64(x[r:r + 1]), "mxfp8")
        assert np.array_equal(m.q[r:r + 1].cpu().numpy(), wq) and np.array_equal(m.s[:, r:r + 1].cpu().numpy(), ws)
    h = dg.dequantize_mx(m, dtype=torch.bfloat16)
    assert torch.equal(h[-1:], dg.dequantize_mx(dg.MxMatrix("mxfp8", 1, cols, m.q[-1:], m.s[:, -1:]), dtype=torch.bfloat16))
    # columns of the last group against all rows: sum over 9000 rows of A^T
    tail = dg.MxMatrix("mxfp8", rows, cols % 256, m.q[:, cols // 256 * 256:], m.s[-1:])
    A = torch.zeros(2, rows, dtype=torch.bfloat16, device=DEV)
    A[0, -1], A[1, 0] = 1, 1
    got = dg.gemm_dq(A, tail, out_dtype=torch.float32)
    assert torch.equal(got, torch.stack([h[-1, cols // 256 * 256:], h[0, cols // 256 * 256:]]).float())


@pytest.mark.parametrize("rows,cols", [(8, 9), (33, 8), (511, 5631), (4096 * 8 + 5, 24), (131072 + 37, 8)])
def test_backward_bands_and_slices(rows, cols):
    # a band short of its eight waves, 16- and 32-row bands, more bands than slices
    g = torch.Generator(device="cuda").manual_seed(rows + cols)
    z = torch.randn(rows, cols, generator=g, device="cuda")
    d = torch.randn(rows, cols, generator=g, device="cuda").to(torch.bfloat16)
    m = dg.quantize_mx(z, format="mxfp8")
    db = torch.empty(cols, device="cuda")
    out = dg.act_backward(d, m, "relu", dbias=db)
    want = torch.where(dg.dequantize_mx(m, dtype=torch.float32) > 0, d.double(), 0.0)
    assert torch.equal(out.double(), want)
    assert torch.equal(dg.act_backward(d, m, "relu"), out)
    # fp32 sums: below one rounding per row added
    bound = rows * 2.0 ** -24 * want.abs().sum(0)
    assert ((db.double() - want.sum(0)).abs() <= bound + 1e-30).all()


@pytest.mark.parametrize("ty", list(T))
@pytest.mark.parametrize("kernel", range(len(dg.mx_kernel_names())))
def test_product_keeps_small_beside_large(kernel, ty):
    """Each row of A holds one group of 8 neighbouring k with elements from 2^-9
    to 2^7, in every other row with two of 128 that cancel.  Sums are multiples of
    2^-10 below 8 * 128 * 6 < 2^13, so an fp32 sum is exact in any order: an fp32
    C and the row kernels keep all of it.  The tiled kernels with a 16-bit C cut
    each product to 2^-13 of the group's largest, 8 of them at most."""
    rng = np.random.default_rng(24)
    codes = np.flatnonzero(np.isfinite(mx_ref.FP8) & (np.abs(mx_ref.FP8) <= 128))
    for M, N, K in ((1, 40, 2048), (5, 17, 64), (33, 65, 300), (130, 270, 1030)):
        ca = np.zeros((M, mx_ref.groups(K) * 256), np.int64)
        for m in range(M):
            at = 8 * rng.integers(0, K // 8)
            ca[m, at:at + 8] = codes[rng.integers(0, len(codes), 8)]
            if m % 2 == 0:
                ca[m, at:at + 2] = np.flatnonzero(mx_ref.FP8 == 128)[0], np.flatnonzero(mx_ref.FP8 == -128)[0]
        cb = rng.integers(0, 16, (N, mx_ref.groups(K) * 256))
        cb[:, 1::2] = cb[:, ::2]
        cb[:, K:] = 0
        qa, qb = mx_ref.pack(ca, "mxfp8"), mx_ref.pack(cb, "mxfp4")
        sa, sb = (np.full((mx_ref.groups(K), n, 8), 127, np.uint8) for n in (M, N))
        a, b = mx_ref.values(qa, sa, "mxfp8", K), mx_ref.values(qb, sb, "mxfp4", K)
        A = dg.MxMatrix("mxfp8", M, K, torch.from_numpy(qa).to(DEV), torch.from_numpy(sa).to(DEV))
        B = dg.MxMatrix("mxfp4", N, K, torch.from_numpy(qb).to(DEV), torch.from_numpy(sb).to(DEV))
        got = dg.gemm_mx(A, B, out_dtype=T[ty], kernel=kernel)
        want = a @ b.T
        if ty == "f32" or dg.mx_kernel_names()[kernel].endswith("_rows"):
            assert torch.equal(got.cpu(), torch.from_numpy(want).to(T[ty])), (M, N, K)
        else:
            cut = 8 * 2.0 ** -13 * np.stack([(np.abs(r) * np.abs(b)).max(1) for r in a])
            assert (np.abs(np64(got) - want) <= cut * (1 + HALF[T[ty]]) + HALF[T[ty]] * np.abs(want) + TINY[T[ty]]).all(), (M, N, K)


@pytest.mark.parametrize("ty", list(T))
def test_relu_gradient_of_infinities(ty):
    """An overflowed gradient at a unit that relu switched off does not reach dZ
    or the bias gradient; at one that is on it does; a NaN z gives NaN."""
    z = torch.tensor([[-1.0, 0.0, -0.0, 2.0], [-3.0, -1e-30, 1.0, 2.0]], device=DEV).repeat(1, 8)
    d = torch.tensor([[math.inf, -math.inf, math.nan, 1.0], [math.nan, math.inf, -math.inf, math.nan]], device=DEV, dtype=T[ty]).repeat(1, 8)
    for fmt in ("mxfp8", "mxint8"):
        m = dg.quantize_mx(z, format=fmt)
        db = torch.empty(32, device=DEV)
        got = np64(dg.act_backward(d, m, "relu", dbias=db))
        want = np.tile([[0, 0, 0, 1], [0, 0, -math.inf, math.nan]], 8)
        assert np.array_equal(got, want, equal_nan=True)
        assert np.array_equal(np64(db), want.sum(0), equal_nan=True)
        m.s[0, 0, 0] = 255
        got = np64(dg.act_backward(d, m, "relu"))
        assert np.isnan(got[0]).all() and np.array_equal(got[1], want[1], equal_nan=True)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxint8"])
@pytest.mark.parametrize("ty", list(T))
def test_relu_mask_is_kept(ty, fmt):
    """keep_positive: the slope that act_backward finds is that of Z itself, down
    to the type's least positive value beside its block's largest; only codes of
    zero change, to 1; H, the scales and in-place use are as without."""
    rng = np.random.default_rng(42)
    for rows, cols, pad in ((1, 1, 0), (5, 33, 1), (70, 300, 0), (257, 1030, 3)):
        x = rng.standard_normal((rows, cols)) * 10.0 ** rng.uniform(-6, 2, (rows, cols))
        x[::2, ::5] = float(torch.finfo(T[ty]).smallest_normal * torch.finfo(T[ty]).eps)
        x[::3, ::7] = 0.0
        x[1::3, 3::7] = -0.0
        x[rows // 2:, ::64] = 500.0
        z = plain(rng, rows, cols, T[ty], pad)
        z.copy_(torch.from_numpy(x).to(T[ty]))
        h0, m0 = dg.act_checkpoint(z, "relu", format=fmt)
        h, m = dg.act_checkpoint(z, "relu", format=fmt, keep_positive=True)
        assert torch.equal(h, h0) and torch.equal(m.s, m0.s)
        q0, q, v = m0.q[:, :cols], m.q[:, :cols], z.float()
        assert torch.equal(q, torch.where((v > 0) & (q0 == 0), torch.ones_like(q0), q0)), (rows, cols)
        assert not m.q[:, cols:].any()
        d = torch.ones(rows, cols, dtype=T[ty], device=DEV)
        assert torch.equal(dg.act_backward(d, m, "relu"), (v > 0).to(T[ty])), (rows, cols)
        _, mi = dg.act_checkpoint(z, "relu", H=z, out=m0, keep_positive=True)
        assert torch.equal(z, h) and torch.equal(mi.q, m.q) and torch.equal(mi.s, m.s)
    z = torch.randn(4, 64, device=DEV, dtype=T[ty])      # a NaN block stays one
    z[2, 40] = math.nan
    _, m = dg.act_checkpoint(z, "relu", format=fmt, keep_positive=True)
    assert m.s[0, 2, 1] == 255 and not m.q[2, 32:64].any()


@pytest.mark.parametrize("transA", [False, True])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("ty", ["f16", "bf16"])
@pytest.mark.parametrize("kernel", range(len(dg.dq_kernel_names())))
def test_dq_product_exact_on_every_tile(kernel, ty, fmt, transA):
    """Every tile with sums that are exact in fp32 (as in test_dq_product_exact):
    five and more slabs of 64 k in each K range, whole and ragged ends of M, N and
    K, A by direct loads and (not on the 256 x 256 tile) through registers, one K
    range and three."""
    rng = np.random.default_rng(34)
    for M, N, K, pads in ((304, 391, 1000, (0, 1)), (512, 256, 960, (2, 3)), (37, 545, 1985, (0,)), (8, 130, 1088, (8, 1))):
        B, b = stored(rng, K, N, fmt, extra=16, lds=K + 1, spread=1, whole=True)
        a = rng.integers(-8, 9, (M, K)).astype(np.float64)
        want = a @ b
        stored_a = torch.from_numpy(np.ascontiguousarray(a.T) if transA else a).to(T[ty])
        r, c = stored_a.shape
        for pad in pads:
            A = torch.full((r, c + pad), math.nan, dtype=T[ty])
            A[:, :c] = stored_a
            A = A.to(DEV)[:, :c]
            direct = (c + pad) % 2 == 0 and (not transA or M % 8 == 0)
            for splits in (1, 3):
                C = torch.full((M + 1, N + 1), math.nan, device=DEV)
                if kernel == 3 and not direct:
                    with pytest.raises(dg.MxError, match="support"):
                        dg.gemm_dq(A, B, C=C[:M, :N], transA=transA, splits=splits, kernel=kernel)
                    continue
                dg.gemm_dq(A, B, C=C[:M, :N], transA=transA, splits=splits, kernel=kernel)
                assert np.array_equal(np64(C[:M, :N]), want), (M, N, K, pad, splits)
                assert torch.isnan(C[M:]).all() and torch.isnan(C[:, N:]).all()


@pytest.mark.parametrize("ty", ["f16", "bf16"])
@pytest.mark.parametrize("kernel", range(len(dg.dq_kernel_names())))
def test_dq_product_epilogue_on_every_tile(kernel, ty):
    """alpha, beta and 16-bit and fp32 outputs with even and odd row strides, in
    one K range and joined from three: two fp32 operations, then half a step."""
    rng = np.random.default_rng(35)
    for M, N, K in ((300, 389, 704), (257, 640, 385)):
        B, b = stored(rng, K, N, "mxfp4", spread=1, whole=True)
        a = rng.integers(-4, 5, (M, K)).astype(np.float64)
        A = torch.from_numpy(a).to(T[ty])
        A = torch.cat([A, A[:, :K % 2]], 1).to(DEV)[:, :K]
        s = a @ b
        for to in (ty, "f32"):
            for pad in (0, 1):
                for splits in (1, 3):
                    c0 = plain(rng, M, N, T[to], pad)
                    base, full = np64(c0), c0.as_strided((M, N + pad), (N + pad, 1))
                    dg.gemm_dq(A, B, C=c0, alpha=0.375, beta=-1.5, splits=splits, kernel=kernel)
                    want = 0.375 * s - 1.5 * base
                    tol = 2 * 2.0 ** -24 * (np.abs(0.375 * s) + np.abs(1.5 * base))
                    tol = tol * (1 + HALF[T[to]]) + (HALF[T[to]] if to != "f32" else 0) * np.abs(want) + TINY[T[to]]
                    assert (np.abs(np64(c0) - want) <= tol).all(), (M, N, to, pad, splits)
                    if pad:
                        assert torch.isnan(full[:, N:]).all()


@pytest.mark.parametrize("ty", list(T))
@pytest.mark.parametrize("fa", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("kernel", range(len(dg.mx_kernel_names())))
def test_product_epilogue_on_every_kernel(kernel, fa, ty):
    """bias, activation, alpha and beta with even and odd row strides of C on each
    kernel, on exact sums; the bound is test_product_epilogue's."""
    rng = np.random.default_rng(25)
    for M, N, K in ((5, 50, 256), (150, 389, 520), (257, 264, 300)):
        A, a = stored(rng, M, K, fa, spread=1, whole=True)
        B, b = stored(rng, N, K, "mxfp4", spread=1, whole=True)
        s = a @ b.T
        alpha, beta = 1.0 / 64, -0.5
        for act in ("none", "relu", "gelu"):
            for pad in (0, 1, 2):
                c0 = plain(rng, M, N, T[ty], pad)
                bias = plain(rng, 1, N, T[ty])[0]
                base = np64(c0)
                full = c0.as_strided((M, N + pad), (N + pad, 1))
                dg.gemm_mx(A, B, C=c0, alpha=alpha, beta=beta, bias=bias, activation=act, kernel=kernel)
                pre = alpha * s + beta * base + np64(bias)
                mag = np.abs(alpha * s) + np.abs(beta * base) + np.abs(np64(bias))
                want = act64(pre, act)
                tol = 1.13 * 4 * 2.0 ** -24 * mag + (1e-6 * np.abs(pre) if act == "gelu" else 0)
                tol = tol * (1 + HALF[T[ty]]) + HALF[T[ty]] * np.abs(want) + TINY[T[ty]]
                assert (np.abs(np64(c0) - want) <= tol).all(), (M, N, act, pad)
                if pad:
                    assert torch.isnan(full[:, N:]).all()


def test_ranges_joined_over_many_rows():
    """The join of two K ranges over more rows than its launch holds workgroups of
    256 threads (2^24 of one row each): equal to the product in one range, whose
    sums are exact too."""
    M, N, K = (1 << 24) + 3, 516, 128
    if torch.cuda.mem_get_info()[0] < 150 << 30:
        pytest.skip("needs 150 GiB of free GPU memory")
    rng = np.random.default_rng(36)
    B, b = stored(rng, K, N, "mxfp4", spread=1, whole=True)
    g = torch.Generator(device=DEV).manual_seed(36)
    A = torch.randint(-4, 5, (M, K), generator=g, device=DEV, dtype=torch.int8).to(torch.float16)
    one = dg.gemm_dq(A, B, splits=1)
    two = dg.gemm_dq(A, B, C=torch.full_like(one, math.nan), splits=2)
    for i in range(0, M, 1 << 22):
        assert torch.equal(one[i:i + (1 << 22)], two[i:i + (1 << 22)]), i
    for r in (0, (1 << 23) - 1, 1 << 23, (1 << 24) - 1, M - 1):
        want = torch.from_numpy(np64(A[r:r + 1]) @ b).to(torch.float16)
        assert torch.equal(two[r:r + 1].cpu(), want), r
    del A, one, two
    torch.cuda.empty_cache()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("ty", ["f16", "bf16"])
def test_dq_operand_values_under_every_scale(ty, fmt):
    """One k and one block per scale byte, 2^-127 to 2^127: the product by 1 is B's
    value rounded once to A's type (subnormals included, infinite past its range)."""
    rng = np.random.default_rng(37)
    n = 255 * 32
    for kernel in range(len(dg.dq_kernel_names())):
        q, s = mx_ref.random_stored(rng, 1, n, fmt)
        s.reshape(-1)[:255] = np.arange(255)
        B = dg.MxMatrix(fmt, 1, n, torch.from_numpy(q).to(DEV), torch.from_numpy(s).to(DEV))
        A = torch.ones(8, 1, dtype=T[ty], device=DEV)
        A = torch.cat([A, A], 1)[:, :1]
        got = dg.gemm_dq(A, B, out_dtype=torch.float32, kernel=kernel)
        want = torch.from_numpy(mx_ref.values(q, s, fmt, n)).to(T[ty]).float()
        assert torch.equal(got.cpu(), want.expand(8, n)), kernel


def test_captured_exact_product_and_mask():
    """An fp32 C of an mxfp8 A (rows and tiles), relu with keep_positive and its
    backward, captured once and replayed on other inputs with eager work between."""
    rng = np.random.default_rng(55)
    w, _ = stored(rng, 200, 512, "mxfp4")

    def chain(x, d):
        a = dg.quantize_mx(x, format="mxfp8")
        z = dg.gemm_mx(a, w, out_dtype=torch.float32)
        one = dg.gemm_mx(dg.quantize_mx(x[:1], format="mxfp8"), w)
        h, kept = dg.act_checkpoint(z, "relu", keep_positive=True)
        db = torch.empty(200, device=DEV)
        dz = dg.act_backward(d, kept, "relu", dbias=db)
        return [z, one, h, dz, db, dg.gemm_dq(dz.to(torch.bfloat16), w, splits=2)]

    sets = [(plain(rng, 150, 512, torch.bfloat16), plain(rng, 150, 200, torch.float32)) for _ in range(3)]
    x, d = (t.clone() for t in sets[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        chain(x, d)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = chain(x, d)
    for k in (1, 2, 0, 1):
        want = [t.clone() for t in chain(*sets[k])]
        assert torch.equal(want[3], torch.where(want[0] > 0, sets[k][1], 0.0))
        x.copy_(sets[k][0]), d.copy_(sets[k][1])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), k


@pytest.mark.parametrize("ty", list(T))
@pytest.mark.parametrize("kernel", range(len(dg.mx_kernel_names())))
def test_product_bound_with_outlier_blocks(kernel, ty):
    """Full-range mxfp8 elements under block scales 2^-6 to 2^6, every other row
    with neighbours that cancel.  Each product of 8 neighbouring k is cut by less
    than 2^-13 of the largest among them (tiled kernels with a 16-bit C; else not at
    all); then at most one fp32 rounding per k, of a partial sum no larger than the
    sum of magnitudes; then half a step of C."""
    rng = np.random.default_rng(26)
    codes = np.flatnonzero(np.isfinite(mx_ref.FP8))
    for M, N, K in ((7, 33, 512), (131, 140, 520)):
        G = mx_ref.groups(K)
        ca = codes[rng.integers(0, len(codes), (M, G * 256))]
        ca[::2, 1::2] = ca[::2, ::2] ^ 0x80
        cb = rng.integers(0, 16, (N, G * 256))
        cb[:, 1::2] = cb[:, ::2]
        ca[:, K:], cb[:, K:] = 0, 0
        qa, qb = mx_ref.pack(ca, "mxfp8"), mx_ref.pack(cb, "mxfp4")
        sa, sb = (rng.integers(121, 134, (G, n, 8)).astype(np.uint8) for n in (M, N))
        a, b = mx_ref.values(qa, sa, "mxfp8", K), mx_ref.values(qb, sb, "mxfp4", K)
        A = dg.MxMatrix("mxfp8", M, K, torch.from_numpy(qa).to(DEV), torch.from_numpy(sa).to(DEV))
        B = dg.MxMatrix("mxfp4", N, K, torch.from_numpy(qb).to(DEV), torch.from_numpy(sb).to(DEV))
        got = np64(dg.gemm_mx(A, B, out_dtype=T[ty], kernel=kernel))
        want, mag = a @ b.T, np.abs(a) @ np.abs(b).T
        assert not want[::2].any() and want[1::2].any()
        tol = K * 2.0 ** -24 * mag
        if ty != "f32" and dg.mx_kernel_names()[kernel].endswith("_tile"):
            for k in range(0, K, 8):
                tol += 8 * 2.0 ** -13 * (np.abs(a[:, None, k:k + 8]) * np.abs(b[None, :, k:k + 8])).max(2)
        big = torch.finfo(T[ty]).max
        fits = np.abs(want) + tol < big
        tol = tol * (1 + HALF[T[ty]]) + HALF[T[ty]] * np.abs(want) + TINY[T[ty]]
        assert fits.mean() > 0.4 and (np.abs(got - want) <= tol)[fits].all(), (M, N, K)
