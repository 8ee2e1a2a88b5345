"""A layer's products on an MI355X, against their formulas in 64 bits (layer_ref):
every type, orientation and kernel at the sizes where tiles, slabs and pieces
end; groups of every size, none among them; special values; the calls as a
program makes them (views, streams, graphs, a whole expert layer)."""
import math

import numpy as np
import pytest
import torch

import dense_gemm_amd as dg
import layer_ref
from layer_ref import T, check, np64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
PAIRS = [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("f16", "f32"), ("bf16", "f32")]
KERNELS = list(range(len(dg.layer_kernel_names())))
SENTINEL = -77.0


def matrix(rng, rows, cols, dtype, pad=0, std=1.0, shift=0):
    """A random matrix on the GPU with `pad` NaN columns behind its rows, its first
    element `shift` elements into its memory."""
    x = torch.full((rows, cols + pad), math.nan, dtype=dtype)
    x[:, :cols] = torch.from_numpy(rng.standard_normal((rows, cols)) * std).to(dtype)
    if shift:
        whole = torch.full((rows * (cols + pad) + shift,), math.nan, dtype=dtype, device=DEV)
        whole[shift:] = x.flatten().to(DEV)
        return whole[shift:].view(rows, cols + pad)[:, :cols]
    return x.to(DEV)[:, :cols]


def output(rows, cols, dtype, pad=0):
    return torch.full((rows, cols + pad), SENTINEL, dtype=dtype, device=DEV)[:, :cols]


def padding_kept(*views):
    for v in views:
        if v is not None and v._base is not None:
            whole = v._base if v._base.dim() == 2 else v._base.view(-1, v._base.shape[-1])
            assert (whole[:, v.shape[-1]:] == SENTINEL).all(), "padding written"


def runs(kernel, call):
    """call(), or None where the forced kernel does not take the problem."""
    try:
        return call()
    except dg.LayerError as e:
        if kernel != dg.DG_KERNEL_AUTO and e.status == dg.DG_ERR_UNSUPPORTED:
            return None
        raise


def fused_case(seed, M, N, K, ty, out, transB, activation="none", bias=False, res=False, keep=False, pad=0, shift=0, alpha=1.0,
               beta=1.0, offsets=None, kernel=-1, splits=1):
    rng = np.random.default_rng(seed)
    t, o = T[ty], T[out]
    G = None if offsets is None else len(offsets) - 1
    A = matrix(rng, M, K, t, pad, shift=shift)
    wr, wc = (N, K) if transB else (K, N)
    W = matrix(rng, (G or 1) * wr, wc, t, pad, std=1 / math.sqrt(max(K, 1)), shift=shift)
    B = W if G is None else W.as_strided((G, wr, wc), (wr * W.stride(0), W.stride(0), 1), W.storage_offset())
    b = matrix(rng, G or 1, N, o, pad) if bias else None
    R = matrix(rng, M, N, o, pad) if res else None
    C, Z = output(M, N, o, pad), output(M, N, o, pad) if keep else None
    kw = dict(transB=transB, alpha=alpha, bias=b if b is None or G is not None else b[0], activation=activation, R=R, beta=beta, Z=Z,
              kernel=kernel)
    if G is None:
        got = runs(kernel, lambda: dg.gemm_fused(A, B, C, splits=splits, **kw))
    else:
        got = runs(kernel, lambda: dg.gemm_grouped(A, B, torch.tensor(offsets, dtype=torch.int32, device=DEV), C, **kw))
    if got is None:
        return False
    want = layer_ref.forward(np64(A), np64(B), offsets, transB, alpha, None if b is None else (np64(b) if G is not None else np64(b[0])),
                             activation, None if R is None else np64(R), beta, o)
    return verify(want, {"C": C, "Z": Z}, offsets, M)


def verify(want, got, offsets, M):
    for name, t in got.items():
        if t is None:
            continue
        ref, bound = want[name]
        if offsets is not None:                       # rows of no group are as they were
            for a, b in ((0, offsets[0]), (offsets[-1], M)):
                assert (t[a:b] == SENTINEL).all(), f"{name}: rows of no group written"
            t, ref, bound = (x[offsets[0]:offsets[-1]] for x in (t, ref, bound))
        check(t, (ref, bound), name)
    padding_kept(*got.values())
    return True


def grad_case(seed, M, N, K, ty, out, transB, activation="gelu", res=False, keep=False, pad=0, alpha=1.0, beta=1.0, offsets=None,
              kernel=-1, splits=1, Z=None, A=None):
    rng = np.random.default_rng(seed)
    t, o = T[ty], T[out]
    G = None if offsets is None else len(offsets) - 1
    A = matrix(rng, M, K, t, pad) if A is None else A
    wr, wc = (N, K) if transB else (K, N)
    W = matrix(rng, (G or 1) * wr, wc, t, pad, std=1 / math.sqrt(max(K, 1)))
    B = W if G is None else W.as_strided((G, wr, wc), (wr * W.stride(0), W.stride(0), 1), W.storage_offset())
    Z = matrix(rng, M, N, o, pad, std=2.0) if Z is None else Z
    R = matrix(rng, M, N, o, pad) if res else None
    C, H = output(M, N, o, pad), output(M, N, o, pad) if keep else None
    kw = dict(transB=transB, alpha=alpha, activation=activation, R=R, beta=beta, H=H, kernel=kernel)
    if G is None:
        got = runs(kernel, lambda: dg.gemm_act_grad(A, B, Z, C, splits=splits, **kw))
    else:
        got = runs(kernel, lambda: dg.gemm_grouped_act_grad(A, B, torch.tensor(offsets, dtype=torch.int32, device=DEV), Z, C, **kw))
    if got is None:
        return False
    want = layer_ref.act_grad(np64(A), np64(B), np64(Z), offsets, transB, alpha, activation, None if R is None else np64(R), beta, o)
    return verify(want, {"C": C, "H": H}, offsets, M)


def dw_case(seed, rows, M, N, ty, out, bias=False, pad=0, shift=0, alpha=1.0, beta=0.0, offsets=None, kernel=-1, splits=1):
    rng = np.random.default_rng(seed)
    t, o = T[ty], T[out]
    G = 1 if offsets is None else len(offsets) - 1
    A, B = matrix(rng, rows, M, t, pad, shift=shift), matrix(rng, rows, N, t, pad, shift=shift)
    whole = output(G * M, N, o, pad)
    if beta:
        whole.copy_(torch.from_numpy(rng.standard_normal((G * M, N))))
    C = whole if offsets is None else whole.as_strided((G, M, N), (M * whole.stride(0), whole.stride(0), 1))
    d = torch.from_numpy(rng.standard_normal((G, M) if offsets is not None else (M,))).float().to(DEV) if bias else None
    c0, d0 = np64(C), None if d is None else np64(d)
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device=DEV)
    if runs(kernel, lambda: dg.gemm_dw(A, B, C, offsets=off, alpha=alpha, beta=beta, dbias=d, kernel=kernel, splits=splits)) is None:
        return False
    want = layer_ref.dw(np64(A), np64(B), offsets, alpha, beta, c0, d0, o)
    check(C, want["C"], "C")
    if bias:
        check(d, want["dbias"], "dbias")
    padding_kept(whole)
    return True


# ---- every kernel, type and orientation at sizes where something ends ----------------------
SIZES = [(1, 1, 1), (1, 130, 64), (2, 17, 3), (5, 64, 100), (16, 16, 16), (17, 257, 129), (33, 8, 65), (64, 64, 64), (65, 129, 200),
         (128, 128, 128), (130, 250, 191), (257, 300, 320), (300, 515, 72), (31, 1032, 512)]


def pads(kernel, i):
    """Row paddings: all with the library's choice, in turn with a forced kernel."""
    return (0, 1, 8) if kernel < 0 else ((0, 1, 8)[i % 3], (0, 8)[i % 2])


@pytest.mark.parametrize("transB", [False, True])
@pytest.mark.parametrize("ty,out", PAIRS)
@pytest.mark.parametrize("kernel", [-1] + KERNELS)
def test_fused(kernel, ty, out, transB):
    ran = 0
    for i, (M, N, K) in enumerate(SIZES):
        for pad in pads(kernel, i):
            o = (i + pad) % 6
            ran += fused_case(100 * i + pad, M, N, K, ty, out, transB, ("none", "relu", "gelu")[o % 3], bias=o in (0, 2, 3), res=o in (1, 2, 4),
                              keep=o in (2, 3, 5), pad=pad, shift=(0, 1, 0)[i % 3] * (pad > 0), alpha=(1.0, -0.5)[i % 2],
                              beta=(1.0, 0.25, 0.0)[i % 3], kernel=kernel)
    assert ran or kernel >= 0


@pytest.mark.parametrize("transB", [False, True])
@pytest.mark.parametrize("ty,out", PAIRS)
@pytest.mark.parametrize("kernel", [-1] + KERNELS)
def test_act_grad(kernel, ty, out, transB):
    for i, (M, N, K) in enumerate(SIZES):
        for pad in pads(kernel, i):
            o = (i + pad) % 4
            grad_case(7000 + 100 * i + pad, M, N, K, ty, out, transB, ("gelu", "relu")[o % 2], res=o in (1, 2), keep=o in (2, 3), pad=pad,
                      alpha=(1.0, 2.0)[i % 2], beta=(1.0, -0.5)[i % 2], kernel=kernel)


@pytest.mark.parametrize("ty,out", PAIRS)
@pytest.mark.parametrize("kernel", [-1] + KERNELS)
def test_dw(kernel, ty, out):
    for i, (M, N, K) in enumerate(SIZES):
        for pad in pads(kernel, i):
            o = (i + pad) % 4
            dw_case(9000 + 100 * i + pad, K, M, N, ty, out, bias=o in (0, 1), pad=pad, shift=(0, 1, 0)[i % 3] * (pad > 0),
                    alpha=(1.0, 0.5)[i % 2], beta=(0.0, 1.0, 0.5)[o % 3], kernel=kernel)


@pytest.mark.parametrize("ty,out", PAIRS)
def test_no_sum(ty, out):
    """K = 0, alpha = 0: the epilogue of zero; A and B are not read (NaN there)."""
    nan = torch.full((40, 24), math.nan, dtype=T[ty], device=DEV)
    R = torch.randn(40, 48, device=DEV).to(T[out])
    bias = torch.randn(48, device=DEV).to(T[out])
    for A, B, alpha in ((nan[:, :0], torch.empty(0, 48, dtype=T[ty], device=DEV), 1.0), (nan, torch.full((24, 48), math.nan, dtype=T[ty], device=DEV), 0.0)):
        C = dg.gemm_fused(A, B, alpha=alpha, bias=bias, activation="relu", R=R, beta=2.0, out_dtype=T[out])
        check(C, layer_ref.forward(np.zeros((40, 1)), np.zeros((1, 48)), bias=np64(bias), activation="relu", R=np64(R), beta=2.0, out=T[out])["C"])
        Z = torch.randn(40, 48, device=DEV).to(T[out])
        C = dg.gemm_act_grad(A, B, Z, alpha=alpha, R=R)
        check(C, layer_ref.act_grad(np.zeros((40, 1)), np.zeros((1, 48)), np64(Z), R=np64(R), out=T[out])["C"])
    x = torch.randn(24, 40, device=DEV).to(T[ty])
    C, d = torch.randn(40, 48, device=DEV).to(T[out]), torch.full((40,), math.nan, device=DEV)
    c0 = np64(C)
    dg.gemm_dw(x, torch.full((24, 48), math.nan, dtype=T[ty], device=DEV), C, alpha=0.0, beta=0.5, dbias=(e := torch.randn(40, device=DEV)))
    check(C, (0.5 * c0, layer_ref.rounding(c0, T[out])))
    dg.gemm_dw(x[:0], torch.empty(0, 48, dtype=T[ty], device=DEV), C, dbias=d)
    assert (C == 0).all() and (d == 0).all() and torch.isfinite(e).all()


def test_empty():
    e = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    off = torch.zeros(4, dtype=torch.int32, device=DEV)
    assert dg.gemm_fused(e(0, 8), e(8, 5)).shape == (0, 5)
    assert dg.gemm_fused(e(3, 8), e(8, 0), bias=e(0)).shape == (3, 0)
    assert dg.gemm_grouped(e(0, 8), e(3, 8, 5), off).shape == (0, 5)
    assert dg.gemm_grouped(e(0, 8), e(0, 8, 5), off[:1]).shape == (0, 5)
    assert dg.gemm_act_grad(e(0, 8), e(8, 5), e(0, 5)).shape == (0, 5)
    C = torch.ones(3, 8, 5, dtype=torch.bfloat16, device=DEV)
    assert (dg.gemm_dw(e(0, 8), e(0, 5), C, offsets=off) == 0).all()
    assert dg.gemm_dw(e(4, 0), e(4, 5)).shape == (0, 5)
    # no column, but a bias gradient
    d = torch.full((8,), math.nan, device=DEV)
    x = torch.randn(50, 8, device=DEV).bfloat16()
    dg.gemm_dw(x, e(50, 0), dbias=d)
    check(d, layer_ref.dw(np64(x), np.zeros((50, 1)))["dbias"])


# ---- groups ------------------------------------------------------------------------------
GROUPS = {
    "one": [0, 40], "none": [0, 0, 0], "empty first and last": [0, 0, 7, 7, 40, 40], "single rows": list(range(21)),
    "tail and head free": [5, 20, 20, 33], "uneven": [0, 1, 130, 131, 400, 417], "two tiles each": [0, 129, 258, 387],
    "a hundred": [int(x) for x in np.cumsum([0] + [(7 * i * i) % 11 for i in range(100)])],
    "two hundred, mostly empty": [int(x) for x in np.cumsum([0] + [70 * (i in (0, 63, 64, 127, 199)) for i in range(200)])],
}


@pytest.mark.parametrize("name", list(GROUPS))
@pytest.mark.parametrize("ty,out", PAIRS)
def test_grouped(ty, out, name):
    offsets = GROUPS[name]
    M = offsets[-1] + (7 if "free" in name or name == "none" else 0)
    for i, kernel in enumerate([-1] + KERNELS):
        for transB in (False, True):
            N, K, pad = ((72, 96, 0), (131, 70, 1), (40, 130, 8))[(i + transB) % 3]
            fused_case(i, M, N, K, ty, out, transB, ("none", "gelu", "relu")[i % 3], bias=True, res=i % 2 == 0, keep=i % 3 == 0,
                       pad=pad, offsets=offsets, kernel=kernel)
            grad_case(i + 50, M, N, K, ty, out, transB, ("gelu", "relu")[i % 2], res=i % 2 == 1, keep=i % 3 == 1, pad=pad, offsets=offsets,
                      kernel=kernel)


@pytest.mark.parametrize("name", list(GROUPS))
@pytest.mark.parametrize("ty,out", PAIRS)
def test_grouped_dw(ty, out, name):
    offsets = GROUPS[name]
    rows = offsets[-1] + (7 if "free" in name else 0)
    for i, kernel in enumerate([-1] + KERNELS):
        M, N, pad = ((72, 40, 0), (131, 70, 1), (40, 130, 8))[i % 3]
        for splits in (1, 0, 3):
            dw_case(i + 10 * splits, rows, M, N, ty, out, bias=True, pad=pad, beta=(0.0, 1.0)[i % 2], offsets=offsets, kernel=kernel,
                    splits=splits)


def test_rows_of_no_group_are_not_read():
    rng = np.random.default_rng(3)
    offsets = [4, 9, 30]
    A, Z = matrix(rng, 40, 64, torch.float16), matrix(rng, 40, 48, torch.float16)
    for t in (A, Z):
        t[:4], t[30:] = math.nan, math.nan
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    B = torch.randn(2, 64, 48, device=DEV).half()
    assert torch.isfinite(dg.gemm_grouped(A, B, off, C=torch.zeros(40, 48, dtype=torch.float16, device=DEV))).all()
    assert torch.isfinite(dg.gemm_grouped_act_grad(A, B, off, Z, C=torch.zeros(40, 48, dtype=torch.float16, device=DEV))).all()
    d = torch.empty(2, 64, device=DEV)
    assert torch.isfinite(dg.gemm_dw(A, Z, offsets=off, dbias=d)).all() and torch.isfinite(d).all()


def test_offsets_outside_the_matrices():
    """Clamped by the kernels: nothing outside is touched, and groups that are in order are right."""
    M, N, K = 50, 40, 64
    rng = np.random.default_rng(4)
    A, B = matrix(rng, M, K, torch.bfloat16), torch.randn(4, K, N, device=DEV).bfloat16()
    for given, means in (([-5, 20, 20, 70, 90], [0, 20, 20, 50, 50]), ([10, 30, 25, 40, 2 ** 31 - 1], None), ([-2 ** 31, -1, 0, 5, 50], [0, 0, 0, 5, 50])):
        whole = torch.full((M + 40, N), SENTINEL, dtype=torch.bfloat16, device=DEV)
        off = torch.tensor(given, dtype=torch.int32, device=DEV)
        C = dg.gemm_grouped(A, B, off, C=whole[20:20 + M])
        assert (whole[:20] == SENTINEL).all() and (whole[20 + M:] == SENTINEL).all()
        if means:
            ref, bound = layer_ref.forward(np64(A), np64(B), means, out=torch.bfloat16)["C"]
            check(C[means[0]:means[-1]], (ref[means[0]:means[-1]], bound[means[0]:means[-1]]))
            check(dg.gemm_dw(A, A, offsets=off), layer_ref.dw(np64(A), np64(A), means, out=torch.bfloat16)["C"])
        else:
            dg.gemm_dw(A, A, offsets=off)
        torch.cuda.synchronize()


def test_rows_claimed_by_many_groups():
    """Offsets that go up and down claim the same rows many times over, more tiles than the
    launch holds: it ends, and writes nothing outside the claimed rows."""
    M, N, K = 150, 72, 64
    rng = np.random.default_rng(5)
    for ty in ("f32", "bf16"):
        A = matrix(rng, M, K, T[ty])
        for pairs in (3, 40, 300):
            off = torch.tensor([20, M - 10] * pairs, dtype=torch.int32, device=DEV)
            B = torch.randn(1, K, N, device=DEV).to(T[ty]).expand(2 * pairs - 1, K, N)
            for kernel in [-1] + KERNELS:
                whole = output(M, N, T[ty], 8)
                if runs(kernel, lambda: dg.gemm_grouped(A, B, off, C=whole, kernel=kernel)) is not None:
                    assert (whole[:20] == SENTINEL).all() and (whole[M - 10:] == SENTINEL).all()
                    padding_kept(whole)
            want = layer_ref.dw(np64(A[20:M - 10]), np64(A[20:M - 10]), None, out=T[ty])["C"]
            got = dg.gemm_dw(A, A, offsets=off)              # every other group has the same rows, the rest none
            for g in (0, pairs - pairs % 2, 2 * pairs - 2):
                check(got[g], want)
            assert (got[1] == 0).all()
            torch.cuda.synchronize()


# ---- K ranges -------------------------------------------------------------------------------
@pytest.mark.parametrize("ty,out", PAIRS)
@pytest.mark.parametrize("splits", [0, 2, 5, 16])
def test_splits(splits, ty, out):
    for M, N, K in ((3, 40, 1000), (70, 130, 700), (1, 9, 64), (40, 200, 2048)):
        fused_case(splits, M, N, K, ty, out, True, "gelu", bias=True, res=True, keep=True, pad=1, splits=splits)
        grad_case(splits, M, N, K, ty, out, False, "relu", res=True, keep=True, splits=splits)
        dw_case(splits, K, M, N, ty, out, bias=True, pad=2, beta=0.5, splits=splits)


def test_caller_workspace_and_bounds():
    """A caller's workspace is used inside its size, and what it held does not matter."""
    A, B = torch.randn(20, 1024, device=DEV).half(), torch.randn(1024, 48, device=DEV).half()
    need = dg.dg_layer_workspace_size(1, 20, 48, 4)
    ws = torch.full((need // 4 + 64,), math.nan, device=DEV)
    got = dg.gemm_fused(A, B, splits=4, workspace=ws[:need // 4])
    assert torch.isnan(ws[need // 4:]).all()
    assert torch.equal(got, dg.gemm_fused(A, B, splits=4))
    with pytest.raises(dg.LayerError, match="workspace_bytes"):
        dg.gemm_fused(A, B, splits=4, workspace=ws[:need // 4 - 1])
    with pytest.raises(dg.LayerError, match=r"\(workspace\)"):
        dg.gemm_fused(A, B, splits=4, workspace=ws[1:])


# ---- special values ---------------------------------------------------------------------------
@pytest.mark.parametrize("ty,out", PAIRS)
def test_special_values(ty, out):
    M, N, K = 20, 24, 32
    g = torch.Generator().manual_seed(1)
    A, B = torch.randn(M, K, generator=g).to(T[ty]), torch.randn(K, N, generator=g).to(T[ty])
    low, big = torch.finfo(T[out]).min, torch.finfo(T[out]).max
    Z = torch.randn(M, N, generator=g).to(T[out])
    Z[:, 0], Z[:, 1], Z[:, 2], Z[:, 3], Z[:, 4], Z[:, 5], Z[:, 6] = math.nan, math.inf, -math.inf, low, big, 0.0, -0.0
    Ad, Bd, Zd = A.to(DEV), B.to(DEV), Z.to(DEV)
    for name in ("relu", "gelu"):
        C = dg.gemm_act_grad(Ad, Bd, Zd, activation=name)
        check(C, layer_ref.act_grad(np64(A), np64(B), np64(Z), activation=name, out=T[out])["C"], name)
    # infinite and NaN gradients: relu stops them where the unit is off
    A[3, 0], A[4, 0], A[5, 0] = math.inf, -math.inf, math.nan
    C = dg.gemm_act_grad(A.to(DEV), Bd, Zd, activation="relu")
    off = (Z <= 0)
    assert (C.cpu()[off] == 0).all()
    on = Z[3:6] > 0
    assert not torch.isfinite(C.cpu()[3:6][on]).any()
    # forward: infinities and NaN in the residual and the bias
    R = torch.zeros(M, N, dtype=T[out])
    R[0, 0], R[1, 1], R[2, 2] = math.inf, -math.inf, math.nan
    A = torch.randn(M, K, generator=g).to(T[ty])
    for name in ("none", "relu", "gelu"):
        C = dg.gemm_fused(A.to(DEV), Bd, activation=name, R=R.to(DEV), out_dtype=T[out])
        want = layer_ref.forward(np64(A), np64(B), activation=name, R=np64(R), out=T[out])["C"]
        want[1][~np.isfinite(want[0])] = 0
        check(C, want, name)
    # beta = 0 does not read R, nor C as R
    nan = torch.full((M, N), math.nan, dtype=T[out], device=DEV)
    assert torch.isfinite(dg.gemm_fused(A.to(DEV), Bd, nan, R=nan, beta=0.0)).all()


def test_far_gelu():
    """gelu and its slope far out on both sides keep their relative accuracy."""
    x = torch.linspace(-13, 13, 4096, dtype=torch.float64)
    for ty, out in PAIRS:
        if ty == "f16" and out == "f32":
            continue
        v = x.to(T[ty])
        A, B = v[:, None].to(DEV), torch.ones(1, 3, dtype=T[ty], device=DEV)
        check(dg.gemm_fused(A, B, activation="gelu", out_dtype=T[out]), layer_ref.forward(np64(A), np64(B), activation="gelu", out=T[out])["C"])
        Z = v[:, None].expand(-1, 3).contiguous().to(T[out]).to(DEV)
        one = torch.ones(4096, 1, dtype=T[ty], device=DEV)
        check(dg.gemm_act_grad(one, B, Z), layer_ref.act_grad(np64(one), np64(B), np64(Z), out=T[out])["C"])


# ---- as a program calls them --------------------------------------------------------------------
def test_residual_in_place():
    A, B = torch.randn(50, 70, device=DEV).bfloat16(), torch.randn(70, 90, device=DEV).bfloat16()
    C = torch.randn(50, 90, device=DEV).bfloat16()
    want = dg.gemm_fused(A, B, activation="relu", R=C.clone())
    assert torch.equal(dg.gemm_fused(A, B, C, activation="relu", R=C), want)
    Z, R = torch.randn(50, 90, device=DEV).bfloat16(), torch.randn(50, 90, device=DEV).bfloat16()
    H = R.clone()
    want = dg.gemm_act_grad(A, B, Z, R=R, H=(h := torch.empty_like(R)))
    assert torch.equal(dg.gemm_act_grad(A, B, Z, R=H, H=H), want) and torch.equal(H, h)
    assert torch.equal(dg.gemm_act_grad(A, B, Z, C=R, R=R), want)


def test_shared_matrix_and_views():
    """One matrix for every group (stride 0), columns of a wider matrix, every other matrix."""
    A = torch.randn(60, 200, device=DEV).half()[:, 8:72]
    off = torch.tensor([0, 20, 21, 60], dtype=torch.int32, device=DEV)
    B = torch.randn(64, 48, device=DEV).half()
    assert torch.equal(dg.gemm_grouped(A, B.expand(3, 64, 48), off), dg.gemm_fused(A, B))
    W = torch.randn(6, 64, 48, device=DEV).half()
    got = dg.gemm_grouped(A, W[::2], off)
    check(got, layer_ref.forward(np64(A), np64(W[::2]), off.tolist(), out=torch.float16)["C"])


def test_results_repeat():
    A, B = torch.randn(700, 512, device=DEV).bfloat16(), torch.randn(700, 260, device=DEV).bfloat16()
    off = torch.tensor([0, 300, 300, 650], dtype=torch.int32, device=DEV)
    first = [(dg.gemm_dw(A, B, offsets=off, dbias=(d := torch.empty(3, 512, device=DEV)), splits=s), d) for s in (0, 1, 4)]
    for _ in range(3):
        for (c, d0), s in zip(first, (0, 1, 4)):
            assert torch.equal(dg.gemm_dw(A, B, offsets=off, dbias=(d := torch.empty(3, 512, device=DEV)), splits=s), c)
            assert torch.equal(d, d0)


def layer_step(x, w1, b1, w2, b2, off, dy, bufs, stream=None):
    """One expert layer with its residual, forward and backward."""
    z, h, y, dz, dx, dw1, db1, dw2, db2 = bufs
    dg.gemm_grouped(x, w1, off, h, transB=True, bias=b1, activation="gelu", Z=z, stream=stream)
    dg.gemm_grouped(h, w2, off, y, transB=True, bias=b2, R=x, stream=stream)
    dg.gemm_grouped_act_grad(dy, w2, off, z, dz, activation="gelu", stream=stream)
    dg.gemm_dw(dy, h, dw2, offsets=off, dbias=db2, stream=stream)
    dg.gemm_grouped(dz, w1, off, dx, R=dy, stream=stream)
    dg.gemm_dw(dz, x, dw1, offsets=off, dbias=db1, stream=stream)


def layer_inputs(seed, M, D, F, G, dtype):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(dtype).to(DEV)  # noqa: E731
    ins = (r(M, D), r(G, F, D, std=D ** -0.5), r(G, F, std=0.3), r(G, D, F, std=F ** -0.5), r(G, D, std=0.3))
    cuts = [0] + sorted(torch.randint(0, M + 1, (G - 1,), generator=g).tolist()) + [M]
    return ins, torch.tensor(cuts, dtype=torch.int32, device=DEV), r(M, D)


def layer_buffers(M, D, F, G, dtype):
    e = lambda *s, dt=dtype: torch.empty(*s, dtype=dt, device=DEV)  # noqa: E731
    f = torch.float32
    return (e(M, F), e(M, F), e(M, D), e(M, F), e(M, D), e(G, F, D, dt=f), e(G, F, dt=f), e(G, D, F, dt=f), e(G, D, dt=f))


def layer_plain(ins, off, dy):
    """The step in 64 bits by torch's differentiation, from rounded inputs."""
    x, w1, b1, w2, b2 = (t.double().cpu().requires_grad_() for t in ins)
    parts = []
    for g, (a, b) in enumerate(zip(off[:-1], off[1:])):
        z = x[a:b] @ w1[g].T + b1[g]
        h = z * 0.5 * torch.special.erfc(-z / math.sqrt(2))
        parts.append(h @ w2[g].T + b2[g] + x[a:b])
    y = torch.cat(parts)
    y.backward(dy.double().cpu())
    return [y] + [t.grad for t in (x, w1, b1, w2, b2)]


@pytest.mark.parametrize("dtype,tol", [(torch.float32, 1e-5), (torch.float16, 4e-3), (torch.bfloat16, 3e-2)])
def test_expert_layer(dtype, tol):
    """All of them together as a training step uses them, against differentiation in 64
    bits.  Tolerance by norm: a value passes at most six roundings (z, h, dz, x, dy and
    the output), each half a step, so 6 eps / 2 and the sums' (a few 1e-6)."""
    M, D, F, G = 150, 96, 200, 5
    ins, off, dy = layer_inputs(3, M, D, F, G, dtype)
    bufs = layer_buffers(M, D, F, G, dtype)
    layer_step(*ins, off, dy, bufs)
    z, h, y, dz, dx, dw1, db1, dw2, db2 = bufs
    assert tol >= 6 * torch.finfo(dtype).eps / 2 + 5e-6
    for got, want, name in zip((y, dx, dw1, db1, dw2, db2), layer_plain(ins, off.tolist(), dy), ("y", "dx", "dw1", "db1", "dw2", "db2")):
        err = (got.double().cpu() - want).norm() / want.norm()
        assert err < tol, (name, float(err))


def test_captured_step():
    """The step in a graph, replayed with other inputs and other group sizes between eager work."""
    M, D, F, G, dtype = 200, 128, 256, 4, torch.bfloat16
    ins, off, dy = layer_inputs(1, M, D, F, G, dtype)
    bufs, eager = layer_buffers(M, D, F, G, dtype), layer_buffers(M, D, F, G, dtype)
    layer_step(*ins, off, dy, bufs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer_step(*ins, off, dy, bufs)
    for seed in range(2, 6):
        new, noff, ndy = layer_inputs(seed, M, D, F, G, dtype)
        for t, n in zip((*ins, off, dy), (*new, noff, ndy)):
            t.copy_(n)
        for b in bufs:
            b.fill_(math.nan)
        graph.replay()
        layer_step(*ins, off, dy, eager)
        torch.cuda.synchronize()
        for a, b in zip(bufs, eager):
            assert torch.equal(a, b)


def test_two_graphs_of_split_sums():
    """Two graphs whose split sums have workspaces of their own, replayed in turn and on two streams at once."""
    A, B = [torch.randn(40, 2048, device=DEV).half() for _ in range(2)], torch.randn(2048, 72, device=DEV).half()
    C = [torch.empty(40, 72, dtype=torch.float16, device=DEV) for _ in range(2)]
    D = [torch.empty(2048, 2048, device=DEV) for _ in range(2)]
    d = [torch.empty(2048, device=DEV) for _ in range(2)]
    dg.gemm_fused(A[0], B, C[0], splits=4)
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            dg.gemm_fused(A[i], B, C[i], splits=4)
            dg.gemm_dw(A[i], A[i], D[i], dbias=d[i], splits=2)
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for seed in range(4):
        for a in A:
            a.copy_(torch.randn(40, 2048, device=DEV))
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            if seed % 2:
                with torch.cuda.stream(s):
                    g.replay()
            else:
                g.replay()
        torch.cuda.synchronize()
        for i in range(2):
            e = torch.empty(2048, device=DEV)
            assert torch.equal(C[i], dg.gemm_fused(A[i], B, splits=4))
            assert torch.equal(D[i], dg.gemm_dw(A[i], A[i], dbias=e, splits=2, out_dtype=torch.float32)) and torch.equal(d[i], e)


def test_streams():
    """Calls on two streams at once, each with its own outputs; the caller's stream orders them."""
    M, D, F, G, dtype = 300, 256, 512, 4, torch.float16
    sets = []
    for seed in (1, 2):
        ins, off, dy = layer_inputs(seed, M, D, F, G, dtype)
        ref = layer_buffers(M, D, F, G, dtype)
        layer_step(*ins, off, dy, ref)
        sets.append((ins, off, dy, ref, layer_buffers(M, D, F, G, dtype), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(3):
        for ins, off, dy, ref, bufs, s in sets:
            layer_step(*ins, off, dy, bufs, stream=s)
    torch.cuda.synchronize()
    for ins, off, dy, ref, bufs, s in sets:
        for a, b in zip(ref, bufs):
            assert torch.equal(a, b)


def test_allocated_results_on_a_given_stream():
    A, B = torch.randn(64, 2048, device=DEV).half(), torch.randn(2048, 64, device=DEV).half()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = dg.gemm_fused(A, B, splits=4, stream=s)
    dw = dg.gemm_dw(A, A, stream=s)
    s.synchronize()
    assert torch.equal(got, dg.gemm_fused(A, B, splits=4)) and torch.equal(dw, dg.gemm_dw(A, A))
    with pytest.raises(ValueError, match="one device"):
        dg.gemm_fused(A, B.cpu())
    with pytest.raises(ValueError, match="one device"):
        dg.gemm_grouped(A, B[None], torch.tensor([0, 64], dtype=torch.int32))


# ---- large -----------------------------------------------------------------------------------------
def test_large_rows_against_a_sample():
    """Products whose matrices pass 2^31 elements: sampled rows against 64 bits."""
    M, N, K = 70000, 32768, 64
    g = torch.Generator(device=DEV).manual_seed(1)
    A = torch.randn(M, K, generator=g, device=DEV).bfloat16()
    B = torch.randn(2, N, K, generator=g, device=DEV).bfloat16()
    off = torch.tensor([0, 40001, M], dtype=torch.int32, device=DEV)
    Z = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    C = dg.gemm_grouped(A, B, off, transB=True, activation="gelu", Z=Z)
    rows = [0, 1, 40000, 40001, 65535, 65536, 69998, 69999]
    a = np64(A[rows])
    for r0, grp in ((slice(0, 3), 0), (slice(3, 8), 1)):
        want = layer_ref.forward(a[r0], np64(B[grp]), transB=True, activation="gelu", out=torch.bfloat16)
        check(C[rows[r0]], want["C"])
        check(Z[rows[r0]], want["Z"])
    del C
    d = torch.empty(2, N, device=DEV)
    W = dg.gemm_dw(Z, A, offsets=off, dbias=d, out_dtype=torch.float32)
    cols = [0, 5, 16384, 32767]
    want = layer_ref.dw(np64(Z[:, cols]), np64(A), off.tolist())
    check(W[:, cols], want["C"])
    check(d[:, cols], want["dbias"])


@pytest.mark.parametrize("ty", ["f16", "bf16"])
@pytest.mark.parametrize("kernel", KERNELS)
def test_outputs_past_the_caches(kernel, ty):
    """Outputs above 64 MB, with ragged ends and rows padded: sampled rows against 64 bits, and every element
    against the first kernel's (whose own bound, of the same sums, doubles the tolerance)."""
    M, N, K, t = 8200, 4099, 72, T[ty]
    g = torch.Generator(device=DEV).manual_seed(7)
    A, B = torch.randn(M, K, generator=g, device=DEV).to(t), (torch.randn(N, K, generator=g, device=DEV) / 9).to(t)
    b, R = torch.randn(N, generator=g, device=DEV).to(t), torch.randn(M, N, generator=g, device=DEV).to(t)
    kw = dict(transB=True, bias=b, activation="gelu", R=R)
    C, Z = output(M, N, t, 5), output(M, N, t, 5)
    if runs(kernel, lambda: dg.gemm_fused(A, B, C, Z=Z, kernel=kernel, **kw)) is None:
        pytest.skip("the kernel does not take the problem")
    padding_kept(C, Z)
    rows = [0, 1, 255, 256, 4097, 8191, 8192, 8199]
    want = layer_ref.forward(np64(A[rows]), np64(B), transB=True, bias=np64(b), activation="gelu", R=np64(R[rows]), beta=1.0, out=t)
    check(C[rows], want["C"])
    check(Z[rows], want["Z"])
    # two roundings (half a step each) of fp32 values that differ by both sums' errors, each at most K 2^-24 times
    # the sum of |a b| (K = 72 terms of 0.07 on average, 10 at the most), times gelu's slope 1.13: 1e-4
    C0, Z0 = torch.empty(M, N, dtype=t, device=DEV), torch.empty(M, N, dtype=t, device=DEV)
    dg.gemm_fused(A, B, C0, Z=Z0, kernel=0, **kw)
    for x, y in ((C, C0), (Z, Z0)):
        off = (x.float() - y.float()).abs() - torch.finfo(t).eps * torch.maximum(x.float().abs(), y.float().abs())
        assert float(off.max()) < 2e-4


def test_row_strides_past_32_bits():
    """Row strides at which 256 rows span more than 2^31 bytes."""
    ld = 5_000_000
    big = torch.zeros(300 * ld, dtype=torch.float16, device=DEV).view(300, ld)
    rng = np.random.default_rng(2)
    A = big[:, :96]
    A.copy_(torch.from_numpy(rng.standard_normal((300, 96))))
    B = matrix(rng, 40, 96, torch.float16, std=0.1)
    C = big[:, 1000:1040]
    got = dg.gemm_fused(A, B, C, transB=True, bias=matrix(rng, 1, 40, torch.float16)[0], activation="relu", R=C)
    assert torch.isfinite(got).all()
    want = dg.gemm_fused(A.contiguous(), B, transB=True)
    check(dg.gemm_fused(A, B, transB=True), layer_ref.forward(np64(A), np64(B), transB=True, out=torch.float16)["C"])
    check(want, layer_ref.forward(np64(A), np64(B), transB=True, out=torch.float16)["C"])
    check(dg.gemm_dw(A, big[:, 2000:2033]), layer_ref.dw(np64(A), np.zeros((300, 33)), out=torch.float16)["C"])
