"""More of a layer's products on an MI355X, against their formulas in 64 bits (layer_ref):
the paths that depend on how operands lie, how long a sum is and how uneven groups are."""
import numpy as np
import pytest
import torch

import dense_gemm_amd as dg
import layer_ref
from layer_ref import T, check, np64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


# ---- long sums ------------------------------------------------------------------------------
@pytest.mark.parametrize("splits", [2048, 4096])
def test_longest_sum_in_many_ranges(splits):
    """The longest sum that the calls take, in more ranges than 2^31 leaves room to round up by:
    ones against zeros and a few ones, so that the sum counts every range's part exactly."""
    K = 2 ** 31 - 1025
    chunk = -(-(-(-K // splits)) // 64) * 64
    ends = [i * chunk + d for i in (1, 2, splits // 2) for d in (-1, 0) if i * chunk + d < K]
    at = sorted(set([0, 1, K - 65, K - 2, K - 1] + ends + np.random.default_rng(splits).integers(0, K, 90).tolist()))
    one = torch.ones(K, dtype=torch.bfloat16, device=DEV)
    few = torch.zeros(K, dtype=torch.bfloat16, device=DEV)
    few[torch.tensor(at, device=DEV)] = 1
    print(f"forward, {splits} ranges", flush=True)
    assert dg.gemm_fused(one[None], few[None], transB=True, splits=splits).item() == len(at)
    torch.cuda.synchronize()
    print(f"weights, {splits} ranges", flush=True)
    d = torch.empty(1, device=DEV)
    assert dg.gemm_dw(few[:, None], one[:, None], dbias=d, splits=splits).item() == len(at) and d.item() == len(at)


# ---- the library's choice of ranges -----------------------------------------------------------
def fused_call(A, B, C, splits, workspace, nbytes):
    """dg_gemm_fused, C = A B^T, with a workspace of `nbytes` bytes."""
    (M, K), N = A.shape, B.shape[0]
    code = {torch.float16: dg.DG_F16_F32ACC, torch.bfloat16: dg.DG_BF16_F32ACC, torch.float32: dg.DG_F32}[A.dtype]
    return dg.dg_gemm_fused(1, 1, None, M, N, K, 1.0, A.data_ptr(), A.stride(0), B.data_ptr(), B.stride(0), 0, None, 0, dg.DG_EPI_NONE,
                            None, N, 0.0, None, N, C.data_ptr(), C.stride(0), code, splits, workspace.data_ptr(), nbytes,
                            torch.cuda.current_stream().cuda_stream)


@pytest.mark.parametrize("ty", ["f16", "f32"])
@pytest.mark.parametrize("M,N,K", [(64, 2047, 5631), (16, 96, 5631), (40, 130, 2049), (3, 1000, 4095)])
def test_choice_within_the_workspace(M, N, K, ty):
    """splits = 0 takes no more ranges than the workspace holds, whatever its size and however the
    operands lie (the query's answer is for aligned ones)."""
    rng = np.random.default_rng(K)
    t = T[ty]
    n = dg.dg_gemm_fused_choose(M, N, K, 1, dg.DG_F16_F32ACC if ty == "f16" else dg.DG_F32)
    A, B = (torch.from_numpy(rng.standard_normal(s) / 8).to(t).to(DEV) for s in ((M, K), (N, K)))
    want = layer_ref.forward(np64(A), np64(B), transB=True, out=t)["C"]
    for ranges in (n, 0, 1, 2, 3, 16):
        nbytes = dg.dg_layer_workspace_size(1, M, N, ranges) or 16
        for less in (0, 4):
            ws = torch.full((nbytes // 4 + 64,), float("nan"), device=DEV)
            C = torch.full((M, N), float("nan"), dtype=t, device=DEV)
            assert fused_call(A, B, C, 0, ws, nbytes - less) == dg.DG_OK, (ranges, less)
            check(C, want)
            assert torch.isnan(ws[(nbytes - less) // 4:]).all()
    assert fused_call(A, B, C, 3, ws, dg.dg_layer_workspace_size(1, M, N, 3) - 4) == -26


@pytest.mark.parametrize("transB", [False, True])
@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("ty", ["f16", "bf16", "f32"])
def test_the_library_s_choice(ty, pad, transB):
    """The torch functions with splits = 0 give, bit for bit, what the library's choice of kernel and ranges
    within a large enough workspace gives, aligned operands or not."""
    t, code = T[ty], {"f16": dg.DG_F16_F32ACC, "bf16": dg.DG_BF16_F32ACC, "f32": dg.DG_F32}[ty]
    g = torch.Generator(device=DEV).manual_seed(1)
    r = lambda a, b: (torch.randn(a, b + pad, generator=g, device=DEV) / 8).to(t)[:, :b]  # noqa: E731
    ws = torch.empty(1 << 26, dtype=torch.uint8, device=DEV)
    several = 0
    for M, N, K in ((512, 1032, 5632), (64, 2048, 5632), (24, 300, 4096), (163, 328, 4202), (2, 2048, 5632), (8, 1184, 4464)):
        A, B, X, Y = r(M, K), r(*((N, K) if transB else (K, N))), r(K, M), r(K, N)
        n = dg.dg_gemm_fused_choose_for(M, N, K, transB, code, A.data_ptr(), A.stride(0), B.data_ptr(), B.stride(0))
        got = dg.gemm_fused(A, B, transB=transB)
        assert torch.equal(got, dg.gemm_fused(A, B, transB=transB, workspace=ws))
        check(got, layer_ref.forward(np64(A), np64(B), transB=transB, out=t)["C"])
        m = dg.dg_gemm_dw_choose_for(1, K, M, N, code, X.data_ptr(), X.stride(0), Y.data_ptr(), Y.stride(0))
        got = dg.gemm_dw(X, Y)
        assert torch.equal(got, dg.gemm_dw(X, Y, workspace=ws))
        check(got, layer_ref.dw(np64(X), np64(Y), out=t)["C"])
        several += (n > 1) + (m > 1)
    assert several


# ---- row strides past 32 bits -------------------------------------------------------------------
@pytest.mark.parametrize("kernel", [-1, 0, 1, 7])
@pytest.mark.parametrize("ty", ["f16", "f32"])
def test_far_rows(ty, kernel):
    """Rows so far apart that 256 of them span more than 2^31 bytes, which the direct loads do not take: A, B
    or both through registers, and every matrix of the epilogue, each by value."""
    t, ld = T[ty], 5_000_000 // (torch.finfo(T[ty]).bits // 16)
    rng = np.random.default_rng(2)
    big = torch.full((300 * ld,), float("nan"), dtype=t, device=DEV).view(300, ld)
    at = [0]

    def far(rows, cols, std=1.0):
        """Columns of their own of the wide matrix, with values."""
        v = big[:rows, at[0]:at[0] + cols]
        at[0] += cols + 64
        return v.copy_(torch.from_numpy(rng.standard_normal((rows, cols)) * std))

    def near(rows, cols, std=1.0):
        return torch.from_numpy(rng.standard_normal((rows, cols)) * std).to(t).to(DEV)

    M, N, K = 300, 44, 96
    for a_far, b_far in ((1, 0), (0, 1), (1, 1)):
        for transB in (False, True):
            A, B = (far if a_far else near)(M, K), (far if b_far else near)(*((N, K) if transB else (K, N)), 0.1)
            R, Z, C, K2, bias = far(M, N), far(M, N), far(M, N), far(M, N), near(1, N)[0]
            kw = dict(transB=transB, kernel=kernel)
            want = layer_ref.forward(np64(A), np64(B), transB=transB, bias=np64(bias), activation="gelu", R=np64(R), beta=0.5, out=t)
            dg.gemm_fused(A, B, C, bias=bias, activation="gelu", R=R, beta=0.5, Z=Z, **kw)
            check(C, want["C"], (a_far, b_far, transB))
            check(Z, want["Z"], (a_far, b_far, transB))
            want = layer_ref.forward(np64(A), np64(B), transB=transB, activation="relu", R=np64(R), out=t)
            check(dg.gemm_fused(A, B, R, activation="relu", R=R, **kw), want["C"])            # the residual in place
            want = layer_ref.act_grad(np64(A), np64(B), np64(Z), transB=transB, R=np64(R), beta=2.0, out=t)
            dg.gemm_act_grad(A, B, Z, C, R=R, beta=2.0, H=K2, **kw)
            check(C, want["C"])
            check(K2, want["H"])
            torch.cuda.synchronize()
        if kernel == 7:
            continue                                  # (few rows: no weight gradients)
        X, Y, W = (far if a_far else near)(M, 40), (far if b_far else near)(M, 33), far(40, 33)
        d = torch.randn(40, device=DEV)
        want = layer_ref.dw(np64(X), np64(Y), beta=0.5, alpha=0.25, C=np64(W), dbias=np64(d), out=t)
        check(dg.gemm_dw(X, Y, W, alpha=0.25, beta=0.5, dbias=d, kernel=kernel), want["C"])
        check(d, want["dbias"])
        off = torch.tensor([3, 100, 100, 290], dtype=torch.int32, device=DEV)
        check(dg.gemm_dw(X, Y, offsets=off, kernel=kernel), layer_ref.dw(np64(X), np64(Y), off.tolist(), out=t)["C"])
        torch.cuda.synchronize()


# ---- few rows in K ranges ---------------------------------------------------------------------------
@pytest.mark.parametrize("transB", [False, True])
@pytest.mark.parametrize("ty,out", [("f16", "f16"), ("bf16", "bf16"), ("f16", "f32"), ("f32", "f32")])
def test_few_rows_in_ranges(ty, out, transB):
    """The few-rows kernel on a range of K: bias, residual, Z and what is kept belong to the join alone (the
    kernel's sums are fp32 where those are 16 bits wide, so that it must not read them by its own type)."""
    t, o = T[ty], T[out]
    rows = dg.layer_kernel_names().index("layer_16_rows")
    for i, (M, N, K) in enumerate([(1, 40, 512), (5, 40, 514), (16, 100, 300), (24, 68, 1100), (3, 260, 129)]):
        rng = np.random.default_rng(i)
        r = lambda a, b, d, s=1.0: torch.from_numpy(rng.standard_normal((a, b)) * s).to(d).to(DEV)  # noqa: E731
        A, B, R, Z, bias = r(M, K, t), r(*((N, K) if transB else (K, N)), t, K ** -0.5), r(M, N, o), r(M, N, o), r(1, N, o)[0]
        for kernel in (rows, -1):
            for splits in (2, 3, 16, 0, 1):
                keep = torch.empty(M, N, dtype=o, device=DEV)
                want = layer_ref.forward(np64(A), np64(B), transB=transB, bias=np64(bias), activation="gelu", R=np64(R), beta=0.5, out=o)
                got = dg.gemm_fused(A, B, transB=transB, bias=bias, activation="gelu", R=R, beta=0.5, Z=keep, out_dtype=o, splits=splits,
                                    kernel=kernel)
                check(got, want["C"], (M, N, K, kernel, splits))
                check(keep, want["Z"])
                want = layer_ref.act_grad(np64(A), np64(B), np64(Z), transB=transB, R=np64(R), out=o)
                check(dg.gemm_act_grad(A, B, Z, transB=transB, R=R, H=keep, splits=splits, kernel=kernel), want["C"], (M, N, K, kernel, splits))
                check(keep, want["H"])
    torch.cuda.synchronize()


# ---- operands that lie differently ----------------------------------------------------------------
PAIRS = [("f16", "f16"), ("bf16", "bf16"), ("f16", "f32"), ("bf16", "f32")]
EVEN = [(65, 130, 200), (300, 516, 72), (17, 258, 192), (129, 64, 130), (5, 40, 514), (64, 64, 64)]      # rows that are aligned without padding
SENTINEL = -77.0


def placed(rng, rows, cols, dtype, odd, std=1.0):
    """A matrix whose rows the direct loads take, or ("stride", "address") do not; NaN around it."""
    pad, shift = (8 if odd is None else 1 if odd == "stride" else 8), (1 if odd == "address" else 0)
    whole = torch.full((rows * (cols + pad) + shift,), float("nan"), dtype=dtype, device=DEV)
    v = whole[shift:].view(rows, cols + pad)[:, :cols]
    v.copy_(torch.from_numpy(rng.standard_normal((rows, cols)) * std))
    bits = v.data_ptr() | v.stride(0) * v.element_size()
    assert (bits % 4 != 0) == (odd is not None)
    return v


def output(rows, cols, dtype):
    return torch.full((rows, cols + 3), SENTINEL, dtype=dtype, device=DEV)[:, :cols]


def same_rows(t, want, offsets, M):
    """Rows of the groups within their bounds, the others and the padding untouched."""
    ref, bound = want
    a, b = (0, M) if offsets is None else (offsets[0], offsets[-1])
    check(t[a:b], (ref[a:b], bound[a:b]))
    assert (t[:a] == SENTINEL).all() and (t[b:] == SENTINEL).all() and (t._base[:, t.shape[1]:] == SENTINEL).all()


@pytest.mark.parametrize("odd_a,odd_b", [("stride", None), (None, "stride"), ("address", None), (None, "address"), ("stride", "address")])
@pytest.mark.parametrize("transB", [False, True])
@pytest.mark.parametrize("ty,out", PAIRS)
def test_one_operand_unaligned(ty, out, transB, odd_a, odd_b):
    """A or B alone through registers, dense and grouped, forward and backward."""
    t, o = T[ty], T[out]
    for kernel in (-1, 0, 1):
        for i, (M, N, K) in enumerate(EVEN):
            rng = np.random.default_rng(i)
            A, B = placed(rng, M, K, t, odd_a), placed(rng, *((N, K) if transB else (K, N)), t, odd_b, 0.1)
            R, C, Z = placed(rng, M, N, o, None), output(M, N, o), output(M, N, o)
            kw = dict(transB=transB, R=R, kernel=kernel)
            want = layer_ref.forward(np64(A), np64(B), transB=transB, activation="gelu", R=np64(R), out=o)
            dg.gemm_fused(A, B, C, activation="gelu", Z=Z, splits=(1, 0, 3)[i % 3], **kw)
            same_rows(C, want["C"], None, M)
            same_rows(Z, want["Z"], None, M)
            want = layer_ref.act_grad(np64(A), np64(B), np64(Z), transB=transB, R=np64(R), out=o)
            dg.gemm_act_grad(A, B, Z, C, splits=(0, 2, 1)[i % 3], **kw)
            same_rows(C, want["C"], None, M)
            # groups, a matrix each (rows of odd length: every other matrix is aligned otherwise)
            offsets = [M // 9, M // 3, M // 3, M // 2 + 1, M - M // 8]
            rows = B.shape[0]
            W = placed(rng, 4 * rows, B.shape[1], t, odd_b, 0.1)
            W3 = W.as_strided((4, rows, B.shape[1]), (rows * W.stride(0), W.stride(0), 1), W.storage_offset())
            off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
            C, H = output(M, N, o), output(M, N, o)
            want = layer_ref.act_grad(np64(A), np64(W3), np64(Z), offsets, transB=transB, R=np64(R), out=o)
            dg.gemm_grouped_act_grad(A, W3, off, Z, C, H=H, **kw)
            same_rows(C, want["C"], offsets, M)
            same_rows(H, want["H"], offsets, M)
            C = output(M, N, o)
            dg.gemm_grouped(A, W3, off, C, **kw)
            same_rows(C, layer_ref.forward(np64(A), np64(W3), offsets, transB=transB, R=np64(R), out=o)["C"], offsets, M)
            if transB:
                continue
            X, Y = placed(rng, M, N, t, odd_a), placed(rng, M, K, t, odd_b)
            for off3, splits in ((None, (1, 3, 0)[i % 3]), (off, (2, 1, 0)[i % 3])):
                G = 1 if off3 is None else 4
                d = torch.empty((N,) if off3 is None else (G, N), device=DEV)
                want = layer_ref.dw(np64(X), np64(Y), None if off3 is None else offsets, out=o)
                check(dg.gemm_dw(X, Y, offsets=off3, dbias=d, splits=splits, out_dtype=o, kernel=kernel), want["C"])
                check(d, want["dbias"])
    torch.cuda.synchronize()


@pytest.mark.parametrize("ty,out", PAIRS + [("f32", "f32")])
@pytest.mark.parametrize("kernel", dg.layer_kernel_names())
def test_every_kernel_runs(kernel, ty, out):
    """Forced on aligned operands of whole tiles, a kernel runs every operator but those it does not know:
    no 256 tile and no deep 128 tile in fp32, no weights with few rows, no stream over a B stored K x N."""
    k, t, o = dg.layer_kernel_names().index(kernel), T[ty], T[out]
    never = ty == "f32" and kernel in ("layer_256x256", "layer_128x128_deep")
    rows, stream = "rows" in kernel, "stream" in kernel
    A, B = torch.randn(64, 256, device=DEV).to(t), (torch.randn(64, 256, device=DEV) / 16).to(t)
    W, Z = B.t().contiguous(), torch.randn(64, 64, device=DEV).to(o)
    off = torch.tensor([0, 20, 64], dtype=torch.int32, device=DEV)
    for splits in (1, 2):
        calls = {"fused nt": lambda: dg.gemm_fused(A, B, transB=True, out_dtype=o, splits=splits, kernel=k),
                 "fused nn": lambda: dg.gemm_fused(A, W, out_dtype=o, splits=splits, kernel=k),
                 "grad nt": lambda: dg.gemm_act_grad(A, B, Z, transB=True, splits=splits, kernel=k),
                 "grad nn": lambda: dg.gemm_act_grad(A, W, Z, splits=splits, kernel=k),
                 "dw": lambda: dg.gemm_dw(A, B, out_dtype=o, splits=splits, kernel=k),
                 "grouped nt": lambda: dg.gemm_grouped(A, B.expand(2, 64, 256), off, transB=True, out_dtype=o, kernel=k),
                 "grouped nn": lambda: dg.gemm_grouped(A, W.expand(2, 256, 64), off, out_dtype=o, kernel=k),
                 "grouped dw": lambda: dg.gemm_dw(A, B, offsets=off, out_dtype=o, splits=splits, kernel=k)}
        for name, call in calls.items():
            if never or (rows and "dw" in name) or (stream and "nn" in name):
                with pytest.raises(dg.LayerError) as e:
                    call()
                assert e.value.status == dg.DG_ERR_UNSUPPORTED
                continue
            got = call()
            if "grad" in name:
                want = layer_ref.act_grad(np64(A), np64(B), np64(Z), transB=True, out=o)["C"]
            elif "dw" in name:
                want = layer_ref.dw(np64(A), np64(B), off.tolist() if "grouped" in name else None, out=o)["C"]
            else:
                want = layer_ref.forward(np64(A), np64(B), transB=True, out=o)["C"]
            check(got, want, name)
    torch.cuda.synchronize()


# ---- few rows over long sums ------------------------------------------------------------------------
@pytest.mark.parametrize("ty,out", PAIRS + [("f32", "f32")])
@pytest.mark.parametrize("K", [2048, 4352, 5632, 6170])
def test_streamed_rows_over_many_chunks(K, ty, out):
    """Weights through LDS, several 512-byte chunks a wave (K = 4352: waves with two and with three of them in
    16 bits; 6170: a last step that is not whole), with up to four rows and with more."""
    t, o = T[ty], T[out]
    stream = dg.layer_kernel_names().index("layer_16_rows_stream")
    rng = np.random.default_rng(K)
    r = lambda a, b, d, s=1.0: torch.from_numpy(rng.standard_normal((a, b)) * s).to(d).to(DEV)  # noqa: E731
    N = 40
    B, bias = r(N, K, t, K ** -0.5), r(1, N, o)[0]
    W = r(3 * N, K, t, K ** -0.5).view(3, N, K)
    for M in (1, 2, 4, 5, 15, 16, 24):
        A, R, Z = r(M, K + 2, t)[:, :K], r(M, N, o), r(M, N, o)
        off = torch.tensor([0, M // 3, M // 3, M], dtype=torch.int32, device=DEV)
        for kernel in (stream, -1):
            keep = torch.empty(M, N, dtype=o, device=DEV)
            want = layer_ref.forward(np64(A), np64(B), transB=True, bias=np64(bias), activation="gelu", R=np64(R), out=o)
            check(dg.gemm_fused(A, B, transB=True, bias=bias, activation="gelu", R=R, Z=keep, out_dtype=o, kernel=kernel), want["C"], (M, kernel))
            check(keep, want["Z"])
            want = layer_ref.act_grad(np64(A), np64(B), np64(Z), transB=True, activation="relu", out=o)
            check(dg.gemm_act_grad(A, B, Z, transB=True, activation="relu", kernel=kernel), want["C"])
            want = layer_ref.forward(np64(A), np64(W), off.tolist(), transB=True, R=np64(R), beta=0.5, out=o)
            check(dg.gemm_grouped(A, W, off, transB=True, R=R, beta=0.5, out_dtype=o, kernel=kernel), want["C"])
        want = layer_ref.forward(np64(A), np64(B), transB=True, out=o)["C"]
        for splits in (2, 3):
            check(dg.gemm_fused(A, B, transB=True, out_dtype=o, splits=splits, kernel=stream), want, splits)
    torch.cuda.synchronize()


# ---- weight gradients of long groups, the longest first --------------------------------------------------
ORDERS = {
    "ascending": [500, 1000, 1500, 2000, 2500], "descending": [2500, 2000, 1500, 1000, 500], "one first behind": [900, 900, 900, 4000],
    "equal": [1024] * 6, "ties and none": [0, 2100, 700, 2100, 0, 700, 2100], "all in one": [0, 0, 5000, 0], "two": [1000, 1300],
    "sixty-four": [(97 * i * i) % 2077 + 200 * (i % 3) for i in range(64)], "sixty-five": [(97 * i * i) % 2077 + 200 * (i % 3) for i in range(65)],
    "one row more": [1024, 1025, 1024, 1025],
}


@pytest.mark.parametrize("ty,out", [("f16", "f16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("name", list(ORDERS))
def test_dw_in_order_of_length(name, ty, out):
    """Groups of 1024 rows and more on average, up to 64 of them, go longest first: every order, ties, groups
    without rows, rows of no group, on every kernel, in one range and more."""
    sizes, t, o = ORDERS[name], T[ty], T[out]
    head, tail = (3, 70) if name in ("ascending", "equal") else (0, 0)
    offsets = [head + sum(sizes[:i]) for i in range(len(sizes) + 1)]
    rows, G, M, N = offsets[-1] + tail, len(sizes), 72, 40
    assert rows >= 1024 * G and (G <= 64) == (name != "sixty-five")
    rng = np.random.default_rng(len(name))
    X, Y = (torch.from_numpy(rng.standard_normal((rows, n))).to(t).to(DEV) for n in (M, N))
    X[:head], X[rows - tail:] = float("nan"), float("nan")
    C0, d0 = torch.randn(G, M, N, device=DEV).to(o), torch.randn(G, M, device=DEV)
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    want = layer_ref.dw(np64(X), np64(Y), offsets, beta=0.5, C=np64(C0), dbias=np64(d0), out=o)
    for k, kernel in [(-1, "auto")] + list(enumerate(dg.layer_kernel_names())):
        if "rows" in kernel or (ty == "f32" and kernel in ("layer_256x256", "layer_128x128_deep")):
            continue
        for splits in (0, 1, 3):
            C, d = C0.clone(), d0.clone()
            dg.gemm_dw(X, Y, C, offsets=off, beta=0.5, dbias=d, splits=splits, kernel=k)
            check(C, want["C"], (kernel, splits))
            check(d, want["dbias"], (kernel, splits))
    torch.cuda.synchronize()


# ---- rounding of long fp32 sums -----------------------------------------------------------------------
@pytest.mark.parametrize("kernel", [k for k in dg.layer_kernel_names() if k not in ("layer_256x256", "layer_128x128_deep")])
def test_long_fp32_sums(kernel):
    """fp32 sums go in chains of 1024 products at the most, and their sums in another, in every kernel.

    The bound, by norm, for products that are random with mean zero: after j of them a chain holds sqrt(j) of their
    size, and a rounding adds an error of at most 2^-24 / sqrt(3) of that by root mean square (uniform within half a
    step, the step at most 2^-23 of the value). Over a chain of L: sqrt(L / 2) 2^-24 / sqrt(3) of the sum, over n chains'
    sums sqrt(n / 2) more of it, and a rounding or two behind. A single chain of 8192 has 1.6e-6 to 2.2e-6, this bound 9.6e-7."""
    k, K, M, N = dg.layer_kernel_names().index(kernel), 8192, 130, 72
    rms = 2.0 ** -24 / 3 ** 0.5
    bound = ((1024 / 2) ** 0.5 + (K / 1024 / 2) ** 0.5 + 3) * rms
    g = torch.Generator(device=DEV).manual_seed(1)
    r = lambda a, b: torch.randn(a, b, generator=g, device=DEV)  # noqa: E731
    far = lambda got, want: float((got.double() - want).norm() / want.norm())  # noqa: E731
    A, W, X = r(M, K), r(N, K), r(K, M)
    want = A.double() @ W.double().t()
    assert far(dg.gemm_fused(A, W, transB=True, kernel=k, splits=1), want) < bound
    if "stream" not in kernel:
        assert far(dg.gemm_fused(A, W.t().contiguous(), kernel=k, splits=1), want) < bound
    if "rows" not in kernel:
        Y = r(K, N)
        assert far(dg.gemm_dw(X, Y, kernel=k, splits=1), X.double().t() @ Y.double()) < bound
