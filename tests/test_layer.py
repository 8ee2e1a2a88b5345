"""A layer's products on the CPU: argument checks of the C ABI, in position order,
and of the torch functions, none of which reaches a GPU; the reference of the GPU
tests against differences."""
import numpy as np
import pytest
import torch

import dense_gemm_amd as dg
import layer_ref

P = 1 << 20      # an address that is aligned and never read: every call here is refused or has nothing to do

FUSED = dict(transB=0, groups=1, offsets=None, M=8, N=16, K=32, alpha=1.0, A=P, lda=32, B=P, ldb=16, strideB=0, bias=P,
             strideBias=0, epilogue=2, Z=P, ldz=16, beta=1.0, R=P, ldr=16, C=P, ldc=16, dtype=1, splits=1, workspace=None,
             workspace_bytes=0, stream=None, kernel=-1)
GRAD = dict(transB=0, groups=1, offsets=None, M=8, N=16, K=32, alpha=1.0, A=P, lda=32, B=P, ldb=16, strideB=0, beta=1.0, R=P,
            ldr=16, H=P, ldh=16, activation=2, Z=P, ldz=16, C=P, ldc=16, dtype=1, splits=1, workspace=None,
            workspace_bytes=0, stream=None, kernel=-1)
DW = dict(groups=1, offsets=None, rows=8, M=16, N=32, alpha=1.0, A=P, lda=16, B=P, ldb=32, beta=0.0, C=P, ldc=32, strideC=0,
          dbias=P, dtype=1, splits=1, workspace=None, workspace_bytes=0, stream=None, kernel=-1)
BIG = 2 ** 31


def bad(base, changes, name):
    """(changed arguments, position of the argument that is refused)"""
    return changes, -(list(base).index(name) + 1)


COMMON = [({"transB": 2}, "transB"), ({"groups": -1}, "groups"), ({"groups": 2}, "groups"), ({"groups": 65536, "offsets": P}, "groups"),
          ({"offsets": P + 2}, "offsets"), ({"M": -1}, "M"), ({"M": BIG}, "M"), ({"N": -1}, "N"), ({"N": BIG}, "N"),
          ({"K": -1}, "K"), ({"K": BIG}, "K"), ({"A": None}, "A"), ({"A": P + 1}, "A"), ({"lda": 31}, "lda"), ({"B": None}, "B"),
          ({"B": P + 1}, "B"), ({"ldb": 15}, "ldb"), ({"transB": 1, "ldb": 31}, "ldb"), ({"strideB": -1}, "strideB"),
          ({"R": P + 1}, "R"), ({"ldr": 15}, "ldr"), ({"C": None}, "C"), ({"C": P + 1}, "C"), ({"C": P + 2, "dtype": 3, "bias": P, "R": None, "Z": P, "H": None}, "C"),
          ({"ldc": 15}, "ldc"), ({"dtype": 5}, "dtype"), ({"dtype": -1}, "dtype"), ({"splits": -1}, "splits"),
          ({"splits": 4097}, "splits"), ({"splits": 2}, "workspace"), ({"splits": 2, "workspace": P + 8}, "workspace"),
          ({"splits": 2, "workspace": P, "workspace_bytes": 2 * 8 * 17 * 4 - 1}, "workspace_bytes")]


@pytest.mark.parametrize("changes,name", COMMON + [
    ({"bias": P + 1}, "bias"), ({"strideBias": -1}, "strideBias"), ({"epilogue": 3}, "epilogue"), ({"epilogue": 4}, "epilogue"),
    ({"Z": P + 1}, "Z"), ({"ldz": 15}, "ldz")])
def test_fused_refusals(changes, name):
    args = {**FUSED, **{k: v for k, v in changes.items() if k in FUSED}}
    assert dg.dg_gemm_fused_with_kernel(*args.values()) == -(list(FUSED).index(name) + 1)
    del args["kernel"]
    assert dg.dg_gemm_fused(*args.values()) == -(list(FUSED).index(name) + 1)


@pytest.mark.parametrize("changes,name", COMMON + [
    ({"activation": 0}, "activation"), ({"activation": 4}, "activation"), ({"H": P + 1}, "H"), ({"ldh": 15}, "ldh"),
    ({"Z": None}, "Z"), ({"Z": P + 1}, "Z"), ({"ldz": 15}, "ldz")])
def test_act_grad_refusals(changes, name):
    args = {**GRAD, **{k: v for k, v in changes.items() if k in GRAD}}
    assert dg.dg_gemm_act_grad_with_kernel(*args.values()) == -(list(GRAD).index(name) + 1)
    del args["kernel"]
    assert dg.dg_gemm_act_grad(*args.values()) == -(list(GRAD).index(name) + 1)


@pytest.mark.parametrize("changes,name", [
    ({"groups": -1}, "groups"), ({"groups": 2}, "groups"), ({"groups": 65536, "offsets": P}, "groups"), ({"offsets": P + 1}, "offsets"),
    ({"rows": -1}, "rows"), ({"rows": BIG}, "rows"), ({"M": -1}, "M"), ({"N": BIG}, "N"), ({"A": None}, "A"), ({"A": P + 1}, "A"),
    ({"lda": 15}, "lda"), ({"B": None}, "B"), ({"B": P + 1}, "B"), ({"ldb": 31}, "ldb"), ({"C": None}, "C"), ({"C": P + 1}, "C"),
    ({"ldc": 31}, "ldc"), ({"strideC": -1}, "strideC"), ({"groups": 2, "offsets": P, "strideC": 511}, "strideC"),
    ({"dbias": P + 2}, "dbias"), ({"dtype": 7}, "dtype"), ({"splits": 5000}, "splits"), ({"splits": 2}, "workspace"),
    ({"splits": 2, "workspace": P, "workspace_bytes": 2 * 16 * 33 * 4 - 1}, "workspace_bytes"),
    ({"alpha": 0.0, "B": None, "A": None}, "A")])
def test_dw_refusals(changes, name):
    args = {**DW, **changes}
    assert dg.dg_gemm_dw_with_kernel(*args.values()) == -(list(DW).index(name) + 1)
    del args["kernel"]
    assert dg.dg_gemm_dw(*args.values()) == -(list(DW).index(name) + 1)


def test_nothing_to_do_needs_no_gpu():
    for change in ({"M": 0}, {"N": 0}, {"groups": 0, "offsets": P}):
        assert dg.dg_gemm_fused_with_kernel(*{**FUSED, **change, "A": None, "B": None, "C": None}.values()) == dg.DG_OK
        assert dg.dg_gemm_act_grad_with_kernel(*{**GRAD, **change, "A": None, "B": None, "C": None, "Z": None}.values()) == dg.DG_OK
    for change in ({"M": 0}, {"groups": 0, "offsets": P}, {"N": 0, "dbias": None}):
        assert dg.dg_gemm_dw_with_kernel(*{**DW, **change, "A": None, "B": None, "C": None}.values()) == dg.DG_OK


def test_too_large_is_unsupported():
    u = dg.DG_ERR_UNSUPPORTED
    assert dg.dg_gemm_fused_with_kernel(*{**FUSED, "M": BIG - 1, "bias": None}.values()) == u
    assert dg.dg_gemm_fused_with_kernel(*{**FUSED, "M": 1 << 30, "N": 1 << 30, "ldb": 1 << 30, "ldc": 1 << 30, "ldz": 1 << 30, "ldr": 1 << 30}.values()) == u
    assert dg.dg_gemm_dw_with_kernel(*{**DW, "rows": BIG - 1}.values()) == u
    assert dg.dg_gemm_fused_with_kernel(*{**FUSED, "kernel": 1000}.values()) == u
    assert dg.dg_gemm_dw_with_kernel(*{**DW, "kernel": -2}.values()) == u


def test_choice_of_a_refused_shape():
    """The library's choice of ranges never hides why a call is refused."""
    huge = 2 ** 31 - 1
    assert dg.dg_gemm_fused_choose(huge, 1, 8, 0, 1) == dg.DG_ERR_UNSUPPORTED
    assert dg.layer._fused_splits(huge, 1, 8, 0, 1) == 1 and dg.layer._dw_splits(1, huge, 8, 8, 1) == 1


def test_select():
    names = dg.layer_kernel_names()
    for dtype in range(5):
        for M in (1, 16, 17, 500, 16384):
            for groups in (0, 1, 8, 300):
                for splits in (0, 1, 4):
                    k = dg.dg_gemm_fused_select(M, 2048, 5632, 1, dtype, groups, splits)
                    assert 0 <= k < len(names) and "any" not in names[k]
                    k = dg.dg_gemm_dw_select(max(groups, 1), M, 512, 300, dtype, splits)
                    assert 0 <= k < len(names) and "rows" not in names[k]
    # one token reads its weights once; many rows go to large tiles (not in fp32: no such tile)
    assert "16_rows" in names[dg.dg_gemm_fused_select(1, 2048, 5632, 1, dg.DG_BF16_F32ACC, 0, 0)]
    assert names[dg.dg_gemm_fused_select(16384, 5632, 2048, 1, dg.DG_BF16_F32ACC, 0, 0)] == "layer_256x256"
    assert dg.dg_gemm_fused_select(1, 1, 1, 0, 0, -1, 0) == -6 and dg.dg_gemm_fused_select(1, 1, 1, 0, 0, 0, 5000) == -7
    assert dg.dg_gemm_dw_select(-1, 1, 1, 1, 0, 0) == -1 and dg.dg_gemm_dw_select(1, 1, 1, 1, 0, -1) == -6


def test_error_names_the_argument():
    e = dg.LayerError("dg_gemm_fused", -13)
    assert "13 (bias)" in str(e) and e.status == -13
    assert "17 (ldh)" in str(dg.LayerError("dg_gemm_act_grad_with_kernel", -17))
    assert "14 (strideC)" in str(dg.LayerError("dg_gemm_dw", -14))
    assert "does not support" in str(dg.LayerError("dg_gemm_dw", dg.DG_ERR_UNSUPPORTED))


def test_kernel_names_and_choices():
    names = dg.layer_kernel_names()
    assert len(names) == len(set(names)) and dg.dg_layer_kernel_name(-1) is None
    assert dg.dg_gemm_fused_choose(-1, 1, 1, 0, 0) == -1 and dg.dg_gemm_fused_choose(1, 1, 1, 2, 0) == -4
    assert dg.dg_gemm_dw_choose(1, 1, 1, 1, 9) == -5 and dg.dg_gemm_dw_choose(70000, 1, 1, 1, 0) == -1
    assert dg.dg_gemm_fused_choose(0, 5, 5, 0, 0) == 1
    for M, N, K in ((1, 16, 16), (64, 2048, 8192), (16384, 5632, 2048)):
        assert 1 <= dg.dg_gemm_fused_choose(M, N, K, 1, 1) <= 4096
        assert 1 <= dg.dg_gemm_dw_choose(4, K, M, N, 1) <= 4096
    assert dg.dg_layer_workspace_size(3, 5, 7, 4) == 3 * 5 * 8 * 4 * 4 and dg.dg_layer_workspace_size(3, 5, 7, 1) == 0


def test_torch_refusals():
    f = lambda *s, dtype=torch.float16: torch.zeros(*s, dtype=dtype)  # noqa: E731
    A, B, off = f(4, 8), f(8, 6), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="inner dimensions"):
        dg.gemm_fused(A, f(7, 6))
    with pytest.raises(TypeError, match="share one dtype"):
        dg.gemm_fused(A, B.float())
    with pytest.raises(TypeError, match="unsupported"):
        dg.gemm_fused(A, B, f(4, 6, dtype=torch.bfloat16))
    with pytest.raises(TypeError, match="bias"):
        dg.gemm_fused(A, B, bias=f(6, dtype=torch.float32))
    with pytest.raises(ValueError, match="bias"):
        dg.gemm_fused(A, B, bias=f(5))
    with pytest.raises(ValueError, match="activation"):
        dg.gemm_fused(A, B, activation="silu")
    with pytest.raises(ValueError, match="activation"):
        dg.gemm_act_grad(A, B, f(4, 6), activation="none")
    with pytest.raises(ValueError, match="R must be"):
        dg.gemm_fused(A, B, R=f(4, 5))
    with pytest.raises(TypeError, match="Z must have C's dtype"):
        dg.gemm_fused(A, B, Z=f(4, 6, dtype=torch.float32))
    with pytest.raises(ValueError, match="unit column stride"):
        dg.gemm_fused(f(8, 4).t(), B)
    with pytest.raises(ValueError, match="overlapping rows"):
        dg.gemm_fused(A, B, C=f(6).expand(4, 6))
    with pytest.raises(ValueError, match="3-D"):
        dg.gemm_grouped(A, B, off)
    with pytest.raises(ValueError, match=r"B must be \[2, 8, 6\]"):
        dg.gemm_grouped(A, f(3, 8, 6), off)
    with pytest.raises(TypeError, match="int32"):
        dg.gemm_grouped(A, f(2, 8, 6), off.long())
    with pytest.raises(ValueError, match="offsets"):
        dg.gemm_grouped(A, f(2, 8, 6), torch.zeros(6, dtype=torch.int32)[::2])
    with pytest.raises(ValueError, match="bias must be"):
        dg.gemm_grouped(A, f(2, 8, 6), off, bias=f(6))
    with pytest.raises(ValueError, match="differ in rows"):
        dg.gemm_dw(A, f(5, 6))
    with pytest.raises(ValueError, match="beta"):
        dg.gemm_dw(A, f(4, 6), beta=1.0)
    with pytest.raises(ValueError, match="C must be"):
        dg.gemm_dw(A, f(4, 6), f(8, 6), offsets=off)
    with pytest.raises(ValueError, match="dbias"):
        dg.gemm_dw(A, f(4, 6), dbias=f(8))
    with pytest.raises(ValueError, match="on a GPU"):
        dg.gemm_fused(A, B)
    with pytest.raises(ValueError, match="contiguous"):
        dg.gemm_fused(A, B, splits=2, workspace=torch.zeros(64, 2, dtype=torch.uint8)[:, 0])


def test_reference_gradients_against_differences():
    """layer_ref's act_grad and dw are the gradients of its forward: central differences of
    sum(V * C) in 64 bits, over two grouped layers with a residual."""
    rng = np.random.default_rng(5)
    off, M, K, N = [0, 3, 3, 7], 7, 5, 4
    x, w, b = rng.standard_normal((M, K)), rng.standard_normal((3, K, N)), rng.standard_normal((3, N))
    w2, r, v = rng.standard_normal((3, N, K)), rng.standard_normal((M, K)), rng.standard_normal((M, K))

    def loss(x, w, b, w2):
        f = layer_ref.forward(x, w, off, alpha=0.7, bias=b, activation="gelu")
        return (v * layer_ref.forward(f["C"][0], w2, off, R=r, beta=0.5)["C"][0]).sum()

    z = layer_ref.forward(x, w, off, alpha=0.7, bias=b, activation="gelu")["Z"][0]
    h = layer_ref.act(z, "gelu")
    dz = layer_ref.act_grad(v, w2, z, off, transB=True)["C"][0]
    g2 = layer_ref.dw(h, v, off)["C"][0]
    g1 = layer_ref.dw(dz, x, off, alpha=0.7)
    dw, db = g1["C"][0].transpose(0, 2, 1), g1["dbias"][0]
    dx = layer_ref.product(dz, w, off, True, 0.7)[0]
    for value, grad in ((x, dx), (w, dw), (b, db), (w2, g2)):
        for _ in range(6):
            at = tuple(rng.integers(0, n) for n in value.shape)
            keep, e = value[at], 1e-5
            value[at] = keep + e
            up = loss(x, w, b, w2)
            value[at] = keep - e
            down = loss(x, w, b, w2)
            value[at] = keep
            assert abs((up - down) / (2 * e) - grad[at]) < 1e-8 * max(1, abs(grad[at]))
