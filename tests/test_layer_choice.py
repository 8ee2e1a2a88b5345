"""The choice of kernel and K ranges for a layer's products, on the CPU (nothing here reaches a
GPU: the queries only compute)."""
import random

import pytest
import torch

import dense_gemm_amd as dg


def test_ranges_do_not_change_a_grouped_choice():
    """Groups of rows always have one range: asking for more leaves the kernel the one of one range."""
    rng = random.Random(0)
    for _ in range(3000):
        shape = rng.randint(1, 4000), rng.randint(16, 6000), rng.randint(16, 6000), rng.randrange(2), rng.randrange(5), rng.randint(1, 64)
        want = dg.dg_gemm_fused_select(*shape, 1)
        for splits in (0, 2, 8, 4096):
            assert dg.dg_gemm_fused_select(*shape, splits) == want, (shape, splits)


def test_choice_for_operands():
    """The query for given operands: as the one for aligned ones where they are aligned, another where not;
    the rows' distance and the address count."""
    rng, other = random.Random(1), 0
    for _ in range(3000):
        M, N, K, tb, dtype = rng.randint(1, 600), rng.randint(16, 6000), rng.randint(16, 6000), rng.randrange(2), rng.randrange(5)
        lda, ldb = -(-K // 2) * 2, -(-(K if tb else N) // 2) * 2
        n = dg.dg_gemm_fused_choose(M, N, K, tb, dtype)
        assert dg.dg_gemm_fused_choose_for(M, N, K, tb, dtype, 256, lda, 256, ldb) == n
        odd = dg.dg_gemm_fused_choose_for(M, N, K, tb, dtype, 258, lda, 256, ldb)
        assert 1 <= odd <= 16 and (dtype or odd == dg.dg_gemm_fused_choose_for(M, N, K, tb, dtype, 258, lda, 256, ldb))
        assert odd == dg.dg_gemm_fused_choose_for(M, N, K, tb, dtype, 256, 1 << 23, 256, ldb)
        if dtype:
            assert odd == dg.dg_gemm_fused_choose_for(M, N, K, tb, dtype, 256, lda + 1, 256, ldb)
        other += odd != n
        groups = rng.randint(1, 40)
        n = dg.dg_gemm_dw_choose(groups, K, M, N, dtype)
        assert dg.dg_gemm_dw_choose_for(groups, K, M, N, dtype, 0, M + M % 2, 4, N + N % 2) == n
        assert 1 <= dg.dg_gemm_dw_choose_for(groups, K, M, N, dtype, 0, M + M % 2, 2, N + N % 2) <= 16
    assert other > 100
    assert dg.dg_gemm_fused_choose_for(-1, 1, 1, 0, 0, 0, 1, 0, 1) == -1 and dg.dg_gemm_fused_choose_for(1, 1, 1, 0, 9, 0, 1, 0, 1) == -5
    assert dg.dg_gemm_fused_choose_for(1, 1, 1, 0, 0, 0, -1, 0, 1) == -7 and dg.dg_gemm_fused_choose_for(1, 1, 1, 0, 0, 0, 1, 0, -1) == -9
    assert dg.dg_gemm_dw_choose_for(70000, 1, 1, 1, 0, 0, 1, 0, 1) == -1 and dg.dg_gemm_dw_choose_for(1, 1, 1, 1, 0, 0, 1, 0, -1) == -9
    assert dg.dg_gemm_fused_choose_for(2 ** 31 - 1, 1, 8, 0, 1, 0, 8, 0, 1) == dg.DG_ERR_UNSUPPORTED


@pytest.mark.parametrize("shift,pad", [(0, 0), (1, 0), (0, 1), (1, 1)])
def test_binding_takes_the_choice_of_its_operands(monkeypatch, shift, pad):
    """For splits = 0 the torch functions leave the choice to the library, beside a workspace that holds the
    ranges that it makes of the operands given, or without one pass one range.  A caller's workspace is
    passed as it is."""
    calls = []
    monkeypatch.setattr(dg.layer, "_stream_of", lambda stream, tensors: (0, None))
    monkeypatch.setattr(dg.layer, "_run", lambda function, index, args: calls.append(dict(zip(dg.layer._SIGNATURES[function][2].split(), args))))

    def matrix(rows, cols):
        whole = torch.zeros(rows * (cols + pad) + shift, dtype=torch.float16)
        return whole[shift:].view(rows, cols + pad)[:, :cols]

    ws, changed = torch.zeros(1 << 16, dtype=torch.uint8), False

    def passes(f, want, aligned, size):
        nonlocal changed
        f()
        c = calls.pop()
        assert (c["splits"], c["workspace_bytes"]) == ((0, dg.dg_layer_workspace_size(*size, want)) if want > 1 else (1, 0))
        f(workspace=ws)
        c = calls.pop()
        assert (c["splits"], c["workspace_bytes"]) == (0, 1 << 16)
        for splits in (1, 2):
            f(splits=splits)
            c = calls.pop()
            assert (c["splits"], c["workspace_bytes"]) == (splits, dg.dg_layer_workspace_size(*size, splits))
        changed |= want != aligned

    for M, N, K in ((512, 1032, 5632), (24, 2048, 5632), (64, 2048, 5632), (100, 300, 2048), (2, 2048, 5632)):
        for transB in (False, True):
            A, B, Z = matrix(M, K), matrix(N, K) if transB else matrix(K, N), torch.zeros(M, N, dtype=torch.float16)
            want = dg.dg_gemm_fused_choose_for(M, N, K, transB, 1, A.data_ptr(), A.stride(0), B.data_ptr(), B.stride(0))
            aligned = dg.dg_gemm_fused_choose(M, N, K, transB, 1)
            passes(lambda **kw: dg.gemm_fused(A, B, transB=transB, **kw), want, aligned, (1, M, N))
            passes(lambda **kw: dg.gemm_act_grad(A, B, Z, transB=transB, **kw), want, aligned, (1, M, N))
        X, Y = matrix(K, M), matrix(K, N)
        want = dg.dg_gemm_dw_choose_for(1, K, M, N, 1, X.data_ptr(), X.stride(0), Y.data_ptr(), Y.stride(0))
        passes(lambda **kw: dg.gemm_dw(X, Y, **kw), want, dg.dg_gemm_dw_choose(1, K, M, N, 1), (1, M, N))
    assert changed == bool(shift or pad)
