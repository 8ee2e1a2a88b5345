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
