"""The choice of kernel and K ranges for a layer's products, on the CPU (nothing here reaches a
GPU: the queries only compute)."""
import random

import dense_gemm_amd as dg


def test_ranges_do_not_change_a_grouped_choice():
    """Groups of rows always have one range: asking for more leaves the kernel the one of one range."""
    rng = random.Random(0)
    for _ in range(3000):
        shape = rng.randint(1, 4000), rng.randint(16, 6000), rng.randint(16, 6000), rng.randrange(2), rng.randrange(5), rng.randint(1, 64)
        want = dg.dg_gemm_fused_select(*shape, 1)
        for splits in (0, 2, 8, 4096):
            assert dg.dg_gemm_fused_select(*shape, splits) == want, (shape, splits)
