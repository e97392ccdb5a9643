"""The memory that archead_reserve_backward takes: a workspace as large as the
launches of any call of up to the reserved rows need, and no larger."""
import pytest

import backward_plan
from gpu_util import say
from packed_quantized_lm_amd.synth import random_small_head


def test_the_ranges_sums_of_a_large_head():
    """151936 x 4096 with k = 256, r = 64 and 2048 rows: G takes 622 MB, the
    ranges' sums of the largest plans less than half of that."""
    rows = 2048
    total = backward_plan.workspace_bytes(151936, 4096, 256, 64, rows)
    G = rows * 151936 * 2
    assert G < total < G * 3 / 2


@pytest.mark.gpu
@pytest.mark.parametrize("V,d,k,r,g", [(9001, 640, 40, 20, 32), (16411, 384, 0, 8, 96), (300, 1024, 33, 0, 128)])
def test_reserved_bytes(V, d, k, r, g):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from packed_quantized_lm_amd import PackedHead
    say(f"backward workspace V={V} d={d} k={k} r={r}")
    head = PackedHead(random_small_head(V, d, k, r, g, 1, seed=V))
    held = []
    for rows in (1, 17, 133, 700, 5000):
        head.reserve_backward(rows)
        held.append(head.device_bytes() - backward_plan.workspace_bytes(V, d, k, r, rows))
    head.close()
    assert len(set(held)) == 1, held  # what is left is the head and its second layout
