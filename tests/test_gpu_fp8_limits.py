"""The 8-bit quantiser on the GPU at the largest number of row blocks that a
launch holds; its last elements lie just below 2^32."""
import pytest

from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from packed_quantized_lm_amd import load_library
    load_library()


def test_most_row_blocks_of_a_launch():
    import torch
    from packed_quantized_lm_amd import fp8_quantize
    from packed_quantized_lm_amd.binding import ESHAPE, ArcheadError
    rows, n = (1 << 28) - 16, 1000
    say(f"quantise {rows} x 16")
    x = torch.zeros(rows + 1, 16, dtype=torch.bfloat16, device="cuda")
    for at in (0, rows // 2, rows - n):
        x[at:at + n] = torch.randn(n, 16, device="cuda")
    q, s = fp8_quantize(x[:rows])
    for at in (0, rows // 2, rows - n):
        want_q, want_s = fp8_quantize(x[at:at + n].clone())
        assert torch.equal(q[at:at + n].view(torch.uint8), want_q.view(torch.uint8))
        assert torch.equal(s[:, at:at + n], want_s)
    assert int(torch.count_nonzero(s)) == 3 * n
    with pytest.raises(ArcheadError) as e:
        fp8_quantize(x)
    assert e.value.status == ESHAPE
