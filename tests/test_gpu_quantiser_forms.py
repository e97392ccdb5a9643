"""The quantiser on either side of its forms' border: bf16 matrices of up to 4096
workgroups of sixteen row blocks (512 of a 128 x 128 block) take exact quotients at
once, larger ones a quick way first.  Codes and scales of the same rows are the same
bits in both, and the oracle's, with blocks that hold true ties, NaN, infinities, zeros
and the ends of the scales' range."""
import numpy as np
import pytest

from oracle import fp8

pytestmark = pytest.mark.gpu


def _rows(rows, cols, seed):
    """bf16 values, as fp32: ordinary blocks, and blocks whose largest is a power of two or 7 of one, so that
    many quotients are exact middles of two codes."""
    import torch
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.normal(0, 1, (rows, cols)).astype(np.float32)).to(torch.bfloat16)
    for r in range(0, rows, 3):
        for b in range(0, cols, 128):
            x[r, b:b + 128] = torch.from_numpy((rng.integers(-112, 113, min(128, cols - b)) / 64).astype(np.float32))
            x[r, b] = 1.75 if (r // 3) % 2 else 2.0
    return x


def _check(codes, scales, x, block_rows):
    import torch
    want_q, want_s = fp8.quantize(x.double().numpy(), block_rows)
    assert np.array_equal(scales.cpu().numpy(), want_s)
    got = codes.view(torch.uint8).cpu().numpy()
    want_q = np.where((want_q & 127) == 0, got & 128 | want_q, want_q)  # the sign of a zero code is free
    assert np.array_equal(got, want_q)


@pytest.mark.parametrize("rows,cols", [(2048, 4096), (65536, 128), (512, 16384), (4096, 2048)])  # 4096 workgroups
def test_rows(rows, cols):
    import torch
    from packed_quantized_lm_amd import fp8_quantize
    some = _rows(96, cols, cols)
    x = some.repeat(-(-(rows + 96) // 96), 1)[:rows + 96].cuda()
    at_once, s1 = fp8_quantize(x[:rows])
    quick, s2 = fp8_quantize(x)
    assert torch.equal(at_once.view(torch.uint8), quick[:rows].view(torch.uint8)) and torch.equal(s1, s2[:, :rows])
    _check(at_once[:96], s1[:, :96].contiguous(), some, 1)


@pytest.mark.parametrize("rows,cols", [(4096, 2048), (65536, 128), (128, 65536)])  # 512 blocks
def test_blocks(rows, cols):
    import torch
    from packed_quantized_lm_amd import fp8_quantize
    some = _rows(128, min(cols, 2048), cols + 1)
    x = some.repeat(rows // 128 + 1, -(-cols // some.shape[1])).cuda()
    at_once, s1 = fp8_quantize(x[:rows], 128)
    quick, s2 = fp8_quantize(x, 128)
    assert torch.equal(at_once.view(torch.uint8), quick[:rows].view(torch.uint8)) and torch.equal(s1, s2[:rows // 128])
    _check(at_once[:128, :256], s1[:1, :2].contiguous(), some[:, :256] if cols > 128 else some, 128)


def test_values_at_the_ends():
    import torch
    from packed_quantized_lm_amd import fp8_quantize
    x = _rows(4200, 2048, 5)
    x[0, 3], x[1, 200], x[2] = float("nan"), float("inf"), 0.0
    x[4] *= 2.0 ** -110
    x[5] *= 2.0 ** 110
    x[6, :128] = 2.0 ** -133
    x[7, 5] = -0.0
    x = x.cuda()
    at_once, s1 = fp8_quantize(x[:4096])
    quick, s2 = fp8_quantize(x)
    assert torch.equal(at_once.view(torch.uint8), quick[:4096].view(torch.uint8))
    assert np.array_equal(s1.cpu().numpy(), s2[:, :4096].cpu().numpy(), equal_nan=True)
