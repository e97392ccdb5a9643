"""The 8-bit quantiser's largest sizes: what a launch cannot hold is refused
before any device work (no GPU here: the pointers are never followed)."""
import ctypes

import pytest

from packed_quantized_lm_amd import binding

B = ctypes.c_void_p(4096)
MOST = (1 << 28) - 16  # row blocks: (2^24 - 1) workgroups of 256 threads, 16 lanes a block


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


def quant(lib, rows, cols, block_rows, x=B):
    return lib.archead_fp8_quantize(rows, cols, x, 0, cols, block_rows, B, cols, B, max(rows, 1 << 14), None)


@pytest.mark.parametrize("rows,cols", [(MOST + 1, 16), (MOST + 15, 128), ((1 << 28) - 1, 16), (MOST // 16 + 1, 2048)])
def test_row_blocks_beyond_a_launch_are_refused(lib, rows, cols):
    groups = -(-rows * -(-cols // 128) // 16)
    assert groups * 256 >= 1 << 32
    assert quant(lib, rows, cols, 1) == binding.ESHAPE
    assert b"2^28" in lib.archead_last_error()


@pytest.mark.parametrize("rows,cols,block_rows", [(MOST, 16, 1), (MOST // 16, 2048, 1), ((1 << 28) - 1, 16, 128)])
def test_the_largest_sizes_pass_the_check(lib, rows, cols, block_rows):
    """Refused for the missing matrix, behind the check of sizes."""
    assert quant(lib, rows, cols, block_rows, x=None) == binding.EINVAL
    assert b"required" in lib.archead_last_error()
