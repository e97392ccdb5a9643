"""archead_backward and archead_reserve_backward refuse bad handles before any
device work (every other refusal needs a loaded head, on the GPU)."""
import ctypes

import pytest

from packed_quantized_lm_amd import binding

B = ctypes.c_void_p(4096)


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


def test_bad_handles(lib):
    for h in (None, ctypes.c_void_p(0x1234560)):
        assert lib.archead_reserve_backward(h, 4, None) == binding.EINVAL
        assert lib.archead_backward(h, 1, B, 1, 8, B, None) == binding.EINVAL
        assert b"handle" in lib.archead_last_error()
