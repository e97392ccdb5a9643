"""The embedding gradient's last launch takes a workgroup of 256 threads for every four of
n ceil(d / 512) waves, and a launch holds fewer than 2^32 threads: more than 2^26 - 4 waves
are refused, before any device work."""
import ctypes

import pytest

from packed_quantized_lm_amd import binding

AT = [ctypes.c_void_p(1 << (40 + i)) for i in range(4)]


def _grad(n, d):
    return binding.load_library().archead_embed_backward(n, 8, d, AT[0], 1, d, AT[1], -1, 1.0, 0, AT[2], 1, d, AT[3], 0, None)


@pytest.mark.parametrize("n,tiles", [(111662, 601), (1 << 16, 1 << 10), (1 << 20, 64)])  # 2^26 - 2, 2^26, 2^26
def test_too_many(n, tiles):
    assert n * tiles > (1 << 26) - 4
    assert _grad(n, 512 * tiles) == binding.ESHAPE


@pytest.mark.parametrize("n,tiles", [(932067, 72), (111661, 601), ((1 << 20) - 1, 64)])
def test_the_most(n, tiles):
    assert (1 << 26) - 4 - 700 <= n * tiles <= (1 << 26) - 4
    assert _grad(n, 512 * tiles) == binding.EINVAL  # its workspace of no bytes is refused, its size is not
