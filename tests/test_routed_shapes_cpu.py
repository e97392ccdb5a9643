"""The shapes that the GPU tests take for sorted histories are sorted, in slices of the
width they are meant to have: told by the workspace, which holds a word a slice and two
bytes a token for them and nothing else where no token is drawn."""
import ctypes

import pytest

import routed_shapes
from packed_quantized_lm_amd import binding


def _bytes(M, V, L, K=0):
    n = ctypes.c_uint64()
    assert binding.load_library().archead_rules_workspace(M, V, L, K, ctypes.byref(n)) == binding.OK
    return n.value


@pytest.mark.parametrize("M,V,L,B,columns", routed_shapes.SHAPES)
def test_sorted_by_slices(M, V, L, B, columns):
    slices = -(-V // columns)
    assert -(-V // 2048) != -(-V // 4096) or columns == 4096
    assert _bytes(M, V, L) == M * slices * 4 + 2 * M * L
    assert _bytes(M, V, L, 7) == M * slices * (7 * 8 + 4) + 2 * M * L


def test_borders():
    assert _bytes(127, 20000, 7000) == 0 and _bytes(128, 20000, 6553) == 0 and _bytes(128, 20000, 6554) > 0
    assert _bytes(128, 4096 * 1024 + 1, 1000) == 0  # more slices than are counted
