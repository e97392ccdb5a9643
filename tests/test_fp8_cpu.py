"""The 8-bit head's entry points refuse bad arguments before any device work
(no GPU here: the pointers are never followed)."""
import ctypes

import pytest

from packed_quantized_lm_amd import binding

B, ODD = ctypes.c_void_p(4096), ctypes.c_void_p(4104)


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


def _quant(lib, rows=4, cols=64, x=B, type=0, ldx=64, br=1, q=B, ldq=64, s=B, lds=4):
    return lib.archead_fp8_quantize(rows, cols, x, type, ldx, br, q, ldq, s, lds, None)


@pytest.mark.parametrize("over,status", [
    (dict(rows=-1), binding.EINVAL), (dict(rows=1 << 31), binding.ESHAPE), (dict(cols=24), binding.ESHAPE),
    (dict(cols=0), binding.ESHAPE), (dict(cols=(1 << 20) + 16), binding.ESHAPE),
    (dict(rows=(1 << 31) - 1, cols=1 << 20, ldx=1 << 20, ldq=1 << 20, lds=1 << 31), binding.ESHAPE),
    (dict(rows=1 << 28, lds=1 << 28), binding.ESHAPE), (dict(rows=1 << 21, br=128, cols=1 << 14, ldx=1 << 14, ldq=1 << 14), binding.ESHAPE),
    (dict(type=2), binding.EINVAL), (dict(br=64), binding.EINVAL), (dict(ldx=63), binding.EINVAL),
    (dict(lds=3), binding.EINVAL), (dict(br=128, lds=0), binding.EINVAL), (dict(x=None), binding.EINVAL),
    (dict(q=None), binding.EINVAL), (dict(s=None), binding.EINVAL), (dict(q=ODD), binding.EINVAL),
    (dict(ldq=72), binding.EINVAL), (dict(ldq=48), binding.EINVAL), (dict(x=ctypes.c_void_p(4098)), binding.EINVAL)])
def test_quantize_refusals(lib, over, status):
    assert _quant(lib, **over) == status
    assert lib.archead_last_error().decode()


def _mm(lib, M=4, N=8, K=64, a=B, lda=64, sa=B, ldsa=4, b=B, ldb=64, sb=B, ldsb=1, out=B, type=0, ldo=8):
    return lib.archead_fp8_matmul(M, N, K, a, lda, sa, ldsa, b, ldb, sb, ldsb, out, type, ldo, None)


@pytest.mark.parametrize("over,status", [
    (dict(M=-1), binding.EINVAL), (dict(N=-1), binding.EINVAL), (dict(M=(1 << 20) + 1), binding.ESHAPE),
    (dict(N=1 << 31), binding.ESHAPE), (dict(K=0), binding.ESHAPE), (dict(K=24), binding.ESHAPE),
    (dict(N=(1 << 30) + 1, ldo=1 << 31), binding.ESHAPE),
    (dict(M=1 << 20, N=(1 << 16) + 1, ldsa=1 << 20, ldo=1 << 17), binding.ESHAPE),
    (dict(type=7), binding.EINVAL), (dict(ldsa=3), binding.EINVAL), (dict(ldsb=0), binding.EINVAL),
    (dict(ldo=7), binding.EINVAL), (dict(a=None), binding.EINVAL), (dict(sa=None), binding.EINVAL),
    (dict(b=None), binding.EINVAL), (dict(sb=None), binding.EINVAL), (dict(out=None), binding.EINVAL),
    (dict(a=ODD), binding.EINVAL), (dict(b=ODD), binding.EINVAL), (dict(lda=72), binding.EINVAL),
    (dict(ldb=48), binding.EINVAL), (dict(lda=1 << 23), binding.ESHAPE), (dict(ldb=1 << 23), binding.ESHAPE),
    (dict(out=ctypes.c_void_p(4098)), binding.EINVAL)])
def test_matmul_refusals(lib, over, status):
    assert _mm(lib, **over) == status
    assert lib.archead_last_error().decode()


def test_empty_calls_succeed(lib):
    assert _quant(lib, rows=0, x=None, q=None, s=None) == binding.OK
    assert _mm(lib, M=0, a=None, out=None) == binding.OK
    assert _mm(lib, N=0, b=None, out=None) == binding.OK
