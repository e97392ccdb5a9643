"""The post-training loss entry points refuse bad arguments before any device
work (no GPU here: the pointers are never followed)."""
import ctypes

import pytest

from packed_quantized_lm_amd import binding

B = ctypes.c_void_p(4096)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


def _logp(lib, M=2, V=8, y=B, type=0, ld=8, t=B, logp=B, lse=B, ws=B, n=BIG):
    return lib.archead_token_logp(M, V, y, type, ld, t, logp, lse, ws, n, None)


@pytest.mark.parametrize("over,status", [
    (dict(M=-1), binding.EINVAL), (dict(M=(1 << 20) + 1), binding.ESHAPE), (dict(V=0), binding.ESHAPE),
    (dict(V=1 << 31, ld=1 << 31), binding.ESHAPE), (dict(type=2), binding.EINVAL), (dict(ld=7), binding.EINVAL),
    (dict(y=None), binding.EINVAL), (dict(t=None), binding.EINVAL), (dict(logp=None, lse=None), binding.EINVAL),
    (dict(ws=None), binding.EINVAL), (dict(ws=ctypes.c_void_p(4100)), binding.EINVAL), (dict(n=8), binding.EINVAL),
    (dict(y=ctypes.c_void_p(4098)), binding.EINVAL)])
def test_token_logp_refusals(lib, over, status):
    assert _logp(lib, **over) == status
    assert lib.archead_last_error().decode()


def _policy(lib, M=2, V=8, y=B, type=0, ld=8, t=B, old=B, ref=B, adv=B, w=B, el=0.2, eh=0.2, beta=0.1, loss=B, dy=B,
            gt=0, ldg=8, ws=B, n=BIG):
    return lib.archead_policy_loss(M, V, y, type, ld, t, old, ref, adv, w, el, eh, beta, None, loss, None, dy, gt, ldg,
                                   ws, n, None)


@pytest.mark.parametrize("over", [
    dict(M=-1), dict(type=5), dict(old=None), dict(ref=None), dict(adv=None), dict(w=None), dict(el=-0.1),
    dict(el=1.1), dict(el=float("nan")), dict(eh=-0.1), dict(eh=float("inf")), dict(beta=-1.0),
    dict(beta=float("nan")), dict(loss=None), dict(gt=3), dict(ldg=7), dict(dy=ctypes.c_void_p(4097), gt=1),
    dict(gt=1), dict(ldg=9), dict(n=16)])  # gt=1, ldg=9: in place (dy == y) with another type or stride
def test_policy_loss_refusals(lib, over):
    assert _policy(lib, **over) == binding.EINVAL
    assert lib.archead_last_error().decode()


def _pref(lib, M=2, V=8, y=B, P=1, off=B, w=B, beta=0.1, sm=0.0, loss=B, dy=None, n=BIG):
    return lib.archead_preference_loss(M, V, y, 0, 8, B, w, P, off, None, beta, sm, None, loss, None, None, dy, 0, 8, B,
                                       n, None)


@pytest.mark.parametrize("over,status", [
    (dict(P=0), binding.EINVAL), (dict(P=(1 << 20) + 1), binding.ESHAPE), (dict(off=None), binding.EINVAL),
    (dict(w=None), binding.EINVAL), (dict(beta=0.0), binding.EINVAL), (dict(beta=float("inf")), binding.EINVAL),
    (dict(sm=0.5), binding.EINVAL), (dict(sm=float("nan")), binding.EINVAL), (dict(loss=None), binding.EINVAL),
    (dict(n=255), binding.EINVAL)])
def test_preference_loss_refusals(lib, over, status):
    assert _pref(lib, **over) == status
    assert lib.archead_last_error().decode()


def test_workspace_sizes(lib):
    n = ctypes.c_uint64()
    assert lib.archead_loss_workspace(0, 1, 0, ctypes.byref(n)) == binding.OK and n.value >= 256
    assert lib.archead_loss_workspace(2048, 151936, 8, ctypes.byref(n)) == binding.OK
    assert 2048 * 4 * 2 < n.value < 1 << 22
    assert lib.archead_loss_workspace(-1, 8, 0, ctypes.byref(n)) == binding.EINVAL
    assert lib.archead_loss_workspace(1, 8, -1, ctypes.byref(n)) == binding.EINVAL
    assert lib.archead_loss_workspace(1, 0, 0, ctypes.byref(n)) == binding.ESHAPE
    assert lib.archead_loss_workspace(1, 8, 0, None) == binding.EINVAL
