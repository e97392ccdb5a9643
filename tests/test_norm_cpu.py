"""The norm's entry points refuse bad arguments before any device work (no GPU
here: the pointers are never followed)."""
import ctypes

import pytest
import torch

import packed_quantized_lm_amd as pq
from packed_quantized_lm_amd import binding

B, C, D, E = (ctypes.c_void_p(4096 * i) for i in (1, 2, 3, 4))
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


def _norm(lib, M=2, d=16, x=B, xt=1, ldx=16, res=C, rt=1, ldr=16, h=D, ldh=16, w=B, wt=1, eps=1e-6, off=0.0, y=E, yt=1,
          ldy=16, q=E, ldq=16, s=E, lds=2):
    return lib.archead_rms_norm(M, d, x, xt, ldx, res, rt, ldr, h, ldh, w, wt, eps, off, y, yt, ldy, q, ldq, s, lds,
                                None)


@pytest.mark.parametrize("over,status", [
    (dict(M=-1), binding.EINVAL), (dict(M=1 << 22), binding.ESHAPE), (dict(d=0), binding.ESHAPE),
    (dict(d=(1 << 20) + 16), binding.ESHAPE), (dict(eps=-1e-6), binding.EINVAL), (dict(eps=NAN), binding.EINVAL),
    (dict(eps=INF), binding.EINVAL), (dict(off=INF), binding.EINVAL), (dict(xt=2), binding.EINVAL),
    (dict(rt=-1), binding.EINVAL), (dict(wt=3), binding.EINVAL), (dict(yt=2), binding.EINVAL),
    (dict(y=None, q=None, s=None), binding.EINVAL), (dict(res=None), binding.EINVAL), (dict(h=None), binding.EINVAL),
    (dict(q=None), binding.EINVAL), (dict(s=None), binding.EINVAL), (dict(x=None), binding.EINVAL),
    (dict(w=None), binding.EINVAL), (dict(d=24, ldx=24, ldr=24, ldh=24, ldy=24, ldq=32), binding.ESHAPE),
    (dict(ldx=15), binding.EINVAL), (dict(ldr=15), binding.EINVAL), (dict(ldh=15), binding.EINVAL),
    (dict(ldy=15), binding.EINVAL), (dict(ldq=0), binding.EINVAL), (dict(ldq=24), binding.EINVAL),
    (dict(lds=1), binding.EINVAL), (dict(ldx=(1 << 40) + 1), binding.EINVAL),
    (dict(x=ctypes.c_void_p(4097)), binding.EINVAL), (dict(q=ctypes.c_void_p(4104)), binding.EINVAL),
    (dict(s=ctypes.c_void_p(4098)), binding.EINVAL), (dict(res=C, h=C, ldh=32), binding.EINVAL),
    (dict(y=B, ldy=32), binding.EINVAL), (dict(y=B, yt=0), binding.EINVAL), (dict(h=B, rt=0), binding.EINVAL),
    (dict(y=D), binding.EINVAL)])
def test_refusals(lib, over, status):
    assert _norm(lib, **over) == status
    assert lib.archead_last_error().decode()


def test_no_rows_is_no_work(lib):
    assert _norm(lib, M=0, lds=0) == binding.OK


def _back(lib, M=2, d=16, u=B, ut=1, ldu=16, h=C, ht=1, ldh=16, w=B, wt=1, eps=1e-6, off=0.0, res=D, ldr=16, dh=E,
          ldd=16, dw=B, ws=B, n=1 << 30):
    return lib.archead_rms_norm_backward(M, d, u, ut, ldu, h, ht, ldh, w, wt, eps, off, res, ldr, dh, ldd, dw, ws, n,
                                         None)


@pytest.mark.parametrize("over,status", [
    (dict(M=-1), binding.EINVAL), (dict(M=1 << 22), binding.ESHAPE), (dict(d=0), binding.ESHAPE),
    (dict(eps=-1.0), binding.EINVAL), (dict(off=NAN), binding.EINVAL), (dict(ut=2), binding.EINVAL),
    (dict(ht=2), binding.EINVAL), (dict(wt=2), binding.EINVAL), (dict(u=None), binding.EINVAL),
    (dict(h=None), binding.EINVAL), (dict(w=None), binding.EINVAL), (dict(dh=None), binding.EINVAL),
    (dict(ldu=15), binding.EINVAL), (dict(ldh=15), binding.EINVAL), (dict(ldr=15), binding.EINVAL),
    (dict(ldd=15), binding.EINVAL), (dict(dh=B), binding.EINVAL), (dict(dh=C), binding.EINVAL),
    (dict(res=E, ldr=32), binding.EINVAL), (dict(ws=None), binding.EINVAL), (dict(ws=ctypes.c_void_p(4104)), binding.EINVAL),
    (dict(n=63), binding.EINVAL), (dict(dw=ctypes.c_void_p(4098)), binding.EINVAL),
    (dict(dh=ctypes.c_void_p(4097)), binding.EINVAL)])
def test_backward_refusals(lib, over, status):
    assert _back(lib, **over) == status
    assert lib.archead_last_error().decode()


def test_workspace_sizes(lib):
    n = ctypes.c_uint64()
    assert lib.archead_rms_norm_workspace(0, 1, ctypes.byref(n)) == binding.OK and n.value >= 16
    for M, d in ((1, 16), (8192, 4096), ((1 << 22) - 1, 16), (7, 1 << 20), (4000, 20000)):
        assert lib.archead_rms_norm_workspace(M, d, ctypes.byref(n)) == binding.OK
        assert 4 * d <= n.value <= 4 * d * (1024 + M // 16) + 4 * M + 64
    assert lib.archead_rms_norm_workspace(1, 1, None) == binding.EINVAL
    assert lib.archead_rms_norm_workspace(1 << 22, 1, ctypes.byref(n)) == binding.ESHAPE


def test_python_refuses_host_tensors_and_wrong_arguments():
    x, w = torch.zeros(2, 16), torch.zeros(16)
    with pytest.raises(ValueError):
        pq.rms_norm(x, w)
    with pytest.raises(ValueError):
        pq.rms_norm(torch.zeros(16), w)
    with pytest.raises(ValueError):
        pq.rms_norm(x.half(), w)
    with pytest.raises(ValueError):
        pq.rms_norm_backward(x, x, w)
