"""The embedding's entry points refuse bad arguments before any device work (no
GPU here: the pointers are never followed)."""
import ctypes

import pytest
import torch

import packed_quantized_lm_amd as pq
from packed_quantized_lm_amd import binding

B, C = ctypes.c_void_p(4096), ctypes.c_void_p(8192)
ODD = ctypes.c_void_p(4097)


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


def _look(lib, n=2, V=8, d=16, table=B, tt=1, ldt=16, scales=B, lds=1, tok=B, pad=-1, scale=1.0, out=C, ot=1, ldo=16):
    return lib.archead_embed(n, V, d, table, tt, ldt, scales, lds, tok, pad, scale, out, ot, ldo, None)


@pytest.mark.parametrize("over,status", [
    (dict(n=-1), binding.EINVAL), (dict(n=(1 << 20) + 1), binding.ESHAPE), (dict(V=0), binding.ESHAPE),
    (dict(V=1 << 31), binding.ESHAPE), (dict(d=0), binding.ESHAPE), (dict(d=(1 << 20) + 1), binding.ESHAPE),
    (dict(tt=3), binding.EINVAL), (dict(ot=2), binding.EINVAL), (dict(tt=2, d=8), binding.ESHAPE),
    (dict(scale=float("nan")), binding.EINVAL), (dict(ldt=15), binding.EINVAL), (dict(ldo=15), binding.EINVAL),
    (dict(tt=2, lds=0), binding.EINVAL), (dict(table=None), binding.EINVAL), (dict(tok=None), binding.EINVAL),
    (dict(out=None), binding.EINVAL), (dict(tt=2, scales=None), binding.EINVAL), (dict(table=ODD), binding.EINVAL),
    (dict(tt=2, table=ctypes.c_void_p(4104)), binding.EINVAL), (dict(tt=2, ldt=24), binding.EINVAL),
    (dict(out=B), binding.EINVAL), (dict(table=C), binding.EINVAL), (dict(out=ODD), binding.EINVAL), (dict(tok=ctypes.c_void_p(4098)), binding.EINVAL)])
def test_lookup_refusals(lib, over, status):
    assert _look(lib, **over) == status
    assert lib.archead_last_error().decode()


def _grad(lib, n=2, V=8, d=16, dout=B, dt=1, ldo=16, tok=B, pad=-1, scale=1.0, acc=0, dtable=C, gt=1, ldt=16, ws=B,
          size=1 << 40):
    return lib.archead_embed_backward(n, V, d, dout, dt, ldo, tok, pad, scale, acc, dtable, gt, ldt, ws, size, None)


@pytest.mark.parametrize("over,status", [
    (dict(n=-1), binding.EINVAL), (dict(n=(1 << 20) + 1), binding.ESHAPE), (dict(V=0), binding.ESHAPE),
    (dict(V=(1 << 26) - (1 << 24)), binding.ESHAPE), (dict(n=1 << 20, d=1 << 15, ldo=1 << 15, ldt=1 << 15), binding.ESHAPE),
    (dict(dt=2), binding.EINVAL), (dict(gt=2), binding.EINVAL), (dict(scale=float("inf")), binding.EINVAL),
    (dict(ldo=15), binding.EINVAL), (dict(ldt=15), binding.EINVAL), (dict(dout=None), binding.EINVAL),
    (dict(tok=None), binding.EINVAL), (dict(dtable=None), binding.EINVAL), (dict(dtable=ODD), binding.EINVAL),
    (dict(dout=ODD), binding.EINVAL), (dict(ws=None), binding.EINVAL), (dict(ws=ctypes.c_void_p(4104)), binding.EINVAL),
    (dict(size=15), binding.EINVAL), (dict(dtable=B), binding.EINVAL), (dict(dout=C), binding.EINVAL)])
def test_gradient_refusals(lib, over, status):
    assert _grad(lib, **over) == status
    assert lib.archead_last_error().decode()


def test_no_tokens_is_no_work(lib):
    assert _look(lib, n=0) == binding.OK
    assert _grad(lib, n=0, acc=1) == binding.OK


def test_workspace_sizes(lib):
    n = ctypes.c_uint64()
    for count, V, d in ((0, 1, 1), (31, 100, 7), (8192, 151936, 4096), (1 << 20, 1 << 20, 64)):
        assert lib.archead_embed_workspace(count, V, d, ctypes.byref(n)) == binding.OK
        parts = count // 32 + count // 1024 + count // 32768
        assert 8 * count <= n.value <= 16 * count + 4 * parts * d + count + 2048 + 256
    assert lib.archead_embed_workspace(1, 1, 1, None) == binding.EINVAL
    assert lib.archead_embed_workspace(-1, 1, 1, ctypes.byref(n)) == binding.EINVAL


def test_python_refuses_host_tensors_and_wrong_arguments():
    t, tok = torch.zeros(4, 16), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        pq.embed(t, tok)
    with pytest.raises(ValueError):
        pq.embed(t.half(), tok)
    with pytest.raises(ValueError):
        pq.embed_backward(t, tok, 4)
    from packed_quantized_lm_amd import embedding
    for pad in (2 ** 31, -2 ** 31 - 1):
        with pytest.raises(ValueError):
            embedding._pad(pad)
