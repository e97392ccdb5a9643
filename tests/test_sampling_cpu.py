"""The sampling entry points refuse bad arguments before any device work (no GPU
here: the pointers are never followed)."""
import ctypes

import pytest
import torch

import packed_quantized_lm_amd as pq
from packed_quantized_lm_amd import binding

B, C = ctypes.c_void_p(4096), ctypes.c_void_p(8192)
ODD = ctypes.c_void_p(4098)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


COMMON = dict(M=2, V=40, y=B, type=0, ld=40, hist=B, L=8, ldh=8, lens=B, prompts=B, rep=B, freq=B, pres=B, ids=B, vals=B,
              nb=4, ldb=4, mask=B, R=2, ldm=2, rows=B)


def _common(over):
    c = dict(COMMON, **{k: v for k, v in over.items() if k in COMMON})
    return list(c.values())


def _adjust(lib, over):
    return lib.archead_adjust_logits(*_common(over), over.get("out", C), over.get("ldo", 40), over.get("ws", B),
                                     over.get("n", 1 << 40), None)


def _sample(lib, over):
    o = dict(dict(K=4, tau=1.0, taus=None, u=B, values=B, indices=B, samples=B, ws=B, n=1 << 30),
             **{k: v for k, v in over.items() if k not in COMMON})
    return lib.archead_sample_logits(*_common(over), *o.values(), None)


BAD = [
    (dict(M=-1), binding.EINVAL), (dict(M=(1 << 20) + 1), binding.ESHAPE), (dict(V=0), binding.ESHAPE),
    (dict(V=(1 << 30) + 1, ld=1 << 31, ldm=1 << 26), binding.ESHAPE), (dict(L=(1 << 20) + 1, ldh=1 << 21), binding.ESHAPE),
    (dict(nb=1024, ldb=1024), binding.ESHAPE), (dict(M=1 << 18, V=1 << 20, ld=1 << 20, ldm=1 << 15, R=1 << 18), binding.ESHAPE),
    (dict(type=2), binding.EINVAL), (dict(ld=39), binding.EINVAL), (dict(ld=(1 << 40) + 1), binding.EINVAL),
    (dict(L=-1), binding.EINVAL), (dict(nb=-1), binding.EINVAL), (dict(R=-1), binding.EINVAL),
    (dict(ldh=7), binding.EINVAL), (dict(hist=None), binding.EINVAL), (dict(ids=None), binding.EINVAL),
    (dict(vals=None), binding.EINVAL), (dict(ldb=3), binding.EINVAL), (dict(ldm=1), binding.EINVAL),
    (dict(mask=None), binding.EINVAL), (dict(rows=None, R=1), binding.EINVAL), (dict(y=None), binding.EINVAL),
    (dict(y=ODD), binding.EINVAL), (dict(hist=ODD), binding.EINVAL), (dict(lens=ODD), binding.EINVAL),
    (dict(rep=ODD), binding.EINVAL), (dict(ids=ODD), binding.EINVAL), (dict(mask=ODD), binding.EINVAL)]


@pytest.mark.parametrize("over,status", BAD + [
    (dict(out=None), binding.EINVAL), (dict(out=ODD), binding.EINVAL), (dict(ldo=39), binding.EINVAL),
    (dict(out=B, ldo=41), binding.EINVAL),
    (dict(M=1 << 10, V=1 << 14, ld=1 << 14, ldm=512, R=1 << 10, L=1 << 15, ldh=1 << 15, ldo=1 << 14, n=1 << 20), binding.EINVAL),
    (dict(M=1 << 10, V=1 << 14, ld=1 << 14, ldm=512, R=1 << 10, L=1 << 15, ldh=1 << 15, ldo=1 << 14, ws=None), binding.EINVAL)])
def test_adjust_refusals(lib, over, status):
    assert _adjust(lib, over) == status
    assert lib.archead_last_error().decode()


@pytest.mark.parametrize("over,status", BAD + [
    (dict(K=0), binding.ESHAPE), (dict(K=17), binding.ESHAPE), (dict(V=3, K=4), binding.ESHAPE),
    (dict(tau=0.0), binding.EINVAL), (dict(tau=NAN), binding.EINVAL), (dict(tau=INF), binding.EINVAL),
    (dict(u=None), binding.EINVAL), (dict(values=None, indices=None, samples=None), binding.EINVAL),
    (dict(ws=None), binding.EINVAL), (dict(ws=ctypes.c_void_p(4104)), binding.EINVAL), (dict(n=63), binding.EINVAL),
    (dict(u=ODD), binding.EINVAL), (dict(samples=ODD), binding.EINVAL), (dict(taus=ODD), binding.EINVAL)])
def test_sample_refusals(lib, over, status):
    assert _sample(lib, over) == status
    assert lib.archead_last_error().decode()


def test_no_rows_is_no_work(lib):
    assert _adjust(lib, dict(M=0)) == binding.OK
    assert _sample(lib, dict(M=0)) == binding.OK


def test_workspace_sizes(lib):
    n = ctypes.c_uint64()
    assert lib.archead_rules_workspace(1, 151936, 300, 0, ctypes.byref(n)) == binding.OK and n.value == 0
    for M, V, L, K in ((1, 1, 0, 1), (1, 151936, 0, 16), (256, 151936, 8192, 16), (256, 151936, 8192, 0),
                       (1 << 20, 17, 1 << 20, 1), (1, 1 << 30, 1 << 20, 16)):
        assert lib.archead_rules_workspace(M, V, L, K, ctypes.byref(n)) == binding.OK
        assert M * K * 8 <= n.value <= M * (K * 8 + 4) * -(-V // 2048) + 2 * M * L
    for M, V, L, K, status in ((-1, 8, 0, 1, binding.EINVAL), (1, 8, -1, 1, binding.EINVAL), (1, 0, 0, 1, binding.ESHAPE),
                               (1, 8, 0, 9, binding.ESHAPE), (1, 80, 0, 17, binding.ESHAPE), (1, 8, 0, -1, binding.ESHAPE),
                               (1, 8, (1 << 20) + 1, 0, binding.ESHAPE), (1, (1 << 30) + 1, 0, 1, binding.ESHAPE)):
        assert lib.archead_rules_workspace(M, V, L, K, ctypes.byref(n)) == status
    assert lib.archead_rules_workspace(1, 1, 0, 1, None) == binding.EINVAL


def test_python_refuses_host_tensors_and_wrong_arguments():
    y = torch.zeros(2, 40)
    for call in (lambda: pq.adjust_logits(y), lambda: pq.sample_logits(y, 4), lambda: pq.adjust_logits(y.half()),
                 lambda: pq.adjust_logits(y[0])):
        with pytest.raises(ValueError):
            call()
