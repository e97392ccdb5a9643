"""The norm and its backward against the fp64 oracle.

u(t) is half a step of type t relative to a value.  Forward: n = h r (w + offset)
is four fp32 roundings (r, w + offset, two products) and y one more.  Backward:
g = u (w + offset) is two, the mean of g h is theirs again (its sum is fp64), r,
k and the two fused operations four more: 8 x 2^-24 of the magnitudes dh is formed
from covers them.  dweight: terms of three roundings (r, h r, the fused product's),
summed over at most 64 rows and the workgroup's 16 teams in fp32: 84 x 2^-24 of the
terms' magnitudes.  All bounds carry 1 % for second order."""
import numpy as np
import pytest

from oracle import fp8, norm

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24
HALF = {"f32": U32, "bf16": 2.0 ** -8}

SHAPES = [(1, 1), (3, 7), (5, 8), (1, 16), (33, 48), (7, 127), (2, 128), (19, 129), (3, 512), (5, 640), (2, 1000),
          (70, 2048), (3, 2049), (1, 4096), (9, 4100), (3, 6151), (2, 8192), (2, 8200), (3, 16384), (2, 16400), (1, 40007)]


@pytest.fixture(scope="module")
def pq():
    import packed_quantized_lm_amd as pq
    return pq


def _t(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def _make(rng, shape, type, scale=1.0):
    import torch
    x = rng.normal(0, scale, shape) * np.exp(rng.normal(0, 0.7, shape[-1]))
    return torch.from_numpy(x.astype(np.float32)).to(_t(type)).cuda()


def _np(t):
    return t.double().cpu().numpy()


def _close(got, want, bound, what):
    off = np.abs(got - want)
    assert np.all(np.isfinite(got)), what
    bad = off > bound
    assert not bad.any(), f"{what}: {bad.sum()} values off, worst {np.max(off / np.maximum(bound, 1e-300)):.3g} x bound"


def _codes_are_nearest(n, q, s, rel):
    """codes q with scales s are the nearest to n, which is known to rel."""
    M, d = n.shape
    v = fp8.decode(q)
    spread = np.repeat(s.astype(np.float64).T, 128, axis=1)[:, :d]
    amax = np.stack([np.abs(n[:, b:b + 128]).max(axis=1) for b in range(0, d, 128)])
    assert np.all(np.abs(s - amax / 448) <= 1.01 * (rel + 2 * U32) * amax / 448 + 2.0 ** -126)
    want = n / np.where(spread > 0, spread, 1.0)
    a = np.abs(want)
    step = 2.0 ** (np.clip(np.floor(np.log2(np.maximum(a, 2.0 ** -6))), -6, 8) - 3)
    assert np.all(np.abs(v - np.clip(want, -448, 448)) <= step / 2 * (1 + 1e-9) + 1.01 * (rel + 2 * U32) * a)


@pytest.mark.parametrize("xt,rt,wt,yt,offset", [("bf16", "bf16", "bf16", "bf16", 0.0), ("f32", "f32", "f32", "f32", 1.0),
                                                ("bf16", "f32", "f32", "bf16", 0.0), ("f32", "bf16", "bf16", "f32", 0.0),
                                                ("bf16", None, "f32", "f32", 1.0), ("f32", None, "bf16", "bf16", 0.0)])
def test_forward(pq, xt, rt, wt, yt, offset):
    for M, d in SHAPES:
        rng = np.random.default_rng(M * 100003 + d)
        x, w = _make(rng, (M, d), xt), _make(rng, (d,), wt)
        res = None if rt is None else _make(rng, (M, d), rt, 3.0)
        codes = d % 16 == 0
        y, h, q, s = pq.rms_norm(x, w, residual=res, eps=1e-5, offset=offset, out_dtype=_t(yt), want_codes=codes)
        want_h = _np(x) if rt is None else norm.add(_np(x), _np(res), rt == "bf16")
        assert (h is None) == (rt is None)
        if h is not None:
            assert h.dtype == _t(rt) and np.array_equal(_np(h), want_h), (M, d)
        n = norm.forward(want_h, _np(w), 1e-5, offset)
        rel = 4.04 * U32
        _close(_np(y), n, np.abs(n) * (rel + HALF[yt]) * 1.01 + 2.0 ** -126, f"y at {M} x {d}")
        if codes:
            import torch
            _codes_are_nearest(n, q.view(torch.uint8).cpu().numpy(), s.cpu().numpy(), rel)
            if yt == "f32":  # the same codes as the quantiser's of the same values
                q2, s2 = pq.fp8_quantize(y)
                assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2)


@pytest.mark.parametrize("ut,ht,wt,through,offset", [("bf16", "bf16", "bf16", True, 0.0), ("f32", "f32", "f32", True, 1.0),
                                                     ("bf16", "f32", "f32", False, 0.0), ("f32", "bf16", "bf16", False, 1.0)])
def test_backward(pq, ut, ht, wt, through, offset):
    for M, d in SHAPES + [(1500, 40), (2100, 520), (3000, 16), (1100, 2056)]:
        rng = np.random.default_rng(M * 100003 + d + 1)
        u, h, w = _make(rng, (M, d), ut), _make(rng, (M, d), ht, 3.0), _make(rng, (d,), wt)
        res = _make(rng, (M, d), ht) if through else None
        dh, dw = pq.rms_norm_backward(u, h, w, dres=res, eps=1e-5, offset=offset)
        want, want_dw, size = norm.backward(_np(u), _np(h), _np(w), 1e-5, offset, None if res is None else _np(res))
        _close(_np(dh), want, 1.01 * (8 * U32 * size + HALF[ht] * np.abs(want)) + 2.0 ** -126, f"dh at {M} x {d}")
        terms = np.sum(np.abs(_np(u) * _np(h)) / norm.rms(_np(h), 1e-5), axis=0)
        _close(_np(dw), want_dw, 1.01 * 84 * U32 * terms + 2.0 ** -126, f"dweight at {M} x {d}")


def test_many_rows(pq):
    """More rows than one part of dweight's sum in fp32 takes, and than a launch has workgroups at once."""
    for M, d in ((70001, 24), (70001, 200), (66000, 1032)):
        rng = np.random.default_rng(d)
        u, h, w = _make(rng, (M, d), "bf16"), _make(rng, (M, d), "bf16"), _make(rng, (d,), "f32")
        dh, dw = pq.rms_norm_backward(u, h, w)
        want, want_dw, size = norm.backward(_np(u), _np(h), _np(w), 1e-6, 0.0)
        _close(_np(dh), want, 1.01 * (8 * U32 * size + HALF["bf16"] * np.abs(want)) + 2.0 ** -126, "dh")
        terms = np.sum(np.abs(_np(u) * _np(h)) / norm.rms(_np(h), 1e-6), axis=0)
        _close(_np(dw), want_dw, 1.01 * 84 * U32 * terms, "dweight")
        y, _, _, _ = pq.rms_norm(h, w)
        n = norm.forward(_np(h), _np(w), 1e-6, 0.0)
        _close(_np(y), n, np.abs(n) * (4.04 * U32 + HALF["bf16"]) * 1.01, "y")


def test_strided_rows_and_in_place(pq):
    import torch
    rng = np.random.default_rng(3)
    M, d = 37, 333
    wide = _make(rng, (M, 2 * d + 5), "bf16")
    x, res, w = wide[:, 3:3 + d], wide[:, d + 5:], _make(rng, (d,), "f32")
    y0, h0, _, _ = pq.rms_norm(x.contiguous(), w, residual=res.contiguous())
    kept = wide.clone()
    y, h, _, _ = pq.rms_norm(x, w, residual=res)
    assert torch.equal(y, y0) and torch.equal(h, h0) and torch.equal(wide, kept)
    y, h, _, _ = pq.rms_norm(x, w, residual=res, h_out=res)  # over the residual, nothing beside it
    assert h is res and torch.equal(y, y0) and torch.equal(res, h0)
    kept[:, d + 5:] = h0
    assert torch.equal(wide, kept)
    u, through = _make(rng, (M, d), "bf16"), _make(rng, (M, d), "bf16")
    dh0, dw0 = pq.rms_norm_backward(u, h0, w, dres=through)
    dh, dw = pq.rms_norm_backward(u, res, w, dres=through, dh_out=through)
    assert dh is through and torch.equal(dh, dh0) and torch.equal(dw, dw0)
    for d in (24, 20001):  # long rows in place too
        x, res = _make(rng, (5, d), "bf16"), _make(rng, (5, d), "bf16")
        w = _make(rng, (d,), "bf16")
        y0, h0, _, _ = pq.rms_norm(x, w, residual=res)
        y, _, _, _ = pq.rms_norm(x, w, residual=res, h_out=res)
        assert torch.equal(y, y0) and torch.equal(res, h0)
        u, through = _make(rng, (5, d), "bf16"), _make(rng, (5, d), "bf16")
        dh0, _ = pq.rms_norm_backward(u, h0, w, dres=through)
        dh, _ = pq.rms_norm_backward(u, h0, w, dres=through, dh_out=through)
        assert torch.equal(dh, dh0)


@pytest.mark.parametrize("d", [96, 640, 5000, 20000])
def test_rows_do_not_touch_each_other(pq, d):
    """NaN, infinities, zeros, and the type's largest and smallest values in one row each."""
    import torch
    rng = np.random.default_rng(d)
    h, w = _make(rng, (8, d), "bf16"), _make(rng, (d,), "f32")
    y0, _, _, _ = pq.rms_norm(h, w)
    u = _make(rng, (8, d), "bf16")
    dh0, _ = pq.rms_norm_backward(u, h, w)
    odd = h.clone()
    odd[1, 5] = float("nan")
    odd[2, d - 1] = float("inf")
    odd[3] = 0.0
    odd[4] = 2.0 ** 120  # squares far past fp32's range
    odd[5] = 2.0 ** -130
    y, _, _, _ = pq.rms_norm(odd, w)
    assert torch.isnan(y[1]).all() and torch.isnan(y[2, d - 1])
    assert (y[2, :d - 1] == 0).all() and (y[3] == 0).all()
    assert torch.equal(y[0], y0[0]) and torch.equal(y[6:], y0[6:])
    n = norm.forward(_np(odd[4:6]), _np(w), 1e-6, 0.0)
    _close(_np(y[4:6]), n, np.abs(n) * (4.04 * U32 + HALF["bf16"]) * 1.01 + 2.0 ** -134, "largest and smallest")
    dh, dw = pq.rms_norm_backward(u, odd, w)
    assert torch.isnan(dh[1]).all() and torch.equal(dh[0], dh0[0]) and torch.equal(dh[6:], dh0[6:])
    assert torch.isnan(dw).any()


def test_no_rows_and_no_weight_gradient(pq):
    import torch
    x, w = torch.zeros(0, 32, device="cuda"), torch.ones(32, device="cuda")
    y, h, q, s = pq.rms_norm(x, w, residual=x, want_codes=True)
    assert y.shape == (0, 32) and h.shape == (0, 32) and q.shape == (0, 32) and s.shape == (1, 0)
    dh, dw = pq.rms_norm_backward(x, x, w)
    assert dh.shape == (0, 32) and torch.equal(dw, torch.zeros_like(w))
    h = torch.ones(3, 32, device="cuda")
    dh, dw = pq.rms_norm_backward(h, h, w, want_dweight=False)
    assert dw is None and dh.shape == (3, 32)


def test_refused_on_the_gpu(pq):
    import torch
    x, w = torch.ones(3, 32, device="cuda"), torch.ones(32, device="cuda")
    for call in (lambda: pq.rms_norm(x, w.cpu()), lambda: pq.rms_norm(x, w[:31]), lambda: pq.rms_norm(x.half(), w),
                 lambda: pq.rms_norm(x, w, residual=x[:2]), lambda: pq.rms_norm(x, w, want_y=False),
                 lambda: pq.rms_norm(x[:, :24], w[:24], want_codes=True), lambda: pq.rms_norm(x, w, h_out=x),
                 lambda: pq.rms_norm(x.t(), w[:3]), lambda: pq.rms_norm(x, w, eps=-1.0),
                 lambda: pq.rms_norm_backward(x, x, w, dres=x.bfloat16()), lambda: pq.rms_norm_backward(x[:2], x, w),
                 lambda: pq.rms_norm_backward(x, x, w, dh_out=x)):
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            call()
    torch.cuda.synchronize()


def test_equal_calls_side_stream_and_graph(pq):
    import torch
    rng = np.random.default_rng(9)
    M, d = 300, 1104
    x, res, w = _make(rng, (M, d), "bf16"), _make(rng, (M, d), "bf16"), _make(rng, (d,), "bf16")
    u = _make(rng, (M, d), "bf16")

    def step():
        y, h, q, s = pq.rms_norm(x, w, residual=res, want_codes=True)
        dh, dw = pq.rms_norm_backward(u, h, w, dres=u)
        return y, h, q.view(torch.uint8), s, dh, dw

    first = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(first, second))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for k in range(3):
        x.copy_(_make(rng, (M, d), "bf16"))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        assert all(torch.equal(a, b) for a, b in zip(got, step()))
