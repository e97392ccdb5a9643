"""The embedding lookup and its gradient against the fp64 oracle.

u(t) is half a step of type t relative to a value.  Lookup: scale * table[v] is one
fp32 product (codes: one more, by the block's scale) and one rounding to out's type;
scale is an fp32 number here.  Gradient: a run of equal tokens is
summed as at most 31 entries before and 31 behind the whole parts at each of its
levels (one up to 8223 tokens, two up to 263167, else three) and at most 256 parts at
the last, 33 where there are three; a part of a level has 32 terms in sums of eight,
joined in pairs.  So a term passes through at most 10 additions a level within parts
and 62 a level and 256 beside them: 2 x 10 + 2 x 62 + 256 = 400 fp32 roundings bound all
three, and no more than its row has terms; one with scale and one to the gradient's
type.  All bounds carry 1 % for second order."""
import numpy as np
import pytest

from oracle import embedding, fp8

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24
HALF = {"f32": U32, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module")
def pq():
    import packed_quantized_lm_amd as pq
    return pq


def _t(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def _make(rng, shape, type):
    import torch
    return torch.from_numpy(rng.normal(0, 1, shape).astype(np.float32)).to(_t(type)).cuda()


def _ids(a):
    import torch
    return torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()


def _np(t):
    return t.double().cpu().numpy()


def _close(got, want, bound, what):
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    fine = ~np.isnan(want)
    off, bound = np.abs(got - want)[fine], np.broadcast_to(bound, want.shape)[fine]
    assert np.all(off <= bound), f"{what}: worst {np.max(off / np.maximum(bound, 1e-300)):.3g} x bound"


@pytest.mark.parametrize("tt", ["f32", "bf16"])
@pytest.mark.parametrize("ot", ["f32", "bf16"])
def test_lookup(pq, tt, ot):
    for n, V, d in ((1, 1, 1), (3, 5, 7), (40, 9, 8), (17, 33, 63), (300, 50, 64), (5, 20, 129), (70, 11, 256),
                    (9, 31, 257), (600, 100, 2561), (2, 3, 40001), (2050, 70, 520)):
        rng = np.random.default_rng(n * 1009 + d)
        table, tok = _make(rng, (V, d), tt), rng.integers(-1, V + 1, n)  # padding and one past the end among them
        scale = float(np.float32(rng.choice([1.0, 0.3, 50.6])))
        got = pq.embed(table, _ids(tok), scale=scale, out_dtype=_t(ot))
        assert got.dtype == _t(ot) and got.shape == (n, d)
        want = embedding.lookup(_np(table), tok, scale)
        _close(_np(got), want, 1.01 * np.abs(want) * (U32 + HALF[ot]), f"{n} {V} {d}")


@pytest.mark.parametrize("ot", ["f32", "bf16"])
def test_lookup_of_an_8_bit_head(pq, ot):
    import torch
    for n, V, d in ((1, 1, 16), (9, 129, 48), (50, 300, 128), (33, 257, 144), (400, 500, 2576)):
        rng = np.random.default_rng(n + d)
        head = pq.Fp8Head(_make(rng, (V, d), "f32"))
        tok = rng.integers(-1, V + 1, n)
        got = head.embed(_ids(tok), scale=2.5, out_dtype=_t(ot))
        s = head.scales.double().cpu().numpy()
        w = fp8.decode(head.weight.view(torch.uint8).cpu().numpy())
        w = w * np.repeat(np.repeat(s, 128, axis=0)[:V], 128, axis=1)[:, :d]
        want = embedding.lookup(w, tok, 2.5)
        _close(_np(got), want, 1.01 * np.abs(want) * (2 * U32 + HALF[ot]), f"{n} {V} {d}")


def _lists(rng, n, V):
    """Tokens as they come: spread out, as text has them, one alone, two in turn, with gaps."""
    yield "spread", rng.integers(0, V, n)
    yield "text", np.minimum((V * rng.random(n) ** 4).astype(np.int64), V - 1)
    yield "one", np.full(n, V - 1)
    yield "two", np.where(np.arange(n) % 3 == 0, 0, V // 2)
    yield "lost", rng.integers(-3, V + 3, n)


def _check(pq, n, V, d, dt, gt, tok, scale, what, **kw):
    rng = np.random.default_rng(n + V + d)
    dout = _make(rng, (n, d), dt)
    got = pq.embed_backward(dout, _ids(tok), V, scale=scale, grad_dtype=_t(gt), **kw)
    want, size, count = embedding.gradient(_np(dout), tok, V, scale, pad=kw.get("pad", -1))
    adds = np.minimum(400, np.maximum(count - 1, 0))[:, None]
    _close(_np(got), want, 1.01 * ((adds + 1) * U32 * size + HALF[gt] * np.abs(want)), what)
    return got


@pytest.mark.parametrize("dt,gt", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16")])
def test_gradient(pq, dt, gt):
    for n, V, d in ((1, 1, 1), (5, 3, 7), (31, 40, 8), (33, 17, 65), (64, 64, 16), (257, 100, 513), (700, 3000, 40),
                    (1500, 7, 24), (4097, 513, 9)):
        for name, tok in _lists(np.random.default_rng(n + d), n, V):
            _check(pq, n, V, d, dt, gt, tok, 0.75, f"{name} {n} {V} {d}")


@pytest.mark.parametrize("n", [8192, 8193, 16384, 16385, 40000, 70001])
def test_gradient_of_many_tokens(pq, n):
    for V in (2, 300, 70000):
        for name, tok in _lists(np.random.default_rng(n + V), n, V):
            _check(pq, n, V, 3, "bf16", "f32", tok, 1.0, f"{name} {n} {V}")


def test_gradient_of_the_longest_list(pq):
    rng = np.random.default_rng(5)
    n, V = 1 << 20, 1 << 19
    tok = np.where(rng.random(n) < 0.5, 77, rng.integers(0, V, n))
    dout = rng.normal(0, 1, (n, 1)).astype(np.float32)
    import torch
    got = pq.embed_backward(torch.from_numpy(dout).cuda(), _ids(tok), V)
    want, size = np.zeros(V), np.zeros(V)
    np.add.at(want, tok, dout[:, 0].astype(np.float64))
    np.add.at(size, tok, np.abs(dout[:, 0].astype(np.float64)))
    adds = np.minimum(400, np.maximum(np.bincount(tok, minlength=V) - 1, 0))
    _close(_np(got)[:, 0], want, 1.01 * ((adds + 2) * U32 * size), "longest")


def test_pad_in_the_table_and_nan_rows_of_lost_tokens(pq):
    import torch
    rng = np.random.default_rng(1)
    tok = np.array([4, 0, 4, 2, -1, 9, 0])
    table = _make(rng, (5, 33), "f32")
    out = pq.embed(table, _ids(tok), pad=4)
    assert (out[0] == 0).all() and torch.isnan(out[4]).all() and torch.isnan(out[5]).all()
    _check(pq, 7, 5, 33, "f32", "f32", tok, 1.0, "pad", pad=4)
    dout = _make(rng, (7, 33), "f32")
    dout[4:6] = float("nan")
    got = pq.embed_backward(dout, _ids(tok), 5)
    assert torch.isfinite(got).all()


@pytest.mark.parametrize("gt", ["f32", "bf16"])
def test_accumulate_and_strides(pq, gt):
    import torch
    rng = np.random.default_rng(2)
    for n, V, d in ((50, 30, 37), (20000, 40, 8)):
        tok = rng.integers(0, V - 4, n)  # the last rows do not occur
        wide, held = _make(rng, (n, 2 * d + 1), "bf16"), _make(rng, (V, d + 3), gt)
        dout, before = wide[:, d:2 * d], held.clone()
        held[V - 1, 0] = float("nan")  # left as it was
        target = held[:, 2:2 + d]
        assert pq.embed_backward(dout, _ids(tok), V, scale=0.5, dtable=target, accumulate=True) is target
        want, size, count = embedding.gradient(_np(dout), tok, V, 0.5)
        want += _np(before[:, 2:2 + d])
        adds = np.minimum(400, np.maximum(count - 1, 0))[:, None]
        _close(_np(target)[:V - 4], want[:V - 4], 1.01 * ((adds + 2) * U32 * (size + np.abs(want)) + HALF[gt] * np.abs(want))[:V - 4],
               "accumulated")
        bits = {"f32": torch.int32, "bf16": torch.int16}[gt]  # a NaN is not equal to itself
        kept = torch.ones(V, d + 3, dtype=torch.bool, device="cuda")
        kept[:V - 4, 2:2 + d] = False
        assert torch.isnan(held[V - 1, 0]) and not torch.isnan(before[V - 1, 0])
        kept[V - 1, 0] = False
        assert torch.equal(held.view(bits)[kept], before.view(bits)[kept])
        out = torch.full((n, d + 5), 7.0, device="cuda", dtype=_t(gt))
        pq.embed(before[:, 2:2 + d], _ids(tok), out=out[:, 1:1 + d])
        assert torch.equal(out[:, 1:1 + d], before[:, 2:2 + d][torch.from_numpy(tok).cuda()])
        assert (out[:, 0] == 7).all() and (out[:, 1 + d:] == 7).all()


def test_no_tokens(pq):
    import torch
    none = _ids([])
    assert pq.embed(torch.ones(4, 8, device="cuda"), none).shape == (0, 8)
    grad = pq.embed_backward(torch.ones(0, 8, device="cuda"), none, 4)
    assert torch.equal(grad, torch.zeros(4, 8, device="cuda"))
    held = torch.ones(4, 8, device="cuda")
    pq.embed_backward(torch.ones(0, 8, device="cuda"), none, 4, dtable=held, accumulate=True)
    assert torch.equal(held, torch.ones_like(held))


def test_refused_on_the_gpu(pq):
    import torch
    t, tok = torch.ones(4, 16, device="cuda"), _ids([0, 1])
    f8 = t.to(torch.float8_e4m3fn)
    for call in (lambda: pq.embed(t, tok.cpu()), lambda: pq.embed(t, tok.long()), lambda: pq.embed(f8, tok),
                 lambda: pq.embed(t, tok, scales=t), lambda: pq.embed(t, tok, out=torch.ones(3, 16, device="cuda")),
                 lambda: pq.embed(t, tok, scale=float("nan")), lambda: pq.embed(f8, tok, scales=torch.ones(1, 2, device="cuda")),
                 lambda: pq.embed_backward(t, tok, 4), lambda: pq.embed_backward(t[:2], tok, 0),
                 lambda: pq.embed_backward(t[:2], tok, 4, accumulate=True),
                 lambda: pq.embed_backward(t[:2], tok, 5, dtable=t)):
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            call()
    torch.cuda.synchronize()


@pytest.mark.parametrize("n", [300, 20000])
def test_equal_calls_side_stream_and_graph(pq, n):
    import torch
    rng = np.random.default_rng(n)
    V, d = 5000, 72
    table, dout = _make(rng, (V, d), "bf16"), _make(rng, (n, d), "bf16")
    tok = _ids(np.minimum((V * rng.random(n) ** 4).astype(np.int64), V - 1))

    def step():
        return pq.embed(table, tok, scale=3.0), pq.embed_backward(dout, tok, V, grad_dtype=torch.float32)

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
        tok.copy_(_ids(rng.integers(-1, V, n)))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        assert all(torch.equal(a, b) for a, b in zip(got, step()))
