"""The operators around the head at the ends of their ranges: offsets past 2^32
elements in tables, rows and logits, calls at once on two streams, and sizes next to
the borders between the kernels' forms."""
import numpy as np
import pytest

from oracle import embedding, norm, rules

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24


@pytest.fixture(scope="module")
def pq():
    import packed_quantized_lm_amd as pq
    return pq


def _cuda(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _np(t):
    return t.double().cpu().numpy()


@pytest.fixture
def plenty():
    """16 GiB and more of free GPU memory, given back at the end."""
    import gc
    import torch
    gc.collect()
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 48 << 30:
        pytest.skip("needs 48 GiB of free GPU memory")
    yield
    gc.collect()
    torch.cuda.empty_cache()


def test_tables_past_32_bits(pq, plenty):
    import torch
    V, d = 530000, 8200  # 4.3e9 elements
    rng = np.random.default_rng(0)
    table = torch.empty(V, d, dtype=torch.bfloat16, device="cuda")
    ids = np.array([V - 1, 7, V // 2, 523809, V - 1, 0])
    rows = torch.from_numpy(rng.normal(0, 1, (len(ids), d)).astype(np.float32)).to(torch.bfloat16).cuda()
    for i, v in enumerate(ids):
        table[v] = rows[i]
    got = pq.embed(table, _cuda(ids.astype(np.int32)), scale=2.0)
    assert torch.equal(got, table[torch.from_numpy(ids).cuda()] * 2)
    # the gradient added to the same rows of the same table, and then written whole
    before = table[torch.from_numpy(ids).cuda()].clone()
    pq.embed_backward(rows, _cuda(ids.astype(np.int32)), V, dtable=table, accumulate=True)
    want, size, _ = embedding.gradient(_np(rows), np.searchsorted(np.unique(ids), ids), 5, 1.0)
    for k, v in enumerate(np.unique(ids)):
        old = _np(before[int(np.nonzero(ids == v)[0][0])])
        assert np.all(np.abs(_np(table[v]) - (want[k] + old)) <= 1.01 * (2.0 ** -8 * np.abs(want[k] + old)
                                                                      + 4 * U32 * (size[k] + np.abs(old))))
    pq.embed_backward(rows, _cuda(ids.astype(np.int32)), V, dtable=table)
    for k, v in enumerate(np.unique(ids)):
        assert np.all(np.abs(_np(table[v]) - want[k]) <= 1.01 * (2.0 ** -8 * np.abs(want[k]) + 2 * U32 * size[k]))
    for v in (1, 261000, 262144, 523775, 523808, 529998):
        assert not table[v].any()


def test_rows_far_apart(pq, plenty):
    import torch
    rng = np.random.default_rng(1)
    apart, d = (1 << 31) + 24, 1000
    flat = torch.empty(2 * apart + 8 * d, dtype=torch.bfloat16, device="cuda")

    def view(at):
        return flat.as_strided((3, d), (apart, 1), at)

    x, res, y = view(0), view(d), view(2 * d)
    xs = torch.from_numpy(rng.normal(0, 1, (3, d)).astype(np.float32)).to(torch.bfloat16).cuda()
    x.copy_(xs)
    res.copy_(xs * 3)
    w = torch.ones(d, device="cuda")
    want = pq.rms_norm(xs, w, residual=xs * 3)
    got = pq.rms_norm(x, w, residual=res, h_out=y)
    assert torch.equal(got[0], want[0]) and torch.equal(y, want[1])
    want = pq.rms_norm_backward(xs, xs * 3, w, dres=xs)
    got = pq.rms_norm_backward(x, res, w, dres=x, dh_out=y)
    assert torch.equal(y, want[0]) and torch.equal(got[1], want[1])
    tok = _cuda(np.array([2, 0, 2], dtype=np.int32))
    assert torch.equal(pq.embed(x, tok), xs[tok.long()])
    assert torch.equal(pq.embed_backward(x, tok, 4), pq.embed_backward(xs, tok, 4))
    pq.embed(xs, tok, out=y)
    assert torch.equal(y, xs[tok.long()])
    y.zero_()
    pq.embed_backward(xs, tok, 3, dtable=y)
    assert torch.equal(y, pq.embed_backward(xs, tok, 3))
    pq.adjust_logits(x, repetition=torch.full((3,), 2.0, device="cuda"), history=tok[:, None].contiguous(), out=y)
    assert torch.equal(y, pq.adjust_logits(xs, repetition=torch.full((3,), 2.0, device="cuda"), history=tok[:, None].contiguous()))
    for a, b in zip(pq.sample_logits(x, 5)[:2], pq.sample_logits(xs, 5)[:2]):
        assert torch.equal(a, b)
    del x, res, y, flat


def test_histories_and_masks_far_apart(pq, plenty):
    import torch
    rng = np.random.default_rng(2)
    V, L, apart = 5000, 60, (1 << 31) + 8
    flat = torch.empty(apart + 4096, dtype=torch.int32, device="cuda")
    y = _cuda(rng.normal(0, 1, (2, V)).astype(np.float32))
    h = rng.integers(0, V, (2, L)).astype(np.int32)
    mask = rules.bits(rng.random((2, V)) < 0.5)
    hv, mv = flat.as_strided((2, L), (apart, 1), 0), flat.as_strided((2, mask.shape[1]), (apart, 1), 1000)
    hv.copy_(_cuda(h))
    mv.copy_(_cuda(mask))
    f = torch.full((2,), 0.5, device="cuda")
    assert torch.equal(pq.adjust_logits(y, history=hv, frequency=f, mask=mv),
                       pq.adjust_logits(y, history=_cuda(h), frequency=f, mask=_cuda(mask)))
    del hv, mv, flat


def test_a_vocabulary_of_many_slices(pq, plenty):
    """One row of 2^28 columns: 65536 slices' keys for one draw."""
    import torch
    V = 1 << 28
    y = torch.zeros(1, V, device="cuda")
    ids = [V - 1, 5, V // 2 + 3, 4096 * 777, 4095]
    for k, v in enumerate(ids):
        y[0, v] = 5.0 - k
    values, got, drawn = pq.sample_logits(y, 7, u=torch.zeros(1, device="cuda"))
    assert got[0].tolist() == ids + [0, 1] and values[0].tolist() == [5.0, 4.0, 3.0, 2.0, 1.0, 0.0, 0.0]
    assert int(drawn) == V - 1
    out = pq.adjust_logits(y, bias_ids=_cuda(np.array([V - 1, V - 2], dtype=np.int32)),
                           bias_values=_cuda(np.array([-np.inf, 7.0], dtype=np.float32)), out=y)
    assert float(out[0, V - 1]) == -np.inf and float(out[0, V - 2]) == 7.0 and float(out[0, 5]) == 4.0


@pytest.mark.parametrize("d", [128, 129, 512, 513, 1024, 1025, 2048, 2049, 4096, 4097, 8192, 8193, 16384, 16385])
def test_widths_next_to_the_forms_borders(pq, d):
    rng = np.random.default_rng(d)
    h, u = (rng.normal(0, 2, (5, d)).astype(np.float32) for _ in range(2))
    w = rng.normal(1, 0.2, d).astype(np.float32)
    y, _, _, _ = pq.rms_norm(_cuda(h), _cuda(w))
    n = norm.forward(h.astype(np.float64), w, 1e-6, 0.0)
    assert np.all(np.abs(_np(y) - n) <= 1.01 * 5 * U32 * np.abs(n))
    dh, dw = pq.rms_norm_backward(_cuda(u), _cuda(h), _cuda(w))
    want, want_dw, size = norm.backward(u.astype(np.float64), h.astype(np.float64), w, 1e-6, 0.0)
    assert np.all(np.abs(_np(dh) - want) <= 1.01 * (8 * U32 * size + U32 * np.abs(want)))
    assert np.all(np.abs(_np(dw) - want_dw) <= 1.01 * 84 * U32 * np.sum(np.abs(u * h) / norm.rms(h.astype(np.float64), 1e-6), axis=0))


@pytest.mark.parametrize("M,d", [(256, 2560), (257, 2560), (257, 4096), (256, 4104), (257, 4104), (257, 8192)])
def test_row_counts_next_to_the_forms_borders(pq, M, d):
    """Few wide rows take more threads each than many."""
    import torch
    rng = np.random.default_rng(M + d)
    x, res = (rng.normal(0, 2, (M, d)).astype(np.float32) for _ in range(2))
    w = rng.normal(1, 0.2, d).astype(np.float32)
    codes = d % 16 == 0
    y, h, q, s = pq.rms_norm(_cuda(x), _cuda(w), residual=_cuda(res), out_dtype=torch.float32, want_codes=codes)
    want_h = norm.add(x.astype(np.float64), res.astype(np.float64), False)
    assert np.array_equal(_np(h), want_h)
    n = norm.forward(want_h, w, 1e-6, 0.0)
    assert np.all(np.abs(_np(y) - n) <= 1.01 * 4.04 * U32 * np.abs(n) + 2.0 ** -126)
    if codes:
        q2, s2 = pq.fp8_quantize(y)
        assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2)


@pytest.mark.parametrize("n,V,d", [(1024, 32768, 24), (1025, 32768, 24), (1024, 32769, 24), (1024, 16384, 513),
                                   (1024, 16385, 513), (8223, 40, 8), (8224, 40, 8), (4096, 400, 2048), (4097, 400, 2048)])
def test_token_counts_next_to_the_forms_borders(pq, n, V, d):
    rng = np.random.default_rng(n + V)
    tok = np.where(rng.random(n) < 0.4, V - 1, rng.integers(0, V, n)).astype(np.int32)
    dout = rng.normal(0, 1, (n, d)).astype(np.float32)
    got = _np(pq.embed_backward(_cuda(dout), _cuda(tok), V))
    want, size, count = embedding.gradient(dout.astype(np.float64), tok, V, 1.0)
    assert np.all(np.abs(got - want) <= 1.01 * (np.minimum(400, np.maximum(count - 1, 0))[:, None] + 2) * U32 * size)


def test_calls_at_once_on_two_streams(pq):
    """The operators of two batches, enqueued in turn on two streams, against one after the other."""
    import torch
    rng = np.random.default_rng(3)

    def batch():
        M, d, V = 200, 1200, 20011
        return dict(x=_cuda(rng.normal(0, 1, (M, d)).astype(np.float32)), w=_cuda(rng.normal(1, 0.1, d).astype(np.float32)),
                    tok=_cuda(rng.integers(0, V, M).astype(np.int32)), table=_cuda(rng.normal(0, 1, (V, d)).astype(np.float32)),
                    y=_cuda(rng.normal(0, 1, (M, V)).astype(np.float32)), h=_cuda(rng.integers(0, V, (M, 4000)).astype(np.int32)),
                    f=torch.full((M,), 0.25, device="cuda"), u=_cuda(rng.random(M).astype(np.float32)), V=V)

    def run(b, stream=None):
        e = pq.embed(b["table"], b["tok"], stream=stream)
        y, h, q, s = pq.rms_norm(e, b["w"], residual=b["x"], want_codes=False, stream=stream)
        dh, dw = pq.rms_norm_backward(y, h, b["w"], dres=b["x"], stream=stream)
        g = pq.embed_backward(dh, b["tok"], b["V"], stream=stream)
        a = pq.adjust_logits(b["y"], history=b["h"], frequency=b["f"], stream=stream)
        v, i, t = pq.sample_logits(b["y"], 16, u=b["u"], history=b["h"], frequency=b["f"], stream=stream)
        return e, y, h, dh, dw, g, a, v, i, t

    batches = [batch(), batch()]
    want = [run(b) for b in batches]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = [run(b, s) for b, s in zip(batches, streams)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))
