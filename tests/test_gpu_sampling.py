"""Penalties, biases and masks on logits and the draw from them, against the
oracle: every operation is one fp32 rounding, so adjusted logits, order and
indices are held bit for bit (bf16 outputs are their one rounding), and the draw,
in fp64 on both sides, exactly; uniform numbers next to a border are moved off it
by more than the two sides' exponentials can differ (1e-12)."""
import numpy as np
import pytest

from oracle import rules

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module")
def pq():
    import packed_quantized_lm_amd as pq
    return pq


def _cuda(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Case:
    """Rows with rules of every kind, in numpy and on the GPU."""

    def __init__(self, M, V, L, B, seed, type="f32", history=True, bias=True, mask=True, mask_rows=True, shared=False):
        import torch
        rng = np.random.default_rng(seed)
        y = torch.from_numpy((rng.normal(0, 2.5, (M, V))).astype(np.float32))
        self.M, self.V = M, V
        self.y = (y.to(torch.bfloat16) if type == "bf16" else y).cuda()
        self.values = self.y.float().cpu().numpy()
        self.kw, self.rows = {}, [dict() for _ in range(M)]
        if history:
            h = np.minimum((V * rng.random((M, L)) ** 3).astype(np.int32), V - 1)
            h[rng.random((M, L)) < 0.02] = -1
            h[rng.random((M, L)) < 0.02] = V
            lens = rng.integers(0, L + 1, M).astype(np.int32)
            lens[0] = L
            lens[M // 2] = 0 if M > 1 else L
            prompts = (rng.random(M) * lens).astype(np.int32)
            rho, beta, alpha = (rng.uniform(a, b, M).astype(np.float32) for a, b in ((0.8, 1.5), (-0.3, 0.6), (-0.3, 0.6)))
            self.kw.update(history=_cuda(h), lengths=_cuda(lens), prompt_lengths=_cuda(prompts), repetition=_cuda(rho),
                           frequency=_cuda(beta), presence=_cuda(alpha))
            for m in range(M):
                self.rows[m].update(history=h[m, :lens[m]], prompt=int(prompts[m]), repetition=rho[m], frequency=beta[m],
                                    presence=alpha[m])
        if bias:
            ids = rng.integers(-1, V + 1, (M, B)).astype(np.int32)
            vals = rng.normal(0, 3, (M, B)).astype(np.float32)
            vals[rng.random((M, B)) < 0.2] = -INF
            if shared:
                ids[:], vals[:] = ids[:1], vals[:1]
            self.kw.update(bias_ids=_cuda(ids[0] if shared else ids), bias_values=_cuda(vals[0] if shared else vals))
            for m in range(M):
                self.rows[m]["bias"] = list(zip(ids[m], vals[m]))
        if mask:
            R = 3 if mask_rows else M
            table = rng.random((R, V)) < np.array([[0.5], [3.0 / V], [0.0]])[np.arange(R) % 3]
            at = rng.integers(-1, R + 1, M).astype(np.int32) if mask_rows else np.arange(M)
            self.kw.update(mask=_cuda(rules.bits(table)))
            if mask_rows:
                self.kw.update(mask_rows=_cuda(at))
            for m in range(M):
                if 0 <= at[m] < R:
                    self.rows[m]["mask"] = table[at[m]]
        self.want = np.stack([rules.adjust(self.values[m], **self.rows[m]) for m in range(M)])
        self.u = rng.random(M).astype(np.float32)
        self.tau = rng.uniform(0.3, 2.0, M).astype(np.float32)
        t = [rules.top(row, min(16, V)) for row in self.want]
        self.best = np.stack([v for v, _ in t]), np.stack([i for _, i in t])

    def tops(self, K):
        return self.best[0][:, :K], self.best[1][:, :K]

    def draws(self, K):
        values, ids = self.tops(K)
        out = np.zeros(self.M, dtype=np.int32)
        for m in range(self.M):
            with np.errstate(all="ignore"):
                w = np.exp((values[m].astype(np.float64) - values[m, 0]) / np.float64(self.tau[m]))
            border = np.cumsum(w) / w.sum()
            while np.any(np.abs(border - np.float64(self.u[m])) < 1e-9):
                self.u[m] = np.float32(self.u[m] * 0.99)
            out[m] = rules.draw(values[m], ids[m], self.u[m], self.tau[m])
        return out


def _same(got, want, what):
    assert got.shape == want.shape and np.array_equal(np.isnan(got), np.isnan(want)), what
    fine = ~np.isnan(want)
    assert np.array_equal(got[fine], want[fine]), f"{what}: {np.sum(got[fine] != want[fine])} values differ"


SHAPES = [(1, 1, 1, 1), (2, 7, 5, 3), (3, 8, 40, 8), (1, 33, 9, 2), (5, 1000, 300, 40), (2, 2048, 64, 5), (3, 2049, 2000, 20),
          (1, 50021, 700, 1023), (2, 16390, 5000, 64), (130, 40000, 50, 7), (600, 9000, 33, 3), (1030, 300, 20, 5), (1100, 3, 2, 2), (1100, 9, 5, 2),
          (130, 40000, 8000, 7), (300, 30000, 9000, 4), (130, 20000, 4000, 9)]  # the last three: histories sorted by slices first


@pytest.mark.parametrize("type", ["f32", "bf16"])
@pytest.mark.parametrize("M,V,L,B", SHAPES)
def test_all_rules(pq, M, V, L, B, type):
    import torch
    c = Case(M, V, L, B, seed=M + V, type=type)
    got = pq.adjust_logits(c.y, **c.kw)
    assert got.dtype == c.y.dtype
    want = torch.from_numpy(c.want).to(c.y.dtype).float().numpy()
    _same(got.float().cpu().numpy(), want, "adjusted")
    K = min(16, V)
    draws = c.draws(K)
    values, ids, samples = pq.sample_logits(c.y, K, u=_cuda(c.u), temperature=_cuda(c.tau), **c.kw)
    want_v, want_i = c.tops(K)
    assert np.array_equal(ids.cpu().numpy(), want_i)
    _same(values.cpu().numpy(), want_v, "largest")
    assert np.array_equal(samples.cpu().numpy(), draws)


@pytest.mark.parametrize("rules_of", [dict(history=False), dict(bias=False), dict(mask=False), dict(mask_rows=False),
                                      dict(shared=True), dict(history=False, bias=False),
                                      dict(history=False, mask=False), dict(bias=False, mask=False),
                                      dict(history=False, bias=False, mask=False)])
def test_each_rule_alone_and_every_k(pq, rules_of):
    for M, V in ((4, 3001), (200, 12345)):
        c = Case(M, V, 90, 30, seed=V, **rules_of)
        _same(pq.adjust_logits(c.y, **c.kw).cpu().numpy(), c.want, str(rules_of))
        for K in (1, 2, 5, 15):
            values, ids, none = pq.sample_logits(c.y, K, **c.kw)
            want_v, want_i = c.tops(K)
            assert none is None and np.array_equal(ids.cpu().numpy(), want_i)
            _same(values.cpu().numpy(), want_v, "largest")


@pytest.mark.parametrize("V", [5000, 300000])
def test_ties_sorted_and_equal_rows(pq, V):
    """Orders that are hard on a bound: all equal, few values, rising, falling, one workgroup's, one thread's or fifteen threads' best."""
    rng = np.random.default_rng(V)
    y = np.stack([np.zeros(V), np.full(V, -INF), rng.integers(0, 3, V), np.arange(V), -np.arange(V),
                  np.where(np.arange(V) // 8 % 256 == 7, 5.0, 0.0), np.where(np.arange(V) < V - 9, -INF, 1.0),
                  rng.permutation(V), np.where(np.arange(V) // 8 % 256 < 15, rng.permutation(V), -1)]).astype(np.float32)
    y[0, 3] = -0.0
    for M in (1, 9, 512):
        rows = np.arange(M) % 9
        t = _cuda(y)[_cuda(rows)].contiguous()
        values, ids, samples = pq.sample_logits(t, 16, u=_cuda(np.full(M, 0.999, dtype=np.float32)), temperature=0.7)
        for m in range(min(M, 18)):
            v, i = rules.top(y[rows[m]], 16)
            assert np.array_equal(ids[m].cpu().numpy(), i), (M, m)
            assert np.array_equal(values[m].cpu().numpy(), v)
            if m in (1, 10):
                assert int(samples[m]) == -1


@pytest.mark.parametrize("M,V", [(1, 2048), (1, 5000), (1030, 4096), (300, 20000)])
def test_rows_whose_largest_lie_together(pq, M, V):
    """Few threads hold more of the largest than the list of candidates: a sixteenth of the columns without a
    large value, one wave's sixteen threads rising, and one thread's columns among them."""
    rng = np.random.default_rng(V)
    c = np.arange(V)
    lane, order = c // 8 % 16, rng.permutation(V) / V
    thread = c // 8 % 256
    y = np.stack([np.where(lane == 0, -3.0, np.where(lane < 8, 1 + order, -10 - order)),
                  np.where(lane == 5, -INF, order),
                  np.where(thread < 16, thread + 0.001 * (c // 2048 * 8 + c % 8), -1.0 - order),
                  np.where(thread < 32, 100 - thread + 0.001 * (c % 8), -1.0),
                  np.where(thread % 64 < 16, 7.0, order), np.where(lane < 15, 2.0, -INF)]).astype(np.float32)
    rows = np.arange(M) % len(y)
    for K in (1, 5, 16):
        values, ids, _ = pq.sample_logits(_cuda(y)[_cuda(rows)].contiguous(), K)
        for m in range(min(M, 12)):
            v, i = rules.top(y[rows[m]], K)
            assert np.array_equal(ids[m].cpu().numpy(), i), (K, m)
            assert np.array_equal(values[m].cpu().numpy(), v)
    for r in range(len(y)) if M == 1 else ():  # each row alone
        values, ids, _ = pq.sample_logits(_cuda(y[r:r + 1]), 16)
        assert np.array_equal(ids[0].cpu().numpy(), rules.top(y[r], 16)[1]), r


def test_numbers_that_are_not_numbers(pq):
    V = 700
    y = np.random.default_rng(0).normal(0, 1, (6, V)).astype(np.float32)
    y[0, [9, 600]] = np.nan
    y[1, [77, 5]] = INF
    y[2, 33] = -np.nan
    y[3] = np.nan
    y[4, 10] = np.nan  # behind the mask
    y[5, 10] = INF
    mask = np.ones((6, V), dtype=bool)
    mask[4:, 10] = False
    u = np.full(6, 0.5, dtype=np.float32)
    values, ids, samples = pq.sample_logits(_cuda(y), 4, u=_cuda(u), mask=_cuda(rules.bits(mask)))
    adjusted = pq.adjust_logits(_cuda(y), mask=_cuda(rules.bits(mask))).cpu().numpy()
    for m in range(6):
        row = rules.adjust(y[m], mask=mask[m])
        _same(adjusted[m], row, "adjusted")
        v, i = rules.top(row, 4)
        assert np.array_equal(ids[m].cpu().numpy(), i)
        _same(values[m].cpu().numpy(), v, "largest")
        assert int(samples[m]) == rules.draw(v, i, 0.5, 1.0)
    # a ban takes +inf and NaN too, and biases of other kinds follow fp32
    ids = _cuda(np.array([5, 77, 3], dtype=np.int32))
    vals = _cuda(np.array([-INF, -INF, INF], dtype=np.float32))
    _same(pq.adjust_logits(_cuda(y), bias_ids=ids, bias_values=vals).cpu().numpy(),
          np.stack([rules.adjust(r, bias=[(5, -INF), (77, -INF), (3, INF)]) for r in y]), "bans")


def test_draw_at_its_ends(pq):
    y = np.zeros((5, 64), dtype=np.float32)
    y[:, 20:] = -INF
    u = np.array([0.0, 1.0 - 2.0 ** -24, 0.5, 1.0, np.nan], dtype=np.float32)
    _, ids, samples = pq.sample_logits(_cuda(y), 16, u=_cuda(u), temperature=2.0)
    assert samples.cpu().tolist() == [0, 15, 8, 15, 15]
    tau = np.array([0.0, -1.0, np.nan, INF, 1e-30], dtype=np.float32)
    y[:, 3] = 1.0
    _, _, samples = pq.sample_logits(_cuda(y), 16, u=_cuda(np.full(5, 0.99, dtype=np.float32)), temperature=_cuda(tau))
    assert samples.cpu().tolist() == [3, 3, 3, 15, 3]


def test_strides_and_in_place(pq):
    import torch
    c = Case(37, 3001, 70, 20, seed=5)
    wide = torch.full((37, 3100), 7.0, device="cuda")
    wide[:, 50:3051] = c.y
    kw = dict(c.kw)
    for name in ("history", "bias_ids", "bias_values", "mask"):  # rows with something beside them
        t = kw[name]
        kw[name] = torch.cat([t, t], dim=1)[:, :t.shape[1]]
    out = torch.full((37, 3050), 9.0, device="cuda")
    got = pq.adjust_logits(wide[:, 50:3051], out=out[:, 4:3005], **kw)
    _same(got.cpu().numpy(), c.want, "strided")
    assert (out[:, :4] == 9).all() and (out[:, 3005:] == 9).all() and torch.equal(wide[:, 50:3051], c.y)
    values, ids, _ = pq.sample_logits(wide[:, 50:3051], 9, **kw)
    assert np.array_equal(ids.cpu().numpy(), c.tops(9)[1])
    view = wide[:, 50:3051]
    assert pq.adjust_logits(view, out=view, **kw) is view
    _same(view.cpu().numpy(), c.want, "in place")
    assert (wide[:, :50] == 7).all() and (wide[:, 3051:] == 7).all()
    for rules_of in (dict(mask=False), dict(history=False, mask=False), dict(bias=False, mask=False)):
        c = Case(5, 3001, 70, 20, seed=6, **rules_of)
        pq.adjust_logits(c.y, out=c.y, **c.kw)
        _same(c.y.cpu().numpy(), c.want, "in place")


def test_lengths_outside_the_history(pq):
    V, L = 100, 10
    h = np.arange(2 * L, dtype=np.int32).reshape(2, L)
    y = np.ones((2, V), dtype=np.float32)
    rho = _cuda(np.full(2, 2.0, dtype=np.float32))
    got = pq.adjust_logits(_cuda(y), history=_cuda(h), lengths=_cuda(np.array([-5, 99], dtype=np.int32)), repetition=rho,
                           prompt_lengths=_cuda(np.array([-1, 1000], dtype=np.int32))).cpu().numpy()
    assert (got[0] == 1).all() and (got[1, 10:20] == 0.5).all() and (np.delete(got[1], range(10, 20)) == 1).all()
    got = pq.adjust_logits(_cuda(y), history=_cuda(h), repetition=rho).cpu().numpy()  # all of it, all generated
    assert (got[0, :10] == 0.5).all() and (got[0, 10:] == 1).all()


def test_a_long_history_of_one_token(pq):
    V, L = 4000, 1 << 20
    h = np.full((1, L), 1234, dtype=np.int32)
    y = np.zeros((1, V), dtype=np.float32)
    got = pq.adjust_logits(_cuda(y), history=_cuda(h), frequency=_cuda(np.array([1.0], dtype=np.float32))).cpu().numpy()
    assert got[0, 1234] == -(2.0 ** 20) and np.count_nonzero(got) == 1


def test_no_rows_and_empty_lists(pq):
    import torch
    y = torch.ones(0, 50, device="cuda")
    assert pq.adjust_logits(y).shape == (0, 50)
    v, i, s = pq.sample_logits(y, 3, u=torch.ones(0, device="cuda"))
    assert v.shape == (0, 3) and i.shape == (0, 3) and s.shape == (0,)
    y = torch.randn(3, 50, device="cuda")
    none, nof = torch.zeros(3, 0, dtype=torch.int32, device="cuda"), torch.zeros(3, 0, device="cuda")
    got = pq.adjust_logits(y, history=none, bias_ids=none, bias_values=nof,
                           mask=torch.zeros(0, 2, dtype=torch.int32, device="cuda"),
                           mask_rows=torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert torch.equal(got, y)


def test_refused_on_the_gpu(pq):
    import torch
    y, h = torch.ones(3, 64, device="cuda"), torch.zeros(3, 8, dtype=torch.int32, device="cuda")
    vec, ids = torch.ones(3, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    for kw in (dict(history=h.long()), dict(history=h[:2]), dict(history=h.cpu()), dict(lengths=ids),
               dict(history=h, lengths=ids[:2]), dict(history=h, lengths=vec), dict(repetition=vec.double()),
               dict(bias_ids=h), dict(bias_ids=h, bias_values=vec), dict(bias_ids=h, bias_values=h),
               dict(mask=h), dict(mask=h[:2, :2]), dict(mask_rows=ids), dict(mask=h[:, :2], mask_rows=vec),
               dict(bias_ids=torch.zeros(1024, dtype=torch.int32, device="cuda"), bias_values=torch.zeros(1024, device="cuda"))):
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            pq.adjust_logits(y, **kw)
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            pq.sample_logits(y, 4, **kw)
    for call in (lambda: pq.sample_logits(y, 0), lambda: pq.sample_logits(y, 17), lambda: pq.sample_logits(y[:, :3], 4),
                 lambda: pq.sample_logits(y, 4, u=vec[:2]), lambda: pq.sample_logits(y, 4, u=vec, temperature=0.0),
                 lambda: pq.sample_logits(y, 4, u=vec, temperature=vec[:2]),
                 lambda: pq.adjust_logits(y, out=torch.ones(3, 63, device="cuda")),
                 lambda: pq.adjust_logits(y, out=y.bfloat16())):
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            call()
    torch.cuda.synchronize()


def test_equal_calls_side_stream_and_graph(pq):
    import torch
    c = Case(40, 30011, 500, 64, seed=11)
    u, tau = _cuda(c.u), _cuda(c.tau)

    def step():
        return (pq.adjust_logits(c.y, **c.kw), *pq.sample_logits(c.y, 16, u=u, temperature=tau, **c.kw))

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
    rng = np.random.default_rng(0)
    for k in range(3):  # the history, its lengths and the masks move on between replays
        c.kw["history"].copy_(_cuda(rng.integers(0, 30011, (40, 500)).astype(np.int32)))
        c.kw["lengths"].copy_(_cuda(rng.integers(0, 501, 40).astype(np.int32)))
        c.kw["mask"].copy_(_cuda(rules.bits(rng.random((3, 30011)) < 0.3)))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        assert all(torch.equal(a, b) for a, b in zip(got, step()))
