"""Histories sorted by slices before the rules are applied, in slices of 2048 and of 4096
columns, held to the oracle bit for bit as the other forms are; from two streams at once,
and replayed from graphs, alone and two at a time, whose histories and lengths move on."""
import numpy as np
import pytest

import routed_shapes
from test_gpu_sampling import Case, _cuda, _same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pq():
    import packed_quantized_lm_amd as pq
    return pq


@pytest.mark.parametrize("type", ["f32", "bf16"])
@pytest.mark.parametrize("M,V,L,B,columns", [s for s in routed_shapes.SHAPES if s[0] * s[2] < 1e7])
def test_all_rules(pq, M, V, L, B, columns, type):
    import torch
    c = Case(M, V, L, B, seed=M + V + L, type=type)
    got = pq.adjust_logits(c.y, **c.kw)
    _same(got.float().cpu().numpy(), torch.from_numpy(c.want).to(c.y.dtype).float().numpy(), "adjusted")
    for K in (1, 16):
        draws = c.draws(K)
        values, ids, samples = pq.sample_logits(c.y, K, u=_cuda(c.u), temperature=_cuda(c.tau), **c.kw)
        want_v, want_i = c.tops(K)
        assert np.array_equal(ids.cpu().numpy(), want_i)
        _same(values.cpu().numpy(), want_v, "largest")
        assert np.array_equal(samples.cpu().numpy(), draws)
    out = c.y.clone()
    assert pq.adjust_logits(out, out=out, **c.kw) is out and torch.equal(out, got)


@pytest.mark.parametrize("M,V,L,B,columns", [s for s in routed_shapes.SHAPES if s[0] * s[2] >= 1e7])
def test_longest(pq, M, V, L, B, columns):
    """Long histories of many rows: counts by scatter, each step in fp32 as the oracle takes it."""
    import torch
    gen = torch.Generator(device="cuda")
    gen.manual_seed(M)
    y = 2 * torch.randn(M, V, generator=gen, device="cuda")
    h = (V * torch.rand(M, L, generator=gen, device="cuda").pow(3)).int() - 1
    n = (torch.rand(M, generator=gen, device="cuda") * (L + 1)).int()
    n[0], n[1] = L, 0
    f = torch.rand(M, generator=gen, device="cuda")
    held = torch.arange(L, device="cuda") < n[:, None]
    count = torch.zeros(M, V + 1, device="cuda")
    count.scatter_add_(1, torch.where(held & (h >= 0), h, V).long(), torch.ones(M, L, device="cuda"))
    want = y - f[:, None] * count[:, :V]
    got = pq.adjust_logits(y, history=h, lengths=n, frequency=f)
    assert torch.equal(got, torch.where(count[:, :V] > 0, want, y))
    values, ids, _ = pq.sample_logits(y, 16, history=h, lengths=n, frequency=f)
    order = torch.sort(got, dim=1, descending=True, stable=True)
    assert torch.equal(values, order.values[:, :16]) and torch.equal(ids.long(), order.indices[:, :16])


class Step:
    def __init__(self, pq, M, V, L, B, seed, type="f32"):
        self.pq, self.c = pq, Case(M, V, L, B, seed=seed, type=type)
        self.u, self.tau = _cuda(self.c.u), _cuda(self.c.tau)
        self.M, self.V, self.L, self.rng = M, V, L, np.random.default_rng(seed)

    def __call__(self, stream=None):
        c = self.c
        return (self.pq.adjust_logits(c.y, stream=stream, **c.kw),
                *self.pq.sample_logits(c.y, 16, u=self.u, temperature=self.tau, stream=stream, **c.kw))

    def move_on(self):
        rng, kw = self.rng, self.c.kw
        kw["history"].copy_(_cuda(rng.integers(-1, self.V + 1, (self.M, self.L)).astype(np.int32)))
        lens = rng.integers(0, self.L + 1, self.M).astype(np.int32)
        lens[:2] = 0, self.L
        kw["lengths"].copy_(_cuda(lens))
        kw["prompt_lengths"].copy_(_cuda((rng.random(self.M) * lens).astype(np.int32)))


def _equal(a, b):
    import torch
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_two_streams_at_once(pq):
    import torch
    steps = [Step(pq, 200, 20011, 8000, 5, 1), Step(pq, 260, 20011, 14000, 5, 2), Step(pq, 200, 20011, 8000, 5, 3, "bf16")]
    want = [s() for s in steps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(3):
        got = [s(stream=t) for s, t in zip(steps, streams)]
        torch.cuda.synchronize()
        assert all(_equal(a, b) for a, b in zip(got, want))


def test_graph_replayed_as_histories_move_on(pq):
    import torch
    for shape in ((130, 20000, 7000, 9), (260, 20011, 14000, 40)):
        step = Step(pq, *shape, seed=4)
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = step()
        for _ in range(4):
            step.move_on()
            graph.replay()
            torch.cuda.synchronize()
            got = [t.clone() for t in held]
            assert _equal(got, step())
        del graph


def test_two_graphs_at_once(pq):
    import torch
    steps = [Step(pq, 130, 20000, 7000, 9, 5), Step(pq, 130, 20000, 7000, 9, 6)]
    for s in steps:
        s()
    torch.cuda.synchronize()
    graphs, held = [], []
    for s in steps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held.append(s())
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        for s in steps:
            s.move_on()
        torch.cuda.synchronize()
        for g, t in zip(graphs, streams):
            with torch.cuda.stream(t):
                g.replay()
        torch.cuda.synchronize()
        got = [[t.clone() for t in h] for h in held]
        assert all(_equal(a, s()) for a, s in zip(got, steps))
