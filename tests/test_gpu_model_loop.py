"""The operators around the head in the order a model runs them: serving (embedding,
residual sum and norm, the packed or the 8-bit head, rules and draw, and the token
back into the history), eager and as a captured graph, each step against the
oracle; and training (the gradients of norm and embedding around the losses and
the head's backward)."""
import numpy as np
import pytest

from oracle import embedding, forward, losses, norm, rules

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24
V, D, M, STEPS, LONG = 3000, 512, 6, 5, 40


@pytest.fixture(scope="module")
def parts():
    import torch
    import packed_quantized_lm_amd as pq
    from packed_quantized_lm_amd.synth import random_small_head
    fields = random_small_head(V, D, 32, 16, 128, M, seed=21)
    dense = forward.dense_rows(fields, np.arange(V))
    rng = np.random.default_rng(3)
    tied = pq.Fp8Head(torch.from_numpy(dense.astype(np.float32)).cuda())
    table = torch.from_numpy(rng.normal(0, 1, (V, D)).astype(np.float32)).to(torch.bfloat16).cuda()
    weight = torch.from_numpy((1 + 0.1 * rng.normal(0, 1, D)).astype(np.float32)).cuda()
    return pq, fields, dense, tied, table, weight


class Loop:
    """A batch of requests in the middle of their answers; step() draws each one's next token."""

    def __init__(self, pq, head, table, weight, codes, seed):
        import torch
        rng = np.random.default_rng(seed)
        self.pq, self.head, self.table, self.weight, self.codes = pq, head, table, weight, codes
        cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
        self.history = cuda(rng.integers(0, V, (M, LONG)).astype(np.int32))
        self.lengths = cuda(rng.integers(3, LONG - STEPS, M).astype(np.int32))
        self.prompts = (self.lengths - 2).contiguous()
        self.stream = torch.zeros(M, D, dtype=torch.bfloat16, device="cuda")
        self.token = cuda(rng.integers(0, V, M).astype(np.int32))
        self.rep, self.freq = cuda(np.full(M, 1.2, np.float32)), cuda(np.full(M, 0.3, np.float32))
        grammar = rng.random((2, V)) < 0.2
        self.grammar = grammar
        self.mask, self.mask_rows = cuda(rules.bits(grammar)), cuda(np.array([-1, 0, 1, 1, -1, 0], dtype=np.int32))
        self.u = cuda(rng.random(M).astype(np.float32))

    def step(self):
        import torch
        pq = self.pq
        if self.codes:  # a tied 8-bit head: its rows are the embedding, the norm writes what it reads
            x = self.head.embed(self.token, scale=0.5)
            _, h, q, s = pq.rms_norm(x, self.weight, residual=self.stream, want_y=False, want_codes=True,
                                     h_out=self.stream)
            self.logits = self.head.forward_codes(q, s)
        else:
            x = pq.embed(self.table, self.token, scale=0.5)
            y, h, _, _ = pq.rms_norm(x, self.weight, residual=self.stream, h_out=self.stream)
            self.y = y
            self.head.forward_into(y, self.logits, None)
        self.x = x
        values, ids, token = pq.sample_logits(self.logits, 8, u=self.u, temperature=0.9, history=self.history,
                                              lengths=self.lengths, prompt_lengths=self.prompts, repetition=self.rep,
                                              frequency=self.freq, mask=self.mask, mask_rows=self.mask_rows)
        self.token.copy_(token)
        self.history.scatter_(1, self.lengths.long()[:, None], token[:, None])
        self.lengths += 1
        return values, ids, token


def _np(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("codes", [False, True])
def test_serving_loop(parts, codes):
    import torch
    pq, fields, dense, tied, table, weight = parts
    head = tied if codes else pq.PackedHead(fields)
    if not codes:
        head.reserve(M)
    loops = [Loop(pq, head, table, weight, codes, seed=4) for _ in range(2)]
    for lp in loops:
        lp.logits = torch.empty(M, V, device="cuda")
    eager, other = loops
    drawn = []
    rows = None
    if codes:
        from oracle import fp8
        s = np.repeat(np.repeat(_np(tied.scales), 128, axis=0)[:V], 128, axis=1)[:, :D]
        rows = fp8.decode(tied.weight.view(torch.uint8).cpu().numpy()) * s
    for _ in range(STEPS):
        before, token = eager.stream.clone(), eager.token.cpu().numpy()
        h, n = eager.history.cpu().numpy().copy(), eager.lengths.cpu().numpy().copy()
        values, ids, got = eager.step()
        drawn.append(got.cpu().numpy())
        # every step's operators against the oracle on what the one before gave them
        want = embedding.lookup(rows if codes else _np(table), token, 0.5)
        assert np.all(np.abs(_np(eager.x) - want) <= 1.01 * np.abs(want) * (2 * U32 + 2.0 ** -8))
        assert np.array_equal(_np(eager.stream), norm.add(_np(eager.x), _np(before), True))
        want = norm.forward(_np(eager.stream), _np(weight), 1e-6, 0.0)
        if not codes:
            assert np.all(np.abs(_np(eager.y) - want) <= 1.01 * np.abs(want) * (4 * U32 + 2.0 ** -8))
        y = eager.logits.cpu().numpy()
        at = eager.mask_rows.cpu().numpy()
        for m in range(M):
            row = rules.adjust(y[m], history=h[m, :n[m]], prompt=int(eager.prompts[m]), repetition=np.float32(1.2),
                               frequency=np.float32(0.3), mask=eager.grammar[at[m]] if at[m] >= 0 else None)
            v, i = rules.top(row, 8)
            assert np.array_equal(ids[m].cpu().numpy(), i) and np.array_equal(values[m].cpu().numpy(), v)
            assert drawn[-1][m] == rules.draw(v, i, float(eager.u[m]), 0.9)
    # the same loop as a graph: its own warm-up on another state first
    warm = Loop(pq, head, table, weight, codes, seed=5)
    warm.logits = torch.empty(M, V, device="cuda")
    warm.step()
    state = [t.clone() for t in (other.stream, other.token, other.history, other.lengths)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = other.step()
    for t, was in zip((other.stream, other.token, other.history, other.lengths), state):
        t.copy_(was)
    for k in range(STEPS):
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(held[2].cpu().numpy(), drawn[k])
        warm.step()  # eager work between the replays
    for a, b in ((eager.history, other.history), (eager.lengths, other.lengths), (eager.stream, other.stream),
                 (eager.logits, other.logits)):
        assert torch.equal(a, b)
    if not codes:
        torch.cuda.synchronize()
        del graph
        head.close()


def test_training_step(parts):
    """loss(embedding -> residual sum -> norm -> packed head): the chain of the
    operators' gradients against the chain of the oracle's, each within what bf16
    hidden states and gradients (2^-8 each, a few of them) leave of the whole."""
    import torch
    pq, fields, dense, _, table, weight = parts
    rng = np.random.default_rng(8)
    n = 48
    tok = torch.from_numpy(np.minimum((V * rng.random(n) ** 4).astype(np.int32), V - 1)).cuda()
    res = torch.from_numpy(rng.normal(0, 1, (n, D)).astype(np.float32)).to(torch.bfloat16).cuda()
    target = torch.from_numpy(rng.integers(0, V, n).astype(np.int32)).cuda()
    adv = torch.from_numpy(rng.normal(0, 1, n).astype(np.float32)).cuda()
    w = torch.full((n,), 1.0 / n, device="cuda")
    head = pq.PackedHead(fields)
    head.reserve_backward(n)
    x = pq.embed(table, tok, scale=0.5)
    y, h, _, _ = pq.rms_norm(x, weight, residual=res)
    logits, _ = head.forward(y)
    old, _ = pq.token_logp(logits, target)
    loss, logp, dlogits = pq.policy_loss(logits, target, old, adv, w, grad_dtype=torch.bfloat16)
    dy = head.backward(dlogits)
    dh, dweight = pq.rms_norm_backward(dy, h, weight)
    dtable = pq.embed_backward(dh, tok, V, scale=0.5, grad_dtype=torch.float32)
    torch.cuda.synchronize()
    wy = losses.policy(logits.cpu().numpy().astype(np.float64), target.cpu().numpy(), old.cpu().numpy(), adv.cpu().numpy(),
                       w.cpu().numpy(), None, 0.0, 0.2, 0.2)
    want_dh, want_dw, _ = norm.backward(wy[2] @ dense, _np(h), _np(weight), 1e-6, 0.0)
    want_dt, _, _ = embedding.gradient(want_dh, tok.cpu().numpy(), V, 0.5)
    for got, want in ((dh, want_dh), (dweight, want_dw), (dtable, want_dt)):
        off = np.linalg.norm(_np(got) - want) / np.linalg.norm(want)
        assert off < 4 * 2.0 ** -8, off
    head.close()
