"""From the norm's codes to an 8-bit head's logits, against the oracle: forward_codes of
given codes and scales, the norm's codes as they reach it, and the serving loop with both
heads, whose logits are checked in every step.

Bounds: the product's are test_gpu_fp8.py's; codes are the nearest to n, which is known to
four fp32 roundings (test_gpu_norm.py's); a packed head's logits are held to 2e-3 of their
row's root mean square, as everywhere."""
import numpy as np
import pytest

from gpu_util import assert_logits_close
from oracle import embedding, fp8, norm
from test_gpu_fp8 import codes_of, tolerance
from test_gpu_model_loop import D, M, STEPS, V, Loop, parts  # noqa: F401
from test_gpu_norm import U32, _codes_are_nearest

pytestmark = pytest.mark.gpu

SHAPES = [(1, 37, 48), (2, 129, 144), (16, 300, 256), (65, 1030, 272), (130, 4097, 1024), (7, 3001, 2576)]


def _np(t):
    return t.double().cpu().numpy()


def _product(q, s, head, out):
    """out is the product of these codes and scales with the head's, within its bound."""
    want, terms = fp8.matmul(codes_of(q), s.cpu().numpy(), codes_of(head.weight), head.scales.cpu().numpy())
    dtype = str(out.dtype).split(".")[1]
    off = np.abs(_np(out) - want) / tolerance(q.shape[0], q.shape[1], dtype, want, terms)
    assert off.max() <= 1, off.max()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("rows,cols,d", SHAPES)
def test_codes_of_hidden_states(rows, cols, d, dtype):
    """forward_codes of the quantiser's codes is forward, bit for bit, and the product of both."""
    import torch
    import packed_quantized_lm_amd as pq
    rng = np.random.default_rng(rows + d)
    head = pq.Fp8Head(torch.from_numpy(rng.normal(0, 0.05, (cols, d)).astype(np.float32)).cuda())
    x = torch.from_numpy((rng.normal(0, 1, (rows, d)) * np.exp(rng.normal(0, 1, (rows, 1)))).astype(np.float32)).cuda()
    q, s = pq.fp8_quantize(x)
    t = getattr(torch, dtype)
    got = head.forward_codes(q, s, out_dtype=t)
    assert got.dtype == t and torch.equal(got, head.forward(x, out_dtype=t))
    _product(q, s, head, got)
    out = torch.full((rows, cols + 5), 3.0, dtype=t, device="cuda")
    assert torch.equal(head.forward_codes(q, s, out=out[:, :cols]), got) and (out[:, cols:] == 3.0).all()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("rows,cols,d", SHAPES)
def test_codes_of_the_norm(rows, cols, d, dtype):
    """The norm's codes are those of its oracle's values, and the logits their product."""
    import torch
    import packed_quantized_lm_amd as pq
    rng = np.random.default_rng(rows * 7 + d)
    head = pq.Fp8Head(torch.from_numpy(rng.normal(0, 0.05, (cols, d)).astype(np.float32)).cuda())
    make = lambda *shape: torch.from_numpy(rng.normal(0, 1, shape).astype(np.float32)).to(torch.bfloat16).cuda()
    x, res, w = make(rows, d), make(rows, d) * 3, make(d)
    _, h, q, s = pq.rms_norm(x, w, residual=res, want_y=False, want_codes=True)
    n = norm.forward(norm.add(_np(x), _np(res), True), _np(w), 1e-6, 0.0)
    _codes_are_nearest(n, codes_of(q), s.cpu().numpy(), 4.04 * U32)
    _product(q, s, head, head.forward_codes(q, s, out_dtype=getattr(torch, dtype)))


class Watched(Loop):
    """The loop, with what the 8-bit head is given kept."""

    def step(self):
        forward_codes = self.head.forward_codes if self.codes else None

        def kept(q, s, **kw):
            self.q, self.s = q, s
            return forward_codes(q, s, **kw)

        if self.codes:
            self.head.forward_codes = kept
        try:
            return super().step()
        finally:
            if self.codes:
                del self.head.forward_codes


@pytest.mark.parametrize("codes", [False, True])
def test_serving_loop_logits(parts, codes):  # noqa: F811
    import torch
    pq, fields, dense, tied, table, weight = parts
    head = tied if codes else pq.PackedHead(fields)
    if not codes:
        head.reserve(M)
    lp = Watched(pq, head, table, weight, codes, seed=6)
    lp.logits = torch.empty(M, V, device="cuda")
    for _ in range(STEPS):
        before, token = lp.stream.clone(), lp.token.cpu().numpy()
        lp.step()
        if codes:
            rows = fp8.decode(codes_of(tied.weight)) * np.repeat(np.repeat(_np(tied.scales), 128, axis=0)[:V], 128,
                                                                 axis=1)[:, :D]
            assert np.all(np.abs(_np(lp.x) - embedding.lookup(rows, token, 0.5)) <= np.abs(_np(lp.x)) * 2.0 ** -7)
            n = norm.forward(norm.add(_np(lp.x), _np(before), True), _np(weight), 1e-6, 0.0)
            _codes_are_nearest(n, codes_of(lp.q), lp.s.cpu().numpy(), 4.04 * U32)
            _product(lp.q, lp.s, tied, lp.logits)
        else:
            assert_logits_close(lp.logits.cpu().numpy(), _np(lp.y) @ dense.T, what="packed head")
    if not codes:
        head.close()
