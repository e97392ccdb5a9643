"""Results that lie in what a call reads are refused through the Python calls, too, and
leave it as it was; results between its rows, columns of one wider matrix, are written."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pq():
    import packed_quantized_lm_amd as pq
    return pq


def _make(*shape):
    import torch
    return torch.from_numpy(np.random.default_rng(len(shape)).normal(0, 1, shape).astype(np.float32)).cuda()


def test_refused(pq):
    import torch
    M, d = 6, 64
    room = _make(40, d)
    w, tok = torch.ones(d, device="cuda"), torch.arange(M, dtype=torch.int32, device="cuda")
    flat = room.view(-1)
    shifted = flat[d // 2:d // 2 + M * d].view(M, d)
    before = room.clone()
    for call in (lambda: pq.rms_norm(_make(M, d), w, residual=room[:M], h_out=room[1:M + 1]),
                 lambda: pq.rms_norm(room[:M], w, residual=_make(M, d), h_out=shifted),
                 lambda: pq.rms_norm(_make(M, d), room[2], residual=_make(M, d), h_out=room[:M]),
                 lambda: pq.rms_norm_backward(room[:M], _make(M, d), w, dh_out=shifted),
                 lambda: pq.rms_norm_backward(_make(M, d), room[:M], w, dh_out=room[1:M + 1]),
                 lambda: pq.rms_norm_backward(_make(M, d), _make(M, d), w, dres=room[:M], dh_out=room[1:M + 1]),
                 lambda: pq.embed(room, tok, out=room[3:3 + M]), lambda: pq.embed(room[:20], tok, out=room[19:19 + M]),
                 lambda: pq.embed_backward(room[:M], tok, 8, dtable=room[4:12]),
                 lambda: pq.embed_backward(room[:M], tok, 8, dtable=room[4:12], accumulate=True),
                 lambda: pq.adjust_logits(room[:M], out=room[1:M + 1]), lambda: pq.adjust_logits(room[:M], out=shifted)):
        with pytest.raises(RuntimeError, match="overlap"):
            call()
    torch.cuda.synchronize()
    assert torch.equal(room, before)


def test_columns_of_one_matrix(pq):
    """Every operand a range of columns of the same rows, results among them."""
    import torch
    M, d = 9, 40
    room = _make(M, 8 * d)
    part = [room[:, i * d:(i + 1) * d] for i in range(8)]
    w, tok = torch.ones(d, device="cuda"), torch.arange(M, dtype=torch.int32, device="cuda") % 5
    want = pq.rms_norm(part[0].contiguous(), w, residual=part[1].contiguous())
    got = pq.rms_norm(part[0], w, residual=part[1], h_out=part[2])
    assert torch.equal(got[0], want[0]) and torch.equal(part[2], want[1])
    want = pq.rms_norm_backward(part[0].contiguous(), part[2].contiguous(), w, dres=part[1].contiguous())
    got = pq.rms_norm_backward(part[0], part[2], w, dres=part[1], dh_out=part[3])
    assert torch.equal(part[3], want[0]) and torch.equal(got[1], want[1])
    want = pq.embed(part[0].contiguous(), tok)
    pq.embed(part[0], tok, out=part[4])
    assert torch.equal(part[4], want)
    want = pq.embed_backward(part[4].contiguous(), tok, M)
    pq.embed_backward(part[4], tok, M, dtable=part[5])
    assert torch.equal(part[5], want)
    kw = dict(history=tok[:, None].contiguous(), repetition=torch.full((M,), 3.0, device="cuda"))
    want = pq.adjust_logits(part[0].contiguous(), **kw)
    pq.adjust_logits(part[0], out=part[6], **kw)
    assert torch.equal(part[6], want)
    # rows of the result between the input's, with another stride
    flat = _make(2, 4096).view(-1)
    x, y = flat.as_strided((3, 40), (1000, 1), 0), flat.as_strided((4, 40), (950, 1), 100)
    want = pq.adjust_logits(x.contiguous())
    between = flat.as_strided((3, 40), (920, 1), 200)  # at 200, 1120 and 2040: x's last row ends there
    pq.adjust_logits(x, out=between)
    assert torch.equal(between, want)
    with pytest.raises(RuntimeError, match="overlap"):
        pq.adjust_logits(y, out=flat.as_strided((4, 40), (940, 1), 110))
    for t in (part[0], part[1]):  # the results themselves, in place
        assert pq.adjust_logits(t, out=t, **kw) is t
