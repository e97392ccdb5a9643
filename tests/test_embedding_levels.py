"""The levels of partial sums of the embedding's gradient: a further one wherever a run of
one token could be left with more than 256 parts of the last, so that no term passes through
more than 400 additions.  Counted by the workspace's size, on the CPU; and on the GPU on both
sides of each switch, with one token that holds all but the first entry of the list."""
import ctypes

import numpy as np
import pytest

U32 = 2.0 ** -24
# tokens, levels
SWITCHES = [(31, 0), (32, 1), (8192, 1), (8223, 1), (8224, 2), (9215, 2), (9216, 2), (263167, 2), (263168, 3),
            (294911, 3), (294912, 3), (1 << 20, 3)]


def _up16(b):
    return -(-b // 16) * 16


@pytest.mark.parametrize("n,levels", SWITCHES)
def test_levels(n, levels):
    from packed_quantized_lm_amd import binding
    d, size = 40, ctypes.c_uint64()
    assert binding.load_library().archead_embed_workspace(n, 1 << 20, d, ctypes.byref(size)) == binding.OK
    want = _up16(8 * n)
    if n > 8192:  # sorted by passes: another list, and the tiles' counts of 512 digits
        want += _up16(8 * n) + -(-n // 2048) * 512 * 4
    want += sum(_up16(4 * d * (n // 32 ** (level + 1))) for level in range(levels))
    assert size.value == max(want, 16)


def _additions(n, levels, first):
    """The most additions a term of a run of entries first .. n - 1 passes through: as the kernels add them."""
    parts_beside = 0  # entries or parts that the run's wave adds by itself
    lo, hi = first, n
    for level in range(levels + 1):
        nlo, nhi = -(-lo // 32), hi // 32
        if level == levels or nlo >= nhi:
            parts_beside += hi - lo
            break
        parts_beside += (nlo * 32 - lo) + (hi - nhi * 32)
        lo, hi = nlo, nhi
    return parts_beside + 10 * levels  # within a part eight terms a wave and two joins


@pytest.mark.parametrize("n,levels", SWITCHES)
def test_no_term_passes_through_more_than_400_additions(n, levels):
    assert max(_additions(n, levels, first) for first in range(64)) <= 400


@pytest.mark.gpu
@pytest.mark.parametrize("type", ["f32", "bf16"])
@pytest.mark.parametrize("n", [8223, 8224, 9215, 9216, 263167, 263168, 294911, 294912])
def test_one_token_holds_all_but_the_first(n, type):
    import torch
    from packed_quantized_lm_amd import embed_backward
    d, V = 24, 70000
    rng = np.random.default_rng(n)
    dout = torch.from_numpy(rng.normal(0, 1, (n, d)).astype(np.float32)).cuda()
    dout = dout.to(torch.bfloat16) if type == "bf16" else dout
    tok = torch.full((n,), 6789, dtype=torch.int32, device="cuda")
    tok[n // 2] = 3  # the list's first, once sorted
    got = embed_backward(dout, tok, V, grad_dtype=torch.float32)
    x = dout.double()
    one = x[n // 2].clone()
    x[n // 2] = 0
    want, size = x.sum(0), x.abs().sum(0)
    assert torch.equal(got[3].double(), one)
    assert bool(((got[6789].double() - want).abs() <= 1.01 * 402 * U32 * size).all())
    got[3] = got[6789] = 0
    assert not got.any()
