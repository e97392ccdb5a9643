"""Log probabilities of ordinary rows on the GPU against fp64, within what the
kernels' own sums allow: terms in fp32, sums of eight in fp32, everything else
in fp64.

Tolerance, absolute in logp, in units of u = 2^-24: a term exp(-x) of Z is off by
2 x u for its difference of two logits and its exponent, 2 u for the
exponential and 2 u for each link that rescales it (a thread's vectors, 6
merges of lanes, one of waves, one for eight slices); eight terms are added by
three roundings; the result is rounded once.  So
  |d logp| <= (2 E[x] + 2 + 2 links + 3 + |logp|) u,  E under the row's probabilities.
"""
import numpy as np
import pytest

from gpu_util import say

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from packed_quantized_lm_amd import load_library
    load_library()


#    M, V, vectors a thread meets at most, slices at most
SIZES = [(2, 151936, 3, 37), (100, 151936, 3, 37), (240, 151936, 19, 1), (2047, 32000, 16, 2), (40, 9001, 2, 1),
         (300, 4097, 3, 1), (64, 257, 1, 1)]


@pytest.mark.parametrize("M,V,vectors,slices", SIZES)
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("spread", [1.0, 4.0])
def test_log_probabilities_of_ordinary_rows(M, V, vectors, slices, dtype, spread):
    import torch
    from packed_quantized_lm_amd import policy_loss, token_logp
    say(f"logp precision M={M} V={V} {dtype} spread={spread}")
    gen = torch.Generator(device="cuda").manual_seed(V + M)
    y = (torch.randn(M, V, generator=gen, device="cuda") * spread).to(getattr(torch, dtype))
    t = torch.randint(0, V, (M,), generator=gen, device="cuda")
    got = {"token_logp": token_logp(y, t.int())[0]}
    if M < 150 or V < 10000:  # the policy loss cuts its rows by rules of its own
        one = torch.ones(M, device="cuda")
        got["policy_loss"] = policy_loss(y, t.int(), one, one, one, grad_dtype=torch.bfloat16)[1]
    for m in range(0, M, 128):
        part = y[m:m + 128].double()
        x = part.amax(1, keepdim=True) - part
        e = torch.exp(-x)
        z = e.sum(1)
        want = -x.gather(1, t[m:m + 128, None])[:, 0] - torch.log(z)
        links = vectors + 6 + 1 + -(-slices // 8)
        tol = U * (2 * (e * x).sum(1) / z + 2 + 2 * links + 3 + want.abs())
        for name, g in got.items():
            off = (g[m:m + 128].double() - want).abs()
            assert (off <= tol).all(), (name, (off / tol).max())
