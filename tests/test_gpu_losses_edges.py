"""The post-training losses on the GPU where an input is not a number, infinite
or nothing, against what include/archead.h says of such rows and the fp64
oracle; in one workgroup per row, in one slice and in several."""
import math

import numpy as np
import pytest

from gpu_util import say
from oracle import losses

pytestmark = pytest.mark.gpu

SIZES = [(8, 5), (8, 64), (300, 1000), (8, 9001), (6, 50021), (200, 33001)]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from packed_quantized_lm_amd import load_library
    load_library()


def dev(a, dtype="float32"):
    import torch
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype=dtype))).to("cuda")


def batch(M, V):
    """Logits, targets and the other inputs of a policy step on the host, the
    ratios away from the clip's borders."""
    rng = np.random.default_rng(M + V)
    y = rng.normal(0, 2, (M, V)).astype(np.float32)
    t = rng.integers(0, V, M)
    logp = losses.token_logp(y, t)
    old = (logp - rng.uniform(-0.15, 0.15, M)).astype(np.float32)
    ref = (logp + rng.normal(0, 0.3, M)).astype(np.float32)
    adv = np.where(np.arange(M) % 2 == 0, 1.0, -1.0).astype(np.float32)
    return y, t, old, ref, adv, np.full(M, 1.0 / M, np.float32)


def step(y, t, old, ref, adv, w, beta):
    """(loss, logp, gradient) as fp64 on the host, the loss alone checked to be the same."""
    import torch
    from packed_quantized_lm_amd import policy_loss
    args = (dev(y), dev(t, "int32"), dev(old), dev(adv), dev(w), dev(ref))
    loss, logp, dy = policy_loss(*args, beta=beta, grad_dtype=torch.float32)
    alone = policy_loss(*args, beta=beta)[0]
    # with and without a gradient rows may be cut differently
    assert torch.allclose(alone, loss, rtol=1e-5, atol=1e-6, equal_nan=True)
    return float(loss), logp.double().cpu().numpy(), dy.double().cpu().numpy()


@pytest.mark.parametrize("M,V", SIZES)
@pytest.mark.parametrize("beta", [0.0, 0.1])
def test_unknown_advantages(M, V, beta):
    say(f"NaN advantage M={M} V={V} beta={beta}")
    y, t, old, ref, adv, w = batch(M, V)
    whole = step(y, t, old, ref, adv, w, beta)
    adv[0] = np.nan
    adv[2], w[2] = np.nan, 0.0  # a row without weight may hold anything
    adv[3], old[3] = np.inf, np.inf  # an infinite advantage at a ratio of zero
    adv[4], old[4] = 0.0, -np.inf  # no advantage at an infinite ratio: no gain, the KL term alone
    loss, logp, g = step(y, t, old, ref, adv, w, beta)
    with np.errstate(over="ignore"):
        want = losses.policy(y, t, old, adv, w, ref, beta)
    assert math.isnan(loss) and math.isnan(want[0])
    assert np.isnan(g[0]).all() and np.isnan(g[3]).all() and np.isnan(want[2][[0, 3]]).all()
    assert not g[2].any() and logp[2] == 0.0
    assert g[4].any() == (beta > 0)
    # fp32's exponentials and sums are within 1e-4 of any entry here
    assert np.allclose(g[4], want[2][4], rtol=1e-4, atol=1e-12)
    rest = np.setdiff1d(np.arange(M), [0, 2, 3, 4])
    assert np.array_equal(g[rest], whole[2][rest]) and np.array_equal(logp[rest], whole[1][rest])


@pytest.mark.parametrize("V", [5, 64, 4099, 50021])
@pytest.mark.parametrize("smoothing", [0.0, 0.1])
def test_infinite_margins(V, smoothing):
    """Pairs with a masked token in the rejected answer (h = inf), in the chosen
    one (h = -inf), in both (NaN) and in none."""
    import torch
    from packed_quantized_lm_amd import preference_loss
    say(f"infinite margins V={V} smoothing={smoothing}")
    rng = np.random.default_rng(V)
    off = np.array([0, 2, 4, 6, 8, 10, 12, 14, 16])
    y = rng.normal(0, 2, (16, V)).astype(np.float32)
    t = rng.integers(0, V, 16)
    for m in (2, 5, 9, 10):
        y[m, t[m]] = -np.inf
    y[0, (t[0] + 1) % V] = -np.inf  # and a mask beside a token
    w = np.ones(16, np.float32)

    def both(rows, offsets):
        got = preference_loss(dev(y[rows]), dev(t[rows], "int32"), dev(w[rows]), dev(offsets, "int32"), beta=0.2,
                              smoothing=smoothing, grad_dtype=torch.float32)
        with np.errstate(invalid="ignore"):
            want = losses.preference(y[rows], t[rows], w[rows], offsets, None, 0.2, smoothing)
        return [x.double().cpu().numpy() for x in got], want
    # fp32's exponentials and sums are within 1e-4 of anything here
    for pair, margin in ((0, np.inf), (1, -np.inf), (2, np.nan), (3, None)):
        rows = slice(4 * pair, 4 * pair + 4)
        (loss, h, logp, g), (wl, wh, wp, wg, _) = both(rows, off[:3])
        if margin is None:
            assert np.isfinite(h).all()
        else:
            assert np.array_equal(h, [margin], equal_nan=True) and np.array_equal(wh, [margin], equal_nan=True)
        assert np.allclose(loss, wl, rtol=1e-4, equal_nan=True), (loss, wl)
        assert np.allclose(logp, wp, rtol=1e-4, atol=1e-4)
        assert np.allclose(g, wg, rtol=1e-4, atol=1e-9, equal_nan=True)
        if margin == np.inf and not smoothing:
            assert loss == 0.0 and not g.any()
    rows = np.r_[0:4, 12:16]
    (loss, h, _, g), (wl, wh, _, wg, _) = both(rows, off[:5])
    assert np.allclose(loss, wl, rtol=1e-4) and np.isfinite(loss) == (smoothing == 0.0)
    assert np.allclose(g, wg, rtol=1e-4, atol=1e-9)


@pytest.mark.parametrize("M,V", SIZES)
def test_masked_tokens_under_a_kl_term(M, V):
    """A token masked by the policy (an infinite KL term), by the reference (too,
    with a finite gradient) and by both (unknown)."""
    say(f"masked tokens M={M} V={V}")
    for kind, expected in (("policy", np.inf), ("reference", np.inf), ("both", np.nan)):
        y, t, old, ref, adv, w = batch(M, V)
        whole = step(y, t, old, ref, adv, w, 0.1)
        if kind != "reference":
            y[0, t[0]] = -np.inf
        if kind != "policy":
            ref[0] = -np.inf
        loss, logp, g = step(y, t, old, ref, adv, w, 0.1)
        with np.errstate(invalid="ignore"):
            want = losses.policy(y, t, old, adv, w, ref, 0.1)
        assert np.array_equal(loss, expected, equal_nan=True) and np.array_equal(want[0], expected, equal_nan=True)
        assert np.allclose(logp, want[1], rtol=1e-4, atol=1e-4)
        if kind == "reference":
            assert np.allclose(g[0], want[2][0], rtol=1e-4, atol=1e-12)
        elif kind == "policy":
            assert g[0, t[0]] == -np.inf and (np.delete(g[0], t[0]) == np.inf).all()
        else:
            assert np.isnan(g[0]).all()
        assert np.array_equal(g[1:], whole[2][1:])
