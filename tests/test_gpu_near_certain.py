"""Tokens of probability near 1, the usual ones of a rollout, on the GPU: what a
row has beside its largest logit decides the log probability -log(1 + rest)
and the gradient at the token, and has to keep its own precision next to 1.

Tolerance of rest, relative, in units of u = 2^-24: a term exp(-x) is off by
u x for its difference of two logits, u x for the exponent's rounding and 2 u
for the exponential; where it is rescaled to a new maximum the differences add
up to x again, with 2 u for each such link; a thread meets V / 2048 vectors at
most and the merges are 6 of lanes, one of waves, one for eight slices of at most
37: links <= V / 2048 + 16.  Eight terms are added in fp32 by three roundings;
what follows is fp64.  The result's rounding adds u.
"""
import numpy as np
import pytest

from gpu_util import say
from oracle import losses

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


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


def rows_of(M, V, kind, dtype="f32"):
    """(logits on the device, the same in fp64, targets, rest, its relative
    tolerance): rest from 1e-3 down to 1e-9.  spread: all other columns share it;
    beside, apart: one runner-up in the target's aligned eight columns or in
    others, what is left far below."""
    import torch
    rng = np.random.default_rng(M * 1000003 + V)
    y = rng.uniform(-3, 0, (M, V))
    t = rng.integers(0, V, M)
    gap = rng.uniform(7, 19.5, M)
    rows = np.arange(M)
    if kind == "spread":
        y[rows, t] = gap + np.log(V)
    else:
        y -= 40 + np.log(V)
        if kind == "beside":
            here = np.minimum(t // 8 * 8 + 8, V) - t // 8 * 8  # columns of the target's eight
            at = t // 8 * 8 + (t % 8 + 1 + rng.integers(0, 7, M) % np.maximum(here - 1, 1)) % here
            at = np.where(here == 1, t - 1, at)
        else:
            at = (t + 8 + rng.integers(0, max(V - 16, 1), M)) % V
        assert (at != t).all()
        y[rows, at] = 0.0
        y[rows, t] = gap
    logits = dev(y)
    if dtype == "bf16":
        logits = logits.to(torch.bfloat16)
    y = logits.double().cpu().numpy()
    x = y[rows, t][:, None] - y
    assert (np.delete(x, t[0], 1)[0] > 0).all()
    e = np.exp(-x)
    e[rows, t] = 0.0
    rest = e.sum(1)
    mean_x = (e * x).sum(1) / rest
    tol = U * (2 * mean_x + 2 + 2 * (V / 2048 + 16) + 3 + 1)
    assert (rest < 2e-3).all() and (rest > 1e-10).all()
    return logits, y, t, rest, tol


# rows in one slice, in a workgroup of 256 or 1024 threads, in slices
SIZES = [(300, 8), (300, 9), (300, 16), (300, 64), (64, 1000), (9, 4097), (40, 9001), (530, 9001), (3, 50021),
         (2, 151936), (240, 40003)]


CASES = [(M, V, kind) for M, V in SIZES for kind in ("spread", "beside", "apart") if kind != "apart" or V >= 24]


@pytest.mark.parametrize("M,V,kind", CASES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_log_probabilities(M, V, kind, dtype):
    import torch
    from packed_quantized_lm_amd import policy_loss, preference_loss, token_logp
    say(f"near certain M={M} V={V} {kind} {dtype}")
    logits, y, t, rest, tol = rows_of(M, V, kind, dtype)
    want = losses.token_logp(y, t)
    assert np.allclose(want, -np.log1p(rest), rtol=1e-14, atol=0)
    ti, zero, one = dev(t, "int32"), dev(np.zeros(M)), dev(np.ones(M))
    got = {"token_logp": token_logp(logits, ti)[0],
           "policy_loss": policy_loss(logits, ti, zero, one, one)[1],
           "policy_loss with a gradient": policy_loss(logits, ti, zero, one, one, grad_dtype=torch.bfloat16)[1],
           "preference_loss": preference_loss(logits, ti, one, dev([0, M // 2, M], "int32"))[2]}
    for name, x in got.items():
        off = np.abs(x.double().cpu().numpy() - want) / np.abs(want)
        assert (off <= tol).all(), (name, (off / tol).max(), off.max() / U)


@pytest.mark.parametrize("M,V,kind", CASES)
@pytest.mark.parametrize("dtype,gtype", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
def test_gradients_at_the_token(M, V, kind, dtype, gtype):
    """c (1 - p) at the target relative to itself.  1 - p = rest / (1 + rest)
    has rest's error and 4 u (its difference's, sum's and quotient's rounding);
    c is taken in fp64 from logp, which is off by at most 2e-3 tol, and rounded,
    as is the product: 3 u; the output's half step.  A scale of 2^12 is exact."""
    import torch
    from packed_quantized_lm_amd import policy_loss, preference_loss
    say(f"gradient near certain M={M} V={V} {kind} {dtype} {gtype}")
    logits, y, t, rest, tol = rows_of(M, V, kind, dtype)
    rng = np.random.default_rng(V)
    rows, used = np.arange(M), np.arange(M)[::max(1, M // 40)]  # the oracle looks at some rows
    adv, w = rng.normal(0, 1, M), rng.uniform(0.5, 1.5, M) / M
    logp = -np.log1p(rest)
    ref = logp + rng.normal(0, 0.3, M)
    adv, w, ref = (a.astype(np.float32) for a in (adv, w, ref))
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}[gtype]
    half = {"f32": U, "bf16": 2.0 ** -8}[gtype]
    ti, scale = dev(t, "int32"), torch.tensor(4096.0, device="cuda")
    _, _, want, coef = losses.policy(y[used], t[used], np.zeros(len(used)), adv[used], w[used], ref[used], 0.04)
    dy = policy_loss(logits, ti, dev(np.zeros(M)), dev(adv), dev(w), dev(ref), beta=0.04, grad_dtype=dt,
                     grad_scale=scale)[2]
    got = dy[torch.from_numpy(rows).cuda(), ti.long()].double().cpu().numpy() / 4096
    own = want[np.arange(len(used)), t[used]]
    assert np.allclose(own, coef * (rest / (1 + rest))[used], rtol=1e-12, atol=0)
    # c = w (-A rho + beta (1 - exp(r))): logp's error moves both terms, which may nearly cancel
    parts = w[used] * (np.abs(adv[used]) + 0.04 * (np.exp(ref[used] - logp[used]) + 1))
    off = np.abs(got[used] - own) / np.abs(own)
    allowed = tol[used] + (7 + 1) * U + half + 2 * parts / np.abs(coef) * np.abs(logp[used]) * tol[used]
    assert (off <= allowed).all(), ((off / allowed).max(), off.max())
    if dtype == gtype:  # over the logits
        over = logits.clone()
        policy_loss(over, ti, dev(np.zeros(M)), dev(adv), dev(w), dev(ref), beta=0.04, dlogits=over, grad_scale=scale)
        assert torch.equal(over, dy)
    offsets = np.array([0, M // 2, M])
    s = (w.astype(np.float64) * (logp - ref))
    margin = 0.3 * (s[:M // 2].sum() - s[M // 2:].sum())
    slope = -0.3 / (1 + np.exp(margin)) * np.where(rows < M // 2, 1, -1) * w
    dy = preference_loss(logits, ti, dev(w), dev(offsets, "int32"), dev(ref), beta=0.3, grad_dtype=dt)[3]
    got = dy[torch.from_numpy(rows).cuda(), ti.long()].double().cpu().numpy()
    own = slope * (rest / (1 + rest))
    off = np.abs(got - own) / np.abs(own)
    # the margin's error, of its rows' log probabilities, moves the slope by at most as much
    allowed = tol + 8 * U + half + 0.3 * (w * np.abs(logp) * tol).sum()
    assert (off <= allowed).all(), ((off / allowed).max(), off.max())


@pytest.mark.parametrize("M,V", [(6, 1), (6, 9), (6, 64), (6, 4097), (6, 9001), (6, 50021), (240, 40003)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_nan_and_infinite_logits_reach_their_row(M, V, dtype):
    """One NaN, or a +inf, anywhere in a row (vectors, the columns behind them,
    beside the largest) makes its results NaN; -inf alone an lse of -inf; other
    rows stay."""
    import torch
    from packed_quantized_lm_amd import policy_loss, token_logp
    say(f"NaN and infinities M={M} V={V} {dtype}")
    rng = np.random.default_rng(V)
    y = rng.normal(0, 3, (M, V))
    t = rng.integers(0, V, M)
    where = [0, V // 2, V - 1]
    bad = [(0, where[0], np.nan), (1, where[1], np.nan), (2, where[2], np.nan), (3, int(t[3]), np.inf),
           (4, where[2], np.inf)]
    for m, v, x in bad:
        y[m, v] = x
    y[5] = -np.inf
    logits = dev(y).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    ti, zero, one = dev(t, "int32"), dev(np.zeros(M)), dev(np.full(M, 1.0))
    logp, lse = (a.cpu().numpy() for a in token_logp(logits, ti))
    assert np.isnan(logp[:6]).all() and np.isnan(lse[:5]).all() and lse[5] == -np.inf
    want = losses.token_logp(logits.double().cpu().numpy(), t)
    assert np.allclose(logp[6:], want[6:], rtol=1e-4, atol=1e-4) and not np.isnan(want[6:]).any()
    for grad in (None, torch.float32):
        loss, lp, dy = policy_loss(logits, ti, zero, one, one, grad_dtype=grad)
        assert torch.isnan(loss) and torch.isnan(lp[:6]).all() and not torch.isnan(lp[6:]).any()
        if grad:
            assert torch.isnan(dy[:6]).all() and not torch.isnan(dy[6:]).any()
