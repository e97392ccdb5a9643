"""Token log probabilities and post-training losses on the GPU against the
fp64 oracle (oracle/losses.py).

Tolerances, in units of u = 2^-24 (fp32) and the output type's half step:
* Z = sum exp(y - top): each term's exponent (y - top) log2(e) takes two
  roundings, so a term exp(-x) is off by 2 x u + 2 u relative (x < 100 for
  terms that matter: smaller ones are below 2^-140 of Z), and a chain of n
  additions by n u; n <= V / 256 + 64 (a workgroup of 256 threads and the
  merges), each merge rescaling with at most 4 u more: rz = (204 + 5 n) u.
* logp = (y_t - top) - log Z: rz + u (2 |y_t - top| + 2 |log Z|) absolute.
* a coefficient moves by its derivative times logp's error, plus 16 u relative.
* dlogits = c (1 - p) or -c p: |dc| + |c| (rz + 204 u) p, and one rounding.
"""
import numpy as np
import pytest

from gpu_util import say
from oracle import losses

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -9 * 2}  # half a step relative to the value


@pytest.fixture(scope="module", autouse=True)
def gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from packed_quantized_lm_amd import load_library
    load_library()


def _dt(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def _rz(V):
    return (204 + 5 * (V / 256 + 64)) * U


def make(M, V, seed, dtype="f32", pad=0, masked=True, kind="normal"):
    """Rows of logits as a strided device tensor, the same values in fp64,
    targets (never on a masked column) and the fp64 logp."""
    import torch
    rng = np.random.default_rng(seed)
    y = rng.normal(0, 3, (M, V))
    t = rng.integers(0, V, M)
    y[np.arange(M), t] += rng.uniform(0, 8, M)
    if kind == "huge":
        y *= 1e4
    if kind == "lowest":  # all columns but the target at the type's lowest value
        y[:] = np.finfo(np.float32).min if dtype == "f32" else -3.3895313892515355e38
        y[np.arange(M), t] = rng.normal(0, 1, M)
    if kind == "flat_lowest":
        y[:] = np.finfo(np.float32).min if dtype == "f32" else -3.3895313892515355e38
    if masked and V > 2 and kind == "normal":
        ban = rng.random((M, V)) < 0.2
        ban[np.arange(M), t] = False
        y[ban] = -np.inf
    buf = torch.full((M, V + pad), float("nan"), dtype=_dt(dtype), device="cuda")
    logits = buf[:, :V]
    logits.copy_(torch.from_numpy(y))
    y64 = logits.double().cpu().numpy()
    return rng, logits, y64, t, losses.token_logp(y64, t)


def dev(a, dtype="float32"):
    import torch
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype=dtype))).to("cuda")


def logp_tol(y64, t, rows, V):
    top = y64[rows].max(1)
    yt = y64[rows, t[rows]]
    lz = np.log(np.exp(y64[rows] - top[:, None]).sum(1))
    return _rz(V) + U * (2 * np.abs(yt - top) + 2 * lz + np.abs(yt))


SHAPES = [(1, 1, "f32", 0), (1, 2, "bf16", 3), (3, 5, "f32", 0), (2, 9, "bf16", 0), (5, 255, "f32", 1),
          (7, 4097, "bf16", 0), (3, 8193, "f32", 7), (1, 50021, "bf16", 0), (2, 151936, "f32", 0),
          (70, 1000, "f32", 0), (301, 2051, "bf16", 1), (2100, 130, "f32", 2), (4099, 3, "bf16", 0)]


@pytest.mark.parametrize("M,V,dtype,pad", SHAPES)
def test_token_logp(M, V, dtype, pad):
    import torch
    from packed_quantized_lm_amd import token_logp
    say(f"token_logp M={M} V={V} {dtype} pad={pad}")
    _, logits, y64, t, want = make(M, V, 100 + V, dtype, pad)
    logp, lse = token_logp(logits, dev(t, "int32"))
    rows = np.arange(M)
    tol = logp_tol(y64, t, rows, V)
    assert (np.abs(logp.double().cpu().numpy() - want) <= tol).all()
    assert (np.abs(lse.double().cpu().numpy() - (y64[rows, t] - want)) <= tol + 2 * U * np.abs(y64.max(1))).all()
    again = token_logp(logits, dev(t, "int32"))
    assert torch.equal(again[0], logp) and torch.equal(again[1], lse)


@pytest.mark.parametrize("kind", ["huge", "lowest", "flat_lowest"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_extreme_logits(kind, dtype):
    from packed_quantized_lm_amd import token_logp
    _, logits, y64, t, want = make(4, 3000, 7, dtype, 1, kind=kind)
    logp, _ = token_logp(logits, dev(t, "int32"))
    tol = _rz(3000) + 2 * U * np.abs(want) + (2 * U * 30 if kind != "huge" else 0)
    assert (np.abs(logp.double().cpu().numpy() - want) <= tol).all()


def test_empty_rows_and_bad_targets():
    import torch
    from packed_quantized_lm_amd import token_logp
    y = torch.zeros(5, 300, device="cuda")
    y[0] = -float("inf")
    y[1, 7] = float("nan")
    logp, lse = (x.cpu() for x in token_logp(y, dev([0, 3, -100, 300, 4], "int32")))
    assert torch.isnan(logp[:4]).all() and lse[0] == -float("inf") and torch.isnan(lse[1])
    assert abs(float(logp[4]) + np.log(300)) < 1e-5 and abs(float(lse[2]) - np.log(300)) < 1e-5
    logp, lse = token_logp(y[:0], dev([], "int32"))
    assert logp.shape == (0,)


@pytest.mark.parametrize("M,V", [(1, 8193), (37, 12289), (512, 9001), (513, 9001), (1, 32768), (2, 32769), (229, 33001),
                                 (231, 33001), (256, 40003)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_token_logp_rows_and_slices(M, V, dtype):
    """Row counts and lengths on both sides of where rows are cut into slices."""
    from packed_quantized_lm_amd import token_logp
    say(f"token_logp M={M} V={V} {dtype}")
    _, logits, y64, t, want = make(M, V, 3 + M + V, dtype, 1)
    logp, lse = token_logp(logits, dev(t, "int32"))
    rows = np.arange(M)
    tol = logp_tol(y64, t, rows, V)
    assert (np.abs(logp.double().cpu().numpy() - want) <= tol).all()
    assert (np.abs(lse.double().cpu().numpy() - (y64[rows, t] - want)) <= tol + 2 * U * np.abs(y64.max(1))).all()


@pytest.mark.parametrize("V", [2, 3, 7])
def test_token_logp_of_near_certain_tokens(V):
    """Probabilities of 1 - 1e-3 and nearer: logp = -log(1 + rest) keeps the
    relative precision of rest.  A term exp(-x), x < 13.5, is off by (2 x + 2) u
    and by 2 u for each of six merges that may rescale it; logp's rounding adds
    u: 42 u relative."""
    from packed_quantized_lm_amd import token_logp
    say(f"token_logp near certain V={V}")
    rng = np.random.default_rng(V)
    M = 300
    y = rng.uniform(-3, 0, (M, V))
    t = rng.integers(0, V, M)
    y[np.arange(M), t] = rng.uniform(5.9, 8.5, M) + np.log(V)
    y = y.astype(np.float32)
    want = losses.token_logp(y.astype(np.float64), t)
    assert (want < 0).all() and (want > -3e-3).all()
    got = token_logp(dev(y), dev(t, "int32"))[0].double().cpu().numpy()
    assert (np.abs(got - want) <= 42 * U * np.abs(want)).all(), (np.abs(got - want) / np.abs(want)).max() / U


def policy_case(M, V, dtype, pad, seed, beta):
    rng, logits, y64, t, logp = make(M, V, seed, dtype, pad)
    step = rng.normal(0, 0.3, M)
    for edge in (np.log(1.28), np.log(0.8)):  # the clip's borders decide a gradient: none within 1e-3 of them
        step = np.where(np.abs(step - edge) < 1e-3, step + 2e-3, step)
    old = (logp - step).astype(np.float32)
    ref = (logp + rng.normal(0, 0.4, M)).astype(np.float32)
    adv = rng.normal(0, 1, M).astype(np.float32)
    w = (rng.uniform(0.5, 1.5, M) * (rng.random(M) < 0.85) / M).astype(np.float32)
    if M > 2:
        w[1] = 0.0
        logits[1] = float("nan")  # a row without weight may hold anything
        t[1] = -100
    want = losses.policy(y64, t, old, adv, w, ref, beta, 0.2, 0.28)
    return logits, y64, t, old, ref, adv, w, want


def check_grad(g, want, t, coef, dcoef, gtype):
    """g against the oracle's gradient with the bound of the module's note."""
    M, V = want.shape
    c = np.abs(coef)[:, None]
    share = np.abs(want) / np.where(c == 0, 1.0, c)  # p, or 1 - p at the target
    err = dcoef[:, None] * share + c * (_rz(V) + 204 * U) * share
    rows = np.nonzero(coef)[0]
    err[rows, t[rows]] = dcoef[rows] + c[rows, 0] * (_rz(V) + 204 * U)  # 1 - p is off by what p < 1 is
    tol = err + np.abs(want) * (HALF[gtype] + 4 * U) + 2.0 ** -126
    got = g.double().cpu().numpy()
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4], tol[bad][:4])


@pytest.mark.parametrize("M,V,dtype,pad", SHAPES)
@pytest.mark.parametrize("gtype,beta", [("f32", 0.04), ("bf16", 0.0)])
def test_policy_loss(M, V, dtype, pad, gtype, beta):
    import torch
    from packed_quantized_lm_amd import policy_loss
    say(f"policy_loss M={M} V={V} {dtype} pad={pad} grad={gtype} beta={beta}")
    logits, y64, t, old, ref, adv, w, (loss, logp, grad, coef) = policy_case(M, V, dtype, pad, 11 + V, beta)
    buf = torch.full((M, V + 5), 7.0, dtype=_dt(gtype), device="cuda")
    got_loss, got_logp, dy = policy_loss(logits, dev(t, "int32"), dev(old), dev(adv), dev(w), dev(ref) if beta else None,
                                         beta=beta, eps_low=0.2, eps_high=0.28, dlogits=buf[:, :V])
    assert (buf[:, V:] == 7.0).all()  # nothing beyond the row
    used = w != 0
    dl = np.zeros(M)
    dl[used] = logp_tol(y64, t, np.nonzero(used)[0], V)
    assert (np.abs(got_logp.double().cpu().numpy() - logp) <= dl).all()
    rho, er = np.exp(logp - old) * used, np.exp(ref - logp) * used
    # derivative of the token loss by logp, times logp's error; 16 u of its terms
    dtok = np.abs(w) * ((np.abs(adv) * rho + beta * (er + 1)) * (dl + 16 * U) + U * 32 * beta * np.abs(ref - logp) * used)
    # logp - old is formed in fp32 from values of up to |logp|
    dtok += np.abs(w) * (np.abs(adv) * rho + beta * er) * 2 * U * np.abs(logp) * used
    assert abs(float(got_loss) - loss) <= dtok.sum() + U * abs(loss)
    dcoef = dtok
    check_grad(dy, grad, t, coef, dcoef, gtype)
    again = policy_loss(logits, dev(t, "int32"), dev(old), dev(adv), dev(w), dev(ref) if beta else None, beta=beta,
                        eps_low=0.2, eps_high=0.28, grad_dtype=_dt(gtype))
    assert torch.equal(again[2], dy) and torch.equal(again[0], got_loss)


@pytest.mark.parametrize("V", [8200, 24575, 32776, 65529, 65545, 98297, 98312, 131077])
@pytest.mark.parametrize("dtype,gtype", [("f32", "f32"), ("f32", "bf16"), ("bf16", "f32"), ("bf16", "bf16")])
def test_policy_loss_long_rows(V, dtype, gtype):
    """Enough rows for a workgroup each, which holds parts of its row: lengths
    at and beyond what is held; most rows without weight, the others against
    the oracle, out of place and in place."""
    import torch
    from packed_quantized_lm_amd import policy_loss
    say(f"policy_loss long rows V={V} {dtype} grad={gtype}")
    M, rows = 190, np.array([0, 1, 57, 128, 189])
    _, y64, t, old, ref, adv, w, _ = policy_case(len(rows), V, dtype, 3, 7 + V, 0.05)
    y = torch.full((M, V + 3), float("nan"), dtype=_dt(dtype), device="cuda")[:, :V]
    y[torch.from_numpy(rows).cuda()] = torch.from_numpy(y64).to("cuda", _dt(dtype))
    want, want_logp, grad, coef = losses.policy(y64, t, old, adv, w, ref, 0.05, 0.2, 0.28)

    def spread(a, dtype="float32"):
        full = np.zeros(M)
        full[rows] = a
        return dev(full, dtype)
    args = (spread(t, "int32"), spread(old), spread(adv), spread(w), spread(ref))
    loss, logp, dy = policy_loss(y, *args, beta=0.05, eps_low=0.2, eps_high=0.28, grad_dtype=_dt(gtype))
    used = w != 0
    dl = np.zeros(len(rows))
    dl[used] = logp_tol(y64, t, np.nonzero(used)[0], V)
    assert (np.abs(logp.double().cpu().numpy()[rows] - want_logp) <= dl).all()
    rho, er = np.exp(want_logp - old) * used, np.exp(ref - want_logp) * used
    dtok = np.abs(w) * ((np.abs(adv) * rho + 0.05 * (er + 1)) * (dl + 16 * U) + U * 1.6 * np.abs(ref - want_logp) * used)
    dtok += np.abs(w) * (np.abs(adv) * rho + 0.05 * er) * 2 * U * np.abs(want_logp) * used
    assert abs(float(loss) - want) <= dtok.sum() + U * abs(want)
    check_grad(dy[torch.from_numpy(rows).cuda()], grad, t, coef, dtok, gtype)
    rest = torch.ones(M, dtype=torch.bool, device="cuda")
    rest[torch.from_numpy(rows).cuda()] = False
    assert not dy[rest].any()
    if dtype == gtype:
        policy_loss(y, *args, beta=0.05, eps_low=0.2, eps_high=0.28, dlogits=y)
        assert torch.equal(y, dy)


def test_policy_gradient_against_differences():
    """The gradient against central differences of the kernel's own loss:
    truncation h^2 / 6 times a third derivative below 8 |c|, and two loss
    roundings over 2 h, with h = 2^-5."""
    import torch
    from packed_quantized_lm_amd import policy_loss
    logits, y64, t, old, ref, adv, w, _ = policy_case(4, 6, "f32", 0, 5, 0.3)
    logits = torch.where(torch.isinf(logits) | torch.isnan(logits), -1.0, logits).contiguous()
    t[1] = 0
    w[:] = 0.25
    old = (losses.token_logp(logits.double().cpu().numpy(), t) - np.array([0.05, -0.05, 0.1, -0.1])).astype(np.float32)
    rest = (dev(t, "int32"), dev(old), dev(adv), dev(w), dev(ref))
    kw = dict(beta=0.3, eps_low=0.5, eps_high=0.9)
    loss, _, g = policy_loss(logits, *rest, grad_dtype=torch.float32, **kw)
    h = 2.0 ** -5
    for i in range(4):
        c = 0.25 * (abs(adv[i]) * 2 + 0.3 * np.exp(abs(float(ref[i]) - float(old[i])) + 1))
        for j in range(6):
            up, down = logits.clone(), logits.clone()
            up[i, j] += h
            down[i, j] -= h
            d = (float(policy_loss(up, *rest, **kw)[0]) - float(policy_loss(down, *rest, **kw)[0])) / (2 * h)
            assert abs(d - float(g[i, j])) <= h * h / 6 * 8 * c + 2 * 40 * U * (abs(float(loss)) + c) / (2 * h)


def test_gradient_in_place_scale_and_streams():
    import torch
    from packed_quantized_lm_amd import policy_loss, preference_loss
    for M, V in ((3, 40961), (600, 1027)):
        logits, y64, t, old, ref, adv, w, _ = policy_case(M, V, "f32", 0, 3, 0.1)
        a = [dev(t, "int32"), dev(old), dev(adv), dev(w), dev(ref)]
        want = policy_loss(logits, *a, beta=0.1, grad_dtype=torch.float32)
        scale = torch.tensor(8.0, device="cuda")
        got = policy_loss(logits, *a, beta=0.1, grad_dtype=torch.float32, grad_scale=scale)
        assert torch.equal(got[2], want[2] * 8.0) and torch.equal(got[0], want[0])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = policy_loss(logits, *a, beta=0.1, grad_dtype=torch.float32, stream=side)
        side.synchronize()
        assert torch.equal(got[2], want[2])
        over = logits.clone()
        got = policy_loss(over, *a, beta=0.1, dlogits=over)
        assert torch.equal(over, want[2]) and torch.equal(got[1], want[1])
        off = dev([0, M // 3, M], "int32")
        want = preference_loss(logits, a[0], a[3], off, a[4], grad_dtype=torch.float32)
        over = logits.clone()
        preference_loss(over, a[0], a[3], off, a[4], dlogits=over)
        assert torch.equal(over, want[3])


PAIRS = [([0, 1, 2], 5, "f32"), ([0, 0, 0], 7, "f32"), ([2, 5, 5, 5, 9], 333, "bf16"), ([0, 40, 71, 72, 200], 2050, "f32"),
         ([0, 3, 4], 50021, "bf16"), ([1, 900, 2300], 67, "f32"), (list(range(0, 1025)), 12, "bf16")]


@pytest.mark.parametrize("offsets,V,dtype", PAIRS)
@pytest.mark.parametrize("gtype,smoothing,with_ref", [("bf16", 0.1, True), ("f32", 0.0, False)])
def test_preference_loss(offsets, V, dtype, gtype, smoothing, with_ref):
    import torch
    from packed_quantized_lm_amd import preference_loss
    M, beta = offsets[-1] + 3, 0.1
    say(f"preference_loss M={M} V={V} P={(len(offsets) - 1) // 2} {dtype}")
    rng, logits, y64, t, lp = make(M, V, 17 + V, dtype, 1)
    ref = (lp + rng.normal(0, 0.2, M)).astype(np.float32) if with_ref else None
    w = (rng.random(M) < 0.9).astype(np.float32)
    outside = np.arange(M)
    outside = (outside < offsets[0]) | (outside >= offsets[-1])
    if outside.any():
        logits[torch.from_numpy(outside).cuda()] = float("nan")  # rows of no answer may hold anything
    loss, h, logp, grad, coef = losses.preference(y64, t, w, offsets, ref, beta, smoothing)
    g_loss, g_h, g_logp, dy = preference_loss(logits, dev(t, "int32"), dev(w), dev(offsets, "int32"),
                                              None if ref is None else dev(ref), beta=beta, smoothing=smoothing,
                                              grad_dtype=_dt(gtype))
    used = (w != 0) & ~outside
    dl = np.zeros(M)
    rows = np.nonzero(used)[0]
    if len(rows):
        dl[rows] = logp_tol(y64, t, rows, V)
    assert (np.abs(g_logp.double().cpu().numpy() - logp) <= dl).all()
    # a margin sums its rows' errors (sums run in 64 bits)
    P = len(h)
    dh = np.array([beta * dl[offsets[2 * p]:offsets[2 * p + 2]].sum() for p in range(P)]) + 2 * U * np.abs(h)
    assert (np.abs(g_h.double().cpu().numpy() - h) <= dh).all()
    assert abs(float(g_loss) - loss) <= dh.mean() + 8 * U * (abs(loss) + np.abs(h).mean())
    dcoef = np.abs(coef) * 16 * U
    for p in range(P):  # |d sigma / dh| <= 1/4
        dcoef[offsets[2 * p]:offsets[2 * p + 2]] += beta / P * (0.25 * dh[p] + 8 * U)
    check_grad(dy, grad, t, coef, dcoef, gtype)
    assert not dy[~torch.from_numpy(used).cuda()].any()


def test_graph_capture_replays():
    """Both losses in one captured graph, replayed with other inputs and eager
    work between the replays."""
    import torch
    from packed_quantized_lm_amd import policy_loss, preference_loss
    M, V = 24, 9001
    logits, y64, t, old, ref, adv, w, _ = policy_case(M, V, "f32", 0, 23, 0.05)
    logits = logits.contiguous()
    a = [dev(t, "int32"), dev(old), dev(adv), dev(w), dev(ref)]
    off = dev([0, 7, 11, 11, 24], "int32")
    step = lambda: (*policy_loss(logits, *a, beta=0.05, grad_dtype=torch.bfloat16),
                    *preference_loss(logits, a[0], a[3], off, a[4], grad_dtype=torch.float32))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        a[2].normal_()
        logits.add_(torch.randn_like(logits) * 0.1 * (torch.arange(M, device="cuda")[:, None] != 1))
        graph.replay()
        torch.cuda.synchronize()
        kept = [x.clone() for x in out]
        for x, y in zip(kept, step()):
            assert torch.equal(torch.nan_to_num(x), torch.nan_to_num(y)), i
        torch.cuda.synchronize()


def test_offsets_past_32_bits():
    """Rows 2^29 elements apart: the last ones past 2^32 elements."""
    import torch
    from packed_quantized_lm_amd import policy_loss, token_logp
    M, V, far = 10, 9001, 1 << 29
    flat = torch.zeros((M - 1) * far + V, dtype=torch.bfloat16, device="cuda")
    y = flat.as_strided((M, V), (far, 1))
    y.copy_(torch.randn(M, V))
    t = torch.randint(0, V, (M,), dtype=torch.int32, device="cuda")
    v = torch.ones(M, device="cuda")
    near = y.contiguous()
    for a, b in zip(token_logp(y, t), token_logp(near, t)):
        assert torch.equal(a, b)
    want = policy_loss(near, t, v, v, v, grad_dtype=torch.bfloat16)
    got = policy_loss(y, t, v, v, v, dlogits=y)  # in place, far apart
    assert torch.equal(got[0], want[0]) and torch.equal(y.contiguous(), want[2])


def test_binding_refuses_bad_tensors():
    import torch
    from packed_quantized_lm_amd import policy_loss, preference_loss, token_logp
    from packed_quantized_lm_amd.binding import ArcheadError
    y = torch.zeros(4, 16, device="cuda")
    t, v = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(4, device="cuda")
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    bad = (ValueError, TypeError)
    for logits in (y.double(), y[0], y.t(), y.cpu(), y[:, ::2], torch.zeros(4, 0, device="cuda"), y[:1].expand(4, 16)):
        with pytest.raises(bad):
            token_logp(logits, t)
    for targets in (t.long(), t[:3], t.cpu(), None):
        with pytest.raises(bad):
            token_logp(y, targets)
    for old in (v.double(), v[:2], None, v.cpu()):
        with pytest.raises(bad):
            policy_loss(y, t, old, v, v)
    with pytest.raises(bad):
        policy_loss(y, t, v, v, v, grad_dtype=torch.float16)
    with pytest.raises(bad):
        policy_loss(y, t, v, v, v, dlogits=torch.zeros(4, 15, device="cuda"))
    for kw in (dict(beta=0.1), dict(beta=-1.0), dict(eps_low=1.5), dict(eps_high=float("inf")), dict(eps_low=float("nan"))):
        with pytest.raises(ArcheadError):
            policy_loss(y, t, v, v, v, **kw)
    with pytest.raises(ArcheadError):  # in place, but of another type
        policy_loss(y, t, v, v, v, dlogits=y.view(torch.bfloat16)[:, :16])
    for o in (off[:2], off.long(), off[:1], off.cpu()):
        with pytest.raises(bad):
            preference_loss(y, t, v, o)
    for kw in (dict(beta=0.0), dict(smoothing=0.5), dict(smoothing=-0.1)):
        with pytest.raises(ArcheadError):
            preference_loss(y, t, v, off, **kw)
    torch.cuda.synchronize()
