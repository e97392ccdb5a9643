"""The post-training operators of the packed head as measured workloads: the
8-bit head (matrix product with a scale per block of 128), token log
probabilities, the clipped policy loss, the preference loss and the packed
head's backward, each in a plain form (elementary torch operations in 32 bits)
and through the framework's entry points.
"""
import math

import torch

own = False  # True: run() calls the framework; False: the plain forms

BLOCK = 128
E4M3_MAX = 448.0


# ---------------------------------------------------------------- cases
def listed():
    return [
        # decoding with an 8-bit head: one token's logits, all of the weights read once
        dict(name="fp8_token", op="fp8", M=1, N=151936, K=4096, out="f32"),
        # a mixed batch on a head with odd sizes; the last block of K is a partial one
        dict(name="fp8_ragged", op="fp8", M=333, N=50021, K=2576, out="bf16"),
        # a prompt's logits from the reference policy's 8-bit head
        dict(name="fp8_prompt", op="fp8", M=2048, N=151936, K=4096, out="f32"),
        # the log probability of the token just drawn
        dict(name="logp_token", op="logp", M=1, V=151936, type="f32", banned=False),
        # scoring a rollout under the reference policy
        dict(name="logp_rollout", op="logp", M=2047, V=151936, type="f32", banned=True),
        # the tiny head's policy step: latency
        dict(name="policy_tiny", op="policy", M=16, V=2048, type="f32", grad="f32", beta=0.04, banned=False),
        # a policy step over a rollout batch, gradient in the hidden states' type
        dict(name="policy_batch", op="policy", M=2048, V=151936, type="f32", grad="bf16", beta=0.04, banned=False),
        # a few answer pairs on an odd vocabulary, logits in 16 bits
        dict(name="preference_few", op="preference", pairs=3, longest=61, V=50021, type="bf16", grad="bf16",
             beta=0.1, smoothing=0.1, banned=True),
        # a batch of ragged answer pairs
        dict(name="preference_batch", op="preference", pairs=8, longest=190, V=151936, type="f32", grad="bf16",
             beta=0.1, smoothing=0.0, banned=False),
        # the hidden states' gradient of a few tokens through the packed head
        dict(name="backward_few", op="backward", M=16, V=151936, d=4096, k=256, r=64, g=128),
        # odd vocabulary, small groups, odd ranks
        dict(name="backward_ragged", op="backward", M=133, V=30011, d=640, k=40, r=20, g=32),
        # a training step's batch through the packed head
        dict(name="backward_batch", op="backward", M=2048, V=151936, d=4096, k=256, r=64, g=128),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["fp8", "logp", "policy", "preference", "backward"])
    if op == "fp8":
        while True:
            c = dict(op=op, M=_log_int(rng, 1, 4096), N=_log_int(rng, 64, 262144), K=16 * _log_int(rng, 1, 512),
                     out=rng.choice(["f32", "bf16"]))
            if c["M"] * c["N"] * c["K"] <= 2048 * 151936 * 4096 and c["N"] * c["K"] <= 151936 * 4096 \
                    and c["M"] * c["N"] <= 2048 * 151936:
                return c
    if op == "backward":
        g = rng.choice([32, 64, 128, 256])
        d = max(128, g) * _log_int(rng, 1, 4096 // max(128, g))
        while True:
            c = dict(op=op, M=_log_int(rng, 1, 2048), V=_log_int(rng, 17, 151936), d=d,
                     k=rng.choice([0, _log_int(rng, 1, 256)]), r=rng.choice([0, _log_int(rng, 1, 64)]), g=g)
            if c["M"] * c["V"] * c["d"] <= 2048 * 151936 * 4096 // 2:
                return c
    c = dict(op=op, V=_log_int(rng, 2, 262144), type=rng.choice(["f32", "bf16"]), banned=rng.random() < 0.5)
    most = 2047 * 151936 // c["V"]
    if op == "preference":
        c["longest"] = _log_int(rng, 1, 512)
        c["pairs"] = _log_int(rng, 1, max(1, min(256, most // (2 * c["longest"]))))
        c.update(beta=rng.choice([0.05, 0.1, 0.5]), smoothing=rng.choice([0.0, 0.1]))
    else:
        c["M"] = _log_int(rng, 1, max(1, min(4096, most)))
    if op == "policy":
        c["beta"] = rng.choice([0.0, 0.01, 0.04])
    if op != "logp":
        c["grad"] = rng.choice(["f32", "bf16"])
    return c


def work(case):
    c = case
    size = {"f32": 4, "bf16": 2}
    if c["op"] == "fp8":
        M, N, K = c["M"], c["N"], c["K"]
        kb, nb = -(-K // BLOCK), -(-N // BLOCK)
        return {"bytes": 2 * M * K + N * K + 4 * nb * kb + size[c["out"]] * M * N, "flops": 2 * M * N * K}
    if c["op"] == "backward":
        M, V, d, k, r, g = (c[n] for n in ("M", "V", "d", "k", "r", "g"))
        packed = V * d // 2 + 2 * V * (d // g) + V * (5 * k // 8 + r) + 4 * V + (k + r) * d + 2 * k + 2 * r * (d // g)
        return {"bytes": packed + 2 * M * V + 2 * M * d, "flops": 2 * M * V * d + 2 * M * (V + d) * (k + r)}
    M = _tokens(c)
    elems = M * c["V"]
    if c["op"] == "logp":
        return {"bytes": elems * size[c["type"]] + 12 * M, "flops": 4 * elems}
    return {"bytes": elems * (size[c["type"]] + size[c["grad"]]) + 24 * M, "flops": 8 * elems}


# ---------------------------------------------------------------- inputs
def _tokens(c):
    """Rows of logits of a case; a preference batch's answers have lengths that
    depend on their number alone, so that the case fixes the work."""
    return sum(_lengths(c)) if c["op"] == "preference" else c["M"]


def _lengths(c):
    return [1 + (i * 7919 + 37) % c["longest"] if i else c["longest"] for i in range(2 * c["pairs"])]


_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _inputs(c, seed):
    """Every input of a case from its seed, on the GPU."""
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def uniform(lo, hi, *shape):
        return lo + (hi - lo) * torch.rand(*shape, generator=gen, device=dev)

    def whole(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=gen, device=dev)

    s = {"case": c}
    if c["op"] == "fp8":
        M, N, K = c["M"], c["N"], c["K"]
        # hidden states with channels of very different sizes; weights as an
        # 8-bit checkpoint holds them: codes and a scale per 128 x 128 block
        s["X"] = (normal(M, K) * torch.exp(normal(K))).to(torch.bfloat16)
        kb, nb = -(-K // BLOCK), -(-N // BLOCK)
        s["w8"] = (normal(N, K) * 100.0).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        s["ws"] = torch.exp(uniform(math.log(1e-4), math.log(1e-3), nb, kb))
        return s
    if c["op"] == "backward":
        M, V, d, k, r, g = (c[n] for n in ("M", "V", "d", "k", "r", "g"))
        G = d // g

        def scales(lo, hi, *shape):
            return torch.exp(uniform(math.log(lo), math.log(hi), *shape)).to(torch.float16)

        s["A5"] = whole(-16, 16, V, k).to(torch.int8)
        s["sA"] = scales(1e-3, 1e-2, V)
        s["B8"] = whole(-128, 128, k, d).to(torch.int8)
        s["sB"] = scales(1e-3, 1e-2, k)
        s["R4"] = whole(0, 256, V, d // 2).to(torch.uint8)
        s["sR"] = scales(1e-4, 1e-3, V, G)
        s["C8"] = whole(-128, 128, V, r).to(torch.int8)
        s["sC"] = scales(1e-3, 1e-2, V)
        s["D8"] = whole(-128, 128, r, d).to(torch.int8)
        s["sD"] = scales(1e-4, 1e-3, r, G)
        # a loss's gradient of the logits: coef (1[v = target] - p), rows of
        # masked tokens zero
        t = whole(0, V, M)
        y = normal(M, V) * 2.5
        grad = torch.softmax(y, dim=1).neg_()
        del y
        rows = torch.arange(M, device=dev)
        grad[rows, t] += 1.0
        coef = normal(M) * (uniform(0, 1, M) > 0.05) / M
        s["dlogits"] = (grad * coef[:, None]).to(torch.bfloat16)
        return s
    M, V = _tokens(c), c["V"]
    y = normal(M, V) * 2.5
    t = whole(0, V, M)
    rows = torch.arange(M, device=dev)
    y[rows, t] += uniform(4.0, 14.0, M)  # drawn tokens are mostly likely ones
    if c["banned"]:  # a vocabulary mask, never over a drawn token
        keep = y[rows, t].clone()
        y.masked_fill_(uniform(0, 1, 1, V) < 0.1, -math.inf)
        y[rows, t] = keep
    s["logits"] = y.to(_TYPES[c["type"]])
    del y
    s["targets"] = t.to(torch.int32)
    if c["op"] == "logp":
        return s
    y64 = torch.cat([part.double().logsumexp(1) for part in s["logits"].split(256)])
    logp = s["logits"][rows, t].double() - y64
    used = uniform(0, 1, M) > 0.05  # padding and prompt tokens carry no loss
    s["ref_logp"] = (logp + 0.2 * normal(M)).float()
    if c["op"] == "policy":
        # log ratios of a few updates, none within 1e-3 of a clip border
        step = 0.15 * normal(M).double()
        for edge in (math.log(1.0 + 0.28), math.log(1.0 - 0.2)):
            step = torch.where((step - edge).abs() < 1e-3, step + 2e-3, step)
        s["old_logp"] = (logp - step).float()
        s["advantages"] = normal(M)
        s["weights"] = used.float() / M
    else:
        s["weights"] = used.float()
        ends = torch.tensor([0] + _lengths(c)).cumsum(0)
        s["offsets"] = ends.to(torch.int32).to(dev)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import packed_quantized_lm_amd as pq
        if case["op"] == "fp8":
            s["head"] = pq.Fp8Head.from_blocks(s["w8"], s["ws"])
        if case["op"] == "backward":
            fields = {n: case[n] for n in ("V", "d", "k", "r", "g")}
            for n in ("A5", "B8", "R4", "C8", "D8"):
                fields[n] = s[n].cpu().numpy()
            for n in ("sA", "sB", "sR", "sC", "sD"):
                fields[n] = s[n].view(torch.int16).cpu().numpy().view("uint16")
            s["head"] = pq.PackedHead(fields)
            s["head"].reserve_backward(case["M"])
    return s


# ---------------------------------------------------------------- one pass
def run(state):
    c = state["case"]
    if own:
        return _run_own(c, state)
    return {"fp8": _plain_fp8, "logp": _plain_logp, "policy": _plain_policy, "preference": _plain_preference,
            "backward": _plain_backward}[c["op"]](c, state)


def _run_own(c, s):
    import packed_quantized_lm_amd as pq
    if c["op"] == "fp8":
        return s["head"].forward(s["X"], out_dtype=_TYPES[c["out"]])
    if c["op"] == "backward":
        return s["head"].backward(s["dlogits"])
    if c["op"] == "logp":
        return pq.token_logp(s["logits"], s["targets"])
    if c["op"] == "policy":
        return pq.policy_loss(s["logits"], s["targets"], s["old_logp"], s["advantages"], s["weights"],
                              ref_logp=s["ref_logp"], beta=c["beta"], eps_low=0.2, eps_high=0.28,
                              grad_dtype=_TYPES[c["grad"]])
    return pq.preference_loss(s["logits"], s["targets"], s["weights"], s["offsets"], s["ref_logp"], beta=c["beta"],
                              smoothing=c["smoothing"], grad_dtype=_TYPES[c["grad"]])


def _plain_fp8(c, s):
    X, w8, ws = s["X"].float(), s["w8"], s["ws"]
    M, K = X.shape
    kb = -(-K // BLOCK)
    # one scale per row and block of 128, then codes: the nearest e4m3 value
    # (ties to even) of the quotient, in 64 bits since 32 round it into ties
    xb = torch.nn.functional.pad(X, (0, kb * BLOCK - K)).view(M, kb, BLOCK)
    amax = xb.abs().amax(2, keepdim=True)
    scale = torch.where(amax > 0, (amax / E4M3_MAX).clamp_min(2.0 ** -126), amax)
    q = torch.where(amax > 0, xb.double() / scale.double().clamp_min(2.0 ** -200), 0.0)
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6))).clamp(-6, 8) - 3)
    q = (torch.round(q / step) * step).clamp(-E4M3_MAX, E4M3_MAX)
    xq = (q.float() * scale).view(M, kb * BLOCK)[:, :K]
    w = w8.float()
    w *= ws.repeat_interleave(BLOCK, 0)[:w.shape[0]].repeat_interleave(BLOCK, 1)[:, :K]
    return (xq @ w.t()).to(_TYPES[c["out"]])


def _softmax_parts(s):
    y = s["logits"].float()
    top = y.amax(1, keepdim=True)
    e = torch.exp(y - top)
    total = e.sum(1, keepdim=True)
    rows = torch.arange(y.shape[0], device=y.device)
    t = s["targets"].long()
    lse = (top + torch.log(total))[:, 0]
    logp = ((y[rows, t] - top[:, 0]) - torch.log(total[:, 0]))
    return e, total, rows, t, logp, lse


def _plain_logp(c, s):
    _, _, _, _, logp, lse = _softmax_parts(s)
    return logp, lse


def _logit_gradient(e, total, rows, t, coef, dtype):
    g = e.mul_(-coef[:, None] / total)
    g[rows, t] += coef
    return g.to(dtype)


def _plain_policy(c, s):
    e, total, rows, t, logp, _ = _softmax_parts(s)
    A, w = s["advantages"], s["weights"]
    ratio = torch.exp(logp - s["old_logp"])
    clipped = ratio.clamp(1.0 - 0.2, 1.0 + 0.28)
    gap = s["ref_logp"] - logp
    kl = torch.exp(gap) - gap - 1.0
    loss = (w * (-torch.minimum(ratio * A, clipped * A) + c["beta"] * kl)).sum()
    inside = ratio * A <= clipped * A
    coef = w * (-A * ratio * inside + c["beta"] * (1.0 - torch.exp(gap)))
    logp = torch.where(w != 0, logp, 0.0)
    return loss, logp, _logit_gradient(e, total, rows, t, coef, _TYPES[c["grad"]])


def _plain_preference(c, s):
    e, total, rows, t, logp, _ = _softmax_parts(s)
    w, off = s["weights"], s["offsets"].long()
    P = c["pairs"]
    diff = torch.where(w != 0, w * (logp - s["ref_logp"]), 0.0).double()
    run_sum = torch.nn.functional.pad(diff.cumsum(0), (1, 0))
    S = run_sum[off[1:]] - run_sum[off[:-1]]
    margin = (c["beta"] * (S[0::2] - S[1::2])).float()
    sm = c["smoothing"]
    neg = torch.log1p(torch.exp(-margin.abs()))
    loss = ((1 - sm) * (neg + (-margin).clamp_min(0)) + sm * (neg + margin.clamp_min(0))).mean()
    dS = -(c["beta"] / P) * ((1 - sm) * torch.sigmoid(-margin) - sm * torch.sigmoid(margin))
    per_seq = torch.stack([dS, -dS], 1).reshape(-1)
    coef = per_seq[torch.searchsorted(off, rows, right=True) - 1] * w
    logp = torch.where(w != 0, logp, 0.0)
    return loss, margin, logp, _logit_gradient(e, total, rows, t, coef, _TYPES[c["grad"]])


def _residual(s, dtype):
    c = s["case"]
    lo, hi = (s["R4"] & 15).to(torch.int8), (s["R4"] >> 4).to(torch.int8)
    codes = torch.stack([lo, hi], 2).view(c["V"], c["d"])
    codes = torch.where(codes > 7, codes - 16, codes)
    return codes.to(dtype).view(c["V"], -1, c["g"]).mul_(s["sR"].to(dtype)[:, :, None]).view(c["V"], c["d"])


def _plain_backward(c, s):
    G = s["dlogits"].float()
    dX = G @ _residual(s, torch.float32)
    if c["k"]:
        T = G @ (s["A5"].float() * s["sA"].float()[:, None])
        dX += T @ (s["B8"].float() * s["sB"].float()[:, None])
    if c["r"]:
        S = G @ (s["C8"].float() * s["sC"].float()[:, None])
        dX += S @ (s["D8"].float().view(c["r"], -1, c["g"]) * s["sD"].float()[:, :, None]).view(c["r"], c["d"])
    return dX.to(torch.bfloat16)


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = _inputs(case, seed)
    f64 = torch.float64
    if case["op"] == "fp8":
        return _exact_fp8(s)
    if case["op"] == "backward":
        What = _residual(s, f64)
        if case["k"]:
            What += (s["A5"].to(f64) * s["sA"].to(f64)[:, None]) @ (s["B8"].to(f64) * s["sB"].to(f64)[:, None])
        if case["r"]:
            spread = s["sD"].to(f64).repeat_interleave(case["g"], 1)
            What += (s["C8"].to(f64) * s["sC"].to(f64)[:, None]) @ (s["D8"].to(f64) * spread)
        return s["dlogits"].to(f64) @ What
    y = s["logits"].to(f64)
    M, V = y.shape
    t = s["targets"].long()
    logq = torch.log_softmax(y, 1)
    lse = torch.logsumexp(y, 1)
    del y
    logp = logq.gather(1, t[:, None])[:, 0]
    if case["op"] == "logp":
        return logp, lse
    w = s["weights"].to(f64)
    ref = s["ref_logp"].to(f64)
    if case["op"] == "policy":
        A = s["advantages"].to(f64)
        ratio = (logp - s["old_logp"].to(f64)).exp()
        low, high = 0.8, 1.28
        stopped = ((A > 0) & (ratio > high)) | ((A < 0) & (ratio < low))
        surrogate = torch.where(A >= 0, torch.minimum(ratio, torch.full_like(ratio, high)),
                                torch.maximum(ratio, torch.full_like(ratio, low))) * A
        kl = (ref - logp).expm1() - (ref - logp)
        head = ((w * (case["beta"] * kl - surrogate)).sum(),)
        coef = w * (torch.where(stopped, 0.0, -A * ratio) - case["beta"] * (ref - logp).expm1())
    else:
        bounds = s["offsets"].tolist()
        sums = [(w[a:b] * (logp - ref)[a:b]).sum() for a, b in zip(bounds[:-1], bounds[1:])]
        h = case["beta"] * torch.stack([x - z for x, z in zip(sums[0::2], sums[1::2])])
        sm, P = case["smoothing"], case["pairs"]
        losses = -(1 - sm) * torch.nn.functional.logsigmoid(h) - sm * torch.nn.functional.logsigmoid(-h)
        head = (losses.mean(), h)
        slope = case["beta"] / P * (torch.sigmoid(h) - (1 - sm))
        coef = torch.zeros(M, dtype=f64, device=w.device)
        for p in range(P):
            coef[bounds[2 * p]:bounds[2 * p + 1]] = slope[p]
            coef[bounds[2 * p + 1]:bounds[2 * p + 2]] = -slope[p]
        coef = coef * w
    grad = logq.exp_().neg_()
    grad.scatter_add_(1, t[:, None], torch.ones(M, 1, dtype=f64, device=grad.device))
    grad.mul_(coef[:, None])
    return (*head, torch.where(w != 0, logp, 0.0), grad)


def _exact_fp8(s):
    f64 = torch.float64
    X = s["X"].to(f64)
    M, K = X.shape
    N = s["w8"].shape[0]
    # every non-negative e4m3 value in order; its index is its code, whose last bit settles a tie
    values = torch.arange(127, dtype=torch.uint8, device=X.device).view(torch.float8_e4m3fn).to(f64)
    middles = (values[1:] + values[:-1]) / 2
    xq = torch.zeros_like(X)
    for k0 in range(0, K, BLOCK):
        x = X[:, k0:k0 + BLOCK]
        top = x.abs().amax(1)
        scale = (top.float() / E4M3_MAX).clamp_min(2.0 ** -126).to(f64)
        q = (x / scale[:, None]).abs().contiguous()
        low, high = torch.searchsorted(middles, q), torch.searchsorted(middles, q, right=True)
        code = torch.where(low % 2 == 0, low, high)
        xq[:, k0:k0 + BLOCK] = values[code] * torch.sign(x) * scale[:, None]
    out = torch.empty(M, N, dtype=f64, device=X.device)
    spread = s["ws"].to(f64).repeat_interleave(BLOCK, 1)[:, :K]
    for n0 in range(0, N, 64 * BLOCK):
        w = s["w8"][n0:n0 + 64 * BLOCK].to(f64)
        w *= spread[n0 // BLOCK:n0 // BLOCK + 64].repeat_interleave(BLOCK, 0)[:w.shape[0]]
        out[:, n0:n0 + 64 * BLOCK] = xq @ w.t()
    return out
