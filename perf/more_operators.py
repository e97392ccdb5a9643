"""The operators around the output head as measured workloads: the RMS norm
with the residual's addition and an 8-bit output, its backward, the embedding
lookup and its gradient, and the logits' penalties, biases and grammar masks
with and without the top-k draw, each in a plain form (elementary torch
operations in 32 bits) and through the framework's entry points.
"""
import math

import torch

own = False  # True: run() calls the framework; False: the plain forms

BLOCK = 128
E4M3_MAX = 448.0
EPS = 1e-6


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one token's final norm in a decode step: latency
        dict(name="norm_token", op="norm", M=1, d=4096, type="bf16", weight="bf16", residual=True, out="bf16",
             offset=0.0),
        # a prompt's final norm, written as the 8-bit head's codes and scales
        dict(name="norm_prompt", op="norm", M=8192, d=4096, type="bf16", weight="bf16", residual=True, out="codes",
             offset=0.0),
        # a training batch: gradients of norm, residual stream and weight
        dict(name="norm_grad_batch", op="norm_grad", M=8192, d=4096, type="bf16", weight="bf16", through=True,
             offset=0.0),
        # odd sizes in 32 bits, no gradient through the residual stream, weights stored around zero
        dict(name="norm_grad_ragged", op="norm_grad", M=777, d=2571, type="f32", weight="f32", through=False,
             offset=1.0),
        # the drawn tokens of a batch, looked up in a tied 8-bit head
        dict(name="embed_tokens", op="embed", n=32, V=151936, d=4096, table="e4m3", out="bf16", scale=1.0),
        # a prompt's rows of a large vocabulary, scaled by the root of the width
        dict(name="embed_prompt", op="embed", n=8192, V=262144, d=2560, table="bf16", out="bf16", scale=50.6),
        # a training batch's gradient of the whole table
        dict(name="embed_grad_batch", op="embed_grad", n=8192, V=151936, d=4096, type="bf16", grad="bf16", scale=1.0),
        # a small odd table, gradient in 32 bits, more tokens than rows
        dict(name="embed_grad_ragged", op="embed_grad", n=4099, V=2048, d=257, type="f32", grad="f32", scale=16.0),
        # the next token of one request with a short history and a grammar
        dict(name="sample_token", op="sample", M=1, V=151936, type="f32", K=16, history=300, bias=0, mask=True),
        # the next tokens of a full batch with long histories, biases and grammars
        dict(name="sample_batch", op="sample", M=256, V=151936, type="f32", K=16, history=8192, bias=64, mask=True),
        # adjusted logits for a caller's own sampler, odd vocabulary, 16 bits
        dict(name="adjust_ragged", op="adjust", M=33, V=50021, type="bf16", history=2000, bias=300, mask=False),
        # the same for a large batch under grammars
        dict(name="adjust_batch", op="adjust", M=256, V=151936, type="f32", history=1024, bias=0, mask=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "embed", "embed_grad", "sample", "adjust"])
    if op in ("norm", "norm_grad"):
        c = dict(op=op, d=_log_int(rng, 16, 16384), type=rng.choice(["f32", "bf16"]),
                 weight=rng.choice(["f32", "bf16"]), offset=rng.choice([0.0, 1.0]))
        if op == "norm":
            c.update(residual=rng.random() < 0.7, out=rng.choice(["f32", "bf16", "codes"]))
            if c["out"] == "codes":
                c["d"] = 16 * max(1, c["d"] // 16)
        else:
            c["through"] = rng.random() < 0.7
        c["M"] = _log_int(rng, 1, min(65536, 8192 * 4096 // c["d"] // (2 if c["type"] == "f32" else 1)))
        return c
    if op in ("embed", "embed_grad"):
        c = dict(op=op, d=16 * _log_int(rng, 1, 512), scale=rng.choice([1.0, 0.5, 50.6]))
        c["n"] = _log_int(rng, 1, min(65536, 8192 * 4096 // c["d"]))
        if op == "embed":
            c.update(table=rng.choice(["f32", "bf16", "e4m3"]), out=rng.choice(["f32", "bf16"]))
        else:
            c.update(type=rng.choice(["f32", "bf16"]), grad=rng.choice(["f32", "bf16"]))
        if c.get("table") != "e4m3" and rng.random() < 0.5:
            c["d"] = max(1, c["d"] - rng.randrange(16))
        c["V"] = _log_int(rng, 17, min(262144, 151936 * 4096 // c["d"] // 2))
        return c
    c = dict(op=op, V=_log_int(rng, 17, 262144), type=rng.choice(["f32", "bf16"]), history=_log_int(rng, 1, 32768),
             bias=rng.choice([0, _log_int(rng, 1, 300)]), mask=rng.random() < 0.5)
    c["M"] = _log_int(rng, 1, max(1, min(1024, 256 * 151936 // c["V"], 256 * 8192 // c["history"])))
    if op == "sample":
        c["K"] = rng.randint(1, 16)
    return c


_SIZE = {"f32": 4, "bf16": 2, "e4m3": 1}


def work(case):
    c = case
    if c["op"] == "norm":
        e, s = c["M"] * c["d"], _SIZE[c["type"]]
        out = e + 4 * c["M"] * -(-c["d"] // BLOCK) if c["out"] == "codes" else e * _SIZE[c["out"]]
        return {"bytes": e * s * (3 if c["residual"] else 1) + out + c["d"] * _SIZE[c["weight"]], "flops": 6 * e}
    if c["op"] == "norm_grad":
        e, s = c["M"] * c["d"], _SIZE[c["type"]]
        return {"bytes": e * s * (4 if c["through"] else 3) + c["d"] * (_SIZE[c["weight"]] + 4), "flops": 12 * e}
    if c["op"] == "embed":
        return {"bytes": c["n"] * (4 + c["d"] * (_SIZE[c["table"]] + _SIZE[c["out"]])), "flops": c["n"] * c["d"]}
    if c["op"] == "embed_grad":
        return {"bytes": c["n"] * (4 + c["d"] * _SIZE[c["type"]]) + c["V"] * c["d"] * _SIZE[c["grad"]],
                "flops": c["n"] * c["d"]}
    e, s = c["M"] * c["V"], _SIZE[c["type"]]
    lists = c["M"] * (2 * c["history"] + 8 * c["bias"] + 20)  # histories are half full at the mean
    masks = _grammars(c) * -(-c["V"] // 32) * 4 if c["mask"] else 0
    out = 8 * c["M"] * c["K"] if c["op"] == "sample" else e * s
    return {"bytes": e * s + lists + masks + out, "flops": 4 * e}


# ---------------------------------------------------------------- inputs
_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _grammars(c):
    """Grammar states of a batch: some requests share one, some have none."""
    return max(1, c["M"] // 2)


def _inputs(c, seed):
    """Every input of a case from its seed, on the GPU."""
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device=dev)

    def frequent(n, *shape):
        """Tokens as text has them: a few ids hold much of it."""
        return (n * uniform(*shape).pow_(4)).long().clamp_(0, n - 1)

    s = {"case": c}
    if c["op"] in ("norm", "norm_grad"):
        M, d, t = c["M"], c["d"], _TYPES[c["type"]]
        channels = torch.exp(0.5 * normal(d))
        s["weight"] = (1.0 - c["offset"] + 0.2 * normal(d)).to(_TYPES[c["weight"]])
        if c["op"] == "norm":
            s["x"] = (normal(M, d) * channels).to(t)
            if c["residual"]:
                s["residual"] = (4.0 * normal(M, d) * channels).to(t)
            return s
        s["h"] = (4.0 * normal(M, d) * channels).to(t)
        s["dy"] = (normal(M, d) / M).to(t)
        s["dres"] = (normal(M, d) / M).to(t) if c["through"] else None
        return s
    if c["op"] == "embed":
        n, V, d = c["n"], c["V"], c["d"]
        s["tokens"] = frequent(V, n).to(torch.int32)
        if c["table"] == "e4m3":
            s["table"] = (normal(V, d) * 100.0).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
            s["scales"] = torch.exp(math.log(1e-4) + math.log(10.0) * uniform(-(-V // BLOCK), -(-d // BLOCK)))
        else:
            s["table"] = torch.empty(V, d, dtype=_TYPES[c["table"]], device=dev).normal_(0.0, 0.02, generator=gen)
        s["tokens"].masked_fill_(uniform(n) < 0.05, -1)  # padding
        return s
    if c["op"] == "embed_grad":
        n, V, d = c["n"], c["V"], c["d"]
        s["tokens"] = frequent(V, n).to(torch.int32)
        s["tokens"].masked_fill_(uniform(n) < 0.05, -1)
        s["dout"] = (normal(n, d) / n).to(_TYPES[c["type"]])
        return s
    M, V, L = c["M"], c["V"], c["history"]
    s["logits"] = (normal(M, V) * 2.5).to(_TYPES[c["type"]])
    s["history"] = frequent(V, M, L).to(torch.int32)
    s["lengths"] = (uniform(M) * (L + 1)).to(torch.int32).clamp_(0, L)
    s["prompt_lengths"] = (uniform(M) * s["lengths"]).to(torch.int32)
    s["repetition"] = 1.0 + 0.3 * uniform(M)
    s["frequency"] = 0.5 * uniform(M)
    s["presence"] = 0.5 * uniform(M)
    if c["bias"]:
        s["bias_ids"] = (V * uniform(M, c["bias"])).to(torch.int32).clamp_(0, V - 1)
        s["bias_values"] = 5.0 * normal(M, c["bias"])
        s["bias_values"].masked_fill_(uniform(M, c["bias"]) < 0.2, -math.inf)
        s["bias_ids"].masked_fill_(uniform(M, c["bias"]) < 0.2, -1)  # lists of different lengths
    if c["mask"]:
        R, W = _grammars(c), -(-V // 32)
        bits = torch.randint(-2 ** 31, 2 ** 31, (R, W), generator=gen, device=dev)
        sparse = bits & torch.randint(-2 ** 31, 2 ** 31, (R, W), generator=gen, device=dev) \
            & torch.randint(-2 ** 31, 2 ** 31, (R, W), generator=gen, device=dev)
        s["mask"] = torch.where(uniform(R, 1) < 0.5, bits, sparse).to(torch.int32)
        if R > 2:
            s["mask"][R - 1] = 0  # a grammar that has come to its end
        s["mask_rows"] = torch.randint(0 if M == 1 else -1, R, (M,), generator=gen, device=dev).to(torch.int32)
    if c["op"] == "sample":
        s["u"] = uniform(M)
        s["temperature"] = 0.5 + uniform(M)
    return s


def prepare(case, seed):
    return _inputs(case, seed)


# ---------------------------------------------------------------- one pass
def run(state):
    c = state["case"]
    if own:
        return _run_own(c, state)
    return {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "embed": _plain_embed,
            "embed_grad": _plain_embed_grad, "sample": _plain_sample, "adjust": _plain_adjust}[c["op"]](c, state)


def _run_own(c, s):
    import packed_quantized_lm_amd as pq
    if c["op"] == "norm":
        codes = c["out"] == "codes"
        y, h, q, qs = pq.rms_norm(s["x"], s["weight"], residual=s.get("residual"), eps=EPS, offset=c["offset"],
                                  want_y=not codes, out_dtype=None if codes else _TYPES[c["out"]], want_codes=codes)
        return y, h, q, qs
    if c["op"] == "norm_grad":
        return pq.rms_norm_backward(s["dy"], s["h"], s["weight"], dres=s["dres"], eps=EPS, offset=c["offset"])
    if c["op"] == "embed":
        return pq.embed(s["table"], s["tokens"], scale=c["scale"], out_dtype=_TYPES[c["out"]], scales=s.get("scales"))
    if c["op"] == "embed_grad":
        return pq.embed_backward(s["dout"], s["tokens"], c["V"], scale=c["scale"], grad_dtype=_TYPES[c["grad"]])
    rules = {k: s.get(k) for k in ("history", "lengths", "prompt_lengths", "repetition", "frequency", "presence",
                                   "bias_ids", "bias_values", "mask", "mask_rows")}
    if c["op"] == "sample":
        return pq.sample_logits(s["logits"], c["K"], u=s["u"], temperature=s["temperature"], **rules)
    return pq.adjust_logits(s["logits"], **rules)


def _plain_norm(c, s):
    x = s["x"].float()
    h = None
    if c["residual"]:
        h = (x + s["residual"].float()).to(s["x"].dtype)
        x = h.float()
    n = x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * (s["weight"].float() + c["offset"])
    if c["out"] != "codes":
        return n.to(_TYPES[c["out"]]), h, None, None
    M, d = n.shape
    nb = -(-d // BLOCK)
    nb_ = torch.nn.functional.pad(n, (0, nb * BLOCK - d)).view(M, nb, BLOCK)
    amax = nb_.abs().amax(2, keepdim=True)
    scale = torch.where(amax > 0, (amax * (1.0 / E4M3_MAX)).clamp_min(2.0 ** -126), amax)
    # the nearest e4m3 value (ties to even) of the quotient, in 64 bits since
    # 32 round it into ties
    q = torch.where(amax > 0, nb_.double() / scale.double().clamp_min(2.0 ** -200), 0.0)
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6))).clamp(-6, 8) - 3)
    q = (torch.round(q / step) * step).clamp(-E4M3_MAX, E4M3_MAX)
    q = q.view(M, nb * BLOCK)[:, :d].to(torch.float32).to(torch.float8_e4m3fn)
    return None, h, q, scale[:, :, 0].t().contiguous()


def _plain_norm_grad(c, s):
    h, dy = s["h"].float(), s["dy"].float()
    r = torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
    g = dy * (s["weight"].float() + c["offset"])
    dh = r * (g - h * (r * r * (g * h).mean(1, keepdim=True)))
    if s["dres"] is not None:
        dh = dh + s["dres"].float()
    return dh.to(s["h"].dtype), (dy * (h * r)).sum(0)


def _plain_embed(c, s):
    t = s["tokens"].long()
    held = t >= 0
    rows = s["table"][t.clamp_min(0)].float() if c["table"] != "e4m3" \
        else s["table"].view(torch.uint8)[t.clamp_min(0)].view(torch.float8_e4m3fn).float()
    if c["table"] == "e4m3":
        rows = rows * s["scales"][t.clamp_min(0) // BLOCK].repeat_interleave(BLOCK, 1)[:, :c["d"]]
    return torch.where(held[:, None], rows * c["scale"], 0.0).to(_TYPES[c["out"]])


def _plain_embed_grad(c, s):
    t = s["tokens"].long()
    rows = torch.where((t >= 0)[:, None], s["dout"].float(), 0.0)
    grad = torch.zeros(c["V"], c["d"], device=rows.device)
    grad.index_add_(0, t.clamp_min(0), rows)
    return grad.mul_(c["scale"]).to(_TYPES[c["grad"]])


def _plain_rules(c, s):
    """The adjusted logits in 32 bits."""
    y = s["logits"].float()
    M, V = y.shape
    t = s["history"].long()
    at = torch.arange(t.shape[1], device=t.device)
    held = at < s["lengths"].long()[:, None]
    drawn = held & (at >= s["prompt_lengths"].long()[:, None])
    zero = torch.zeros(M, V + 1, device=t.device)
    seen = zero.scatter(1, torch.where(held, t, V), 1.0)[:, :V]
    count = zero.scatter_add(1, torch.where(drawn, t, V), torch.ones_like(t, dtype=torch.float32))[:, :V]
    rho = s["repetition"][:, None]
    y = torch.where(seen > 0, torch.where(y > 0, y / rho, y * rho), y)
    y = torch.where(count > 0, (y - s["frequency"][:, None] * count) - s["presence"][:, None], y)
    if c["bias"]:
        ids = s["bias_ids"].long()
        last = torch.full((M, V + 1), -1, dtype=torch.long, device=t.device)
        last.scatter_reduce_(1, torch.where(ids >= 0, ids, V), torch.arange(c["bias"], device=t.device).expand(M, -1),
                             "amax")
        last = last[:, :V]
        bias = torch.gather(s["bias_values"], 1, last.clamp_min(0))
        y = torch.where(last >= 0, y + bias, y)
    if c["mask"]:
        v = torch.arange(V, device=t.device)
        r = s["mask_rows"].long()
        allowed = (s["mask"][r.clamp_min(0)][:, v // 32] >> (v % 32).to(torch.int32)) & 1
        y = torch.where((allowed != 0) | (r < 0)[:, None], y, -math.inf)
    return y


def _plain_adjust(c, s):
    return _plain_rules(c, s).to(s["logits"].dtype)


def _pick(values, ids, s):
    """The draw from the candidates, in 64 bits: it lies next to a border."""
    v = values.double()
    w = torch.exp((v - v[:, :1].clamp_min(-1e30)) / s["temperature"].double()[:, None])
    run_sum = w.cumsum(1)
    over = run_sum > s["u"].double()[:, None] * run_sum[:, -1:]
    first = over.float().argmax(1, keepdim=True)
    return torch.where(v[:, 0] > -math.inf, ids.gather(1, first)[:, 0], -1).to(torch.int32)


def _plain_sample(c, s):
    # equal values stay in the order of their indices
    values, ids = torch.sort(_plain_rules(c, s), dim=1, descending=True, stable=True)
    values, ids = values[:, :c["K"]].contiguous(), ids[:, :c["K"]].to(torch.int32)
    return values, ids, _pick(values, ids, s)


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = _inputs(case, seed)
    return {"norm": _exact_norm, "norm_grad": _exact_norm_grad, "embed": _exact_embed,
            "embed_grad": _exact_embed_grad, "sample": _exact_sample, "adjust": _exact_rules}[case["op"]](case, s)


def _exact_norm(c, s):
    f64 = torch.float64
    h, d = s["x"].to(f64), c["d"]
    given = None
    if c["residual"]:
        given = h + s["residual"].to(f64)
        h = given.to(s["x"].dtype).to(f64)  # the norm is the stored sum's
    rms = (torch.linalg.vector_norm(h, dim=1) ** 2 / d + EPS).sqrt()
    n = h / rms[:, None] * (s["weight"].to(f64) + c["offset"])
    if c["out"] != "codes":
        return n, given, None, None
    # every non-negative e4m3 value in order; its index is its code, whose last bit settles a tie
    values = torch.arange(127, dtype=torch.uint8, device=n.device).view(torch.float8_e4m3fn).to(f64)
    middles = (values[1:] + values[:-1]) / 2
    q, scales = torch.zeros_like(n), []
    for k0 in range(0, d, BLOCK):
        part = n[:, k0:k0 + BLOCK]
        scale = part.abs().amax(1) / E4M3_MAX
        scales.append(scale)
        a = (part / scale.clamp_min(2.0 ** -126)[:, None]).abs().contiguous()
        low, high = torch.searchsorted(middles, a), torch.searchsorted(middles, a, right=True)
        q[:, k0:k0 + BLOCK] = values[torch.where(low % 2 == 0, low, high)] * torch.sign(part)
    return None, given, q, torch.stack(scales)


def _exact_norm_grad(c, s):
    # the derivative of sum(dy n(h)) by h: n = w h / rms, drms/dh_j = h_j / (d rms)
    f64 = torch.float64
    h, w = s["h"].to(f64), s["weight"].to(f64) + c["offset"]
    up = s["dy"].to(f64)
    rms = ((h * h).sum(1) / c["d"] + EPS).sqrt()[:, None]
    unit = h / rms
    dh = (up * w - unit * ((up * w * unit).sum(1, keepdim=True) / c["d"])) / rms
    if s["dres"] is not None:
        dh += s["dres"].to(f64)
    return dh, torch.einsum("md,md->d", up, unit)


def _exact_embed(c, s):
    f64 = torch.float64
    out = torch.zeros(c["n"], c["d"], dtype=f64, device="cuda")
    at = torch.nonzero(s["tokens"] >= 0)[:, 0]
    t = s["tokens"][at].long()
    if c["table"] == "e4m3":
        codes = s["table"].view(torch.uint8)
        every = torch.arange(256, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn).to(f64)
        col = torch.arange(c["d"], device="cuda") // BLOCK
        out[at] = every[codes[t].long()] * s["scales"].to(f64)[(t // BLOCK)[:, None], col[None, :]] * c["scale"]
    else:
        out[at] = s["table"][t].to(f64) * c["scale"]
    return out


def _exact_embed_grad(c, s):
    at = torch.nonzero(s["tokens"] >= 0)[:, 0]
    t = s["tokens"][at].long()
    ids, which = torch.unique(t, return_inverse=True)
    sums = torch.zeros(ids.numel(), c["d"], dtype=torch.float64, device="cuda")
    sums.index_add_(0, which, s["dout"][at].double())
    out = torch.zeros(c["V"], c["d"], dtype=torch.float64, device="cuda")
    out[ids] = sums * c["scale"]
    return out


def _exact_rules(c, s):
    f64 = torch.float64
    y = s["logits"].to(f64)
    M, V = y.shape
    rows = torch.arange(M, device=y.device)[:, None].expand_as(s["history"])
    at = torch.arange(c["history"], device=y.device)[None, :]
    flat = rows * V + s["history"].long()
    inside = at < s["lengths"][:, None]
    seen = torch.bincount(flat[inside], minlength=M * V).view(M, V) > 0
    times = torch.bincount(flat[inside & (at >= s["prompt_lengths"][:, None])], minlength=M * V).view(M, V).to(f64)
    rho = s["repetition"].to(f64)[:, None].expand(M, V)
    y[seen] = torch.where(y[seen] > 0, y[seen] / rho[seen], y[seen] * rho[seen])
    y -= s["frequency"].to(f64)[:, None] * times + s["presence"].to(f64)[:, None] * (times > 0)
    for j in range(c["bias"]):  # a later entry of an id replaces an earlier one
        if j == 0:
            bias = torch.zeros_like(y)
        r = torch.nonzero(s["bias_ids"][:, j] >= 0)[:, 0]
        bias[r, s["bias_ids"][r, j].long()] = s["bias_values"][r, j].to(f64)
    if c["bias"]:
        y += bias
    if c["mask"]:
        bit = torch.arange(32, device=y.device, dtype=torch.int32)
        table = ((s["mask"][:, :, None] >> bit) & 1).view(s["mask"].shape[0], -1)[:, :V].bool()
        r = s["mask_rows"].long()
        y.masked_fill_(~table[r.clamp_min(0)] & (r >= 0)[:, None], -math.inf)
    return y


def _exact_sample(c, s):
    values = _exact_rules(c, s).topk(c["K"], dim=1).values
    return values, None, None  # the indices and the draw are whole numbers
