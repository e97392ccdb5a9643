"""The post-training operators on the GPU at the ends of their documented
ranges: 2^20 rows, rows of 2^31 - 1 logits, sums over 2^20 columns, 2^29
columns of a product; against fp64 on the same device.

Tolerances are those of the other tests of each operator, in units of u = 2^-24:
log probabilities within (2 E[x] + 2 + 2 links + 3 + |logp|) u (a thread of the
longest row meets 512 vectors: links <= 1100), gradients 8 u more and the
output's half step; products (K + 8) 2^-23 of the terms' magnitudes; the
backward as in test_gpu_backward.py.
"""
import numpy as np
import pytest

from gpu_util import say
from oracle import forward

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from packed_quantized_lm_amd import load_library
    load_library()


def test_most_rows():
    """2^20 rows of 5 logits; as many rows through both losses and back."""
    import torch
    from packed_quantized_lm_amd import policy_loss, preference_loss, token_logp
    say("2^20 rows")
    M, V = 1 << 20, 5
    gen = torch.Generator(device="cuda").manual_seed(1)
    y = torch.randn(M, V, generator=gen, device="cuda") * 2
    t = torch.randint(0, V, (M,), generator=gen, device="cuda")
    logq = torch.log_softmax(y.double(), 1)
    want = logq.gather(1, t[:, None])[:, 0]
    # x < 30; one scalar link a logit and the merges
    tol = U * (2 * 30 + 2 + 2 * 16 + 3 + want.abs())
    got, lse = token_logp(y, t.int())
    assert ((got.double() - want).abs() <= tol).all()
    adv = torch.randn(M, generator=gen, device="cuda")
    w = torch.full((M,), 2.0 ** -20, device="cuda")
    old = (want - 0.05).float()
    loss, logp, dy = policy_loss(y, t.int(), old, adv, w, eps_low=0.2, eps_high=0.2, grad_dtype=torch.float32)
    assert torch.equal(logp, got)
    rho = torch.exp(want - old.double())
    value = -(adv.double() * rho) * w.double()
    assert abs(float(loss) - float(value.sum())) <= float((value.abs() * (tol + 8 * U)).sum()) + U * abs(float(loss))
    coef = -adv.double() * rho * w.double()
    grad = -logq.exp() * coef[:, None]
    grad.scatter_add_(1, t[:, None], coef[:, None])
    assert ((dy.double() - grad).abs() <= coef.abs()[:, None] * (2 * tol + 16 * U)[:, None]).all()
    # pairs of two answers of one row each
    off = torch.arange(M + 1, dtype=torch.int32, device="cuda")
    loss, h, _, dy = preference_loss(y, t.int(), torch.ones(M, device="cuda"), off, beta=0.5, grad_dtype=torch.float32)
    margin = 0.5 * (want[0::2] - want[1::2])
    both = 0.5 * (tol[0::2] + tol[1::2])
    assert ((h.double() - margin).abs() <= both + U * margin.abs()).all()
    value = torch.nn.functional.softplus(-margin)
    assert abs(float(loss) - float(value.mean())) <= float(both.mean()) + 8 * U * float(value.mean())
    slope = -0.5 / (M // 2) * torch.sigmoid(-margin)
    coef = torch.stack([slope, -slope], 1).reshape(-1)
    grad = -logq.exp() * coef[:, None]
    grad.scatter_add_(1, t[:, None], coef[:, None])
    assert ((dy.double() - grad).abs() <= coef.abs()[:, None] * (4 * tol + 16 * U)[:, None] + 1e-30).all()


def test_longest_rows():
    """Two rows of 2^31 - 1 logits; the second one's lie past 2^31 elements."""
    import torch
    from packed_quantized_lm_amd import policy_loss, token_logp
    say("rows of 2^31 - 1 logits")
    M, V = 2, (1 << 31) - 1
    y = torch.empty(M, V, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(2)
    part = 1 << 28
    for m in range(M):
        for v in range(0, V, part):
            n = min(part, V - v)
            y[m, v:v + n] = torch.randn(n, generator=gen, device="cuda")
    t = torch.tensor([V - 1, 1 << 30], device="cuda")
    y[0, V - 1], y[1, 1 << 30] = 25.0, 30.0
    z, zx = torch.zeros(M, dtype=torch.float64), torch.zeros(M, dtype=torch.float64)
    top = torch.tensor([25.0, 30.0], dtype=torch.float64)
    for m in range(M):
        for v in range(0, V, part):
            x = float(top[m]) - y[m, v:v + part].double()
            e = torch.exp(-x)
            z[m] += e.sum().cpu()
            zx[m] += (e * x).sum().cpu()
    want = -torch.log(z)
    tol = U * (2 * zx / z + 2 + 2 * 1100 + 3 + want.abs())
    got = token_logp(y, t.int())[0].double().cpu()
    assert ((got - want).abs() <= tol).all(), (got, want)
    one = torch.ones(M, device="cuda")
    old = want.float().cuda()
    _, logp, dy = policy_loss(y, t.int(), old, one, one, grad_dtype=torch.bfloat16)
    assert ((logp.double().cpu() - want).abs() <= tol).all()
    for m in range(M):
        p_t = 1.0 / float(z[m])
        for v in [0, 1 << 29, (1 << 30) - 4, V - 1000]:
            n = min(1000, V - v)
            x = float(top[m]) - y[m, v:v + n].double().cpu()
            grad = torch.exp(-x) * p_t  # c = -1
            if v <= int(t[m]) < v + n:
                grad[int(t[m]) - v] = p_t - 1
            off = (dy[m, v:v + n].double().cpu() - grad).abs()
            rel = float(tol[m]) * 2 + 2 * U * 40 + 16 * U + 2.0 ** -8
            assert (off <= rel * grad.abs() + 2.0 ** -133).all(), (m, v, (off / grad.abs()).max())


@pytest.mark.parametrize("M,N,K,dtype", [(3, 200, 1 << 20, "float32"), (100, 130, 1 << 20, "float32"),
                                         (100, 130, 1 << 20, "bfloat16"), (1 << 20, 16, 16, "float32"),
                                         ((1 << 20) - 1, 17, 32, "bfloat16"), (1, 1 << 29, 16, "bfloat16"),
                                         (17, (1 << 27) + 5, 16, "bfloat16")])
def test_products_at_the_ends_of_their_sizes(M, N, K, dtype):
    import torch
    from packed_quantized_lm_amd import fp8_matmul
    say(f"product {M} x {N} x {K} {dtype}")
    gen = torch.Generator(device="cuda").manual_seed(K)
    f8 = torch.float8_e4m3fn

    def codes(rows, cols):
        out = torch.empty(rows, cols, dtype=f8, device="cuda")
        step = max(1, (1 << 28) // cols)
        for r in range(0, rows, step):
            n = min(step, rows - r)
            out[r:r + n] = (torch.randn(n, cols, generator=gen, device="cuda") * 60).to(f8)
        return out
    a, b = codes(M, K), codes(N, K)
    nb = -(-K // 128)
    sa = torch.exp(torch.randn(nb, M, generator=gen, device="cuda"))
    sb = torch.exp(torch.randn(-(-N // 128), nb, generator=gen, device="cuda"))
    got = fp8_matmul(a, sa, b, sb, out_dtype=getattr(torch, dtype))
    rows = torch.arange(M, device="cuda") if M <= 4096 else torch.cat([torch.arange(0, 600), torch.arange(M - 600, M)]).cuda()
    cols = torch.arange(N, device="cuda") if N <= 4096 else torch.cat([torch.arange(0, 600), torch.arange(N - 600, N)]).cuda()
    A = a.view(torch.uint8)[rows].view(f8).double() * sa[:, rows].double().repeat_interleave(128, 0)[:K].t()
    B = b.view(torch.uint8)[cols].view(f8).double() * sb[cols // 128].double().repeat_interleave(128, 1)[:, :K]
    want, terms = A @ B.t(), A.abs() @ B.abs().t()
    cut = 7 * 2.0 ** -13 if dtype == "bfloat16" and M > 64 else 0.0
    tol = ((K + 8) * 2.0 ** -23 + cut) * terms + (2.0 ** -8 if dtype == "bfloat16" else U) * want.abs()
    assert ((got[rows][:, cols].double() - want).abs() <= tol).all()


def test_most_rows_through_the_packed_head():
    """2^20 rows in parts of 2048."""
    import torch
    import test_gpu_backward
    from packed_quantized_lm_amd import PackedHead
    from packed_quantized_lm_amd.synth import random_small_head
    say("2^20 rows through the packed head")
    V, M = 40, 1 << 20
    f = random_small_head(V, 128, 5, 3, 32, 1, seed=30)
    head = PackedHead(f)
    head.reserve_backward(M)
    gen = torch.Generator(device="cuda").manual_seed(4)
    G = torch.randn(M, V, generator=gen, device="cuda").to(torch.bfloat16)
    dX = head.backward(G)
    head.close()
    W = torch.from_numpy(forward.dense_rows(f, np.arange(V))).to("cuda")
    R, A, B, C, D = test_gpu_backward.magnitudes(f)
    terms_of = torch.from_numpy(R + A @ B + C @ D).to("cuda")
    for m in range(0, M, 1 << 16):
        want = G[m:m + (1 << 16)].double() @ W
        terms = G[m:m + (1 << 16)].double().abs() @ terms_of
        tol = (2.0 ** -11 + (V + 8) * 2.0 ** -23 + 2.0 ** -16) * terms + 2.0 ** -8 * want.abs() + 2.0 ** -133
        assert ((dX[m:m + (1 << 16)].double() - want).abs() <= tol).all()
