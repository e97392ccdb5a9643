"""The packed head's backward at the sizes whose launches differ from those of
few rows: tiles of 256 rows, the finish by 64 x 64, whole parts of the most
rows held at a time; against dX = G W_hat in fp64.

Tolerance, that of test_gpu_backward.py: codes times scales are rounded once to
fp16 (2^-11), fp32 entries of G too; a sum of n terms in fp32 is off by n 2^-23
of their magnitudes; T and U carry 16 bits on; small entries of a row lose
2^-39 of its largest; dX is rounded once (2^-8).
"""
import numpy as np
import pytest

import backward_plan
import test_gpu_backward
from gpu_util import say
from oracle import forward
from packed_quantized_lm_amd.synth import random_small_head

#        V, d, k, r, g, M, rows reserved
SHAPES = [(65537, 384, 40, 20, 96, 1500, 1500), (33001, 640, 100, 70, 32, 2047, 2048),
          (16411, 2048, 256, 128, 256, 1500, 1500), (65537, 2048, 0, 0, 64, 511, 511), (600, 8192, 20, 0, 128, 2048, 2048),
          (100, 6144, 0, 0, 64, 1500, 1500), (9001, 128, 8, 4, 32, 2300, 4000), (3001, 256, 33, 16, 32, 601, 601),
          (1000, 384, 64, 64, 96, 700, 300), (500, 4224, 32, 96, 32, 31, 31), (257, 128, 64, 64, 128, 16, 16)]


@pytest.fixture(autouse=True)
def gpu(request):
    if request.node.get_closest_marker("gpu"):
        import torch
        if not torch.cuda.is_available():
            pytest.skip("no GPU")


def test_the_shapes_reach_every_launch():
    """Of both lists of shapes together, by the rules in csrc/backward.hip: every
    kind of tile with full and padded low-rank tiles, one and several ranges,
    every finish, every conversion, one launch and two, parts of either size."""
    found = set()
    for V, d, k, r, g, M in test_gpu_backward.SHAPES:
        for dtype in ("bfloat16", "float32"):
            found |= backward_plan.of_call(V, d, k, r, M, M, dtype)
    for V, d, k, r, g, M, reserved in SHAPES:
        for dtype in ("bfloat16", "float32"):
            found |= backward_plan.of_call(V, d, k, r, M, reserved, dtype)
    kinds = [rows for rows, _, _ in backward_plan.C["kTiles"]]
    want = {f"low tiles {b}, {s}" for b in kinds for s in ("full", "partly padding")}
    want |= {f"tiles {b}, {s}" for b in kinds for s in ("one range", "several ranges")}
    want |= {f"finish {f}" for f in ("split", "16 x 16", "64 x 64")}
    want |= {f"tiles {kinds[-1]}, finish {f}" for f in ("16 x 16", "64 x 64")}
    want |= {f"convert {s} {t}" for s in ("a row", "slices") for t in ("bfloat16", "float32")}
    want |= {"one launch", "two launches", "parts", "parts of kChunkM"}
    assert want <= found, sorted(want - found)


@pytest.mark.gpu
@pytest.mark.parametrize("V,d,k,r,g,M,reserved", SHAPES)
@pytest.mark.parametrize("dtype,pad", [("bfloat16", 0), ("float32", 3)])
def test_backward_of_many_rows(V, d, k, r, g, M, reserved, dtype, pad):
    import torch
    from packed_quantized_lm_amd import PackedHead
    say(f"backward V={V} d={d} k={k} r={r} g={g} M={M} reserved={reserved} {dtype}")
    f = random_small_head(V, d, k, r, g, 1, seed=V + d)
    head = PackedHead(f)
    head.reserve_backward(reserved)
    gen = torch.Generator(device="cuda").manual_seed(V + M)
    p = torch.softmax(torch.randn(M, V, generator=gen, device="cuda") * 3, 1)
    p[torch.arange(M), torch.randint(0, V, (M,), generator=gen, device="cuda")] -= 1
    p *= torch.randn(M, 1, generator=gen, device="cuda") / M
    p[M // 2] = 0
    G = torch.full((M, V + pad), float("nan"), dtype=getattr(torch, dtype), device="cuda")[:, :V]
    G.copy_(p)
    del p
    dX = head.backward(G)
    assert torch.equal(head.backward(G), dX)
    few = slice(M - 3, M)  # a row's result is its own, near enough: other launches take it in a small call
    small = head.backward(G[few])
    head.close()

    def there(a):
        return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float64)).to("cuda")
    W = there(forward.dense_rows(f, np.arange(V)))
    R, A, B, C, D = (there(a) for a in test_gpu_backward.magnitudes(f))
    G = G.double()
    aG = G.abs()
    want = G @ W
    terms = aG @ R + (aG @ A) @ B + (aG @ C) @ D
    rel = 2.0 ** -11 * (2 if dtype == "float32" else 1) + (V + k + r) * 2.0 ** -23 + 2.0 ** -16
    lost = aG.amax(1, keepdim=True) * 2.0 ** -39 * (R.sum(0) + A.sum(0) @ B + C.sum(0) @ D)[None, :]
    tol = rel * terms + lost + 2.0 ** -8 * want.abs() + 2.0 ** -133
    err = (dX.double() - want).abs()
    assert (err <= tol).all(), float((err / tol).max())
    assert not dX[M // 2].any()
    assert ((small.double() - want[few]).abs() <= tol[few]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("V,d,k,r,g,M,reserved", SHAPES)
def test_rows_of_the_head_come_back(V, d, k, r, g, M, reserved):
    """One-hot gradients of different sizes pick rows of W_hat from all over the
    vocabulary: each sum over it has one term, and only the k and r terms of the
    second products are added, so that codes, scales, and the places of rows and
    columns show at 2^-11 of the terms and dX's rounding."""
    import torch
    from packed_quantized_lm_amd import PackedHead
    say(f"backward one-hot V={V} d={d} k={k} r={r} g={g} M={M}")
    f = random_small_head(V, d, k, r, g, 1, seed=V + d + 1)
    head = PackedHead(f)
    head.reserve_backward(reserved)
    v = (np.arange(M) * 7919 + 13) % V
    x = np.where(np.arange(M) % 3 == 0, -1.0, 1.5) * 2.0 ** (np.arange(M) % 17 - 8)
    G = torch.zeros(M, V, dtype=torch.bfloat16, device="cuda")
    G[torch.arange(M), torch.from_numpy(v)] = torch.from_numpy(x).to(torch.bfloat16).cuda()
    got = head.backward(G).double().cpu().numpy()
    head.close()
    # of those rows of the head alone
    part = dict(f, V=M, **{n: f[n][v] for n in ("A5", "sA", "R4", "sR", "C8", "sC")})
    R, A, B, C, D = test_gpu_backward.magnitudes(part)
    want = forward.dense_rows(part, np.arange(M)) * x[:, None]
    terms = (R + A @ B + C @ D) * np.abs(x)[:, None]
    tol = (2.0 ** -11 + (k + r) * 2.0 ** -23 + 2.0 ** -16) * terms + 2.0 ** -8 * np.abs(want) + 2.0 ** -133
    err = np.abs(got - want)
    assert (err <= tol).all(), ((err / tol).max(), np.argwhere(err > tol)[:4])


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["sR", "sA", "sC"])
def test_scales_far_below_the_largest(kind):
    """One scale near fp16's largest value beside ordinary and tiny ones: a code
    times its scale keeps 11 bits, or 2^-31 of the largest code times scale."""
    import torch
    from packed_quantized_lm_amd import PackedHead
    say(f"backward with one large {kind}")
    V, d, k, r, g = 300, 256, 24, 16, 32
    f = random_small_head(V, d, k, r, g, 1, seed=21)
    rng = np.random.default_rng(3)
    for n in ("sR", "sA", "sC"):
        s = 2.0 ** rng.uniform(-20, -8, f[n].shape)
        f[n] = s.astype(np.float16).view(np.uint16)
    f[kind] = f[kind].copy()
    f[kind].reshape(-1)[7] = np.array(60000, np.float16).view(np.uint16)
    head = PackedHead(f)
    head.reserve_backward(V)
    got = head.backward(torch.eye(V, dtype=torch.bfloat16, device="cuda")).double().cpu().numpy()
    head.close()
    R, A, B, C, D = test_gpu_backward.magnitudes(f)
    largest = {n: c * np.abs(test_gpu_backward.half(f[n])).max() for n, c in (("sR", 8), ("sA", 16), ("sC", 128))}
    lost = 2.0 ** -31 * (largest["sR"] + largest["sA"] * B.sum(0) + largest["sC"] * D.sum(0))[None, :]
    want = forward.dense_rows(f, np.arange(V))
    tol = ((2.0 ** -11 + (k + r) * 2.0 ** -23 + 2.0 ** -16) * (R + A @ B + C @ D) + lost + 2.0 ** -8 * np.abs(want)
           + 2.0 ** -133)
    err = np.abs(got - want)
    assert (err <= tol).all(), ((err / tol).max(), np.argwhere(err > tol)[:4])
