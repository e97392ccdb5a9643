"""The packed head's gradient by its hidden states on the GPU against the fp64
oracle: dX = G W_hat with the dense W_hat of oracle/forward.py.

Tolerance: a code times its scale is rounded once to fp16 (2^-11 of it), fp32
entries of G too (bf16 ones are exact within 2^28 of the row's largest, below
that off by 2^-39 of it); a sum of n terms in fp32, each addition rounded or
truncated, is off by n 2^-23 of the terms' magnitudes; T and U carry 16 bits
into the second product (2^-16); dX is rounded once (2^-8).
"""
import numpy as np
import pytest

from gpu_util import say
from oracle import forward, layout
from packed_quantized_lm_amd.synth import random_small_head

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from packed_quantized_lm_amd import load_library
    load_library()


def half(bits):
    return np.asarray(bits).view(np.float16).astype(np.float64)


def magnitudes(f):
    """|sR R4|, the core's two factors' and the correction's."""
    R = np.abs(layout.unpack_r4(f["R4"], f["d"]).astype(float))
    R = R * np.repeat(np.abs(half(f["sR"])), f["g"], axis=1)
    A = np.abs(f["A5"].astype(float)) * np.abs(half(f["sA"]))[:, None]
    B = np.abs(f["B8"].astype(float)) * np.abs(half(f["sB"]))[:, None]
    C = np.abs(f["C8"].astype(float)) * np.abs(half(f["sC"]))[:, None]
    D = np.abs(f["D8"].astype(float)) * np.repeat(np.abs(half(f["sD"])), f["g"], axis=1)
    return R, A, B, C, D


def check(f, dlogits, dX, what=""):
    G = dlogits.double().cpu().numpy()
    want = G @ forward.dense_rows(f, np.arange(f["V"]))
    R, A, B, C, D = magnitudes(f)
    aG = np.abs(G)
    terms = aG @ R + (aG @ A) @ B + (aG @ C) @ D
    rel = 2.0 ** -11 * (2 if str(dlogits.dtype) == "torch.float32" else 1) + (f["V"] + f["k"] + f["r"]) * 2.0 ** -23 + 2.0 ** -16
    # rows of W_hat's magnitudes times what the smallest entries of G lose
    lost = aG.max(1)[:, None] * 2.0 ** -39 * (R.sum(0) + A.sum(0) @ B + C.sum(0) @ D)[None, :]
    tol = rel * terms + lost + 2.0 ** -8 * np.abs(want) + 2.0 ** -133
    got = dX.double().cpu().numpy()
    err = np.abs(got - want)
    assert (err <= tol).all(), (what, (err / tol).max())
    return want, got


def gradient(M, V, seed, dtype="bfloat16", pad=0, kind="softmax"):
    import torch
    rng = np.random.default_rng(seed)
    if kind == "softmax":
        y = rng.normal(0, 3, (M, V))
        p = np.exp(y - y.max(1, keepdims=True))
        g = -p / p.sum(1, keepdims=True)
        g[np.arange(M), rng.integers(0, V, M)] += 1
        g *= rng.normal(0, 1, M)[:, None] * np.exp(rng.normal(0, 3, M))[:, None]
    elif kind == "onehot":
        g = np.zeros((M, V))
        g[np.arange(M), (np.arange(M) * 37) % V] = 1.0
    else:
        g = rng.normal(0, 1, (M, V)) * np.exp(rng.normal(0, 4, (M, V)))
    buf = torch.full((M, V + pad), float("nan"), dtype=getattr(torch, dtype), device="cuda")
    buf[:, :V] = torch.from_numpy(g)
    return buf[:, :V]


#        V, d, k, r, g, M
SHAPES = [(16, 128, 0, 0, 32, 1), (1, 128, 5, 3, 128, 2), (37, 256, 16, 4, 64, 3), (130, 384, 0, 8, 96, 5),
          (1000, 128, 33, 0, 128, 16), (2049, 640, 40, 20, 32, 33), (517, 256, 7, 70, 256, 64),
          (3001, 512, 256, 64, 128, 65), (777, 1024, 100, 16, 64, 129), (300, 256, 16, 16, 128, 257),
          (5003, 384, 24, 12, 32, 31), (9001, 128, 8, 4, 128, 200), (16411, 128, 40, 0, 64, 256), (140003, 128, 0, 8, 64, 180)]


@pytest.mark.parametrize("V,d,k,r,g,M", SHAPES)
@pytest.mark.parametrize("dtype,pad,kind", [("bfloat16", 0, "softmax"), ("float32", 3, "wide")])
def test_backward_matches_the_oracle(V, d, k, r, g, M, dtype, pad, kind):
    import torch
    from packed_quantized_lm_amd import PackedHead
    say(f"backward V={V} d={d} k={k} r={r} g={g} M={M} {dtype} {kind}")
    f = random_small_head(V, d, k, r, g, 1, seed=V + d)
    head = PackedHead(f)
    before = head.device_bytes()
    head.reserve_backward(M)
    assert head.device_bytes() > before
    G = gradient(M, V, V + M, dtype, pad, kind)
    dX = head.backward(G)
    check(f, G, dX)
    assert torch.equal(head.backward(G), dX)
    head.close()


def test_columns_of_the_head_come_back():
    """One-hot gradients pick single rows of W_hat: codes, scales and the order
    of every column (bf16 rounding apart)."""
    from packed_quantized_lm_amd import PackedHead
    for V, d, k, r, g in ((300, 256, 40, 24, 64), (129, 384, 0, 0, 32)):
        f = random_small_head(V, d, k, r, g, 1, seed=5)
        head = PackedHead(f)
        head.reserve_backward(V)
        G = gradient(V, V, 0, kind="onehot")
        check(f, G, head.backward(G))
        head.close()


def test_scales_of_very_different_sizes():
    """Rows and groups whose scales span fp16's range, zero scales, negative ones."""
    from packed_quantized_lm_amd import PackedHead
    f = random_small_head(400, 256, 32, 16, 32, 1, seed=8)
    rng = np.random.default_rng(0)
    for n in ("sR", "sA", "sC"):
        s = 2.0 ** rng.integers(-14, 5, f[n].shape) * rng.uniform(1, 2, f[n].shape) * rng.choice([-1, 1, 0], f[n].shape)
        f[n] = s.astype(np.float16).view(np.uint16)
    head = PackedHead(f)
    head.reserve_backward(40)
    G = gradient(40, 400, 3)
    check(f, G, head.backward(G))
    head.close()


def test_zero_nan_and_infinite_rows():
    import torch
    from packed_quantized_lm_amd import PackedHead
    f = random_small_head(700, 256, 16, 8, 128, 1, seed=2)
    head = PackedHead(f)
    head.reserve_backward(70)
    G = gradient(70, 700, 1)
    want = head.backward(G)
    H = G.clone()
    H[3] = 0
    H[5, 17] = float("nan")
    H[66, 0] = float("inf")
    got = head.backward(H)
    assert not got[3].any()
    assert torch.isnan(got[5]).all() and torch.isnan(got[66]).all()
    rest = [m for m in range(70) if m not in (3, 5, 66)]
    assert torch.equal(got[rest], want[rest])
    head.close()


def test_parts_reserve_streams_and_graphs():
    """More rows than reserved go in parts; a later reserve enlarges; a side
    stream; a captured call replayed with other inputs."""
    import torch
    from packed_quantized_lm_amd import PackedHead
    from packed_quantized_lm_amd.binding import ArcheadError
    f = random_small_head(900, 256, 16, 8, 64, 1, seed=4)
    head = PackedHead(f)
    G = gradient(150, 900, 9)
    with pytest.raises(ArcheadError):
        head.backward(G)
    head.reserve_backward(40)
    parts = head.backward(G)
    check(f, G, parts)
    bytes40 = head.device_bytes()
    head.reserve_backward(10)
    assert head.device_bytes() == bytes40
    head.reserve_backward(200)
    assert head.device_bytes() > bytes40
    whole = head.backward(G)
    check(f, G, whole)
    assert head.backward(G[:0]).shape == (0, 256)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = head.backward(G, stream=side)
    side.synchronize()
    assert torch.equal(out, whole)
    torch.cuda.current_stream().wait_stream(side)
    static = G.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = head.backward(static)
        with pytest.raises(ArcheadError):
            head.reserve_backward(400, stream=torch.cuda.current_stream())
    for i in range(3):
        static.copy_(G * (i + 1))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, head.backward(static))
    # the forward of the same handle is left as it was
    from packed_quantized_lm_amd import x_tensor_from_bits
    y, _ = head.forward(x_tensor_from_bits(f["X"]))
    ref = forward.forward(f, f["X"])
    assert np.abs(y.cpu().numpy() - ref).max() <= 2e-3 * np.sqrt((ref ** 2).mean())
    head.close()


def test_a_refused_reserve_leaves_the_handle_as_it_was(monkeypatch):
    from packed_quantized_lm_amd import PackedHead
    from packed_quantized_lm_amd.binding import ENOMEM, ArcheadError
    f = random_small_head(600, 256, 8, 8, 64, 1, seed=6)
    head = PackedHead(f)
    held = head.device_bytes()
    monkeypatch.setenv("ARCHEAD_TEST_ALLOC_LIMIT", "4096")
    with pytest.raises(ArcheadError) as e:
        head.reserve_backward(8)
    assert e.value.status == ENOMEM and head.device_bytes() == held
    monkeypatch.setenv("ARCHEAD_TEST_ALLOC_LIMIT", "")
    head.reserve_backward(8)
    G = gradient(8, 600, 2)
    want = head.backward(G)
    monkeypatch.setenv("ARCHEAD_TEST_ALLOC_LIMIT", "4096")
    with pytest.raises(ArcheadError):
        head.reserve_backward(300)
    import torch
    assert torch.equal(head.backward(G), want)
    head.close()


def test_offsets_past_32_bits():
    """Rows of dlogits 2^29 elements apart: the last ones past 2^32 elements."""
    import torch
    from packed_quantized_lm_amd import PackedHead
    f = random_small_head(1000, 128, 8, 8, 32, 1, seed=12)
    head = PackedHead(f)
    head.reserve_backward(4)
    M, far = 10, 1 << 29
    flat = torch.zeros((M - 1) * far + 1000, dtype=torch.bfloat16, device="cuda")
    G = flat.as_strided((M, 1000), (far, 1))
    G.copy_(gradient(M, 1000, 3))
    assert torch.equal(head.backward(G), head.backward(G.contiguous()))
    head.close()


def test_binding_refuses_bad_tensors():
    import torch
    from packed_quantized_lm_amd import PackedHead
    f = random_small_head(64, 128, 8, 8, 32, 1, seed=7)
    head = PackedHead(f)
    head.reserve_backward(4)
    g = torch.zeros(4, 64, device="cuda")
    for bad in (g.double(), g.half(), g[0], g[:, :32], g.cpu(), g.t(), None, g[:1].expand(4, 64)):
        with pytest.raises((ValueError, TypeError)):
            head.backward(bad)
    for out in (torch.zeros(4, 128, device="cuda"), torch.zeros(3, 128, dtype=torch.bfloat16, device="cuda")):
        with pytest.raises((ValueError, TypeError)):
            head.backward(g, dX=out)
    head.close()
    with pytest.raises(ValueError):
        head.backward(g)
