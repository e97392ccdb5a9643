"""The 8-bit head on the GPU against the fp64 oracle (oracle/fp8.py).

The quantiser is exact: equal codes and scales.  The product sums n = K terms
in fp32 in some order, each addition rounded or truncated (2^-23 of what has
been added so far, at most the sum of the terms' magnitudes), and takes three
roundings per block for the scales: |error| <= (K + 8) 2^-23 sum |terms|,
and half a step of the output's type.  With more than 64 rows and a bf16
result the products are formed by the fp8 matrix instruction, which aligns
each group of eight to its largest and cuts the others off at 2^-13 of it: a
group loses less than 7 2^-13 of its largest term, so all of them lose at most
7 2^-13 sum |terms|.
"""
import numpy as np
import pytest

from gpu_util import say
from oracle import fp8

pytestmark = pytest.mark.gpu
HALF = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8}


def tolerance(M, K, dtype, want, terms):
    cut = 7 * 2.0 ** -13 if dtype == "bfloat16" and M > 64 else 0.0
    return ((K + 8) * 2.0 ** -23 + cut) * terms + HALF[dtype] * np.abs(want)


@pytest.fixture(scope="module", autouse=True)
def gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from packed_quantized_lm_amd import load_library
    load_library()


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda")


def codes_of(t):
    import torch
    return t.view(torch.uint8).cpu().numpy()


def check_quant(x, block_rows):
    from packed_quantized_lm_amd import fp8_quantize
    q, s = fp8_quantize(x, block_rows)
    want_q, want_s = fp8.quantize(x.double().cpu().numpy(), block_rows)
    assert np.array_equal(s.cpu().numpy(), want_s)
    got = codes_of(q)
    want_q = np.where((want_q & 127) == 0, got & 128 | want_q, want_q)  # the sign of a zero code is free
    assert np.array_equal(got, want_q)


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("rows,cols,pad", [(1, 16, 0), (3, 144, 0), (130, 256, 5), (257, 1040, 1), (1, 4096, 0)])
def test_quantise_matches_the_oracle(rows, cols, pad, dtype, block_rows):
    import torch
    say(f"fp8_quantize {rows} x {cols} {dtype} block_rows={block_rows}")
    rng = np.random.default_rng(rows + cols)
    x = rng.normal(0, 1, (rows, cols + pad)) * np.exp(rng.normal(0, 2, cols + pad))
    x[rows // 2, :16] = 0.0
    x[:, -(cols // 3):] = 0.0 if rows == 130 else x[:, -(cols // 3):]
    t = dev(x.astype(np.float32)).to(getattr(torch, dtype))[:, :cols]
    check_quant(t, block_rows)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_quantise_ties_and_extremes(dtype):
    """Blocks whose quotients are ties, next to ties, subnormal codes, and
    scales from the smallest to the largest."""
    import torch
    v = fp8.decode(np.arange(127, dtype=np.uint8))
    mid = (v[1:] + v[:-1]) / 2
    rows = []
    for scale in (1.0, 0.5, 2.0 ** -20, 2.0 ** -120, 2.0 ** 100, 3.0, 1.1, 7e-3, 2.0 ** -126):
        for x in (np.concatenate([mid, [448.0, -448.0]]), np.concatenate([np.nextafter(mid.astype(np.float32), 0), [448, 1]]),
                  np.concatenate([-np.nextafter(mid.astype(np.float32), np.float32(1e9)), [448, 1]])):
            rows.append(x * scale)
    rows += [np.full(128, 1e-45), np.full(128, 3e38), np.r_[1e-40, np.full(127, 2e-41)]]
    check_quant(dev(np.array(rows).astype(np.float32)).to(getattr(torch, dtype)), 1)


def test_quantise_every_bf16_value():
    """All finite bf16 values, in blocks under a largest value of their own exponent range."""
    import torch
    bits = np.arange(65536, dtype=np.uint16).reshape(512, 128)
    f = (bits.astype(np.uint32) << 16).view(np.float32)
    f = np.where(np.isfinite(f), f, 0)
    check_quant(dev(f).to(torch.bfloat16), 1)
    rng = np.random.default_rng(3)
    check_quant(dev(rng.permutation(f.reshape(-1)).reshape(512, 128)).to(torch.bfloat16), 1)


def test_nan_and_infinity():
    import torch
    from packed_quantized_lm_amd import Fp8Head, fp8_quantize
    x = torch.ones(4, 256, device="cuda")
    x[1, 3], x[2, 200], x[3, :128] = float("nan"), float("inf"), float("nan")
    q, s = fp8_quantize(x)
    assert codes_of(q)[1, 3] == 127 and torch.isinf(s[1, 2]) and (codes_of(q)[3, :128] == 127).all()
    y = Fp8Head(torch.randn(33, 256, device="cuda")).forward(x)
    assert torch.isfinite(y[0]).all() and torch.isnan(y[1:]).all()


SHAPES = [(1, 1, 16), (1, 37, 48), (2, 16, 128), (5, 129, 144), (16, 300, 256), (17, 40, 1040), (33, 1000, 400),
          (64, 257, 512), (65, 130, 272), (127, 515, 640), (128, 256, 256), (129, 257, 384), (200, 700, 1168),
          (300, 1100, 2064), (513, 300, 128), (1, 5000, 4096), (7, 3001, 2576), (16, 300, 4096),
          (9, 200, 16400), (130, 4097, 1024), (600, 2500, 144), (777, 6001, 400), (999, 16290, 272)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_product(M, N, K, dtype):
    import torch
    from packed_quantized_lm_amd import fp8_matmul
    say(f"fp8_matmul M={M} N={N} K={K} {dtype}")
    rng = np.random.default_rng(M + N + K)
    f8 = torch.float8_e4m3fn

    def matrix(rows):  # strided rows; what lies past K is NaN
        buf = torch.full((rows, K + 32), 0x7F, dtype=torch.uint8, device="cuda")
        c = rng.integers(0, 127, (rows, K)).astype(np.uint8) | (rng.integers(0, 2, (rows, K)).astype(np.uint8) << 7)
        buf[:, :K] = dev(c)
        return c, buf.view(f8)[:, :K]
    a, ta = matrix(M)
    b, tb = matrix(N)
    nb = -(-K // 128)
    sa = np.exp(rng.normal(0, 1, (nb, M))).astype(np.float32)
    sb = np.exp(rng.normal(0, 1, (-(-N // 128), nb))).astype(np.float32)
    want, terms = fp8.matmul(a, sa, b, sb)
    buf = torch.full((M, N + 3), 7.0, dtype=getattr(torch, dtype), device="cuda")
    got = fp8_matmul(ta, dev(sa), tb, dev(sb), out=buf[:, :N])
    assert (buf[:, N:] == 7.0).all()
    err = np.abs(got.double().cpu().numpy() - want)
    tol = tolerance(M, K, dtype, want, terms)
    assert (err <= tol).all(), (err / tol).max()
    again = fp8_matmul(ta, dev(sa), tb, dev(sb), out_dtype=getattr(torch, dtype))
    assert torch.equal(again, got)


def test_product_of_integers_is_exact():
    """Small integer codes and power-of-two scales: no rounding anywhere."""
    import torch
    from packed_quantized_lm_amd import fp8_matmul
    rng = np.random.default_rng(9)
    for M, N, K in ((3, 50, 4096), (70, 600, 1024), (300, 520, 640)):
        a, b = (fp8.encode(rng.integers(-3, 4, (n, K)).astype(float)) for n in (M, N))
        sa = 2.0 ** rng.integers(-2, 3, (-(-K // 128), M)).astype(np.float32)
        sb = 2.0 ** rng.integers(-2, 3, (-(-N // 128), -(-K // 128))).astype(np.float32)
        f8 = lambda c: dev(c).view(torch.float8_e4m3fn)
        got = fp8_matmul(f8(a), dev(sa.astype(np.float32)), f8(b), dev(sb.astype(np.float32)))
        assert np.array_equal(got.double().cpu().numpy(), fp8.matmul(a, sa, b, sb)[0])


def test_head_empty_sizes_streams_and_graphs():
    import torch
    from packed_quantized_lm_amd import Fp8Head, fp8_quantize
    W = torch.randn(777, 272, device="cuda").bfloat16()
    head = Fp8Head(W)
    assert head.forward(W[:0]).shape == (0, 777)
    for M in (1, 30, 150):
        X = torch.randn(M, 272, device="cuda").bfloat16()
        want = head.forward(X)
        q, s = fp8_quantize(X)
        ref, terms = fp8.matmul(codes_of(q), s.cpu().numpy(), codes_of(head.weight), head.scales.cpu().numpy())
        assert (np.abs(want.double().cpu().numpy() - ref) <= 281 * 2.0 ** -23 * terms).all()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        y = head.forward(X, stream=side)
        side.synchronize()
        assert torch.equal(y, want)
        with torch.cuda.stream(side):
            head.forward(X)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = head.forward(X)
        for _ in range(3):
            X.normal_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, head.forward(X))


def test_offsets_past_32_bits():
    """Rows of out that lie 2^26 elements apart: the last ones past 2^32."""
    import torch
    from packed_quantized_lm_amd import Fp8Head
    head = Fp8Head(torch.randn(300, 64, device="cuda"))
    for M in (17, 70):
        X = torch.randn(M, 64, device="cuda")
        flat = torch.zeros(M * (1 << 26) + 512, dtype=torch.bfloat16, device="cuda")
        out = flat.as_strided((M, 300), (1 << 26, 1))
        head.forward(X, out=out)
        assert torch.equal(out.contiguous(), head.forward(X, out_dtype=torch.bfloat16))
        del flat, out


def test_binding_refuses_bad_tensors():
    import torch
    from packed_quantized_lm_amd import Fp8Head, fp8_matmul, fp8_quantize
    from packed_quantized_lm_amd.binding import ArcheadError
    x = torch.zeros(8, 64, device="cuda")
    for bad in (x.double(), x[0], x.cpu(), x.t(), x[:, :24], x[:, :8], x[:, ::2], None):
        with pytest.raises((ValueError, TypeError)):
            fp8_quantize(bad)
    with pytest.raises(ValueError):
        fp8_quantize(x, 64)
    q, s = fp8_quantize(x)
    w, ws = fp8_quantize(x, 128)
    for args in ((q.float(), s, w, ws), (q, s[:, :3], w, ws), (q, s.double(), w, ws), (q, s, w[:, :32], ws),
                 (q, s, w, ws.cpu()), (q.cpu(), s, w, ws), (q[:, :24], s, w[:, :24], ws), (q.t(), s, w, ws)):
        with pytest.raises((ValueError, TypeError)):
            fp8_matmul(*args)
    with pytest.raises(ValueError):
        fp8_matmul(q, s, w, ws, out_dtype=torch.float16)
    with pytest.raises(ArcheadError):  # a row stride that is no multiple of 16
        flat = torch.zeros(8 * 72, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        fp8_matmul(flat.as_strided((8, 64), (72, 1)), s, w, ws)
    with pytest.raises(ValueError):
        Fp8Head.from_blocks(w, ws[:, :0])
    with pytest.raises(ValueError):
        Fp8Head(x).forward(torch.zeros(2, 48, device="cuda"))
    torch.cuda.synchronize()
