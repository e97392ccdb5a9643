"""Matrices in 8-bit floating point with a scale per block of 128, their
product, and an output head held that way (the archead_fp8_quantize and
archead_fp8_matmul entry points): argument checks and output allocation; the
work is in the library's HIP kernels."""
from __future__ import annotations

from .binding import _check, _need, load_library
from .losses import _type_code, need_rows, on_stream, ptr

BLOCK = 128


def _blocks(n: int) -> int:
    return -(-n // BLOCK)


def fp8_quantize(x, block_rows: int = 1, stream=None):
    """(codes, scales) of x, fp32 or bf16 rows x cols (cols a multiple of 16,
    rows may be strided): codes float8_e4m3fn rows x cols; scales fp32,
    [ceil(cols / 128), rows] for block_rows = 1 (a scale per row and block of
    128 columns), [ceil(rows / 128), ceil(cols / 128)] for block_rows = 128."""
    import torch
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be a rows x cols tensor")
    rows, cols = (int(n) for n in x.shape)
    code = _type_code(x.dtype, "x")
    if cols < 16 or cols % 16:
        raise ValueError("the columns must be a multiple of 16")
    if block_rows not in (1, BLOCK):
        raise ValueError("block_rows must be 1 or 128")
    ldx = need_rows(x, "x", (x.dtype,), (rows, cols), x.device)
    shape = (_blocks(cols), rows) if block_rows == 1 else (_blocks(rows), _blocks(cols))

    def call(st):
        q = torch.empty((rows, cols), dtype=torch.float8_e4m3fn, device=x.device)
        s = torch.empty(shape, dtype=torch.float32, device=x.device)
        _check(load_library().archead_fp8_quantize(rows, cols, ptr(x), code, ldx, block_rows, ptr(q), cols, ptr(s),
                                                   shape[1], st), "archead_fp8_quantize")
        return q, s
    return on_stream(x.device, stream, call)


def fp8_matmul(a, a_scales, b, b_scales, out_dtype=None, out=None, stream=None):
    """a b^T of a (M x K, scales [ceil(K / 128), M]) and b (N x K, scales
    [ceil(N / 128), ceil(K / 128)]): M x N in out_dtype (float32, the default,
    or bfloat16), or written to out (its rows may be strided)."""
    import torch
    f8 = torch.float8_e4m3fn
    if not isinstance(a, torch.Tensor) or not isinstance(b, torch.Tensor) or a.dim() != 2 or b.dim() != 2:
        raise ValueError("a and b must be matrices")
    M, K = (int(n) for n in a.shape)
    N, dev = int(b.shape[0]), a.device
    if K < 16 or K % 16:
        raise ValueError("K must be a multiple of 16")
    lda = need_rows(a, "a", (f8,), (M, K), dev)
    ldb = need_rows(b, "b", (f8,), (N, K), dev)
    _need(a_scales, "a_scales", (torch.float32,), (_blocks(K), M), dev)
    _need(b_scales, "b_scales", (torch.float32,), (_blocks(N), _blocks(K)), dev)
    if out is not None:
        code = _type_code(out.dtype, "out")
        if out_dtype is not None and out_dtype != out.dtype:
            raise ValueError("out and out_dtype disagree")
        ldo = need_rows(out, "out", (out.dtype,), (M, N), dev)
    else:
        out_dtype = torch.float32 if out_dtype is None else out_dtype
        code, ldo = _type_code(out_dtype, "out_dtype"), max(N, 1)

    def call(st):
        y = torch.empty((M, N), dtype=out_dtype, device=dev) if out is None else out
        _check(load_library().archead_fp8_matmul(M, N, K, ptr(a), lda, ptr(a_scales), M, ptr(b), ldb, ptr(b_scales),
                                                 _blocks(K), ptr(y), code, ldo, st), "archead_fp8_matmul")
        return y
    return on_stream(dev, stream, call)


class Fp8Head:
    """An output head (V x d) in e4m3 with a scale per 128 x 128 block, e.g.
    the reference policy's or a baseline to hold a packed head against.  The
    hidden states are quantised per row and block of 128 on every call."""

    def __init__(self, W, stream=None):
        """Quantises W (fp32 or bf16, V x d, d a multiple of 16)."""
        self.weight, self.scales = fp8_quantize(W, BLOCK, stream=stream)
        self.V, self.d = (int(n) for n in W.shape)

    @classmethod
    def from_blocks(cls, weight, scales):
        """A head from a checkpoint's codes (float8_e4m3fn V x d, contiguous) and block scales
        (fp32 [ceil(V / 128), ceil(d / 128)]), both kept, not copied."""
        import torch
        if not isinstance(weight, torch.Tensor) or weight.dim() != 2 or weight.shape[1] < 16 or weight.shape[1] % 16:
            raise ValueError("weight must be V x d with d a multiple of 16")
        V, d = (int(n) for n in weight.shape)
        _need(weight, "weight", (torch.float8_e4m3fn,), (V, d), weight.device)
        _need(scales, "scales", (torch.float32,), (_blocks(V), _blocks(d)), weight.device)
        self = cls.__new__(cls)
        self.weight, self.scales, self.V, self.d = weight, scales, V, d
        return self

    def forward(self, X, out_dtype=None, out=None, stream=None):
        """Logits M x V (fp32 by default, or bfloat16) of hidden states X (fp32 or bf16, M x d)."""
        import torch
        if not isinstance(X, torch.Tensor) or X.dim() != 2 or X.shape[1] != self.d:
            raise ValueError(f"X must be an M x {self.d} tensor")
        if X.device != self.weight.device:
            raise ValueError(f"X must live on {self.weight.device}, not {X.device}")
        q, s = fp8_quantize(X, 1, stream=stream)
        y = fp8_matmul(q, s, self.weight, self.scales, out_dtype=out_dtype, out=out, stream=stream)
        return y

    def forward_codes(self, codes, scales, out_dtype=None, out=None, stream=None):
        """forward of hidden states that are already codes and scales (rms_norm's with want_codes)."""
        return fp8_matmul(codes, scales, self.weight, self.scales, out_dtype=out_dtype, out=out, stream=stream)

    def embed(self, tokens, scale: float = 1.0, pad: int = -1, out_dtype=None, out=None, stream=None):
        """The head's rows as a tied embedding: scale * weight[tokens], n x d (bfloat16 by default)."""
        from .embedding import embed
        return embed(self.weight, tokens, scale=scale, pad=pad, out_dtype=out_dtype, out=out, scales=self.scales,
                     stream=stream)
