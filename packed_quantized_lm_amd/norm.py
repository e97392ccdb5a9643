"""The root-mean-square norm with the residual's addition and an 8-bit output,
and its backward (the archead_rms_norm and archead_rms_norm_backward entry
points): argument checks and output allocation; the work is in the library's
HIP kernels.  Rows may be strided; outputs and the workspace are allocated on
the call's stream, so the calls can be captured into a graph."""
from __future__ import annotations

import ctypes
import functools

from .binding import _check, _need, load_library
from .fp8 import _blocks
from .losses import _type_code, need_rows, on_stream, ptr


def _matrix(t, name):
    import torch
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be an M x d tensor")
    M, d = t.shape
    return M, d, t.device


def _weight(weight, d, dev):
    import torch
    if not (isinstance(weight, torch.Tensor) and weight.get_device() == dev.index and weight.shape == (d,)
            and weight.is_contiguous()):
        _need(weight, "weight", (torch.float32, torch.bfloat16), (d,), dev)
    return _type_code(weight.dtype, "weight")


def _like(t, shape, dtype):
    """A contiguous tensor of this shape and type on t's device."""
    import torch
    # the cheapest of torch's allocations, where it is the same one
    if t.dtype is dtype and t.shape == shape and t.is_contiguous():
        return torch.empty_like(t)
    return t.new_empty(shape, dtype=dtype)


@functools.lru_cache(maxsize=256)
def _workspace_bytes(M, d):
    n = ctypes.c_uint64()
    _check(load_library().archead_rms_norm_workspace(M, d, ctypes.byref(n)), "archead_rms_norm_workspace")
    return n.value


def rms_norm(x, weight, residual=None, eps: float = 1e-6, offset: float = 0.0, want_y: bool = True, out_dtype=None,
             want_codes: bool = False, h_out=None, stream=None):
    """(y, h, codes, scales) of x + residual (fp32 or bf16, M x d each): the sum
    h, in the residual's type (None without one; h_out, which may be residual
    itself, takes it), its norm y = h / rms(h) * (weight + offset) in out_dtype
    (x's type by default; None for want_y=False) and, with want_codes, the norm
    as fp8_quantize's codes and scales (d a multiple of 16; else None, None),
    quantised from its fp32 values."""
    import torch
    M, d, dev = _matrix(x, "x")
    xc = _type_code(x.dtype, "x")
    ldx = need_rows(x, "x", (x.dtype,), (M, d), dev)
    wc = _weight(weight, d, dev)
    if not want_y and not want_codes:
        raise ValueError("want_y or want_codes is required")
    if not want_y and out_dtype is not None:
        raise ValueError("out_dtype without want_y")
    rc = ldr = ldh = 0
    if residual is not None:
        if not isinstance(residual, torch.Tensor):
            raise TypeError("residual must be a torch tensor")
        rc = _type_code(residual.dtype, "residual")
        ldr = need_rows(residual, "residual", (residual.dtype,), (M, d), dev)
    if h_out is not None:
        if residual is None:
            raise ValueError("h_out without a residual")
        ldh = need_rows(h_out, "h_out", (residual.dtype,), (M, d), dev)
        if h_out.data_ptr() == residual.data_ptr() and M > 1 and ldh != ldr:
            raise ValueError("h_out over residual needs its row stride")
    yt = x.dtype if out_dtype is None else out_dtype
    yc = _type_code(yt, "out_dtype")
    if want_codes and (d < 16 or d % 16):
        raise ValueError("codes need d to be a multiple of 16")

    def call(st):
        y = _like(x, (M, d), yt) if want_y else None
        h, stride = h_out, ldh
        if residual is not None and h is None:
            h, stride = _like(residual, (M, d), residual.dtype), d
        q = s = None
        if want_codes:
            q = x.new_empty((M, d), dtype=torch.float8_e4m3fn)
            s = x.new_empty((_blocks(d), M), dtype=torch.float32)
        if M:  # empty tensors have no addresses to pass on
            _check(load_library().archead_rms_norm(
                M, d, x.data_ptr(), xc, ldx, ptr(residual), rc, ldr, ptr(h), stride, weight.data_ptr(), wc, eps, offset,
                ptr(y), yc, d, ptr(q), d, ptr(s), M, st), "archead_rms_norm")
        return y, h, q, s
    return on_stream(dev, stream, call)


def rms_norm_backward(dy, h, weight, dres=None, eps: float = 1e-6, offset: float = 0.0, want_dweight: bool = True,
                      dh_out=None, stream=None):
    """(dh, dweight): the gradient by h (and so by x and the residual alike), in
    h's type, of what dy = the gradient by y reaches through the norm, plus dres,
    what reaches h through the residual stream (h's type, or None); and the
    weight's, fp32 d (None for want_dweight=False).  dh_out, which may be dres
    itself, takes the former."""
    import torch
    M, d, dev = _matrix(h, "h")
    hc = _type_code(h.dtype, "h")
    if not isinstance(dy, torch.Tensor):
        raise TypeError("dy must be a torch tensor")
    uc = _type_code(dy.dtype, "dy")
    ldh = need_rows(h, "h", (h.dtype,), (M, d), dev)
    ldu = need_rows(dy, "dy", (dy.dtype,), (M, d), dev)
    ldr = 0 if dres is None else need_rows(dres, "dres", (h.dtype,), (M, d), dev)
    wc = _weight(weight, d, dev)
    ldd = d if dh_out is None else need_rows(dh_out, "dh_out", (h.dtype,), (M, d), dev)

    def call(st):
        dh = _like(h, (M, d), h.dtype) if dh_out is None else dh_out
        dw = h.new_empty(d, dtype=torch.float32) if want_dweight else None
        n = _workspace_bytes(M, d)
        ws = h.new_empty(n, dtype=torch.uint8)
        _check(load_library().archead_rms_norm_backward(
            M, d, dy.data_ptr(), uc, ldu, h.data_ptr(), hc, ldh, weight.data_ptr(), wc, eps, offset, ptr(dres), ldr,
            dh.data_ptr(), ldd, ptr(dw), ws.data_ptr(), n, st), "archead_rms_norm_backward")
        return dh, dw
    return on_stream(dev, stream, call)
