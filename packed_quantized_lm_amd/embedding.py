"""Rows of an embedding table by token, from fp32, bf16 or 8-bit tables, and the
table's gradient (the archead_embed and archead_embed_backward entry points):
argument checks and output allocation; the work is in the library's HIP
kernels.  Outputs and the workspace are allocated on the call's stream, so the
calls can be captured into a graph."""
from __future__ import annotations

import ctypes
import functools

from .binding import _check, _need, load_library
from .fp8 import _blocks
from .losses import _need_vector, _type_code, need_rows, on_stream, ptr

E4M3 = 2


@functools.lru_cache(maxsize=256)
def _workspace_bytes(n, V, d):
    need = ctypes.c_uint64()
    _check(load_library().archead_embed_workspace(n, V, d, ctypes.byref(need)), "archead_embed_workspace")
    return need.value


def _tokens(tokens, dev):
    import torch
    if not isinstance(tokens, torch.Tensor) or tokens.dim() != 1:
        raise ValueError("tokens must be a vector")
    _need_vector(tokens, "tokens", torch.int32, tokens.shape[0], dev)
    return tokens.shape[0]


def _pad(pad):
    if not -2 ** 31 <= pad < 2 ** 31:
        raise ValueError("pad must be a 32-bit number")
    return int(pad)


def embed(table, tokens, scale: float = 1.0, pad: int = -1, out_dtype=None, out=None, scales=None, stream=None):
    """scale * table[tokens], n x d in out_dtype (the table's type by default,
    bfloat16 for 8-bit tables) or written to out (its rows may be strided).
    table: V x d, float32, bfloat16, or float8_e4m3fn with scales fp32
    [ceil(V / 128), ceil(d / 128)] (an Fp8Head's); tokens: int32 n.  A token
    equal to pad gives zeros, any other outside [0, V) NaN."""
    import torch
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("table must be a V x d tensor")
    (V, d), dev = table.shape, table.device
    f8 = table.dtype == torch.float8_e4m3fn
    code = E4M3 if f8 else _type_code(table.dtype, "table")
    ldt = need_rows(table, "table", (table.dtype,), (V, d), dev)
    n, pad = _tokens(tokens, dev), _pad(pad)
    if f8:
        if scales is None:
            raise ValueError("an 8-bit table needs its scales")
        _need(scales, "scales", (torch.float32,), (_blocks(V), _blocks(d)), dev)
    elif scales is not None:
        raise ValueError("scales belong to 8-bit tables")
    if out is not None:
        if out_dtype is not None and out_dtype != out.dtype:
            raise ValueError("out and out_dtype disagree")
        oc, ldo = _type_code(out.dtype, "out"), need_rows(out, "out", (out.dtype,), (n, d), dev)
    else:
        out_dtype = (torch.bfloat16 if f8 else table.dtype) if out_dtype is None else out_dtype
        oc, ldo = _type_code(out_dtype, "out_dtype"), d

    def call(st):
        y = table.new_empty((n, d), dtype=out_dtype) if out is None else out
        _check(load_library().archead_embed(n, V, d, table.data_ptr(), code, ldt, ptr(scales), _blocks(d),
                                            tokens.data_ptr(), pad, scale, y.data_ptr(), oc, ldo, st), "archead_embed")
        return y
    return on_stream(dev, stream, call)


def embed_backward(dout, tokens, V: int, scale: float = 1.0, pad: int = -1, grad_dtype=None, dtable=None,
                   accumulate: bool = False, stream=None):
    """The gradient of a V x d table by what embed gave for tokens: row v is
    scale times the sum of the rows of dout (fp32 or bf16, n x d, rows may be
    strided) whose token is v.  Returned in grad_dtype (dout's type by default)
    or written to dtable (rows may be strided); with accumulate it is added to
    dtable, and rows of tokens that do not occur are left alone."""
    import torch
    if not isinstance(dout, torch.Tensor) or dout.dim() != 2:
        raise ValueError("dout must be an n x d tensor")
    (n, d), dev, V = dout.shape, dout.device, int(V)
    code = _type_code(dout.dtype, "dout")
    ldo = need_rows(dout, "dout", (dout.dtype,), (n, d), dev)
    if _tokens(tokens, dev) != n:
        raise ValueError("dout needs a row for every token")
    pad = _pad(pad)
    if dtable is not None:
        if grad_dtype is not None and grad_dtype != dtable.dtype:
            raise ValueError("dtable and grad_dtype disagree")
        gc, ldt = _type_code(dtable.dtype, "dtable"), need_rows(dtable, "dtable", (dtable.dtype,), (V, d), dev)
    else:
        if accumulate:
            raise ValueError("accumulate needs dtable")
        grad_dtype = dout.dtype if grad_dtype is None else grad_dtype
        gc, ldt = _type_code(grad_dtype, "grad_dtype"), d

    def call(st):
        g = dout.new_empty((V, d), dtype=grad_dtype) if dtable is None else dtable
        need = _workspace_bytes(n, V, d)
        ws = dout.new_empty(need, dtype=torch.uint8)
        _check(load_library().archead_embed_backward(
            n, V, d, dout.data_ptr(), code, ldo, tokens.data_ptr(), pad, scale, int(accumulate), g.data_ptr(), gc, ldt,
            ws.data_ptr(), need, st), "archead_embed_backward")
        return g
    return on_stream(dev, stream, call)
