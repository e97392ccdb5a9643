"""Penalties, biases and grammar masks on logits, and the top-k draw from what
they leave (the archead_adjust_logits and archead_sample_logits entry points):
argument checks and output allocation; the work is in the library's HIP
kernels.  Outputs and the workspace are allocated on the call's stream, so the
calls can be captured into a graph."""
from __future__ import annotations

import ctypes
import functools

from .binding import _check, _need, load_library
from .losses import _need_vector, _type_code, need_rows, on_stream, ptr


def _rows_of(t, name, dtype, M, n, dev):
    """A matrix of M rows: its row stride."""
    return need_rows(t, name, (dtype,), (M, n), dev)


def _rules(logits, history, lengths, prompt_lengths, repetition, frequency, presence, bias_ids, bias_values, mask,
           mask_rows):
    """Checks everything the two calls share; (M, V, L, the C arguments from logits to mask_rows)."""
    import torch
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2 or logits.shape[1] < 1:
        raise ValueError("logits must be an M x V tensor")
    (M, V), dev = logits.shape, logits.device
    code = _type_code(logits.dtype, "logits")
    ld = need_rows(logits, "logits", (logits.dtype,), (M, V), dev)
    for name, t, dtype in (("lengths", lengths, torch.int32), ("prompt_lengths", prompt_lengths, torch.int32),
                           ("repetition", repetition, torch.float32), ("frequency", frequency, torch.float32),
                           ("presence", presence, torch.float32), ("mask_rows", mask_rows, torch.int32)):
        if t is not None:
            _need_vector(t, name, dtype, M, dev)
    L = ldh = B = ldb = R = ldm = 0
    if history is not None:
        if not isinstance(history, torch.Tensor) or history.dim() != 2:
            raise ValueError("history must be an M x L tensor")
        L = int(history.shape[1])
        ldh = _rows_of(history, "history", torch.int32, M, L, dev)
    elif lengths is not None or prompt_lengths is not None:
        raise ValueError("lengths and prompt_lengths belong to a history")
    if (bias_ids is None) != (bias_values is None):
        raise ValueError("bias_ids and bias_values come together")
    if bias_ids is not None:
        if not isinstance(bias_ids, torch.Tensor) or bias_ids.dim() not in (1, 2):
            raise ValueError("bias_ids must be a list of B ids, or M of them")
        B = int(bias_ids.shape[-1])
        if bias_ids.dim() == 1:  # one list for all rows
            _need(bias_ids, "bias_ids", (torch.int32,), (B,), dev)
            _need(bias_values, "bias_values", (torch.float32,), (B,), dev)
        else:
            ldb = _rows_of(bias_ids, "bias_ids", torch.int32, M, B, dev)
            if _rows_of(bias_values, "bias_values", torch.float32, M, B, dev) != ldb:
                raise ValueError("bias_ids and bias_values need the same row stride")
        if B == 0:
            bias_ids = bias_values = None
    if mask is not None:
        if not isinstance(mask, torch.Tensor) or mask.dim() != 2:
            raise ValueError("mask must be an R x ceil(V / 32) tensor")
        R, words = int(mask.shape[0]), -(-V // 32)
        ldm = _rows_of(mask, "mask", torch.int32, R, words, dev)
        if mask_rows is None and R != M:
            raise ValueError("without mask_rows the mask has a row for each row of logits")
        if R == 0:
            mask = mask_rows = None
    elif mask_rows is not None:
        raise ValueError("mask_rows belong to a mask")
    if L == 0:
        history = lengths = prompt_lengths = None
    return M, V, L, (M, V, ptr(logits), code, ld, ptr(history), L, ldh, ptr(lengths), ptr(prompt_lengths),
                        ptr(repetition), ptr(frequency), ptr(presence), ptr(bias_ids), ptr(bias_values), B, ldb,
                        ptr(mask), R, ldm, ptr(mask_rows))


@functools.lru_cache(maxsize=256)
def _workspace_bytes(M, V, L, K):
    n = ctypes.c_uint64()
    _check(load_library().archead_rules_workspace(M, V, L, K, ctypes.byref(n)), "archead_rules_workspace")
    return n.value


def _workspace(logits, L, K):
    """The calls' workspace and its size; none where nothing is needed."""
    import torch
    n = _workspace_bytes(*logits.shape, L, K)
    return (logits.new_empty(n, dtype=torch.uint8) if n else None), n


def adjust_logits(logits, history=None, lengths=None, prompt_lengths=None, repetition=None, frequency=None,
                  presence=None, bias_ids=None, bias_values=None, mask=None, mask_rows=None, out=None, stream=None):
    """The logits (fp32 or bf16, M x V) under their requests' rules, in the same
    type, or written to out (logits itself included):
    - history, int32 M x L tokens, of which lengths (int32 M) are in use and
      prompt_lengths (int32 M) of those are the prompt: repetition (fp32 M)
      divides or multiplies the logits of tokens that occur, frequency and
      presence (fp32 M) are taken off those that were generated;
    - bias_ids and bias_values, int32 and fp32 M x B (or B for all rows): added;
    - mask, int32 R x ceil(V / 32) bits of the tokens a grammar allows, row
      mask_rows[m] (int32 M; -1 for none) or row m: all others become -inf."""
    import torch
    M, V, L, args = _rules(logits, history, lengths, prompt_lengths, repetition, frequency, presence, bias_ids,
                              bias_values, mask, mask_rows)
    ldo = V if out is None else need_rows(out, "out", (logits.dtype,), (M, V), logits.device)

    def call(st):
        y = logits.new_empty((M, V)) if out is None else out
        ws, n = _workspace(logits, L, 0)
        _check(load_library().archead_adjust_logits(*args, ptr(y), ldo, ptr(ws), n, st), "archead_adjust_logits")
        return y
    return on_stream(logits.device, stream, call)


def sample_logits(logits, K: int, u=None, temperature=1.0, history=None, lengths=None, prompt_lengths=None,
                  repetition=None, frequency=None, presence=None, bias_ids=None, bias_values=None, mask=None,
                  mask_rows=None, stream=None):
    """(values fp32 M x K, indices int32 M x K, samples int32 M or None): the K <= 16
    largest of the logits under adjust_logits' rules, in order, and with u (fp32 M,
    in [0, 1)) a draw from them at the temperature (a number, or fp32 M; rows whose
    own is not positive take their largest, at inf all that are left weigh the same).  A
    row whose rules leave nothing draws -1."""
    import torch
    M, V, L, args = _rules(logits, history, lengths, prompt_lengths, repetition, frequency, presence, bias_ids,
                              bias_values, mask, mask_rows)
    dev, K = logits.device, int(K)
    if not 1 <= K <= min(16, V):
        raise ValueError("K must lie in [1, min(16, V)]")
    if u is not None:
        _need_vector(u, "u", torch.float32, M, dev)
    tau, taus = 1.0, None
    if isinstance(temperature, torch.Tensor):
        _need_vector(temperature, "temperature", torch.float32, M, dev)
        taus = temperature
    else:
        tau = float(temperature)

    def call(st):
        values = logits.new_empty((M, K), dtype=torch.float32)
        indices = logits.new_empty((M, K), dtype=torch.int32)
        samples = None if u is None else logits.new_empty(M, dtype=torch.int32)
        ws, n = _workspace(logits, L, K)
        _check(load_library().archead_sample_logits(*args, K, tau, ptr(taus), ptr(u), ptr(values), ptr(indices),
                                                    ptr(samples), ptr(ws), n, st), "archead_sample_logits")
        return values, indices, samples
    return on_stream(dev, stream, call)
