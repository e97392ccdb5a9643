"""Token log probabilities and post-training losses over logits (the
archead_token_logp, archead_policy_loss and archead_preference_loss entry
points): argument checks and output allocation; the work is in the library's
HIP kernels.  Rows may be strided (any row stride >= V); outputs and the
workspace are allocated on the call's stream, so the calls can be captured
into a graph."""
from __future__ import annotations

import contextlib
import ctypes

from .binding import _check, _need, load_library

F32, BF16 = 0, 1


def _type_code(dtype, name):
    import torch
    try:
        return {torch.float32: F32, torch.bfloat16: BF16}[dtype]
    except KeyError:
        raise ValueError(f"{name} must be float32 or bfloat16, not {dtype}") from None


@contextlib.contextmanager
def _entered(device, stream):
    import torch
    with torch.cuda.device(device):
        s = torch.cuda.current_stream(device) if stream is None else stream
        if s.device != device:
            raise ValueError(f"the stream belongs to {s.device}, the tensors live on {device}")
        with torch.cuda.stream(s):
            yield s.cuda_stream


def on_stream(device, stream, call):
    """call(hipStream_t) with device current and stream (default: that
    device's current one) the stream of the allocations inside."""
    import torch
    # entering torch's device and stream contexts costs 10 us, more than the
    # smallest calls, and a Stream object 2 us: both are skipped where they
    # would change nothing
    if stream is None and device.index == torch.cuda.current_device():
        return call(torch._C._cuda_getCurrentRawStream(device.index))
    with _entered(device, stream) as st:
        return call(st)


def need_rows(t, name, dtypes, shape, device):
    """As _need, for a matrix whose rows may be strided; returns the row stride."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    # the usual call, in one line; the rest says what is wrong with another
    if device.type == "cuda" and t.device == device and t.dtype in dtypes and t.shape == shape and t.is_contiguous():
        return max(shape[1], 1)
    if t.device.type != "cuda" or t.device != device:
        raise ValueError(f"{name} must live on {device}, not {t.device}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must have dtype {' or '.join(str(d) for d in dtypes)}, not {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if shape[0] <= 1 or shape[1] == 0:
        if shape[1] > 1 and t.stride(1) != 1:
            raise ValueError(f"{name} must have contiguous rows")
        return max(int(shape[1]), 1)
    if (shape[1] > 1 and t.stride(1) != 1) or t.stride(0) < shape[1]:
        raise ValueError(f"{name} must have contiguous rows that do not overlap")
    return int(t.stride(0))


def ptr(t):
    return None if t is None else t.data_ptr()


def _need_vector(t, name, dtype, n, device):
    # what a sound call costs is this one line; _need says what is wrong with another
    if not (hasattr(t, "dtype") and t.dtype == dtype and t.shape == (n,) and t.device == device and t.is_contiguous()):
        _need(t, name, (dtype,), (n,), device)


def _logit_args(logits, targets, **vectors):
    """Checks logits, targets and the fp32 vectors of M values; (M, V, type, ld)."""
    import torch
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
        raise ValueError("logits must be an M x V tensor")
    M, V = logits.shape
    if V < 1:
        raise ValueError("logits need at least one column")
    code = _type_code(logits.dtype, "logits")
    ld = need_rows(logits, "logits", (logits.dtype,), (M, V), logits.device)
    _need_vector(targets, "targets", torch.int32, M, logits.device)
    for name, t in vectors.items():
        if t is not None:
            _need_vector(t, name, torch.float32, M, logits.device)
    return M, V, code, ld


def _workspace(M, V, P, device):
    import torch
    n = ctypes.c_uint64()
    _check(load_library().archead_loss_workspace(M, V, P, ctypes.byref(n)), "archead_loss_workspace")
    return torch.empty(n.value, dtype=torch.uint8, device=device), n.value


def _gradient(logits, M, V, grad_dtype, dlogits):
    """(dlogits, type code, row stride) of a gradient to write, (None, 0, 0) for none."""
    import torch
    if dlogits is None and grad_dtype is None:
        return None, 0, 0
    if dlogits is None:
        code = _type_code(grad_dtype, "grad_dtype")
        return torch.empty(M, V, dtype=grad_dtype, device=logits.device), code, V
    if grad_dtype is not None and dlogits.dtype != grad_dtype:
        raise ValueError("dlogits and grad_dtype disagree")
    code = _type_code(dlogits.dtype, "dlogits")
    return dlogits, code, need_rows(dlogits, "dlogits", (dlogits.dtype,), (M, V), logits.device)


def token_logp(logits, targets, stream=None):
    """(logp, lse), fp32 M each: the log probability of targets (int32 M) and
    the log-normaliser of every row of logits (fp32 or bf16, M x V)."""
    import torch
    M, V, code, ld = _logit_args(logits, targets)
    dev = logits.device

    def call(st):
        logp = torch.empty(M, dtype=torch.float32, device=dev)
        lse = torch.empty(M, dtype=torch.float32, device=dev)
        ws, n = _workspace(M, V, 0, dev)
        _check(load_library().archead_token_logp(M, V, ptr(logits), code, ld, ptr(targets), ptr(logp), ptr(lse),
                                                 ptr(ws), n, st), "archead_token_logp")
        return logp, lse
    return on_stream(dev, stream, call)


def policy_loss(logits, targets, old_logp, advantages, weights, ref_logp=None, beta: float = 0.0,
                eps_low: float = 0.2, eps_high: float = 0.2, grad_dtype=None, dlogits=None, grad_scale=None,
                stream=None):
    """The clipped policy loss with a KL term, sum_m weights_m (...): returns
    (loss fp32 scalar, logp fp32 M, dlogits or None).  The gradient by the
    logits is computed when grad_dtype (float32 or bfloat16) or a tensor
    dlogits to write it to (logits itself included) is given; grad_scale, an
    fp32 device scalar, multiplies it."""
    import torch
    M, V, code, ld = _logit_args(logits, targets, old_logp=old_logp, advantages=advantages, weights=weights,
                                 ref_logp=ref_logp)
    dev = logits.device
    for name, t in (("old_logp", old_logp), ("advantages", advantages), ("weights", weights)):
        if t is None:
            raise ValueError(f"{name} is required")
    if grad_scale is not None:
        _need(grad_scale, "grad_scale", (torch.float32,), (), dev)

    def call(st):
        dy, gcode, ldg = _gradient(logits, M, V, grad_dtype, dlogits)
        loss = torch.empty((), dtype=torch.float32, device=dev)
        logp = torch.empty(M, dtype=torch.float32, device=dev)
        ws, n = _workspace(M, V, 0, dev)
        _check(load_library().archead_policy_loss(
            M, V, ptr(logits), code, ld, ptr(targets), ptr(old_logp), ptr(ref_logp), ptr(advantages), ptr(weights),
            float(eps_low), float(eps_high), float(beta), ptr(grad_scale), ptr(loss), ptr(logp), ptr(dy), gcode, ldg,
            ptr(ws), n, st), "archead_policy_loss")
        return loss, logp, dy
    return on_stream(dev, stream, call)


def preference_loss(logits, targets, weights, offsets, ref_logp=None, beta: float = 0.1, smoothing: float = 0.0,
                    grad_dtype=None, dlogits=None, grad_scale=None, stream=None):
    """The preference loss of P answer pairs; offsets (int32 2P + 1) bound the
    answers' rows, chosen and rejected in turn.  Returns (loss fp32 scalar,
    margins fp32 P, logp fp32 M, dlogits or None), the gradient as for
    policy_loss."""
    import torch
    M, V, code, ld = _logit_args(logits, targets, weights=weights, ref_logp=ref_logp)
    dev = logits.device
    if weights is None:
        raise ValueError("weights is required")
    if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or offsets.shape[0] < 3 or offsets.shape[0] % 2 == 0:
        raise ValueError("offsets must hold 2P + 1 values, P >= 1")
    _need(offsets, "offsets", (torch.int32,), (offsets.shape[0],), dev)
    P = (int(offsets.shape[0]) - 1) // 2
    if grad_scale is not None:
        _need(grad_scale, "grad_scale", (torch.float32,), (), dev)

    def call(st):
        dy, gcode, ldg = _gradient(logits, M, V, grad_dtype, dlogits)
        loss = torch.empty((), dtype=torch.float32, device=dev)
        margins = torch.empty(P, dtype=torch.float32, device=dev)
        logp = torch.empty(M, dtype=torch.float32, device=dev)
        ws, n = _workspace(M, V, P, dev)
        _check(load_library().archead_preference_loss(
            M, V, ptr(logits), code, ld, ptr(targets), ptr(weights), P, ptr(offsets), ptr(ref_logp), float(beta),
            float(smoothing), ptr(grad_scale), ptr(loss), ptr(margins), ptr(logp), ptr(dy), gcode, ldg, ptr(ws), n,
            st), "archead_preference_loss")
        return loss, margins, logp, dy
    return on_stream(dev, stream, call)
