"""Packed ARCHead LM-head forward for MI355X (gfx950).

The forward of the ARCHead packed output head (logits = X W_hat^T with
W_hat = (sA o A5)(sB o B8) + sR o R4 + (sC o C8)(sD o D8), factored so that
W_hat is never materialised) runs in hand-written HIP kernels behind the C
ABI in include/archead.h.  `binding.PackedHead` is the Python face of that
ABI; `binding.build_head` constructs a packed head on the GPU from a dense
head and calibration states; `losses` holds the token log probabilities and
post-training losses over logits; `fp8` holds the 8-bit head (matrices in
e4m3 with a scale per block of 128, and their product); `norm`, `embedding`
and `sampling` hold what stands around a head in a model's loop (the final
norm, the embedding, and the rules and draw of the next token); `synth` draws
seeded synthetic inputs.
"""
from .binding import PackedHead, build_head, load_library, quantize, x_tensor_from_bits  # noqa: F401
from .embedding import embed, embed_backward  # noqa: F401
from .fp8 import Fp8Head, fp8_matmul, fp8_quantize  # noqa: F401
from .losses import policy_loss, preference_loss, token_logp  # noqa: F401
from .norm import rms_norm, rms_norm_backward  # noqa: F401
from .sampling import adjust_logits, sample_logits  # noqa: F401

__all__ = ["Fp8Head", "PackedHead", "adjust_logits", "build_head", "embed", "embed_backward", "fp8_matmul",
           "fp8_quantize", "load_library", "policy_loss", "preference_loss", "quantize", "rms_norm",
           "rms_norm_backward", "sample_logits", "token_logp", "x_tensor_from_bits"]
