"""8-bit activation checkpoints.  Test infrastructure: see ``oracle/__init__``.

The pages keep the layer's input between the forward and the backward for one
product, dA = s (dY B)^T X [P3 "The idea"; P2 "Follow one QLoRA training
step", step 4], and give no storage format for it.  The format taken: a bf16
X [m x k] as int8 codes with one bf16 scale per block of 64 consecutive
elements of a row,

    c     = max |x|
    scale = bf16_rne(c / 127)
    code  = clamp(rint_half_even(x / scale), -127, 127)      (0 when scale == 0)
    X^    = bf16_rne(code * scale)

Quotients are formed in fp64 here: x and scale have 8-bit significands, so a
quotient that is no half integer differs from every half integer by more than
2^-17 relative, and fp64 rounding cannot move it across one.
"""

import numpy as np

from . import quant

BLOCK = 64


def quantize(X) -> tuple:
    """(codes int8 [m x k], scale fp32-held bf16 values [m x k/64])."""
    x = np.asarray(X, dtype=np.float64)
    m, k = x.shape
    b = x.reshape(m, k // BLOCK, BLOCK)
    c = np.max(np.abs(b), axis=2) if m else np.zeros((m, k // BLOCK))
    scale = quant.bf16_bits_to_f32(quant.bf16_rne_bits((c / 127.0).astype(np.float32)))
    s = scale.astype(np.float64)[:, :, None]
    q = np.divide(b, s, out=np.zeros_like(b), where=s > 0)
    codes = np.clip(np.rint(q), -127, 127).astype(np.int8).reshape(m, k)
    return codes, scale.reshape(m, k // BLOCK)


def dequant_bits(codes, scale) -> np.ndarray:
    """bf16 bit patterns of X^ [m x k]."""
    m, k = codes.shape
    v = codes.reshape(m, k // BLOCK, BLOCK).astype(np.float64) * np.asarray(scale, dtype=np.float64)[:, :, None]
    return quant.bf16_rne_bits(v.astype(np.float32)).reshape(m, k)    # 15-bit products are exact in fp32


def dequant_values(codes, scale) -> np.ndarray:
    return quant.bf16_bits_to_f32(dequant_bits(codes, scale)).astype(np.float64)
