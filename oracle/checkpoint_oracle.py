"""Plain reference of the 8-bit activation checkpoint (TEST INFRASTRUCTURE
ONLY), from its definition: a block is 64 consecutive columns of a token, a its
largest |x|, the codes rint(127 x / a), and what they stand for
bf16(fl32(c fl32(a fl32(1/127)))).  Shares no code with the HIP library.
"""

from __future__ import annotations

import numpy as np

from .qlora_oracle import bf16_bits_to_f64, bf16_rne_bits_from_f32

__all__ = ["encode", "decode", "restored"]


def encode(bits):
    """(codes int8 [M, k], constants float64 [M, k/64]) of bf16 bit patterns [M, k]."""
    M, k = bits.shape
    x = bf16_bits_to_f64(bits).reshape(M, k // 64, 64)
    a = np.abs(x).max(axis=2)
    fine = np.isfinite(x).all(axis=2)
    a = np.where(fine, a, np.nan)
    use = fine & (a > 0)
    with np.errstate(invalid="ignore", divide="ignore"):
        c = np.rint(127 * x / np.where(use, a, 1.0)[..., None])
    c = np.where(use[..., None], c, 0.0)
    return c.astype(np.int8).reshape(M, k), a


def decode(codes, a):
    """bf16 bit patterns [M, k] of codes and constants (NaN blocks: a NaN)."""
    M, k = codes.shape
    step = (a.astype(np.float32) * np.float32(1.0 / 127.0)).astype(np.float32)
    v = codes.reshape(M, k // 64, 64).astype(np.float32) * step[..., None]
    return bf16_rne_bits_from_f32(v.astype(np.float32)).reshape(M, k)


def restored(bits):
    """What the checkpoint of bits stands for (bf16 bit patterns)."""
    return decode(*encode(bits))
