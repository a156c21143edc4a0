"""4-bit weights with one power-of-two scale per 32 (oracle; test infrastructure only).

A code's magnitude is one of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (one fraction bit, two
exponent bits), bit 3 its sign; W_ik = value(code_ik) 2^(scale_{i, k/32} - 127).
A row's codes are packed two to a byte, the even column in the low nibble.
Rounding: per 32 weights the least power of two (2^-126 or more) with
max |w| <= 6 scale, then the nearest magnitude, ties to the even code.
"""
from __future__ import annotations

import numpy as np

from .norm import least_exponent

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(W):
    """(packed codes uint8 [rows][cols/2], scale bytes uint8 [rows][cols/32]); W finite."""
    W = np.asarray(W, np.float64)
    b = W.reshape(W.shape[0], -1, 32)
    e = least_exponent(np.max(np.abs(b), axis=2), 6.0)
    m = np.abs(b) * np.exp2(-e.astype(np.float64))[..., None]
    far = np.abs(m[..., None] - MAGNITUDES)
    near = far == far.min(axis=-1, keepdims=True)
    # of two equally near codes one is even
    code = np.argmax(near * (2 - np.arange(8) % 2), axis=-1)
    code = np.where(b < 0, code + 8, code).reshape(W.shape).astype(np.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), (e + 127).astype(np.uint8)


def values(codes, scales):
    """The weights in float64."""
    codes = np.asarray(codes, np.uint8)
    code = np.empty((codes.shape[0], codes.shape[1] * 2), np.uint8)
    code[:, 0::2], code[:, 1::2] = codes & 15, codes >> 4
    v = MAGNITUDES[code & 7] * np.where(code & 8, -1.0, 1.0)
    return v * np.repeat(np.exp2(np.asarray(scales, np.float64) - 127.0), 32, axis=1)
