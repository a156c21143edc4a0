"""RMS norm with the residual's addition (oracle; test infrastructure only).

  rstd_t = (mean_j h_tj^2 + eps)^(-1/2),  v_tj = h_tj rstd_t w_j
and, in 8 bits, per block of 32 columns the least integer e >= -126 with
max |v| <= 448 2^e over the block's finite values, each v 2^-e rounded half to
even onto the e4m3 numbers (three fraction bits, least normal exponent -6,
largest 448).  h = x + residual is the caller's, rounded as it is stored.

Backward of L(v) with g = dL/dv * w, by the quotient rule:
  dL/dh_i = rstd g_i - rstd^3 h_i / H sum_j g_j h_j,  plus the residual stream's
own dL/dh;  dL/dw_j = sum_t dL/dv_tj h_tj rstd_t.
"""
from __future__ import annotations

import numpy as np


def rmsnorm_forward(h, w, eps):
    """(v, rstd) in float64."""
    h = np.asarray(h, np.float64)
    rstd = 1.0 / np.sqrt(np.mean(h * h, axis=1) + eps)
    return h * rstd[:, None] * np.asarray(w, np.float64), rstd


def rmsnorm_backward(dv, h, w, rstd, dh=None):
    """(dL/dh, dL/dw)."""
    dv, h, w, r = (np.asarray(a, np.float64) for a in (dv, h, w, rstd))
    g = dv * w
    out = r[:, None] * g - r[:, None] ** 3 * h * np.mean(g * h, axis=1, keepdims=True)
    if dh is not None:
        out = out + np.asarray(dh, np.float64)
    return out, np.sum(dv * h * r[:, None], axis=0)


def least_exponent(top, largest, least=-126):
    """Elementwise the least integer e >= least with top <= largest * 2^e."""
    top = np.asarray(top, np.float64)
    e = np.full(top.shape, least)
    with np.errstate(divide="ignore"):
        guess = np.where(top > 0, np.floor(np.log2(np.where(top > 0, top, 1.0) / largest)), least)
    for d in (-1, 0, 1, 2):   # log2 may be an ulp off: decide by comparison
        c = np.maximum(guess + d, least).astype(np.int64)
        fits = top <= largest * np.exp2(c.astype(np.float64))
        lower = ~(top <= largest * np.exp2(c - 1.0)) | (c == least)
        e = np.where(fits & lower, c, e)
    return e


def round_to_grid(v, fraction_bits, least_normal):
    """Half to even onto the floats of so many fraction bits (subnormals below 2^least_normal)."""
    v = np.asarray(v, np.float64)
    exp = np.maximum(np.frexp(v)[1] - 1, least_normal)
    step = np.exp2(exp.astype(np.float64) - fraction_bits)
    return np.round(v / step) * step


def quantize8(v):
    """(values of the codes, exponents e [n][H/32]); v finite."""
    v = np.asarray(v, np.float64)
    b = v.reshape(v.shape[0], -1, 32)
    e = least_exponent(np.max(np.abs(b), axis=2), 448.0)
    q = round_to_grid(b * np.exp2(-e.astype(np.float64))[..., None], 3, -6)
    return q.reshape(v.shape), e
