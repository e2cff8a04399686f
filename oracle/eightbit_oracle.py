"""Plain fp64 CPU oracle of the 8-bit operators -- test infrastructure only.

numpy float64 throughout, each function the plain definition of what it
returns; no code shared with the GPU path.
"""
from __future__ import annotations

import numpy as np


def to_codes(v):
    """(p / scale before rounding, scale) of the rows of v: scale = max|v|/127.

    The unrounded quotient is returned so that a code can be held to within
    half a step of it, whichever way a tie falls.  Zero rows give zeros.
    """
    top = np.max(np.abs(v), axis=1) if v.shape[1] else np.zeros(v.shape[0])
    scale = top / 127.0
    quot = np.divide(v, scale[:, None], out=np.zeros_like(v), where=scale[:, None] > 0)
    return quot, scale


def rmsnorm(x, w, eps, residual=None):
    """(h, rstd, y): h = x + residual, rstd = (mean h^2 + eps)^(-1/2), y = h rstd w."""
    h = x if residual is None else x + residual
    rstd = 1.0 / np.sqrt(np.mean(h * h, axis=1) + eps)
    return h, rstd, h * rstd[:, None] * w


def rmsnorm_backward(dy, h, w, eps_rstd, dh=None):
    """(dx, dw) from the kept h and rstd."""
    n = h * eps_rstd[:, None]
    u = dy * w
    dx = eps_rstd[:, None] * (u - n * np.mean(u * n, axis=1, keepdims=True))
    return (dx if dh is None else dx + dh), np.sum(dy * n, axis=0)


def matmul_q8(xq, xs, wq, ws=None, bias=None, g=None, lora=None, s=1.0):
    """(y, size): the product with its composition, and the sum of the absolute
    values of its terms, which rounding errors are measured against."""
    base = (xq.astype(np.float64) @ wq.astype(np.float64).T) * xs[:, None]
    if ws is not None:
        base = base * ws
    y, size = base.copy(), np.abs(base)
    if g is not None:
        y = y + (g - 1.0) * base + g * s * lora
        size = size + np.abs((g - 1.0) * base) + np.abs(g * s * lora)
    if bias is not None:
        y = y + bias
        size = size + np.abs(bias)
    return y, size
