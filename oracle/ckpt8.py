"""8-bit activation checkpoint oracle (fp64).

TEST INFRASTRUCTURE ONLY (see the package docstring).

The row-scaled experts keep [a|b] as MXFP8 rows (quant_mx8_rows of a and of b)
between forward and backward; the backward is the formula's at the values that
read back, the forward's own results are those of the unrounded a and b.
"""
from __future__ import annotations

import numpy as np

from .moe import sigmoid, silu

__all__ = ["rowscaled_fwd", "swiglu_bwd_rowscaled"]


def rowscaled_fwd(xp, offsets, W1, W3, W2, p):
    """a, b, h = p silu(a) b and o = h W2 of the permuted rows."""
    P, f = xp.shape[0], W1.shape[2]
    a, b, h, o = np.zeros((P, f)), np.zeros((P, f)), np.zeros((P, f)), np.zeros((P, W2.shape[2]))
    for e in range(len(offsets) - 1):
        r = slice(int(offsets[e]), int(offsets[e + 1]))
        if r.stop > r.start:
            a[r], b[r] = xp[r] @ W1[e], xp[r] @ W3[e]
            h[r] = p[r, None] * silu(a[r]) * b[r]
            o[r] = h[r] @ W2[e]
    return a, b, h, o


def swiglu_bwd_rowscaled(a, b, p, dh):
    """(da, db, p silu(a) b, dp) of h = p silu(a) b for dh = dO W2^T."""
    s = sigmoid(a)
    g = silu(a) * b
    return (p[:, None] * dh * b * s * (1 + a * (1 - s)), p[:, None] * dh * silu(a), p[:, None] * g,
            (g * dh).sum(1))
