"""Root-mean-square norm with the residual's addition, and its gradients.

TEST INFRASTRUCTURE ONLY (see the package docstring).

s = x + residual as stored (the caller passes the rounding of the storage type),
rstd = (mean(s^2) + eps)^(-1/2), y = s rstd gamma.  With g = dy gamma,
dx = dsum + rstd (g - s rstd^2 mean(g s)) and dgamma = sum over rows of
dy s rstd.
"""
from __future__ import annotations

import numpy as np

__all__ = ["rms_norm", "rms_norm_bwd"]


def rms_norm(s, gamma, eps):
    """(y, rstd) of rows s [T][d]."""
    s = np.asarray(s, np.float64)
    rstd = 1.0 / np.sqrt((s * s).mean(axis=1) + eps)
    return s * rstd[:, None] * np.asarray(gamma, np.float64), rstd


def rms_norm_bwd(dy, s, rstd, gamma, dsum=None):
    """(dx, dgamma) for the upstream gradients dy of y and dsum of s."""
    dy, s = np.asarray(dy, np.float64), np.asarray(s, np.float64)
    r = np.asarray(rstd, np.float64)[:, None]
    g = dy * np.asarray(gamma, np.float64)
    dx = r * (g - s * r * r * (g * s).mean(axis=1, keepdims=True))
    if dsum is not None:
        dx = dx + np.asarray(dsum, np.float64)
    return dx, (dy * s * r).sum(axis=0)
