"""4-bit integer expert weights in groups with a scale and a zero point.

TEST INFRASTRUCTURE ONLY (see the package docstring).

`group` consecutive rows of a column of W [E][R][C] share a scale s and a zero
point z; the weight of code q is bf16(s (q - z)).  s: the smallest number of 20
significant bits, at least 2^-126 (1 for a group of zeros), with max|w| <= 7 s and z
= 8, or (asymmetric) hi - lo <= 15 s, lo = min(w, 0), hi = max(w, 0), z = round(-lo
/ s); q = round(w / s) + z held to 0 .. 15.  Ties to even, quotients exact.  A group that is not finite, or whose
scale would be 2^124 or more, is NaN.
"""
from __future__ import annotations

import numpy as np

from .moe import silu

__all__ = ["bf16_round", "quant_i4", "dequant_i4", "i4_tiles", "i4_untiled", "experts_fwd_i4"]


def bf16_round(v):
    """fp64 -> the nearest bf16 number (8 significant bits, ties to even; normal range)."""
    m, e = np.frexp(np.asarray(v, np.float64))
    return np.ldexp(np.rint(np.ldexp(m, 8)), e - 8)


def _scale_up(need):
    """Smallest number of 20 significant bits >= need, at least 2^-126."""
    m, e = np.frexp(np.maximum(need, 2.0 ** -126))
    return np.ldexp(np.ceil(np.ldexp(m, 20)), e - 20)


def quant_i4(W, group, asymmetric=False):
    """codes uint8 [E][R][C], scales fp64 [E][R/group][C] (NaN: a group that is not finite), zeros uint8."""
    W = np.asarray(W, np.float64)
    E, R, C = W.shape
    w = W.reshape(E, R // group, group, C)
    bad = ~np.isfinite(w).all(axis=2)
    w = np.where(bad[:, :, None], 0.0, w)
    lo, hi = np.minimum(w.min(axis=2), 0), np.maximum(w.max(axis=2), 0)
    span = hi - lo if asymmetric else np.maximum(hi, -lo)
    s = np.where(span == 0, 1.0, _scale_up(span / (15 if asymmetric else 7)))
    z = np.clip(np.rint(-lo / s), 0, 15) if asymmetric else np.full_like(s, 8)
    q = np.clip(np.rint(w / s[:, :, None]) + z[:, :, None], 0, 15)
    bad |= s >= 2.0 ** 124
    return q.astype(np.uint8).reshape(E, R, C), np.where(bad, np.nan, s), z.astype(np.uint8)


def dequant_i4(q, s, z):
    """The weights [E][R][C] (bf16 values, fp64)."""
    q = np.asarray(q).astype(np.float64)
    group = q.shape[1] // s.shape[1]
    return bf16_round(np.repeat(np.asarray(s, np.float64), group, axis=1) *
                      (q - np.repeat(np.asarray(z).astype(np.float64), group, axis=1)))


def i4_tiles(q, s, z, pair=None):
    """Stored codes [E][N/16][R/128][4][16][16] and scale words uint32 [E][N/64][R/128][128/group][16][4]; `pair`:
    (q, s, z) of a matrix whose 16-column groups alternate with this one's."""
    E, R, C = q.shape
    U = 128 * s.shape[1] // R
    srcs = [(q, s, z)] + ([pair] if pair is not None else [])
    N = C * len(srcs)
    codes = np.zeros((E, N // 16, R // 128, 4, 16, 16), np.uint8)
    words = np.zeros((E, N // 64, R // 128, U, 16, 4), np.uint32)
    for p, (q_, s_, z_) in enumerate(srcs):
        bits = np.asarray(s_, np.float32).view(np.uint32)
        bits = np.where(np.isnan(s_), np.uint32(0x7fc00000), bits)
        assert not (bits & 15).any()
        w = bits | np.where(np.isnan(s_), 8, z_).astype(np.uint32)
        for c in range(C):
            n = 16 * (len(srcs) * (c // 16) + p) + c % 16
            for k in range(128):
                j, g, half, b = k // 32, k // 8 % 4, k // 4 % 2, k % 4
                codes[:, n // 16, :, g, n % 16, 4 * j + b] |= (q_[:, k::128, c] << (4 * half)).astype(np.uint8)
            words[:, n // 64, :, :, n % 16, n // 16 % 4] = w[:, :, c].reshape(E, R // 128, U)
    return codes, words


def i4_untiled(codes, words, pair=False):
    """The inverse: (q, s, z), or a pair of them."""
    E, NT, KT = codes.shape[:3]
    U, n_src = words.shape[3], 2 if pair else 1
    R, C = KT * 128, NT * 16 // n_src
    out = []
    for p in range(n_src):
        q, w = np.zeros((E, R, C), np.uint8), np.zeros((E, KT * U, C), np.uint32)
        for c in range(C):
            n = 16 * (n_src * (c // 16) + p) + c % 16
            for k in range(128):
                j, g, half, b = k // 32, k // 8 % 4, k // 4 % 2, k % 4
                q[:, k::128, c] = (codes[:, n // 16, :, g, n % 16, 4 * j + b] >> (4 * half)) & 15
            w[:, :, c] = words[:, n // 64, :, :, n % 16, n // 16 % 4].reshape(E, KT * U)
        out.append((q, (w & np.uint32(0xfffffff0)).view(np.float32).astype(np.float64), (w & 15).astype(np.uint8)))
    return out if pair else out[0]


def experts_fwd_i4(x, offsets, W1, W3, W2):
    """o [P][d] of permuted rows x, from dequantised weights, with h rounded to bf16; also h before its rounding,
    a and b."""
    P, f, d = x.shape[0], W1.shape[2], W2.shape[2]
    a, b, o = np.zeros((P, f)), np.zeros((P, f)), np.zeros((P, d))
    for e in range(len(offsets) - 1):
        r = slice(int(offsets[e]), int(offsets[e + 1]))
        a[r], b[r] = x[r] @ W1[e], x[r] @ W3[e]
        o[r] = bf16_round(silu(a[r]) * b[r]) @ W2[e]
    return o, silu(a) * b, a, b
