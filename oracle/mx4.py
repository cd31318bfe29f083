"""MXFP4 oracle: E2M1 elements with one power-of-two (E8M0) scale per 32 values.

TEST INFRASTRUCTURE ONLY (see the package docstring).

The pages credit FP4 for part of the Blackwell results without a definition;
the storage is the OCP Microscaling one.  Reading used:

* E2M1 code c: sign bit 3, magnitude (0, 0.5, 1, 1.5, 2, 3, 4, 6)[c & 7];
* block of 32 values along the contraction: s is the smallest integer with
  max |v| <= 6 * 2^s, at least -126, 0 for an all-zero block; the stored byte
  is s + 127, or 255 when the block holds a NaN or an infinity;
* code(v) = the nearest E2M1 value to v * 2^-s, ties to the even code, the sign
  kept (a value that rounds to zero keeps its sign bit);
* weights: 128-row x 16-column tiles (quant_mx4_weights states the layout).
"""
from __future__ import annotations

import numpy as np

from .e4m3 import e4m3_decode, e4m3_encode
from .moe import combine, permute_map, route, silu
from .mx import dequant_mx_rows, quant_mx_rows

__all__ = ["E2M1", "mx4_decode", "mx4_encode", "mx_scale_byte", "quant_mx4_rows", "dequant_mx4_rows",
           "quant_mx8_rows", "dequant_mx8_rows", "quant_mx4_weights", "dequant_mx4_weights",
           "experts_mx4", "layer_fwd_mx4"]

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
_TABLE = np.concatenate([E2M1, -E2M1])


def mx4_decode(codes):
    return _TABLE[np.asarray(codes, dtype=np.uint8)]


def mx4_encode(v):
    """Nearest E2M1 code of |v| <= 6, by search on the value table; a tie goes to
    the even code."""
    v = np.asarray(v, dtype=np.float64)
    m = np.abs(v)
    hi = np.clip(np.searchsorted(E2M1, m, side="left"), 0, 7)
    lo = np.maximum(hi - 1, 0)
    dl, dh = m - E2M1[lo], E2M1[hi] - m
    take_lo = (dl < dh) | ((dl == dh) & (lo % 2 == 0))
    return (np.where(take_lo, lo, hi) + 8 * np.signbit(v)).astype(np.uint8)


def mx_scale_byte(V, top):
    """E8M0 byte of every block along V's last axis (top = 6 or 448)."""
    V = np.asarray(V, dtype=np.float64)
    bad = ~np.isfinite(V).all(-1)
    amax = np.max(np.abs(np.where(np.isfinite(V), V, 0.0)), axis=-1)
    s = np.full(amax.shape, -126, dtype=np.int64)
    with np.errstate(divide="ignore"):
        near = np.where(amax > 0, np.floor(np.log2(np.where(amax > 0, amax, 1.0) / top)), 0)
    for off in (3, 2, 1, 0, -1, -2):           # the smallest s that holds amax, by trial
        t = (near + off).astype(np.int64)
        s = np.where((amax <= top * np.exp2(t.astype(np.float64))) & (t >= -126), t, s)
    s = np.where(amax == 0, 0, s)
    return np.where(bad, 255, s + 127).astype(np.uint8)


def _scale(sb):
    sb = np.asarray(sb, np.int64)
    return np.where(sb == 255, np.nan, np.exp2((sb - 127).astype(np.float64)))


def _blocks(A):
    A = np.asarray(A)
    assert A.shape[-1] % 32 == 0
    return A.reshape(*A.shape[:-1], A.shape[-1] // 32, 32)


def quant_mx4_rows(A):
    """1 x 32 blocks along the last axis: packed codes [.., K/2] (lower index in
    the low nibble), scale bytes [.., K/32].  Codes of a NaN block are 0 here
    (they carry no meaning)."""
    V = _blocks(np.asarray(A, dtype=np.float64))
    sb = mx_scale_byte(V, 6.0)
    with np.errstate(invalid="ignore"):
        c = mx4_encode(np.where(sb[..., None] == 255, 0.0, V / np.where(sb == 255, 1.0, _scale(sb))[..., None]))
    c = c.reshape(*A.shape[:-1], A.shape[-1] // 2, 2)
    return c[..., 0] | (c[..., 1] << 4), sb


def dequant_mx4_rows(codes, sb):
    codes = np.asarray(codes, dtype=np.uint8)
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    return mx4_decode(c) * np.repeat(_scale(sb), 32, axis=-1)


def quant_mx8_rows(A):
    """The MXFP8 rows that the 4-bit experts make of h: E4M3 codes, s at least
    -126, scale byte 255 for a block with a NaN or an infinity."""
    V = _blocks(np.asarray(A, dtype=np.float64))
    sb = mx_scale_byte(V, 448.0)
    c = e4m3_encode(np.where(sb[..., None] == 255, 0.0, V / np.where(sb == 255, 1.0, _scale(sb))[..., None]))
    return c.reshape(A.shape), sb


def dequant_mx8_rows(codes, sb):
    return e4m3_decode(codes) * np.repeat(_scale(sb), 32, axis=-1)


def quant_mx4_weights(W, pair=None):
    """Expert matrices W [E][R][C] in the tile layout: codes [E][N/16][R/128][4][16][16]
    (byte b of (group g, column c) of tile (nt, kt): rows 128 kt + 32 g + 2 b and + 1
    of column 16 nt + c), scale bytes [E][N/64][R/128][4][16][4] (byte j of (g, c) of
    (nb, kt): that row group of column 64 nb + 16 j + c).  `pair`: 16-column groups of
    W and pair alternate (N = 2 C)."""
    W = np.asarray(W)
    E, R, C = W.shape
    srcs = [W] if pair is None else [W, np.asarray(pair)]
    N = C * len(srcs)
    codes = np.zeros((E, N // 16, R // 128, 4, 16, 16), np.uint8)
    scales = np.zeros((E, N // 64, R // 128, 4, 16, 4), np.uint8)
    for e in range(E):
        for p, M in enumerate(srcs):
            q, sb = quant_mx4_rows(np.ascontiguousarray(M[e].T))       # [C][R/2], [C][R/32]
            for c in range(C):
                G = (c // 16) * len(srcs) + p
                codes[e, G, :, :, c % 16, :] = q[c].reshape(R // 128, 4, 16)
                scales[e, G // 4, :, :, c % 16, G % 4] = sb[c].reshape(R // 128, 4)
    return codes, scales


def dequant_mx4_weights(codes, scales):
    """Values [E][R][N] of tiled codes and scales."""
    E, NT, KT = codes.shape[:3]
    out = np.empty((E, KT * 128, NT * 16))
    for e in range(E):
        for nt in range(NT):
            for c in range(16):
                out[e, :, 16 * nt + c] = dequant_mx4_rows(
                    codes[e, nt, :, :, c, :].reshape(-1), scales[e, nt // 4, :, :, c, nt % 4].reshape(-1))
    return out


def split_pair(M):
    """[..][2f] with alternating 16-column groups -> the two [..][f]."""
    v = M.reshape(*M.shape[:-1], -1, 2, 16)
    return (v[..., 0, :].reshape(*M.shape[:-1], -1), v[..., 1, :].reshape(*M.shape[:-1], -1))


def experts_mx4(xd, offsets, W13, W2, a8):
    """From dequantised permuted rows xd [P][d] and weights (values): a, b, h and
    o = Q(h) W2; rows from offsets[-1] on stay zero."""
    P, f = xd.shape[0], W13.shape[2] // 2
    a, b = np.zeros((P, f)), np.zeros((P, f))
    o = np.zeros((P, W2.shape[2]))
    h = np.zeros((P, f))
    quant, dequant = (quant_mx8_rows, dequant_mx8_rows) if a8 else (quant_mx4_rows, dequant_mx4_rows)
    for e in range(len(offsets) - 1):
        r = slice(int(offsets[e]), int(offsets[e + 1]))
        if r.stop > r.start:
            a[r], b[r] = split_pair(xd[r] @ W13[e])
            h[r] = silu(a[r]) * b[r]
            o[r] = dequant(*quant(h[r])) @ W2[e]
    return a, b, h, o


def layer_fwd_mx4(logits, x, W1, W3, W2, k, a8):
    """Route, quantise x rows, experts with 4-bit weights, combine."""
    idx, p = route(logits, k)
    counts, offsets, row_of, token_of = permute_map(idx, W1.shape[0])
    xd = dequant_mx_rows(*quant_mx_rows(x)) if a8 else dequant_mx4_rows(*quant_mx4_rows(x))
    W13d = dequant_mx4_weights(*quant_mx4_weights(W1, W3))
    W2d = dequant_mx4_weights(*quant_mx4_weights(W2))
    a, b, h, o = experts_mx4(xd[token_of], offsets, W13d, W2d, a8)
    return dict(idx=idx, p=p, counts=counts, offsets=offsets, row_of=row_of, token_of=token_of, xd=xd,
                W13=W13d, W2=W2d, a=a, b=b, h=h, o=o, y=combine(o, row_of, p))
