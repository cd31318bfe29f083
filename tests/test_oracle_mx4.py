"""Pins of the MXFP4 oracle (oracle/mx4.py), CPU only: the code table by
enumeration, rounding against brute force, the scale rule at its boundaries, the
tile layout element by element, and a whole layer near the unquantised one."""
import numpy as np
import pytest

import oracle
from oracle.mx4 import split_pair

RNG = np.random.default_rng(44)


def test_every_code_is_its_value():
    for c in range(16):
        s, e, m = c >> 3, (c >> 1) & 3, c & 1
        v = (1 + m / 2) * 2.0 ** (e - 1) if e else m / 2
        assert oracle.mx4_decode(c) == (-v if s else v)
    assert np.array_equal(oracle.mx4_encode(oracle.mx4_decode(np.arange(16))),
                          np.where(np.arange(16) == 8, 8, np.arange(16)))


def test_rounding_brute_force():
    v = np.concatenate([RNG.uniform(-6, 6, 4000), np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]),
                        -np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]), [0.0, -0.0, -0.1, 6.0]])
    got = oracle.mx4_encode(v)
    for x, c in zip(v, got):
        d = np.abs(oracle.E2M1 - abs(x))
        best = np.flatnonzero(d == d.min())
        want = best[0] if len(best) == 1 else best[best % 2 == 0][0]
        assert (c & 7) == want and (c >> 3) == np.signbit(x)


@pytest.mark.parametrize("top", [6.0, 448.0])
def test_scale_byte(top):
    for s in (-126, -60, -1, 0, 1, 5, 100):
        edge = top * 2.0 ** s
        for a, want in ((edge, s), (edge * (1 + 2.0 ** -23), s + 1), (edge * (1 - 2.0 ** -23), s)):
            blk = np.zeros(32)
            blk[7] = -a
            if want <= 120:
                assert oracle.mx_scale_byte(blk, top) == want + 127, (a, want)
    assert oracle.mx_scale_byte(np.zeros(32), top) == 127
    tiny = np.zeros(32)
    tiny[0] = 1e-45
    assert oracle.mx_scale_byte(tiny, top) == 1
    for bad in (np.nan, np.inf, -np.inf):
        tiny[3] = bad
        assert oracle.mx_scale_byte(tiny, top) == 255


def test_rows_error_is_half_a_step():
    A = RNG.standard_normal((9, 96)) * np.exp(RNG.uniform(-20, 20, (9, 1)))
    q, sb = oracle.quant_mx4_rows(A)
    v = oracle.dequant_mx4_rows(q, sb)
    sc = np.repeat(np.exp2(sb.astype(float) - 127), 32, axis=1)
    m = np.abs(A) / sc
    step = np.where(m < 2, 0.5, np.where(m < 4, 1.0, 2.0))
    assert (m <= 6).all() and (np.abs(v - A) <= step / 2 * sc * (1 + 1e-12)).all()


def test_tile_layout_element_by_element():
    E, R, C = 2, 256, 128
    W1, W3 = (RNG.standard_normal((E, R, C)) for _ in range(2))
    codes, scales = oracle.quant_mx4_weights(W1, W3)
    W = oracle.dequant_mx4_weights(codes, scales)
    for M, got in zip((W1, W3), split_pair(W)):
        for e in range(E):
            q, sb = oracle.quant_mx4_rows(np.ascontiguousarray(M[e].T))
            assert np.array_equal(got[e], oracle.dequant_mx4_rows(q, sb).T)
    for _ in range(200):
        e, n, k = RNG.integers(E), RNG.integers(2 * C), RNG.integers(R)
        grp, c = n // 16, n % 16
        src = (W1, W3)[grp % 2][e, :, (grp // 2) * 16 + c]
        byte = codes[e, n // 16, k // 128, (k % 128) // 32, c, (k % 32) // 2]
        sc = scales[e, n // 64, k // 128, (k % 128) // 32, c, (n // 16) % 4]
        val = oracle.mx4_decode((byte >> 4) if k % 2 else (byte & 15)) * 2.0 ** (int(sc) - 127)
        blk = src[k // 32 * 32:k // 32 * 32 + 32]
        assert val == oracle.dequant_mx4_rows(*oracle.quant_mx4_rows(blk[None]))[0, k % 32]


@pytest.mark.parametrize("a8", [False, True])
def test_layer_stays_near_the_unquantised_one(a8):
    """E2M1 rounds a value by at most a quarter of itself (half a step of 0.5 in
    [1, 2), of 1 in [2, 4), of 2 in [4, 6]) or of 0.25 scales below that; over
    sums of 128 and more independent roundings the result keeps its direction."""
    T, d, E, k, f = 24, 128, 4, 2, 128
    x, logits = RNG.standard_normal((T, d)), RNG.standard_normal((T, E)).astype(np.float32)
    W1, W3, W2 = (RNG.standard_normal(s) * s[1] ** -0.5 for s in ((E, d, f), (E, d, f), (E, f, d)))
    st = oracle.layer_fwd_mx4(logits, x, W1, W3, W2, k, a8)
    ref = oracle.layer_fwd(logits, x, W1, W3, W2, k)
    y, r = st["y"].ravel(), ref["y"].ravel()
    assert y @ r / np.linalg.norm(y) / np.linalg.norm(r) > 0.95
