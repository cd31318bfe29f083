"""Pins of the 8-bit checkpoint oracle, CPU only: the backward formula against
central differences of the forward, and the kept values within half an E4M3 step."""
import numpy as np

import oracle

RNG = np.random.default_rng(8)


def test_swiglu_backward_against_differences():
    """Central differences at step t err by t^2/6 times the third derivative (below
    2 for silu, times |b p g|) plus 2^-52/t rounding: t = 2^-14 keeps both under 1e-8
    times the terms' magnitude."""
    P, f = 7, 32
    a, b, g = (RNG.standard_normal((P, f)) * 2 for _ in range(3))
    p = RNG.uniform(0.05, 1, P)
    loss = lambda a, b, p: (g * p[:, None] * oracle.moe.silu(a) * b).sum()  # noqa: E731
    da, db, h, dp = oracle.swiglu_bwd_rowscaled(a, b, p, g)
    t = 2.0 ** -14
    for _ in range(60):
        i, j = RNG.integers(P), RNG.integers(f)
        u = np.zeros((P, f))
        u[i, j] = t
        assert abs((loss(a + u, b, p) - loss(a - u, b, p)) / (2 * t) - da[i, j]) < 1e-6
        assert abs((loss(a, b + u, p) - loss(a, b - u, p)) / (2 * t) - db[i, j]) < 1e-6
    for i in range(P):
        u = np.zeros(P)
        u[i] = t
        assert abs((loss(a, b, p + u) - loss(a, b, p - u)) / (2 * t) - dp[i]) < 1e-6
    assert np.array_equal(h, p[:, None] * (oracle.moe.silu(a) * b))


def test_rowscaled_forward_is_the_weighted_plain_one():
    counts, d, f = [3, 0, 5], 32, 64
    off = np.concatenate([[0], np.cumsum(counts)])
    x, p = RNG.standard_normal((8, d)), RNG.uniform(0, 1, 8)
    W1, W3 = RNG.standard_normal((3, d, f)), RNG.standard_normal((3, d, f))
    W2 = RNG.standard_normal((3, f, d))
    a, b, h, o = oracle.rowscaled_fwd(x, off, W1, W3, W2, p)
    for e in range(3):
        for r in range(off[e], off[e + 1]):
            want = (oracle.moe.silu(x[r] @ W1[e]) * (x[r] @ W3[e])) @ W2[e] * p[r]
            assert np.allclose(o[r], want, rtol=1e-12, atol=1e-12)


def test_kept_values_are_within_half_a_step():
    v = RNG.standard_normal((40, 96)) * np.exp(RNG.uniform(-30, 30, (40, 1)))
    q, sb = oracle.quant_mx8_rows(v)
    back = oracle.dequant_mx8_rows(q, sb)
    sc = np.repeat(np.exp2(sb.astype(float) - 127), 32, axis=1)
    m = np.abs(v) / sc
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(m, 1e-300))), -6) - 3)
    assert (m <= 448).all() and (np.abs(back - v) <= step / 2 * sc).all()
