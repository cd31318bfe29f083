"""The integer weights' oracle against exact rational arithmetic, brute force and
round trips."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle


def smallest_scale(need: Fraction) -> Fraction:
    """Smallest k 2^e >= need with k < 2^20, at least 2^-126, by search over e."""
    s = None
    for e in range(-160, 140):
        k = -((-need) // Fraction(2) ** e)
        if k < 2 ** 20 or (k == 2 ** 20):
            s = k * Fraction(2) ** e
            break
    return max(s, Fraction(1, 2 ** 126))


def rint(v: Fraction) -> int:
    return round(v)  # Python rounds fractions half to even


@pytest.mark.parametrize("asym", [False, True])
def test_groups_against_fractions(asym):
    rng = np.random.default_rng(1)
    W = (rng.standard_normal((1, 128, 12)) * np.exp2(rng.integers(-40, 40, (1, 1, 12)))).astype(np.float32)
    W[0, :, 1] = 0
    W[0, :32, 2] = np.abs(W[0, :32, 2])
    W[0, :32, 3] = -np.abs(W[0, :32, 3])
    W[0, :32, 4] = np.arange(32) / 2 - 7                    # halves: ties
    W[0, 32:64, 4] = np.float32(1e-42)
    W[0, 64:96, 5] = np.linspace(-3.4e38, 3.4e38, 32)
    q, s, z = oracle.quant_i4(W, 32, asym)
    for c in range(12):
        for g in range(4):
            w = [Fraction(float(v)) for v in W[0, 32 * g:32 * g + 32, c]]
            lo, hi = min(w + [Fraction(0)]), max(w + [Fraction(0)])
            need = (hi - lo) / 15 if asym else max(hi, -lo) / 7
            sc = Fraction(1) if need == 0 else smallest_scale(need)
            # (fp64 spans: exact unless 2^29 apart)
            if sc >= 2 ** 124:
                assert np.isnan(s[0, g, c])
                continue
            assert Fraction(float(s[0, g, c])) == sc
            zz = min(max(rint(-lo / sc), 0), 15) if asym else 8
            assert z[0, g, c] == zz
            assert [int(v) for v in q[0, 32 * g:32 * g + 32, c]] == [min(max(rint(v / sc) + zz, 0), 15) for v in w]


def test_scale_is_the_smallest():
    for need in (1.0, 1.5, 1 + 2.0 ** -19, 1 + 2.0 ** -20, 2 - 2.0 ** -30, 3e-38, 1e-45):
        s = float(oracle.i4._scale_up(np.array(need)))
        assert s >= need and Fraction(s) == smallest_scale(Fraction(need))


def test_bf16_round_against_torch():
    v = np.random.default_rng(2).standard_normal(4096).astype(np.float32) * 10
    v[:512] = (np.arange(512) + 256.5) / 256                # ties
    assert np.array_equal(oracle.bf16_round(v), torch.from_numpy(v).bfloat16().double().numpy())


@pytest.mark.parametrize("asym", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_error_is_half_a_step(group, asym):
    W = np.random.default_rng(group).standard_normal((2, 256, 16))
    q, s, z = oracle.quant_i4(W, group, asym)
    s_ = np.repeat(s, group, axis=1)
    err = np.abs(s_ * (q - np.repeat(z.astype(float), group, axis=1)) - W)
    # (asymmetric: the zero point's rounding moves the ends by up to half a step more)
    assert (err <= s_ * (1.0 if asym else 0.5) * (1 + 1e-12)).all()
    assert np.abs(oracle.dequant_i4(q, s, z) - W).max() <= (err + 2.0 ** -8 * np.abs(W)).max() + 1e-2


@pytest.mark.parametrize("group", [32, 64, 128])
def test_tiles_round_trip_and_places(group):
    rng = np.random.default_rng(group)
    q = [rng.integers(0, 16, (2, 256, 64)).astype(np.uint8) for _ in range(2)]
    s = [np.exp2(rng.integers(-9, 9, (2, 256 // group, 64))).astype(np.float64) for _ in range(2)]
    z = [rng.integers(0, 16, (2, 256 // group, 64)).astype(np.uint8) for _ in range(2)]
    codes, words = oracle.i4_tiles(q[0], s[0], z[0], (q[1], s[1], z[1]))
    assert codes.shape == (2, 8, 2, 4, 16, 16) and words.shape == (2, 2, 2, 128 // group, 16, 4)
    for p, got in enumerate(oracle.i4_untiled(codes, words, True)):
        assert all(np.array_equal(a, b) for a, b in zip(got, (q[p], s[p], z[p])))
    # row 128 + 32*2 + 8*3 + 4 + 1 of column 17 of the second matrix: stored column 16*(2*1+1) + 1
    assert codes[1, 3, 1, 3, 1, 4 * 2 + 1] >> 4 == q[1][1, 128 + 64 + 24 + 5, 17]
    one = oracle.i4_tiles(q[0], s[0], z[0])
    assert np.array_equal(oracle.i4_untiled(*one)[0], q[0])


def test_experts_match_the_plain_oracle():
    """On weights that are whole multiples the 4-bit experts are the plain ones up to h's rounding."""
    rng = np.random.default_rng(6)
    E, d, f, P = 3, 128, 128, 10
    W = [rng.integers(-8, 8, s).astype(np.float64) / 64 for s in ((E, d, f), (E, d, f), (E, f, d))]
    Wq = []
    for w in W:
        q = (w * 64 + 8).astype(np.uint8)
        Wq.append(oracle.dequant_i4(q, np.full((E, 1, w.shape[2]), 1 / 64), np.full((E, 1, w.shape[2]), 8, np.uint8)))
        assert np.array_equal(Wq[-1], w)
    x, off = rng.standard_normal((P, d)), np.array([0, 4, 4, 10])
    o = oracle.experts_fwd_i4(x, off, *Wq)[0]
    ref = oracle.experts_fwd(x, off, *W)[3]
    h = oracle.experts_fwd_i4(x, off, *Wq)[1]
    bound = np.zeros_like(ref)
    for e in range(E):
        r = slice(off[e], off[e + 1])
        bound[r] = 2.0 ** -8 * np.abs(h[r]) @ np.abs(W[2][e])
    assert (np.abs(o - ref) <= bound + 1e-12).all()
