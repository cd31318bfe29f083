"""The tile orders of the grouped products (csrc/tile_order.h), on the CPU: every
tile is taken once, and rows count as uneven exactly when an eighth of the tile
list holds more than 5/4 of an eighth of them."""
import ctypes
import os
import shutil
import subprocess
from fractions import Fraction

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def order(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("needs a C++ compiler")
    so = str(tmp_path_factory.mktemp("order") / "order.so")
    subprocess.run([cxx, "-O1", "-std=c++17", "-shared", "-fPIC", "-I",
                    os.path.join(os.path.dirname(HERE), "token_routed_expert_amd", "csrc"),
                    os.path.join(HERE, "tile_order_check.cpp"), "-o", so], check=True, capture_output=True, text=True)
    return ctypes.CDLL(so)


@pytest.mark.parametrize("fn", ["remap", "remap_rounds8", "remap_rounds32"])
def test_every_tile_once(order, fn):
    for n in list(range(1, 80)) + [255, 256, 257, 511, 513, 1000, 4099]:
        assert sorted(getattr(order, fn)(i, n) for i in range(n)) == list(range(n))


def offsets(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def uneven(order, counts):
    off = offsets(counts)
    return bool(order.uneven(off.ctypes.data_as(ctypes.c_void_p), len(counts)))


def by_tiles(counts):
    """The rule from its words: every expert has the same number of tiles, an eighth
    of the list takes its tiles, each with its expert's rows."""
    E = len(counts)
    share = [Fraction(0)] * 8
    for t in range(8 * E):                     # 8 tiles an expert: eighths end between tiles
        share[t // E] += Fraction(counts[t // 8], 8)
    return max(share) > Fraction(5, 4) * Fraction(sum(counts), 8)


@pytest.mark.parametrize("rows", [1, 32, 482])
def test_even_rows_are_even_for_every_number_of_experts(order, rows):
    for E in range(1, 257):
        assert not uneven(order, [rows] * E), E


def test_against_the_words(order):
    rng = np.random.default_rng(0)
    seen = set()
    for _ in range(3000):
        E = int(rng.integers(1, 40))
        counts = rng.integers(0, 60, E) + 40 * int(rng.integers(0, 6))
        counts = [int(c) for c in counts]
        if rng.random() < 0.3:
            counts[int(rng.integers(E))] += int(rng.integers(0, 2000))
        assert uneven(order, counts) == by_tiles(counts), counts
        seen.add((by_tiles(counts), E % 8 == 0))
    assert len(seen) == 4


def test_rows_near_the_largest_call(order):
    big = (2 ** 31 - 1) // 64
    assert not uneven(order, [big] * 64)
    assert uneven(order, [2 ** 31 - 64] + [1] * 16)
    assert not uneven(order, [0] * 5)          # no rows at all
