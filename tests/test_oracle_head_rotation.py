"""The oracle of head norms and rotations, pinned to complex arithmetic, to what a
rotation leaves alone, and to values worked out by hand; the library's frequencies
(host code) pinned to it, and its units of 2^-64 turn to exact integers."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest

from oracle import head_rotation as ohr


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_attention_scatter_gb300 as pkv
    pkv.build()
    pkv.load()
    return pkv


def test_one_pair_by_hand():
    x = np.array([[[3.0, 4.0]]])
    got = ohr.norm_rope(x, [2.0, 1.0], 0.0, [2], [math.pi / 4])
    r = math.sqrt(12.5)                                # rms; a quarter turn: (a, b) -> (-b, a)
    assert np.allclose(got, [[[-4 / r, 6 / r]]], atol=1e-15)


@pytest.mark.parametrize("interleaved", [False, True])
def test_complex_product_norms_and_relative_positions(interleaved):
    rng = np.random.default_rng(0)
    x = rng.normal(size=(5, 3, 24))
    freq, _ = ohr.frequencies(16, 100.0)
    pos = np.array([0, 1, 7, 1000, -3])
    y = ohr.norm_rope(x, None, 0.0, pos, freq, interleaved)
    i, j = (np.arange(0, 16, 2), np.arange(1, 16, 2)) if interleaved else (np.arange(8),
                                                                           np.arange(8, 16))
    z = (x[..., i] + 1j * x[..., j]) * np.exp(1j * pos[:, None] * np.asarray(freq))[:, None]
    assert np.allclose(y[..., i], z.real, atol=1e-12)
    assert np.allclose(y[..., j], z.imag, atol=1e-12)
    assert np.array_equal(y[..., 16:], x[..., 16:])
    assert np.array_equal(y[0], x[0])                  # position 0
    # scores depend on the difference of positions
    a, b = ohr.norm_rope(x, None, 0, pos + 11, freq, interleaved), y
    assert np.allclose((a[1] * a[2]).sum(-1), (b[1] * b[2]).sum(-1))


SPECS = [dict(rotary_dim=128, base=1e6), dict(rotary_dim=64, base=1e4, scaling="linear", factor=4),
         dict(rotary_dim=20, base=5e5, scaling="ntk", factor=2.5),
         dict(rotary_dim=128, base=1e6, scaling="yarn", factor=4, original_max_position=32768),
         dict(rotary_dim=16, base=1e4, scaling="yarn", factor=8, original_max_position=20),
         dict(rotary_dim=64, base=1e4, scaling="yarn", factor=8, original_max_position=4096,
              low=2, high=16),
         dict(rotary_dim=128, base=5e5, scaling="bands", factor=8, original_max_position=8192),
         dict(rotary_dim=2, base=10.0, scaling="bands", factor=8, original_max_position=10,
              low=0.5, high=2)]


@pytest.mark.parametrize("spec", SPECS)
def test_library_frequencies(pkv, spec):
    got, mag = pkv.rotary_frequencies(**spec)
    ref, rmag = ohr.frequencies(**spec)
    # powers and products in 64 bits on both sides
    assert np.allclose(got, ref, rtol=1e-14, atol=0) and abs(mag - rmag) <= 2.0 ** -24 * rmag


def test_frequencies_by_hand(pkv):
    assert pkv.rotary_frequencies(4, 100.0) == ([1.0, 0.1], 1.0)
    assert pkv.rotary_frequencies(4, 100.0, "linear", 2)[0] == [0.5, 0.05]
    # 100 positions: w = 1 makes 15.9 turns, 0.1 makes 1.59, between 1 and 4
    got = pkv.rotary_frequencies(4, 100.0, "bands", 2, 100)[0]
    keep = (10 / (2 * math.pi) - 1) / 3
    assert got[0] == 1.0 and abs(got[1] - (0.1 * keep + 0.05 * (1 - keep))) < 1e-16


PI = Fraction(3141592653589793238462643383279502884197169399375105820974944592307816406286,
              10 ** 75)


@pytest.mark.parametrize("f", [0.0, 1.0, 65536.0, 6.283185307179586, 1e-5, 0.1234567890123, 2e-19,
                               1e-300, 5e-324, 2.0 ** -64, 3.0])
def test_turns_are_the_nearest_integers(pkv, f):
    out = (ctypes.c_uint64 * 1)()
    assert pkv.load().pkv_rotary_turns((ctypes.c_double * 1)(f), 1, out) == 0
    exact = Fraction(f) / (2 * PI) * 2 ** 64
    off = (out[0] - exact) % 2 ** 64
    assert min(off, 2 ** 64 - off) <= Fraction(1, 2) + Fraction(1, 10 ** 6)
