"""What the 4-bit format holds at every magnitude, on its 64-bit form (which the
kernels match bit for bit), and that scaling by a power of two brings small rows
into its range."""
import numpy as np
import pytest

import cache_ref as ref


def rows(a, seed):
    """Rows whose groups of 16 have the largest magnitude a."""
    x = np.random.default_rng(seed).uniform(-1, 1, (64, 8, 16))
    x /= np.abs(x).max(-1, keepdims=True)
    return (x * a).reshape(64, 128)


def error(x):
    return np.abs(ref.dequantise(*ref.quantise(x)) - x).max()


@pytest.mark.parametrize("e", range(-16, 12))
def test_bounds(e):
    """The scale is off by 2^-4 of it at most (from 6 * 2^-6 up), or by 2^-10: a code's half
    step of 1, or what is cut above 6, is then below 0.18 a, or a / 6 + 6 * 2^-10.  Above
    2688 the scale stays 448: its half step, or what is cut."""
    for i, f in enumerate(np.linspace(1, 2, 9)[:-1]):
        a = f * 2.0 ** e
        bound = 0.18 * a if a >= 6 * 2.0 ** -6 else a / 6 + 6 * 2.0 ** -10
        assert error(rows(a, i)) <= (bound if a <= 2688 else max(448, a - 2688))


def test_smallest():
    x = rows(2.0 ** -11, 3)
    assert not ref.dequantise(*ref.quantise(x)).any()
    assert ref.dequantise(*ref.quantise(rows(2.0 ** -11 * 1.001, 3))).any()


@pytest.mark.parametrize("a", [3e-5, 0.001, 0.01, 0.05])
def test_scaled_rows(a):
    x = rows(a, 5)
    k = 2.0 ** -np.floor(np.log2(a))
    assert np.abs(ref.dequantise(*ref.quantise(x * k)) / k - x).max() <= 0.18 * a
