"""The pieces that attention over packed rows takes a weight in, in numpy: an f16
number's upper byte rounded to nearest, then that of what is left, and so on."""
import numpy as np
import pytest


def pieces(x, n):
    """The sum of n pieces of f16 numbers, in 64 bits."""
    left, total = x.copy(), np.zeros(x.shape)
    for _ in range(n):
        piece = ((left.view(np.uint16).astype(np.uint32) + 0x80) & 0xFF00).astype(np.uint16).view(np.float16)
        total += piece.astype(np.float64)
        left = (left - piece).astype(np.float16)
    return total


@pytest.mark.parametrize("n", [3, 4])
def test_weights_in_pieces(n):
    """Every weight up to 2^15: exact from 2^-6 on, and never off by more than
    2^-17, half of the smallest e5m2 number; a fourth piece is no nearer."""
    x = np.arange(0, 0x7801, dtype=np.uint16).view(np.float16)
    assert float(x[-1]) == 2.0 ** 15
    off = np.abs(pieces(x, n) - x.astype(np.float64))
    assert not off[x >= 2.0 ** -6].any()
    assert off.max() == 2.0 ** -17
    assert np.array_equal(off, np.abs(pieces(x, 3) - x.astype(np.float64)))
