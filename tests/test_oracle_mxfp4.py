"""Pins of the MXFP4 oracle: worked blocks, ties, the clamped exponents and NaN blocks, and
the routing rule, each against values written out by hand or exact rationals."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import mxfp4_oracle as M4
from workloads import to_bf16_bits


def _codes(packed):
    return np.stack((packed & 15, packed >> 4), axis=-1).reshape(packed.shape[0], -1)


def test_worked_block():
    x = np.zeros((1, 32), dtype=np.float32)
    # amax 6 -> e = 2 - 2 = 0, byte 127
    x[0, :16] = [6, -6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, 0.2, -0.3, 0.5, -0.0, 4, 3, 2]
    p, s = M4.quantize(to_bf16_bits(x))
    assert s[0, 0] == 127
    want = [7, 15, 6, 6, 4, 4, 2, 2, 0, 0, 9, 1, 8, 6, 5, 4]
    assert list(_codes(p)[0, :16]) == want
    assert list(M4.dequantize(p, s)[0, :4]) == [6.0, -6.0, 4.0, 4.0]


@pytest.mark.parametrize("amax, byte", [(1.0, 125), (1.99, 125), (2.0, 126), (7.97, 127), (8.0, 128),
                                        (2.0**-126, 0), (2.0**-124, 1), (2.0**-133, 0), (3.3e38, 252)])
def test_scale_bytes(amax, byte):
    x = np.zeros((1, 32), dtype=np.float32)
    x[0, 5] = -amax
    assert M4.quantize(to_bf16_bits(x))[1][0, 0] == byte


def test_saturation_zero_and_nan_blocks():
    x = np.zeros((1, 96), dtype=np.float32)
    x[0, 0], x[0, 1] = 7.9, -7.0           # above 6 at e = 0: saturate
    x[0, 64], x[0, 65] = np.nan, 1.0
    p, s = M4.quantize(to_bf16_bits(x))
    assert list(s[0]) == [127, 0, 255]
    assert list(_codes(p)[0, :2]) == [7, 15]
    v = M4.dequantize(p, s)
    assert not v[0, 32:64].any() and np.isnan(v[0, 64:]).all()


def test_nearest_even_against_rationals():
    """Every bf16 value of one binade range against the nearest of the 8 magnitudes, by exact
    rational distance."""
    bits = np.arange(0x3E00, 0x40FF, dtype=np.uint16)   # 0.125 .. 7.97
    bits = bits[: bits.size // 31 * 31].reshape(-1, 31)
    x = np.concatenate([np.full((bits.shape[0], 1), 0x40C0, dtype=np.uint16), bits], axis=1)  # 6.0 leads
    p, s = M4.quantize(x)
    assert (s == 127).all()
    codes = _codes(p)
    vals = [Fraction(v) for v in M4.E2M1_POS]
    for row_c, row_b in zip(codes, x):
        for c, b in zip(row_c, row_b):
            v = Fraction(float(np.array([int(b) << 16], dtype=np.uint32).view(np.float32)[0]))
            d = [abs(v - q) for q in vals]
            best = [i for i in range(8) if d[i] == min(d)]
            assert c == (best[0] if len(best) == 1 else [i for i in best if i % 2 == 0][0]), float(v)


def test_routing_rule():
    inf, nan = np.inf, np.nan
    l = np.array([[1, 3, 3, 2], [-inf, 0, -inf, -inf], [-inf] * 4, [0, nan, 5, 1], [0.0, -0.0, -1, -2]],
                 dtype=np.float32)
    ids, w = M4.route(l, 2, True)
    assert ids.tolist() == [[1, 2], [1, -1], [-1, -1], [1, 2], [0, 1]]
    assert w[0].tolist() == [0.5, 0.5] and w[1].tolist() == [1.0, 0.0] and not w[2].any()
    assert np.isnan(w[3]).all()
    _, full = M4.route(l, 2, False)
    z = np.exp([1.0, 3, 3, 2])
    assert np.allclose(full[0], z[1] / z.sum())
